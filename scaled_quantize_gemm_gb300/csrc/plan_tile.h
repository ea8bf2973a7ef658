// plan_tile.h -- where a tile of the experts' products by rows lies, out of the
// plan's words, and which rows of A it loads.  Plain arithmetic, also for a host
// compiler.  Whatever the words hold, a tile begins and ends on whole boxes inside
// the buffers (so a row number stays below rows + 256), and what its loads bring in
// are the bytes that its barrier expects: another routing's plan gives wrong
// numbers, no more.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define FP8SQ_HD __host__ __device__ __forceinline__
#else
#define FP8SQ_HD inline
#endif

namespace fp8sq {

constexpr int kTileHalf = 128;      // rows of a tile that one CTA holds
constexpr int kTileBox = 32;        // rows of a load where a CTA holds fewer

struct PlanTile {
    int row0, end, nb, expert;      // first row, the row its rows end before, column tile, expert
};

// Tile t of num_n column tiles a row tile, of the words of row tile t / num_n:
// {first tile of its group, expert << 8 | tiles in the group, the group's first row,
// the expert's last row + 1}.  rows: of the buffers, a multiple of kTileBox.  half:
// 128 rows further on.
FP8SQ_HD PlanTile plan_tile(int first, int expert_size, int row, int end, int t, int num_n, int E, int rows, int half)
{
    auto low = [](int a, int b) { return a < b ? a : b; };
    auto high = [](int a, int b) { return a > b ? a : b; };
    PlanTile x;
    // (unsigned where foreign words could overflow)
    const int r = (int)((uint32_t)t - (uint32_t)first * (uint32_t)num_n), size = high(expert_size & 0xFF, 1);
    x.nb = low(high(r / size, 0), num_n - 1);
    x.expert = low(high(expert_size >> 8, 0), E - 1);
    const uint32_t at = (uint32_t)row + ((uint32_t)r - (uint32_t)x.nb * (uint32_t)size) * 2u * kTileHalf + (uint32_t)half * kTileHalf;
    x.row0 = low(high((int)at, 0), rows) & ~(kTileBox - 1);
    x.end = low(high(end, 0), rows) & ~(kTileBox - 1);
    return x;
}

// Rows of A that CTA `rank` of a tile loads: the expert's alone, in boxes of
// kTileBox rows, or kTileHalf in one.
FP8SQ_HD int plan_tile_rows(const PlanTile& x, int rank)
{
    const int left = x.end - x.row0 - rank * kTileHalf;
    return left < 0 ? 0 : left < kTileHalf ? left : kTileHalf;
}

}  // namespace fp8sq
