// gemm_common.cuh -- pieces shared by the tensor-core GEMM translation units:
// tile rasterisation, the shared-memory ring layout, the epilogue's staged
// bulk stores, and the host-side tensor-map and descriptor builders.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace fp8sq {

struct TileSched {
    int num_m, num_n, group;
    __device__ __forceinline__ void coords(int t, int& mb, int& nb) const
    {
        const int per_group = group * num_n;
        const int g = t / per_group;
        const int first = g * group;
        const int gs = min(num_m - first, group);
        const int r = t - g * per_group;
        mb = first + r % gs;
        nb = r / gs;
    }
};

// M-tiles per group of the rasterisation.  The concurrent tiles of one wave
// cover `group` M-tiles and about concurrent / group N-tiles, so they hold
// (group x tile_m + concurrent / group x tile_n) rows of K bytes in L2, and
// B is read from DRAM num_m / group times.  The largest group of 32, 16, 8
// whose wave stays within 48 MB (about a third of L2) is taken; 8 otherwise.
// Measured on the GB300 (per-tensor pair kernel, 16384 x 14336 x 4096 / 8192^3
// / 16384 x 4096 x 14336, us): group 8: 533.5 / 302.0 / 529.7; 16: 524.5 /
// 297.5 / 532.3; 32: 522.0 / 307.8 / 552.5.  The MX kernel at 8192^3: 16:
// 355.8, 32: 353.4, 64: 379.2.
inline int raster_group(int64_t K, int tile_m, int tile_n, int concurrent)
{
    for (int g = 32; g > 8; g /= 2) {
        const int64_t rows = (int64_t)g * tile_m + (int64_t)((concurrent + g - 1) / g) * tile_n;
        if (rows * K <= (int64_t)48 << 20) return g;
    }
    return 8;
}

constexpr int BM = 128;
constexpr int BK = 128;  // bytes = elements for 8-bit operands
constexpr int A_BYTES = BM * BK;

// ------------------------------------------------------------------ staged stores
constexpr int kStageBytes = 1024;   // one staging buffer: 32 rows x 32 bytes

// One lane's 32-byte staging row: 16 bf16 or 8 fp32 outputs.
template <bool OUT_BF16>
__device__ __forceinline__ void stage_row(uint8_t* rowp, const float* v)
{
    if (OUT_BF16) {
#pragma unroll
        for (int q4 = 0; q4 < 2; ++q4) {
            uint4 w4;
            __nv_bfloat162 h0 = __floats2bfloat162_rn(v[8 * q4 + 0], v[8 * q4 + 1]);
            __nv_bfloat162 h1 = __floats2bfloat162_rn(v[8 * q4 + 2], v[8 * q4 + 3]);
            __nv_bfloat162 h2 = __floats2bfloat162_rn(v[8 * q4 + 4], v[8 * q4 + 5]);
            __nv_bfloat162 h3 = __floats2bfloat162_rn(v[8 * q4 + 6], v[8 * q4 + 7]);
            w4.x = *reinterpret_cast<uint32_t*>(&h0);
            w4.y = *reinterpret_cast<uint32_t*>(&h1);
            w4.z = *reinterpret_cast<uint32_t*>(&h2);
            w4.w = *reinterpret_cast<uint32_t*>(&h3);
            *reinterpret_cast<uint4*>(rowp + 16 * q4) = w4;
        }
    } else {
        *reinterpret_cast<float4*>(rowp) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(rowp + 16) = make_float4(v[4], v[5], v[6], v[7]);
    }
}
// Bulk tensor store of a 32 x 32-byte staging buffer (one bulk group per call
// site's commit).
__device__ __forceinline__ void bulk_store_2d(const CUtensorMap* m, int x, int y, const uint8_t* buf)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(x), "r"(y), "r"(smem_addr(buf))
                 : "memory");
}

__device__ __forceinline__ void stage_store_drain(int lane)
{
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
}

template <int BN, int STAGES, int NACC, int EPI_STAGE_WARPS = 0>
struct Smem {
    static constexpr int B_BYTES = BN * BK;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int BAR_OFF = STAGES * STAGE;
    static constexpr int NBARS = 2 * STAGES + 2 * NACC + 1;
    static constexpr int STG_OFF = BAR_OFF + 512;                      // epilogue staging (1 KB per warp)
    static constexpr int BYTES = STG_OFF + EPI_STAGE_WARPS * kStageBytes + 1024;   // + alignment slack
    static_assert(NBARS * 8 + 16 <= 512, "barriers and the TMEM holder fit before the staging area");
};

// ------------------------------------------------------------------ giving up
// A producer's or an MMA thread's last act, whether or not a wait of its own
// ran out: another warp of the CTA may leave as soon as the error word is set,
// so a CTA exits only after its copies and its MMAs are known to be done (which
// the last releases of a pair's stages and accumulators say too).
// Issue i of a ring went to stage i % STAGES in phase i / STAGES.

// waits (with a limit) for the last `issued` copies of a ring
template <int STAGES>
__device__ __forceinline__ void drain_ring(uint64_t* full, int issued)
{
    for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
        wait_drain(&full[i % STAGES], (uint32_t)(i / STAGES) & 1u);
}
// CTA pairs: the odd CTA's copies are counted on the leader's barriers beside
// the leader's own, so those of a stage that the leader never issued complete
// no phase.  A producer that gives up writes its count into both CTAs (stop,
// -1 before); after a cluster barrier, the leader expects the odd CTA's bytes
// alone for the stages it was ahead by, `total` of them at most, and waits.
__device__ __forceinline__ void pair_stop(int* stop, uint32_t rank, int issued)
{
    stop[rank] = issued;
    st_shared_cluster_u32(cluster_map(smem_addr(&stop[rank]), rank ^ 1u), (uint32_t)issued);
}
template <int STAGES>
__device__ __forceinline__ void drain_odd(uint64_t* full, const int* stop, int total, uint32_t stage_bytes)
{
    const int odd = stop[1] >= 0 ? stop[1] : total;
    for (int i = stop[0]; i < odd; ++i) mbar_arrive_expect_tx(&full[i % STAGES], stage_bytes);
    for (int i = stop[0]; i < odd; ++i) wait_drain(&full[i % STAGES], (uint32_t)(i / STAGES) & 1u);
}

// ------------------------------------------------------------------ host
// 2-D u8 tensor [rows][inner] (inner contiguous), box box_rows x 128 bytes, 128-byte swizzle
bool make_tmap(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t rows, uint32_t box_rows);
// 2-D tensor map of 8-bit codes Q [M][N] (row pitch `pitch`, N if 0) for the
// staged code stores: box 32 rows x 32 bytes, no swizzle
bool make_tmap_codes(CUtensorMap* m, void* Q, int64_t M, int64_t N, int64_t pitch = 0);
// 2-D tensor map of an output D [M][N] (row pitch `pitch` elements, N if 0)
// for the staged epilogue stores: box 32 rows x 32 bytes, no swizzle (stores
// clip at the matrix edge)
bool make_tmap_out(CUtensorMap* m, void* D, int64_t M, int64_t N, bool bf16, int64_t pitch = 0);
// instruction descriptor, kind::f8f6f4: D fp32, A/B format, both K-major, N, M = 128
uint32_t make_idesc(int a_fmt, int b_fmt, int n);

}  // namespace fp8sq
