// ffn_pair.cuh -- products with their elementwise work in the epilogue on CTA
// pairs: the feed-forward sublayer's (ffn.cu) and the experts' (experts.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act.cuh"
#include "gemm_common.cuh"
#include "internal.h"
#include "plan_tile.h"
#include "ptx.cuh"

namespace fp8sq {

enum { kEpiAct = 0, kEpiGlu = 1, kEpiGluBwd = 2 };
// Experts' products over rows sorted by expert (segments that start and end on
// multiples of 32 rows, zeros in the rows that fill one up):
//   kRows    A's rows by expert, B [E][N][K]: D[r] = A[r] B[e(r)]^T
//   kRowsMn  the same with B [E][K][N]
//   kWgrad   D[e] = A_e^T B_e over the segment's rows, A [R][M], B [R][N]
// 32 rows are what an epilogue warp holds and what one MMA contracts over, so no
// store and no sum crosses a segment and nothing is masked.
enum { kNoGroups = 0, kRows = 1, kRowsMn = 2, kWgrad = 3 };

struct FfnParams {
    int M, N, K;             // N: columns of the accumulators' matrix (glu: features F)
    const float* sA;
    const float* sB;
    int act;
    const float* bias;       // [N] or null
    const void* res;         // [M][N] or null; may be D itself (read coherently, before the same thread writes)
    int res_f32;
    void* D;                 // [M][N] or null
    int d_f32;
    __nv_bfloat16* Z;        // [M][N] (glu: [g | u], [M][2N]) or null
    uint8_t* Q;              // [M][N] (glu_bwd: [M][2N]) or null
    int qfmt;
    float* qstate;           // multiplier at [qH], amax combined into [0]
    int qH;
    const __nv_bfloat16* gu; // glu_bwd: [g | u], [M][2N]
    int* err;
    // experts: the plan's offsets, tile count and tiles; sB then is [E] (kRows, kRowsMn), M the sorted rows (kWgrad:
    // rows of each D[e])
    const int32_t* offsets;
    const int32_t* ntiles;
    const int4* tiles;
    int E, max_tiles, rows;              // rows of the sorted buffers
    // experts, few rows: the plan's blocks of 32 rows, and the weight rows of an expert
    const int4* blocks;
    int max_blocks, wrows;
};

// Ring stages of 32 KB.  Where the epilogue reads rows beside the sums, the
// lines in flight need room in the L1 that shares the SM's memory with the ring:
// five stages, not six (2000 x 1616 -> 5440 with an fp32 residual 40.0 -> 36.8 us;
// gated backward of 1056 tokens, 928 -> 7776, 109 -> 106).  Without such reads
// six are as fast or faster (256 tokens, 4096 -> 2 x 14336: 29.9 against 30.9).
template <int KIND, int GROUP = 0>
constexpr int kFfnStages = KIND == kEpiGlu || (KIND == kEpiAct && GROUP != 0) ? 6 : 5;
// Epilogue warps: two per TMEM lane quarter; four for glu_bwd, whose epilogue is
// the longest (an exponential and a reciprocal an element, two outputs) and has
// more latency to cover than two warps of an SM quarter do.
template <int KIND>
constexpr int kFfnEpiWarps = KIND == kEpiGluBwd ? 16 : 8;
template <int KIND>
constexpr int kFfnThreads = 32 * (2 + kFfnEpiWarps<KIND>);
constexpr int kFfnBN = 256, kFfnBH = 128;
// Staging boxes of 1 KB, shared out among the epilogue warps.
template <int KIND>
constexpr int kFfnBoxes = KIND == kEpiGluBwd ? 64 : 32;
template <int KIND, int GROUP = 0, bool PAIR = true>
struct FfnSmem : Smem<PAIR ? kFfnBH : kFfnBN, PAIR ? kFfnStages<KIND, GROUP> : 4, 2, kFfnBoxes<KIND>> {
    using Base = Smem<PAIR ? kFfnBH : kFfnBN, PAIR ? kFfnStages<KIND, GROUP> : 4, 2, kFfnBoxes<KIND>>;
    // (swizzled staging wants its areas on 1 KB boundaries: stage_lines, the codes of glu_bwd)
    static constexpr int STG_OFF = KIND == kEpiGluBwd || (KIND == kEpiAct && GROUP != 0) ? Base::BAR_OFF + 1024 : Base::STG_OFF;
    static constexpr int BYTES = STG_OFF + Base::BYTES - Base::STG_OFF;
};

// ------------------------------------------------------------------ epilogue pieces
__device__ __forceinline__ uint32_t pack_bf16(float2 v)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// |v| as fp32 bits: their unsigned maximum is the amax, a NaN above everything
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
// the first `left` of 32 columns, nothing where keep is 0
__device__ __forceinline__ void max32(uint32_t& amax, const float2 (&v)[16], int left, uint32_t keep)
{
    float m = 0.0f;
    if (left >= 32) {
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max3_nan(m, fabsf(v[j].x), fabsf(v[j].y));
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (2 * j < left) m = max3_nan(m, fabsf(v[j].x), fabsf(v[j].y));
    }
    amax = max(amax, __float_as_uint(m) & keep);       // not negative: ordered as integers, a NaN above all
}
// 16 and 32 codes of one row
__device__ __forceinline__ uint4 codes16(const float2* v, float m, int fmt)
{
    uint32_t w[4];
    auto all = [&](auto cvt) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 a = __fmul2_rn(v[2 * j], f2(m)), b = __fmul2_rn(v[2 * j + 1], f2(m));
            w[j] = cvt(a.x, a.y) | (cvt(b.x, b.y) << 16);
        }
    };
    if (fmt == kE4M3) all([](float a, float b) { return cvt_e4m3x2(a, b); });
    else all([](float a, float b) { return cvt_e5m2x2(a, b); });
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store32_bf16(__nv_bfloat16* d, int left, const float2 (&v)[16])
{
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (8 * c + 8 <= left)
            *reinterpret_cast<uint4*>(d + 8 * c) = make_uint4(pack_bf16(v[4 * c]), pack_bf16(v[4 * c + 1]),
                                                              pack_bf16(v[4 * c + 2]), pack_bf16(v[4 * c + 3]));
}
__device__ __forceinline__ void store32_codes(uint8_t* q, int left, const float2 (&v)[16], float m, int fmt)
{
    if (16 <= left) *reinterpret_cast<uint4*>(q) = codes16(v, m, fmt);
    if (32 <= left) *reinterpret_cast<uint4*>(q + 16) = codes16(v + 8, m, fmt);
}

// Staged bulk stores of one epilogue warp: 4 KB, four boxes of 32 rows x 32
// bytes.  A row segment of 32 bytes per lane and one bulk store per box write
// whole sectors to L2, where 16-byte stores by lane write each sector twice.
// Boxes go out as they are filled; when the four are used up the warp waits
// until the earlier ones have been read.
struct Stager {
    uint8_t* buf;
    int lane, slot;
    // a chunk's first box waits until the previous chunk's have been read
    __device__ __forceinline__ void next_chunk() { slot = 4; }
    __device__ __forceinline__ void reset()
    {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        slot = 0;
    }
    __device__ __forceinline__ uint8_t* take(int boxes)
    {
        if (slot + boxes > 4) reset();
        uint8_t* p = buf + slot * kStageBytes;
        slot += boxes;
        return p + 32 * lane;
    }
    // bulk stores of `boxes` boxes of `cols` columns each at (col, row0)
    __device__ __forceinline__ void send(const CUtensorMap* m, int boxes, int cols, int col, int row0, int left)
    {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            const uint8_t* p = buf + (slot - boxes) * kStageBytes;
            for (int i = 0; i < boxes; ++i)
                if (i * cols < left) bulk_store_2d(m, col + i * cols, row0, p + i * kStageBytes);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
    __device__ __forceinline__ void bf16(const CUtensorMap* m, const float2 (&v)[16], int col, int row0, int left)
    {
        uint8_t* p = take(2);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(p + (c >> 1) * kStageBytes + (c & 1) * 16) =
                make_uint4(pack_bf16(v[4 * c]), pack_bf16(v[4 * c + 1]), pack_bf16(v[4 * c + 2]), pack_bf16(v[4 * c + 3]));
        send(m, 2, 16, col, row0, left);
    }
    __device__ __forceinline__ void f32(const CUtensorMap* m, const float2 (&v)[16], int col, int row0, int left)
    {
        uint8_t* p = take(4);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            *reinterpret_cast<float4*>(p + (c >> 1) * kStageBytes + (c & 1) * 16) =
                make_float4(v[2 * c].x, v[2 * c].y, v[2 * c + 1].x, v[2 * c + 1].y);
        send(m, 4, 8, col, row0, left);
    }
    __device__ __forceinline__ void codes(const CUtensorMap* m, const float2 (&v)[16], float mult, int fmt, int col,
                                          int row0, int left)
    {
        const uint4 lo = codes16(v, mult, fmt), hi = codes16(v + 8, mult, fmt);
        uint8_t* p = take(1);
        *reinterpret_cast<uint4*>(p) = lo;
        *reinterpret_cast<uint4*>(p + 16) = hi;
        send(m, 1, 32, col, row0, left);
    }
};

// One epilogue warp's 32 rows x 128 bytes of the output (64 bf16 or 32 fp32 columns)
// through its 4 KB staging area and one bulk store, in the tensor map's 128-byte
// swizzle (16-byte piece j of row r at piece j ^ (r & 7): no bank conflicts).  Whole
// 128-byte lines, because the TMA unit takes the stores row by row beside the
// loads: with 32-byte boxes they were as many requests as eight K blocks of loads.
template <bool F32>
__device__ __forceinline__ void stage_lines(uint8_t* buf, int lane, const CUtensorMap* m, const uint32_t* r, float scale,
                                            int col, int row0)
{
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
    uint8_t* row = buf + 128 * lane;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F32) {
                w[i] = __float_as_uint(__fmul_rn(__uint_as_float(r[4 * j + i]), scale));
            } else {
                const int k = 8 * j + 2 * i;
                w[i] = pack_bf16(__fmul2_rn(make_float2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), f2(scale)));
            }
        }
        *reinterpret_cast<uint4*>(row + ((j ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        bulk_store_2d(m, col, row0, buf);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

// a whole 32-byte sector in one load (16-byte loads by row take each twice).
// RO: through the read-only path; not the residual, which the call may be
// overwriting in place (other elements of it, at the time).
template <bool RO>
__device__ __forceinline__ void ldg32(uint4& a, uint4& b, const void* p)
{
    if constexpr (RO)
        asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
            : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
            : "l"(p));
    else
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                     : "l"(p)
                     : "memory");
}
template <bool RO>
__device__ __forceinline__ uint4 ldg16(const uint4* p)
{
    if constexpr (RO) return __ldg(p);
    else return *p;
}
// 32 columns of a row of bf16 (64 bytes) or fp32 (128 bytes) into registers,
// ahead of their use; zeros past `bytes_left`
template <int N, bool RO>
__device__ __forceinline__ void fetch_row(uint4* raw, const void* src, int bytes_left)
{
    const uint4* s = static_cast<const uint4*>(src);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        if (16 * (i + 2) <= bytes_left && (reinterpret_cast<uintptr_t>(src) & 31) == 0) ldg32<RO>(raw[i], raw[i + 1], s + i);
        else {
            raw[i] = 16 * (i + 1) <= bytes_left ? ldg16<RO>(s + i) : make_uint4(0, 0, 0, 0);
            raw[i + 1] = 16 * (i + 2) <= bytes_left ? ldg16<RO>(s + i + 1) : make_uint4(0, 0, 0, 0);
        }
    }
}
__device__ __forceinline__ float2 raw_bf16(const uint4* raw, int j)     // columns 2 j, 2 j + 1
{
    const uint4 w = raw[j >> 2];
    return unpack_bf16((j & 3) == 0 ? w.x : (j & 3) == 1 ? w.y : (j & 3) == 2 ? w.z : w.w);
}
__device__ __forceinline__ float2 raw_f32(const uint4* raw, int j)
{
    const uint4 w = raw[j >> 1];
    return (j & 1) ? make_float2(__uint_as_float(w.z), __uint_as_float(w.w))
                   : make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
}
// Waits for the loads from tensor memory, of which r is one: no use of r is
// moved ahead of it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ uint32_t atomic_add_acq_rel(uint32_t* p, uint32_t v)
{
    uint32_t old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}
// ------------------------------------------------------------------ tiles of 256 x 256
// Bound by the tensor cores where K is long (ncu, 2048 tokens, K 4096: tensor
// pipe active 85 % glu_fwd, 73 % gemm_act with gelu, z and codes, 68 % glu_bwd),
// by the epilogue where it is short: an accumulator's 128 x 256 values a CTA take
// about 8 us through eight warps (gelu, z and codes), which the MMAs of the next
// tile cover from K of about 3000 on.
// One GB300, us, a few passes on a cool GPU / back to back at the power limit:
// glu_fwd 16384 x 4096 -> 2 x 14336 with g, u and codes 1040-1070 / 1170-1240 (3640 /
// 3200 TFLOP/s); gemm_act 16384 x 4096 -> 14336 with bias, gelu_tanh, z and codes
// 553-569 / 632-667; glu_bwd 2048 x 4096 -> 14336 83.
// A tile of a pair's work: its first row (of A and D), the row its rows end
// before, its column tile, its expert, and the range of the contraction: the
// first coordinate, K blocks, 32-wide steps of the last block.
struct PairTile {
    int row0, end, nb, expert, k0, nkb, last;
};
// the plan's words (ordinary loads: the kernel that writes them may still run while
// this one is resident, so they are no constants of its run)
struct LoadPlan {
    template <typename T>
    __device__ __forceinline__ T operator()(const T* q) const { return *q; }
};
// (L2 only: leaves nothing in the SM's own cache)
struct LoadPlanL2 {
    template <typename T>
    __device__ __forceinline__ T operator()(const T* q) const { return __ldcg(q); }
};
template <int GROUP, bool PAIR, typename LOAD = LoadPlan>
__device__ __forceinline__ int pair_tiles(const FfnParams& p, const TileSched& sched)
{
    if constexpr (GROUP == kNoGroups) return sched.num_m * sched.num_n;
    else if constexpr (GROUP == kWgrad) return p.E * sched.num_m * sched.num_n;
    else return (PAIR ? 1 : 2) * min(LOAD()(p.ntiles), p.max_tiles) * sched.num_n;
}
// (One CTA a tile: the plan's tiles in halves of 128 rows, all first halves before
// all second ones, of which those past their expert's rows have no K blocks.)
// num: pair_tiles
template <int GROUP, bool PAIR, typename LOAD = LoadPlan>
__device__ __forceinline__ PairTile pair_tile(const FfnParams& p, const TileSched& sched, int t, int num)
{
    PairTile x;
    [[maybe_unused]] int half = 0;
    if constexpr (!PAIR) {
        const int n = num / 2;
        half = t >= n ? 1 : 0;
        t -= half * n;
    }
    if constexpr (GROUP == kWgrad) {
        const int per = sched.num_m * sched.num_n;
        int mb;
        x.expert = t / per;
        sched.coords(t - x.expert * per, mb, x.nb);
        x.row0 = mb * 2 * BM;
        x.end = p.M;
        // (whatever the plan holds, here and below, the work is bounded and every row inside the buffers)
        x.k0 = min(max(LOAD()(p.offsets + x.expert), 0), p.rows);
        const int rows = max(min(LOAD()(p.offsets + x.expert + 1), p.rows) - x.k0, 0);
        x.nkb = (rows + BK - 1) / BK;
        x.last = (rows - (x.nkb - 1) * BK + 31) / 32;
    } else if constexpr (GROUP != kNoGroups) {
        // a group's tiles share t / num_n with its first num_n * size tiles' range
        const int4 d = LOAD()(p.tiles + t / sched.num_n);
        const PlanTile y = plan_tile(d.x, d.y, d.z, d.w, t, sched.num_n, p.E, p.M, half);
        x.nb = y.nb;
        x.expert = y.expert;
        x.row0 = y.row0;
        x.end = y.end;
        x.k0 = 0;
        x.nkb = PAIR || x.row0 < x.end ? (p.K + BK - 1) / BK : 0;
        x.last = (p.K - (x.nkb - 1) * BK + 31) / 32;
    } else {
        int mb;
        sched.coords(t, mb, x.nb);
        x.row0 = mb * 2 * BM;
        x.end = p.M;
        x.expert = x.k0 = 0;
        x.nkb = (p.K + BK - 1) / BK;
        x.last = BK / 32;
    }
    return x;
}

// Rows of A that CTA `rank` of the pair loads for a tile.  Experts' products by rows:
// those of the expert alone (a multiple of 32, in boxes of 32 rows), as the rest of
// the tile's sums are not stored: an expert of few rows reads little beside its
// weights (on CTA pairs: 4 of 32 experts, 1040 -> 2304, 192 tokens 20.8 -> 18.7 us; 8 of 64, 4096 ->
// 2 x 1792, 256 tokens 158.9 -> 155.4; others within 1 %).
static_assert(kTileHalf == BM && kTileBox == kExpertPad, "plan_tile.h");
template <int GROUP>
__device__ __forceinline__ int pair_rows(const PairTile& x, int rank)
{
    if constexpr (GROUP == kRows || GROUP == kRowsMn) return plan_tile_rows({x.row0, x.end, x.nb, x.expert}, rank);
    else return BM;
}

// PAIR false (experts' rows): the same on one CTA a tile of 128 x 256 with MMAs of its
// own (M = 128), for experts of few rows: with 128 rows or less a pair's second CTA
// multiplies nothing but padding, and 256 rows of it take as long as the weights'
// bytes (experts.cu has both sides measured).
template <int KIND, int GROUP = kNoGroups, bool PAIR = true>
__global__ void __cluster_dims__(PAIR ? 2 : 1, 1, 1) __launch_bounds__(kFfnThreads<KIND>, 1)
    k_ffn_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, FfnParams p,
               uint32_t idesc, TileSched sched, const __grid_constant__ CUtensorMap tmO0,
               const __grid_constant__ CUtensorMap tmO1, const __grid_constant__ CUtensorMap tmO2)
{
    static_assert(PAIR || (GROUP == kRows && KIND != kEpiGluBwd), "one CTA a tile: experts' rows, weights K-major");
    constexpr int BN = kFfnBN, BH = kFfnBH, STAGES = PAIR ? kFfnStages<KIND, GROUP> : 4;
    constexpr bool b_mn = KIND == kEpiGluBwd || GROUP >= kRowsMn;          // (glu_bwd: Wd [K][F])
    constexpr bool a_mn = GROUP == kWgrad;
    using L = FfnSmem<KIND, GROUP, PAIR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t* empty = full + STAGES;
    uint64_t* afull = empty + STAGES;
    uint64_t* aempty = afull + 2;
    uint64_t* drain = aempty + 2;
    uint32_t* holder = reinterpret_cast<uint32_t*>(drain + 1);
    constexpr uint32_t TMEM_COLS = 2 * BN;
    __shared__ int s_skip;
    __shared__ int s_stop[2];                  // stages each CTA's producer had issued when it gave up, else -1
    const uint32_t rank = cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cid = PAIR ? blockIdx.x >> 1 : blockIdx.x, ncl = PAIR ? gridDim.x >> 1 : gridDim.x;
    // a tile's first row of B in this CTA.  glu_fwd: gate rows in the even CTA, the up
    // rows of the same features in the odd one
    auto weight_row = [&](const PairTile& x) {
        int br = KIND == kEpiGlu ? (int)rank * p.N + x.nb * BH : x.nb * BN + (int)rank * BH;
        if constexpr (GROUP == kRows) br += x.expert * (KIND == kEpiGlu ? 2 * p.N : p.N);
        return br;
    };

    // what touches no global memory of the kernel before this one runs ahead
    // of the wait on it
    if (threadIdx.x == 0) {
        s_stop[0] = s_stop[1] = -1;
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&afull[b], 1);
            mbar_init(&aempty[b], (PAIR ? 2 : 1) * kFfnEpiWarps<KIND>);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(holder, TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(holder, TMEM_COLS);
            tmem_relinquish();
        }
    }
    if constexpr (GROUP == kRows) {
        // The first tile's weights into L2 while the kernel before still runs, by the
        // plan as it stands there now: a hint, as a kernel or more lies between the
        // plan's and this one as a rule; for a plan that is not there yet the wrong
        // weights, no more (pair_tile keeps any plan's tiles within them).  A
        // sublayer, us, without / with: 8 of 64 experts, 4096 -> 1792, 1 token 53.8 / 51.2, 32
        // tokens 241 / 237; 2 of 8, 4096 -> 2048, 16 tokens 56.0 / 53.3; 4 of 32, 2304 -> 1040, 16
        // tokens 58.6 / 57.0; 6 of 96, 1024 -> 512, 4 tokens 28.4 / 27.2; on CTA pairs, 1024 tokens, 8
        // of 64 293.6 / 290.0, 2 of 16, 4096 -> 3584 160.2 / 156.8, 4 of 32 82.0 / 81.8.
        constexpr int64_t L2Q = (int64_t)64 << 20;
        const int num = threadIdx.x == 64 ? pair_tiles<GROUP, PAIR, LoadPlanL2>(p, sched) : 0;
        if (cid < num) {
            const PairTile x = pair_tile<GROUP, PAIR, LoadPlanL2>(p, sched, cid, num);
            const int br = weight_row(x), to = min(x.nkb, (int)(L2Q / ((int64_t)gridDim.x * L::B_BYTES)));
            for (int kb = 0; kb < to; ++kb) {
                prefetch_l2_2d(&tmB, kb * BK, br);
                if (!PAIR) prefetch_l2_2d(&tmB, kb * BK, br + (KIND == kEpiGlu ? p.N : BH));
            }
        }
    }
    pdl_enter();
    if (threadIdx.x == 0) s_skip = rank == 0 ? *reinterpret_cast<volatile int*>(p.err) : 0;
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();    // both CTAs' barriers initialised, the leader's flag written
    tc_fence_after();
    int skip = s_skip;
    if (rank != 0) skip = (int)ld_shared_cluster_u32(cluster_map(smem_addr(&s_skip), 0));
    const uint32_t tmem_base = *holder;

    const int num_tiles = pair_tiles<GROUP, PAIR>(p, sched);
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_bounded_err_cluster(bar, parity, p.err); };

    if (skip) {
        // a wait ran out earlier: compute nothing (the same decision in both CTAs)
    } else if (warp == 0) {
        if (lane == 0) {
            const uint32_t full0 = cluster_map(smem_addr(full), 0);
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool aborted = false;
            for (int t = cid; t < num_tiles && !aborted; t += ncl) {
                const PairTile x = pair_tile<GROUP, PAIR>(p, sched, t, num_tiles);
                const int ar = x.row0 + (int)rank * BM;
                const int br = weight_row(x);
                const int bk = GROUP == kRowsMn ? x.expert * p.K : x.k0;
                const int rows = pair_rows<GROUP>(x, (int)rank);
                const uint32_t tx = (uint32_t)((PAIR ? 2 : 1) * L::B_BYTES) +
                                    (uint32_t)(BK * (pair_rows<GROUP>(x, 0) + (PAIR ? pair_rows<GROUP>(x, 1) : 0)));
                for (int kb = 0; kb < x.nkb; ++kb) {
                    if (!wait(&empty[stage], phase ^ 1u)) {
                        aborted = true;
                        break;
                    }
                    uint8_t* sa = smem + stage * L::STAGE;
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], tx);
                    const int ka = x.k0 + kb * BK, kr = bk + kb * BK;
                    if constexpr (PAIR) {
                        if (rows == BM) {
                            tma_load_2d_pair(sa, &tmA, a_mn ? ar : ka, a_mn ? ka : ar, full0 + 8u * stage);
                        } else {
                            for (int i = 0; i < rows; i += 32)         // (experts: tmO2 is A in boxes of 32 rows)
                                tma_load_2d_pair(sa + i * BK, &tmO2, ka, ar + i, full0 + 8u * stage);
                        }
                        tma_load_2d_pair(sa + A_BYTES, &tmB, b_mn ? br : kr, b_mn ? kr : br, full0 + 8u * stage);
                    } else {
                        if (rows == BM) tma_load_2d(sa, &tmA, ka, ar, &full[stage]);
                        else
                            for (int i = 0; i < rows; i += 32) tma_load_2d(sa + i * BK, &tmO2, ka, ar + i, &full[stage]);
                        // gate rows, then up rows; or 256 rows
                        tma_load_2d(sa + A_BYTES, &tmB, kr, br, &full[stage]);
                        tma_load_2d(sa + A_BYTES + BH * BK, &tmB, kr, br + (KIND == kEpiGlu ? p.N : BH), &full[stage]);
                    }
                    ++issued;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // (experts: the next product's CTAs start as this grid's leave their SMs; 4 of
            // 32 experts, 2304 -> 1040 and back, 192 tokens on CTA pairs 56.5 -> 55.3 us)
            if (GROUP != kNoGroups) pdl_trigger();
            if (PAIR && __builtin_expect(aborted, 0)) pair_stop(s_stop, rank, issued);
            bool released = !aborted;
            for (int i = 0; i < STAGES && released; ++i) {     // every stage's last release has landed
                released = wait(&empty[stage], phase ^ 1u);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            // (else the copies, which complete on the leader's barriers)
            if (__builtin_expect(!released && rank == 0, 0)) drain_ring<STAGES>(full, issued);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            auto commit = [](uint64_t* bar) {
                if constexpr (PAIR) mma_pair_commit(bar, 3);
                else mma_commit(bar);
            };
            int stage = 0, lt = 0;
            uint32_t phase = 0;
            bool aborted = false;
            for (int t = cid; t < num_tiles && !aborted; t += ncl) {
                const PairTile x = pair_tile<GROUP, PAIR>(p, sched, t, num_tiles);
                if ((GROUP == kWgrad || !PAIR) && x.nkb == 0) continue;          // an expert without rows: zeros, no product
                const int b = lt & 1;
                const uint32_t u = (uint32_t)(lt >> 1);
                ++lt;
                if (!wait(&aempty[b], (u & 1u) ^ 1u)) {
                    aborted = true;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(b * BN);
                for (int kb = 0; kb < x.nkb; ++kb) {
                    if (!wait(&full[stage], phase)) {
                        aborted = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_addr(smem + stage * L::STAGE);
                    const uint64_t da = a_mn ? sdesc_mn_sw128(sa) : sdesc_kmajor_sw128(sa);
                    const uint64_t db = b_mn ? sdesc_mn_sw128(sa + A_BYTES) : sdesc_kmajor_sw128(sa + A_BYTES);
                    constexpr uint64_t sta = a_mn ? 256 : 2, stb = b_mn ? 256 : 2;
                    // (experts: what the last block holds past the range, rows of the next expert, is not multiplied)
                    const int steps = GROUP != kNoGroups && kb + 1 == x.nkb ? x.last : BK / 32;
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        if (GROUP == kNoGroups || k < steps) {
                            if constexpr (PAIR) mma_pair_f8f6f4(d, da + sta * k, db + stb * k, idesc, (kb | k) != 0 ? 1u : 0u);
                            else mma_f8f6f4(d, da + sta * k, db + stb * k, idesc, (kb | k) != 0 ? 1u : 0u);
                        }
                    commit(&empty[stage]);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!aborted) commit(&afull[b]);
            }
            bool released = !aborted;
            for (int j = 0; j < 2 && released; ++j) {       // both accumulators' last releases have landed
                const int l2 = lt + j;
                released = wait(&aempty[l2 & 1], ((uint32_t)(l2 >> 1) & 1u) ^ 1u);
            }
            if (__builtin_expect(!released, 0)) {
                if constexpr (PAIR) mma_pair_commit(drain, 1);          // completes once every issued MMA is done
                else mma_commit(drain);
                wait_drain(drain, 0);
            }
        }
    } else {
        const int quarter = warp & 3;       // the TMEM lane quarter this warp may read
        const int part = (warp - 2) >> 2;   // share of the columns
        constexpr int PARTS = kFfnEpiWarps<KIND> / 4, BOXES = kFfnBoxes<KIND> / kFfnEpiWarps<KIND>;
        float scale = __ldg(p.sA) * __ldg(p.sB);
        const float qm = p.Q ? p.qstate[p.qH] : 1.0f;
        uint32_t amax = 0;
        const uint32_t aempty0 = PAIR ? cluster_map(smem_addr(aempty), 0) : 0u;
        auto hand_back = [&](int b) {
            if constexpr (PAIR) mbar_arrive_cluster_relaxed(aempty0 + 8u * b);
            else mbar_arrive(&aempty[b]);
        };
        Stager out{smem + L::STG_OFF + (warp - 2) * BOXES * kStageBytes, lane, 0};
        // columns of a tile in this warp's share; what its epilogue reads
        // beside the sums (the residual, or g and u) is fetched one chunk of
        // 32 columns (16 of g and u) ahead, the first chunk's before the tile's
        // sums are done
        constexpr int TN = KIND == kEpiGlu ? BH : BN;
        const int c_begin = part * (TN / PARTS), c_end = c_begin + TN / PARTS;
        uint4 pre[KIND == kEpiGluBwd ? 4 : 8];
        auto fetch = [&](int row, int col, int end) {
            const int left = row < end ? min(p.N - col, 32) : 0;
            if constexpr (KIND == kEpiAct) {
                if (!p.res) return;
                if (p.res_f32) fetch_row<8, false>(pre, static_cast<const float*>(p.res) + (int64_t)row * p.N + col, 4 * left);
                else fetch_row<4, false>(pre, static_cast<const __nv_bfloat16*>(p.res) + (int64_t)row * p.N + col, 2 * left);
            } else if constexpr (KIND == kEpiGluBwd) {
                // 16 columns of g, then of u
                const __nv_bfloat16* s = p.gu + (int64_t)row * 2 * p.N + col;
                fetch_row<2, true>(pre, s, 2 * left);
                fetch_row<2, true>(pre + 2, s + p.N, 2 * left);
            }
        };
        int lt = 0;
        for (int t = cid; t < num_tiles; t += ncl) {
            const PairTile x = pair_tile<GROUP, PAIR>(p, sched, t, num_tiles);
            if (!PAIR && x.nkb == 0) continue;
            const bool some = GROUP != kWgrad || x.nkb > 0;          // (else zeros)
            const int b = lt & 1;
            const uint32_t u = (uint32_t)(lt >> 1);
            if (some) ++lt;
            const int nb = x.nb, end = x.end;
            const int row0 = x.row0 + (int)rank * BM + quarter * 32, row = row0 + lane;
            if constexpr (GROUP == kRows || GROUP == kRowsMn) scale = __ldg(p.sA) * __ldg(p.sB + x.expert);
            const int store0 = GROUP == kWgrad ? x.expert * p.M + row0 : row0;          // of the staged stores
            const uint32_t keep = row < end ? 0xFFFFFFFFu : 0u;
            const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(b * BN);
            fetch(row, nb * TN + c_begin, end);
            // gemm_act: lane l holds the bias of columns 4 l .. 4 l + 3 of the share
            [[maybe_unused]] float4 bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if constexpr (KIND == kEpiAct) {
                const int bc = nb * TN + c_begin + 4 * lane;
                if (p.bias && bc + 4 <= p.N) bias = __ldg(reinterpret_cast<const float4*>(p.bias + bc));
            }
            const bool ok = !some || wait(&afull[b], u & 1u);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
            if constexpr (GROUP != kNoGroups && KIND == kEpiAct) {
                // The product alone: short contractions (a weight gradient's few
                // hundred rows) leave it little time, so it stores whole lines, and
                // hands the accumulator back before its last are on their way.
                constexpr int HALF = TN / PARTS / 2;                   // 64 columns
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t r[2][32];
                    if (some) {
                        __syncwarp();                  // tcgen05.ld takes a converged warp
                        tmem_ld_32x32b_x32(taddr + (uint32_t)(c_begin + HALF * h), r[0]);
                        tmem_ld_32x32b_x32(taddr + (uint32_t)(c_begin + HALF * h + 32), r[1]);
                        tmem_ld_wait_for(r[0]);
                        tmem_ld_wait_for(r[1]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 64; ++j) r[j >> 5][j & 31] = 0;
                    }
                    if (h == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (some && lane == 0) hand_back(b);
                    }
                    const int col = nb * TN + c_begin + HALF * h;
                    if (row0 < end && col < p.N) {
                        const float sc = some ? scale : 0.0f;
                        if (p.d_f32) {
                            stage_lines<true>(out.buf, lane, &tmO1, r[0], sc, col, store0);
                            if (col + 32 < p.N) stage_lines<true>(out.buf, lane, &tmO1, r[1], sc, col + 32, store0);
                        } else {
                            stage_lines<false>(out.buf, lane, &tmO1, &r[0][0], sc, col, store0);
                        }
                    }
                }
            } else {
#pragma unroll 1
                for (int c = c_begin; c < c_end && row0 < end; c += 32) {
                    const int col = nb * TN + c, left = p.N - col;
                    if (left <= 0) break;
                    __syncwarp();                  // tcgen05.ld takes a converged warp
                    float2 v[16];
                    if constexpr (KIND == kEpiGlu) {
                        uint32_t rg[32], ru[32];
                        tmem_ld_32x32b_x32(taddr + (uint32_t)c, rg);
                        tmem_ld_32x32b_x32(taddr + (uint32_t)(BH + c), ru);
                        tmem_ld_wait();
                        float2 g[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            g[j] = __fmul2_rn(make_float2(__uint_as_float(rg[2 * j]), __uint_as_float(rg[2 * j + 1])), f2(scale));
                            v[j] = __fmul2_rn(make_float2(__uint_as_float(ru[2 * j]), __uint_as_float(ru[2 * j + 1])), f2(scale));
                        }
                        if (p.Z) {
                            out.next_chunk();
                            out.bf16(&tmO0, g, col, store0, left);
                            out.bf16(&tmO1, v, col, store0, left);
                        }
                        act_dispatch(p.act, [&](auto tag) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = __fmul2_rn(v[j], act_f2<decltype(tag)::act>(g[j]));
                        });
                        if (p.Q) max32(amax, v, left, keep);
                        if (keep) {
                            if (p.D) store32_bf16(static_cast<__nv_bfloat16*>(p.D) + (int64_t)row * p.N + col, left, v);
                            if (p.Q) store32_codes(p.Q + (int64_t)row * p.N + col, left, v, qm, p.qfmt);
                        }
                        __syncwarp();
                    } else if constexpr (KIND == kEpiAct) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(taddr + (uint32_t)c, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            v[j] = __fmul2_rn(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), f2(scale));
                        out.next_chunk();
                        if (p.bias) {
                            const int from = (c - c_begin) / 4;       // the lane that holds column c
#pragma unroll
                            for (int j = 0; j < 16; j += 2) {
                                const int s = from + j / 2;
                                v[j] = __fadd2_rn(v[j], make_float2(__shfl_sync(0xFFFFFFFFu, bias.x, s),
                                                                    __shfl_sync(0xFFFFFFFFu, bias.y, s)));
                                v[j + 1] = __fadd2_rn(v[j + 1], make_float2(__shfl_sync(0xFFFFFFFFu, bias.z, s),
                                                                            __shfl_sync(0xFFFFFFFFu, bias.w, s)));
                            }
                        }
                        if (p.Z) out.bf16(&tmO0, v, col, store0, left);
                        act_dispatch(p.act, [&](auto tag) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = act_f2<decltype(tag)::act>(v[j]);
                        });
                        if (p.res) {
                            if (p.res_f32) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) v[j] = __fadd2_rn(v[j], raw_f32(pre, j));
                            } else {
#pragma unroll
                                for (int j = 0; j < 16; ++j) v[j] = __fadd2_rn(v[j], raw_bf16(pre, j));
                            }
                            if (c + 32 < c_end) fetch(row, col + 32, end);
                        }
                        if (p.D) {
                            if (p.d_f32) out.f32(&tmO1, v, col, store0, left);
                            else out.bf16(&tmO1, v, col, store0, left);
                        }
                        if (p.Q) {
                            max32(amax, v, left, keep);
                            out.codes(&tmO2, v, qm, p.qfmt, col, store0, left);
                        }
                    } else {
                        // two halves of 16 columns, each a 16-byte piece of the two boxes' rows
                        // (32 rows x 64 codes of dg, then of du, in the maps' 64-byte swizzle:
                        // piece j of row r at j ^ ((r >> 1) & 3)), which go out as the warp's
                        // 64 columns are complete.  Boxes of 32 codes were twice as many
                        // requests to the TMA unit, beside the loads (4096 -> 14336, 8192 tokens 322 ->
                        // 307 us, 2048 tokens 86.4 -> 83.2).
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            uint32_t r[16];
                            __syncwarp();
                            tmem_ld_32x32b_x16(taddr + (uint32_t)(c + 16 * h), r);
                            tmem_ld_wait();
                            float2 dg[8], du[8];
                            act_dispatch(p.act, [&](auto tag) {
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const float2 dh = __fmul2_rn(
                                        make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), f2(scale));
                                    float2 f, d;
                                    act_fd2<decltype(tag)::act>(raw_bf16(pre, j), f, d);
                                    dg[j] = __fmul2_rn(__fmul2_rn(dh, raw_bf16(pre + 2, j)), d);
                                    du[j] = __fmul2_rn(dh, f);
                                }
                            });
                            const int cn = c + 16 * (h + 1);
                            if (cn < c_end) fetch(row, nb * TN + cn, end);
                            float m = 0.0f;
                            if (left > 16 * h) {
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    m = max3_nan(m, fabsf(dg[j].x), fabsf(dg[j].y));
                                    m = max3_nan(m, fabsf(du[j].x), fabsf(du[j].y));
                                }
                            }
                            amax = max(amax, __float_as_uint(m) & keep);
                            const uint4 qg = codes16(dg, qm, p.qfmt), qu = codes16(du, qm, p.qfmt);
                            if (c == c_begin && h == 0) out.reset();        // the last tile's boxes have been read
                            const int piece = (c - c_begin) / 16 + h;
                            uint8_t* q = out.buf + 64 * lane + 16 * (piece ^ ((lane >> 1) & 3));
                            *reinterpret_cast<uint4*>(q) = qg;
                            *reinterpret_cast<uint4*>(q + 2 * kStageBytes) = qu;
                        }
                        if (c + 32 >= c_end || left <= 32) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                bulk_store_2d(&tmO0, nb * TN + c_begin, row0, out.buf);
                                bulk_store_2d(&tmO1, nb * TN + c_begin, row0, out.buf + 2 * kStageBytes);
                                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) hand_back(b);
            }
        }
        stage_store_drain(lane);
        if (p.Q) {
            amax = __reduce_max_sync(0xFFFFFFFFu, amax);
            if (lane == 0) atomicMax(reinterpret_cast<unsigned int*>(p.qstate), amax);
        }
    }
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();
    if (PAIR && __builtin_expect(s_stop[0] >= 0, 0)) {                      // (the same in both CTAs)
        // what the odd CTA had loaded for stages that the leader never issued is
        // expected now, and waited for (with a limit)
        if (rank == 0 && threadIdx.x == 0) {
            auto odd = [&](auto&& f) {
                int i = 0;
                for (int t = cid; t < num_tiles; t += ncl) {
                    const PairTile x = pair_tile<GROUP, PAIR>(p, sched, t, num_tiles);
                    for (int kb = 0; kb < x.nkb; ++kb, ++i) {
                        if (s_stop[1] >= 0 && i >= s_stop[1]) return;
                        if (i >= s_stop[0]) f(i, (uint32_t)(L::B_BYTES + BK * pair_rows<GROUP>(x, 1)));
                    }
                }
            };
            odd([&](int i, uint32_t bytes) { mbar_arrive_expect_tx(&full[i % STAGES], bytes); });
            odd([&](int i, uint32_t) { wait_drain(&full[i % STAGES], (uint32_t)(i / STAGES) & 1u); });
        }
        cluster_sync_all();
    }
    // nothing is pending into either CTA any more
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem_base, TMEM_COLS);
        else tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

}  // namespace fp8sq
