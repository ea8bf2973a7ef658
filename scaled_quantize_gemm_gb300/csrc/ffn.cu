// ffn.cu -- the products of a feed-forward sublayer with their elementwise
// work in the epilogue, on the sm_103a tensor cores (per-tensor FP8 scales).
//
//   gemm_act  z = (sum_k A[m][k] B[n][k]) sA sB + bias[n],
//             y = act(z) + residual[m][n]; z (bf16), y (bf16 / fp32) and the
//             FP8 codes of y under a delayed state, each optional
//   glu_fwd   [g | u] = (A W^T) sA sW with W = [W_gate; W_up] ([2F][K]),
//             h = act(g) u; [g | u] (bf16), h (bf16) and its codes, each optional
//   glu_bwd   dh = (dY Wd) s; dg = dh u act'(g), du = dh act(g) from the
//             forward's [g | u]; the codes of [dg | du] under one delayed state
//
// All three run on CTA pairs (tcgen05 .cta_group::2, M = 256, N = 256; products
// of few rows or few tiles on k_ffn_rows and k_ffn_ksplit, further down): the
// even CTA issues the MMAs over both CTAs' shared memory and each CTA's TMEM
// holds its 128 rows, two accumulators of 256 columns.  In glu_fwd the even
// CTA loads 128 rows of W_gate and the odd one the same 128 rows of W_up, so
// columns 0-127 of an accumulator are g and columns 128-255 the u of the same
// features: one thread holds both and the product needs no exchange and no
// interleaved weight.
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act.cuh"
#include "gemm_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fp8sq {

enum { kEpiAct = 0, kEpiGlu = 1, kEpiGluBwd = 2 };

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
};

// Ring stages of 32 KB.  Where the epilogue reads rows beside the sums, the
// lines in flight need room in the L1 that shares the SM's memory with the ring:
// five stages, not six (2000 x 1616 -> 5440 with an fp32 residual 40.0 -> 36.8 us;
// gated backward of 1056 tokens, 928 -> 7776, 109 -> 106).  Without such reads
// six are as fast or faster (256 tokens, 4096 -> 2 x 14336: 29.9 against 30.9).
template <int KIND>
constexpr int kFfnStages = KIND == kEpiGlu ? 6 : 5;
// Epilogue warps: two per TMEM lane quarter; four for glu_bwd, whose epilogue is
// the longest (an exponential and a reciprocal an element, two outputs) and has
// more latency to cover than two warps of an SM quarter do.
template <int KIND>
constexpr int kFfnEpiWarps = KIND == kEpiGluBwd ? 16 : 8;
template <int KIND>
constexpr int kFfnThreads = 32 * (2 + kFfnEpiWarps<KIND>);
constexpr int kFfnBN = 256, kFfnBH = 128;
template <int KIND>
using FfnSmem = Smem<kFfnBH, kFfnStages<KIND>, 2, 32>;      // 32 staging boxes of 1 KB, shared out among the epilogue warps

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
// 553-569 / 632-667; glu_bwd 2048 x 4096 -> 14336 86 (under the profiler).
template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFfnThreads<KIND>, 1)
    k_ffn_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, FfnParams p,
               uint32_t idesc, TileSched sched, const __grid_constant__ CUtensorMap tmO0,
               const __grid_constant__ CUtensorMap tmO1, const __grid_constant__ CUtensorMap tmO2)
{
    constexpr int BN = kFfnBN, BH = kFfnBH, STAGES = kFfnStages<KIND>;
    constexpr bool b_mn = KIND == kEpiGluBwd;          // Wd [K][F]: MN-major
    using L = FfnSmem<KIND>;
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
            mbar_init(&aempty[b], 2 * kFfnEpiWarps<KIND>);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        tmem_alloc_pair(holder, TMEM_COLS);
        tmem_relinquish_pair();
    }
    pdl_enter();
    if (threadIdx.x == 0) s_skip = rank == 0 ? *reinterpret_cast<volatile int*>(p.err) : 0;
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                        // both CTAs' barriers initialised, the leader's flag written
    tc_fence_after();
    int skip = s_skip;
    if (rank != 0) skip = (int)ld_shared_cluster_u32(cluster_map(smem_addr(&s_skip), 0));
    const uint32_t tmem_base = *holder;

    const int num_tiles = sched.num_m * sched.num_n;
    const int nkb = (p.K + BK - 1) / BK;
    const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_bounded_err_cluster(bar, parity, p.err); };

    if (skip) {
        // a wait ran out earlier: compute nothing (the same decision in both CTAs)
    } else if (warp == 0) {
        if (lane == 0) {
            constexpr uint32_t PAIR_TX = 2u * (uint32_t)L::STAGE;
            const uint32_t full0 = cluster_map(smem_addr(full), 0);
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool aborted = false;
            for (int t = cid; t < num_tiles && !aborted; t += ncl) {
                int mb, nb;
                sched.coords(t, mb, nb);
                const int ar = mb * 2 * BM + (int)rank * BM;
                // glu_fwd: gate rows in the even CTA, the up rows of the same
                // features in the odd one
                const int br = KIND == kEpiGlu ? (int)rank * p.N + nb * BH : nb * BN + (int)rank * BH;
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!wait(&empty[stage], phase ^ 1u)) {
                        aborted = true;
                        break;
                    }
                    uint8_t* sa = smem + stage * L::STAGE;
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], PAIR_TX);
                    tma_load_2d_pair(sa, &tmA, kb * BK, ar, full0 + 8u * stage);
                    tma_load_2d_pair(sa + A_BYTES, &tmB, b_mn ? br : kb * BK, b_mn ? kb * BK : br, full0 + 8u * stage);
                    ++issued;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (__builtin_expect(aborted, 0)) pair_stop(s_stop, rank, issued);
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
            int stage = 0, lt = 0;
            uint32_t phase = 0;
            bool aborted = false;
            for (int t = cid; t < num_tiles && !aborted; t += ncl, ++lt) {
                const int b = lt & 1;
                const uint32_t u = (uint32_t)(lt >> 1);
                if (!wait(&aempty[b], (u & 1u) ^ 1u)) {
                    aborted = true;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(b * BN);
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!wait(&full[stage], phase)) {
                        aborted = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_addr(smem + stage * L::STAGE);
                    const uint64_t da = sdesc_kmajor_sw128(sa);
                    const uint64_t db = b_mn ? sdesc_mn_sw128(sa + A_BYTES) : sdesc_kmajor_sw128(sa + A_BYTES);
                    constexpr uint64_t stb = b_mn ? 256 : 2;
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        mma_pair_f8f6f4(d, da + 2 * k, db + stb * k, idesc, (kb | k) != 0 ? 1u : 0u);
                    mma_pair_commit(&empty[stage], 3);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!aborted) mma_pair_commit(&afull[b], 3);
            }
            bool released = !aborted;
            for (int j = 0; j < 2 && released; ++j) {       // both accumulators' last releases have landed
                const int l2 = lt + j;
                released = wait(&aempty[l2 & 1], ((uint32_t)(l2 >> 1) & 1u) ^ 1u);
            }
            if (__builtin_expect(!released, 0)) {
                mma_pair_commit(drain, 1);                  // completes once every issued MMA is done
                wait_drain(drain, 0);
            }
        }
    } else {
        const int quarter = warp & 3;       // the TMEM lane quarter this warp may read
        const int part = (warp - 2) >> 2;   // share of the columns
        constexpr int PARTS = kFfnEpiWarps<KIND> / 4, BOXES = 32 / kFfnEpiWarps<KIND>;
        const float scale = __ldg(p.sA) * __ldg(p.sB);
        const float qm = p.Q ? p.qstate[p.qH] : 1.0f;
        uint32_t amax = 0;
        const uint32_t aempty0 = cluster_map(smem_addr(aempty), 0);
        Stager out{smem + L::STG_OFF + (warp - 2) * BOXES * kStageBytes, lane, 0};
        // columns of a tile in this warp's share; what its epilogue reads
        // beside the sums (the residual, or g and u) is fetched one chunk of
        // 32 columns (16 of g and u) ahead, the first chunk's before the tile's
        // sums are done
        constexpr int TN = KIND == kEpiGlu ? BH : BN;
        const int c_begin = part * (TN / PARTS), c_end = c_begin + TN / PARTS;
        uint4 pre[KIND == kEpiGluBwd ? 4 : 8];
        auto fetch = [&](int row, int col) {
            const int left = row < p.M ? min(p.N - col, 32) : 0;
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
        for (int t = cid; t < num_tiles; t += ncl, ++lt) {
            const int b = lt & 1;
            const uint32_t u = (uint32_t)(lt >> 1);
            int mb, nb;
            sched.coords(t, mb, nb);
            const int row0 = mb * 2 * BM + (int)rank * BM + quarter * 32, row = row0 + lane;
            const uint32_t keep = row < p.M ? 0xFFFFFFFFu : 0u;
            const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(b * BN);
            fetch(row, nb * TN + c_begin);
            // gemm_act: lane l holds the bias of columns 4 l .. 4 l + 3 of the share
            [[maybe_unused]] float4 bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if constexpr (KIND == kEpiAct) {
                const int bc = nb * TN + c_begin + 4 * lane;
                if (p.bias && bc + 4 <= p.N) bias = __ldg(reinterpret_cast<const float4*>(p.bias + bc));
            }
            const bool ok = wait(&afull[b], u & 1u);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = c_begin; c < c_end && row0 < p.M; c += 32) {
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
                        out.bf16(&tmO0, g, col, row0, left);
                        out.bf16(&tmO1, v, col, row0, left);
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
                    if (p.Z) out.bf16(&tmO0, v, col, row0, left);
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
                        if (c + 32 < c_end) fetch(row, col + 32);
                    }
                    if (p.D) {
                        if (p.d_f32) out.f32(&tmO1, v, col, row0, left);
                        else out.bf16(&tmO1, v, col, row0, left);
                    }
                    if (p.Q) {
                        max32(amax, v, left, keep);
                        out.codes(&tmO2, v, qm, p.qfmt, col, row0, left);
                    }
                } else {
                    // two halves of 16 columns, each 16 bytes of the two boxes' rows
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
                        if (cn < c_end) fetch(row, nb * TN + cn);
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
                        if (h == 0) out.reset();        // the previous chunk's boxes have been read
                        uint8_t* q = out.buf + 32 * lane + 16 * h;
                        *reinterpret_cast<uint4*>(q) = qg;
                        *reinterpret_cast<uint4*>(q + kStageBytes) = qu;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        bulk_store_2d(&tmO0, col, row0, out.buf);
                        bulk_store_2d(&tmO1, col, row0, out.buf + kStageBytes);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(aempty0 + 8u * b);
        }
        stage_store_drain(lane);
        if (p.Q) {
            amax = __reduce_max_sync(0xFFFFFFFFu, amax);
            if (lane == 0) atomicMax(reinterpret_cast<unsigned int*>(p.qstate), amax);
        }
    }
    __syncthreads();
    cluster_sync_all();
    if (__builtin_expect(s_stop[0] >= 0, 0)) {                      // (the same in both CTAs)
        const int total = num_tiles > cid ? (num_tiles - cid + ncl - 1) / ncl * nkb : 0;
        if (rank == 0 && threadIdx.x == 0) drain_odd<STAGES>(full, s_stop, total, (uint32_t)L::STAGE);
        cluster_sync_all();
    }
    // nothing is pending into either CTA any more
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// ================================================================== few rows
// Products too small for 256 x 256 tiles on every SM: few rows (serving:
// single tokens and small batches, where the time is the weights' bytes) or
// few tiles (rows_plan chooses).  The roles are swapped -- 128 weight rows are the M of the MMA
// and NT tokens its N -- and the K loop is split over all SMs.  The work is
// the list of (tile, 128-wide K block) pairs in tile order; CTA i of G takes
// the i-th G-th of it, so every SM streams the same number of bytes whatever
// the sizes, and a tile's K range belongs to one or a few neighbouring CTAs.
// A CTA that holds all of a tile's K blocks finishes it from tensor memory;
// otherwise each writes its fp32 partial sums to the workspace and the last
// one to arrive (a counter per tile, which it sets back to 0) adds them in CTA
// order, so the result does not depend on the order of arrival, and runs the
// epilogue.  No CTA waits for another.
// glu: a tile is the gate and the up rows of 64 features, lanes 0-63 and 64-127
// of one accumulator; the pair meets in shared memory (a whole tile) or in the
// partial sums.
// One GB300, us, weights from DRAM: gated block 4096 -> 2 x 14336, one token
// 22.6-23.1 (117 MB; a probe that did nothing but load the same boxes took
// 22.6), 64 tokens 26.4; 14336 -> 4096 with residual, one token 14.4 (59 MB; the
// probe 12.4; from about 48 tokens k_ffn_ksplit is faster).
//   warp 0 producer, warp 1 MMA, warps 2-17 epilogue (TMEM lane = weight row,
//   four warps per lane quarter, each a quarter of the tokens)
// A lane of a finishing warp holds one output column, so a token's stores are
// 32 consecutive columns: coalesced without staging.  Sixteen epilogue warps,
// because the join is a read of a few partial tiles by one CTA: bytes in
// flight (with eight, 14336 -> 4096 for 64 tokens spent 6.5 us in it).
constexpr int kRowsEpiWarps = 16;
constexpr int kRowsThreads = 32 * (2 + kRowsEpiWarps);
constexpr int kRowsMaxCtas = 192;                 // partial slots in the workspace
constexpr int kRowsMaxTiles = 16384;              // counters in the workspace
constexpr size_t kRowsCounterBytes = kRowsMaxTiles * sizeof(uint32_t);

template <int KIND, int NT>
struct RowsLayout {
    static constexpr bool GLU = KIND == kEpiGlu;
    static constexpr int COLS = GLU ? BM / 2 : BM;                       // output columns of a tile
    static constexpr int STAGE = A_BYTES + NT * BK;
    static constexpr int SUMS = GLU ? BM * NT * 4 : 0;                   // a whole tile's sums
    static constexpr int STAGES = (200 * 1024 - SUMS) / STAGE;
    static constexpr int SUM_OFF = STAGES * STAGE;
    static constexpr int BAR_OFF = SUM_OFF + SUMS;
    static constexpr int BYTES = BAR_OFF + 512 + 1024;
    static constexpr uint32_t TMEM_COLS = 2 * NT;
    static constexpr int SHARE = NT / 4;                                 // tokens of an epilogue warp
    static_assert((2 * STAGES + 5) * 8 + 8 <= 512, "barriers");
    static_assert(TMEM_COLS >= 32 && TMEM_COLS <= 512, "tensor memory");
};

struct RowsParams {
    int wtiles, mtiles, nkb, split;      // tile = weight tile x mtiles + token tile
    uint32_t* counters;
    float* part;                         // [CTA][2][NT / 4][128 weight rows][4 tokens]
};

// first work item of CTA i
__device__ __forceinline__ int rows_start(const RowsParams& w, int i)
{
    const int64_t g = gridDim.x;
    const int tiles = w.wtiles * w.mtiles;
    if (!w.split) return (int)((int64_t)i * tiles / g) * w.nkb;
    return (int)((int64_t)i * ((int64_t)tiles * w.nkb) / g);
}
// the CTA that holds work item u (split work)
__device__ __forceinline__ int rows_owner(const RowsParams& w, int u)
{
    return (int)((((int64_t)u + 1) * gridDim.x - 1) / ((int64_t)w.wtiles * w.mtiles * w.nkb));
}

// The residual of CH tokens of column n as stored bits: the loads of a chunk
// are in flight together, and nothing here waits for them, so a caller fetches
// ahead of its sums (converted at once, or fetched where it is added, the
// latency was up to a third of a small product's time).
template <int CH>
__device__ __forceinline__ void rows_residual(const FfnParams& p, int m0, int n, uint32_t (&r)[CH])
{
    if (!p.res || n >= p.N) return;
    if (p.res_f32) {
#pragma unroll
        for (int j = 0; j < CH; ++j)
            if (m0 + j < p.M) r[j] = static_cast<const uint32_t*>(p.res)[(int64_t)(m0 + j) * p.N + n];
    } else {
#pragma unroll
        for (int j = 0; j < CH; ++j)
            if (m0 + j < p.M) r[j] = static_cast<const uint16_t*>(p.res)[(int64_t)(m0 + j) * p.N + n];
    }
}

// The epilogue of CH tokens (m0 .. m0 + CH - 1) of weight row n: a holds the
// raw sums (glu: of the gate, up those of the up row), r the residual.
template <int KIND, int CH>
__device__ __forceinline__ void rows_epilogue(const FfnParams& p, float (&a)[CH], float (&up)[CH],
                                              const uint32_t (&r)[CH], int m0, int n, float scale, float qm,
                                              uint32_t& amax)
{
    const int live = p.M - m0;                   // tokens of the chunk inside the matrix
    if constexpr (KIND == kEpiAct) {
        const float bias = p.bias ? __ldg(p.bias + n) : 0.0f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            a[j] = a[j] * scale;
            if (p.bias) a[j] += bias;
            if (p.Z && j < live) p.Z[(int64_t)(m0 + j) * p.N + n] = __float2bfloat16_rn(a[j]);
        }
        act_dispatch(p.act, [&](auto tag) {
#pragma unroll
            for (int j = 0; j < CH; j += 2)
                if (j < live) {
                    const float2 y = act_f2<decltype(tag)::act>(make_float2(a[j], a[j + 1]));
                    a[j] = y.x;
                    a[j + 1] = y.y;
                }
        });
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            if (p.res) a[j] += __uint_as_float(p.res_f32 ? r[j] : r[j] << 16);
            if (p.D && j < live) {
                const int64_t o = (int64_t)(m0 + j) * p.N + n;
                if (p.d_f32) static_cast<float*>(p.D)[o] = a[j];
                else static_cast<__nv_bfloat16*>(p.D)[o] = __float2bfloat16_rn(a[j]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            a[j] *= scale;
            up[j] *= scale;
            if (p.Z && j < live) {
                __nv_bfloat16* z = p.Z + (int64_t)(m0 + j) * 2 * p.N + n;
                z[0] = __float2bfloat16_rn(a[j]);
                z[p.N] = __float2bfloat16_rn(up[j]);
            }
        }
        act_dispatch(p.act, [&](auto tag) {
#pragma unroll
            for (int j = 0; j < CH; j += 2)
                if (j < live) {
                    const float2 h = __fmul2_rn(make_float2(up[j], up[j + 1]),
                                                act_f2<decltype(tag)::act>(make_float2(a[j], a[j + 1])));
                    a[j] = h.x;
                    a[j + 1] = h.y;
                }
        });
        if (p.D) {
#pragma unroll
            for (int j = 0; j < CH; ++j)
                if (j < live)
                    static_cast<__nv_bfloat16*>(p.D)[(int64_t)(m0 + j) * p.N + n] = __float2bfloat16_rn(a[j]);
        }
    }
    if (p.Q) {
#pragma unroll
        for (int j = 0; j < CH; ++j)
            if (j < live) {
                amax = max(amax, abs_bits(a[j]));
                const float v = __fmul_rn(a[j], qm);
                p.Q[(int64_t)(m0 + j) * p.N + n] =
                    (uint8_t)(p.qfmt == kE4M3 ? cvt_e4m3x2(v, 0.0f) : cvt_e5m2x2(v, 0.0f));
            }
    }
}

template <int KIND, int NT>
__global__ void __launch_bounds__(kRowsThreads, 1)
    k_ffn_rows(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, FfnParams p,
               RowsParams w, uint32_t idesc)
{
    using L = RowsLayout<KIND, NT>;
    constexpr int STAGES = L::STAGES;
    constexpr bool GLU = L::GLU;
    constexpr int BOX = L::COLS;                 // weight rows of a load (glu: gate rows, then up rows)
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t* empty = full + STAGES;
    uint64_t* afull = empty + STAGES;
    uint64_t* aempty = afull + 2;
    uint64_t* drain = aempty + 2;
    uint32_t* holder = reinterpret_cast<uint32_t*>(drain + 1);
    __shared__ int s_last, s_skip;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // what touches no global memory of the kernel before this one runs ahead
    // of the wait on it
    if (threadIdx.x == 0) {
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&afull[b], 1);
            mbar_init(&aempty[b], kRowsEpiWarps);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(holder, L::TMEM_COLS);
        tmem_relinquish();
    }
    const int u0 = rows_start(w, blockIdx.x), u1 = rows_start(w, blockIdx.x + 1);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Weights into L2 while the kernel before still runs: the ring's first
    // stages by the producer, what follows (up to L2Q bytes) by an epilogue
    // thread, which has nothing to do yet.  L2 is where all SMs meet: should
    // that kernel be writing them, the loads below, after the wait, still see
    // what it wrote.
    {
        constexpr int64_t L2Q = (int64_t)64 << 20;
        const int cap = (int)(L2Q / ((int64_t)gridDim.x * A_BYTES));
        const int from = threadIdx.x == 0 ? 0 : threadIdx.x == 64 ? STAGES : 1 << 30;
        const int to = min(u1 - u0, threadIdx.x == 0 ? STAGES : cap);
        if (from < to) {
            int tile = (u0 + from) / w.nkb, kb = u0 + from - tile * w.nkb;
            int wt = tile / w.mtiles, mt = tile - wt * w.mtiles;
            for (int i = from; i < to; ++i) {
                if (mt == 0) {
                    prefetch_l2_2d(&tmW, kb * BK, wt * BOX);
                    if (GLU) prefetch_l2_2d(&tmW, kb * BK, p.N + wt * BOX);
                }
                if (++kb == w.nkb) {
                    kb = 0;
                    if (++mt == w.mtiles) {
                        mt = 0;
                        ++wt;
                    }
                }
            }
        }
    }
    pdl_enter();
    // One decision for the CTA: the epilogue warps meet in named barriers, which
    // wait for all of them without a limit, so a word that is set between two
    // warps' reads must not send one of them past the others.
    if (threadIdx.x == 0) s_skip = *reinterpret_cast<volatile int*>(p.err);
    __syncthreads();
    const uint32_t tmem_base = *holder;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_bounded_err(bar, parity, p.err); };

    if (s_skip) {
        // a wait ran out earlier: compute nothing
    } else if (warp == 0) {
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            int tile = u0 / w.nkb, kb = u0 - tile * w.nkb;
            int wt = tile / w.mtiles, mt = tile - wt * w.mtiles;
            for (int u = u0; u < u1; ++u) {
                if (!wait(&empty[stage], phase ^ 1u)) break;
                uint8_t* sw = smem + stage * L::STAGE;
                mbar_arrive_expect_tx(&full[stage], (uint32_t)L::STAGE);
                tma_load_2d(sw, &tmW, kb * BK, wt * BOX, &full[stage]);
                if (GLU) tma_load_2d(sw + A_BYTES / 2, &tmW, kb * BK, p.N + wt * BOX, &full[stage]);
                tma_load_2d(sw + A_BYTES, &tmX, kb * BK, mt * NT, &full[stage]);
                ++issued;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++kb == w.nkb) {
                    kb = 0;
                    if (++mt == w.mtiles) {
                        mt = 0;
                        ++wt;
                    }
                }
            }
            // every load is under way: the next kernel's CTAs may take over the
            // SMs as this grid's tail leaves them (all of this grid is resident)
            pdl_trigger();
            drain_ring<STAGES>(full, issued);    // no copy is in flight when the CTA exits, whoever gives up a wait
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0, seg = 0;
            uint32_t phase = 0;
            bool aborted = false;
            for (int u = u0; u < u1 && !aborted; ++seg) {
                const int b = seg & 1;
                const int end = min(u1, (u / w.nkb + 1) * w.nkb);
                if (!wait(&aempty[b], ((uint32_t)(seg >> 1) & 1u) ^ 1u)) {
                    aborted = true;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(b * NT);
                for (uint32_t first = 0; u < end; ++u) {
                    if (!wait(&full[stage], phase)) {
                        aborted = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sw = smem_addr(smem + stage * L::STAGE);
                    const uint64_t dw = sdesc_kmajor_sw128(sw), dx = sdesc_kmajor_sw128(sw + A_BYTES);
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        mma_f8f6f4(d, dw + 2 * k, dx + 2 * k, idesc, k != 0 ? 1u : first);
                    first = 1;
                    mma_commit(&empty[stage]);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!aborted) mma_commit(&afull[b]);
            }
            mma_commit(drain);                   // every MMA issued is done before the tensor memory is freed
            wait_drain(drain, 0);
        }
    } else {
        const int quarter = warp & 3;
        const int part = (warp - 2) >> 2;                   // share of the tokens
        const int wr = quarter * 32 + lane;                 // weight row within the tile
        const float scale = __ldg(p.sA) * __ldg(p.sB);
        const float qm = p.Q ? p.qstate[p.qH] : 1.0f;
        constexpr int ETH = 32 * kRowsEpiWarps;
        const int et = threadIdx.x - 64;
        float* sums = reinterpret_cast<float*>(smem + L::SUM_OFF);
        uint32_t amax = 0;
        int seg = 0;
        // glu: tokens 4 i .. 4 i + 3 of feature et % 64 from the sums of `parts`
        // blocks; the block s is at src(s)
        auto glu_quads = [&](int wt, int m_tile, int left, int parts, auto src, auto load) {
            const int f = et & 63, n = wt * 64 + f;
#pragma unroll 1
            for (int i = et >> 6; 4 * i < left && i < NT / 4; i += ETH / 64) {
                constexpr int SEG = 6;
                float g[4] = {}, up[4] = {};
#pragma unroll 1
                for (int s0 = 0; s0 < parts; s0 += SEG) {
                    float4 vg[SEG], vu[SEG];
#pragma unroll
                    for (int s = 0; s < SEG; ++s)
                        if (s0 + s < parts) {
                            const float4* q = reinterpret_cast<const float4*>(src(s0 + s)) + i * BM + f;
                            vg[s] = load(q);
                            vu[s] = load(q + 64);
                        }
#pragma unroll
                    for (int s = 0; s < SEG; ++s)
                        if (s0 + s < parts) {
                            g[0] += vg[s].x;
                            g[1] += vg[s].y;
                            g[2] += vg[s].z;
                            g[3] += vg[s].w;
                            up[0] += vu[s].x;
                            up[1] += vu[s].y;
                            up[2] += vu[s].z;
                            up[3] += vu[s].w;
                        }
                }
                const uint32_t none[4] = {};
                if (n < p.N) rows_epilogue<KIND, 4>(p, g, up, none, m_tile + 4 * i, n, scale, qm, amax);
            }
        };
        for (int u = u0; u < u1; ++seg) {
            const int b = seg & 1;
            const int tile = u / w.nkb, kb0 = u - tile * w.nkb;
            const int wt = tile / w.mtiles, mt = tile - wt * w.mtiles;
            const int end = min(u1, (tile + 1) * w.nkb);
            const bool whole = kb0 == 0 && end == (tile + 1) * w.nkb;
            u = end;
            const int n = wt * BOX + wr;                    // gemm_act: the lane's output column
            const int t0 = part * L::SHARE;                 // this warp's first token in the tile
            const int left = p.M - mt * NT;                 // tokens of the tile inside the matrix
            const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(b * NT);
            uint32_t rs[L::SHARE];                          // the residual, fetched ahead of the sums
            if (!GLU && whole) rows_residual<L::SHARE>(p, mt * NT + t0, n, rs);
            if (!bar_all(1, ETH, wait(&afull[b], (uint32_t)(seg >> 1) & 1u))) break;
            __syncwarp();                      // tcgen05.ld takes a converged warp, which bar_all does not leave
            tc_fence_after();
            // this CTA's block of sums: in shared memory for a whole glu tile
            // (the barrier above says that the last one has been read)
            float* mine = GLU && whole ? sums : w.part + ((int64_t)blockIdx.x * 2 + (kb0 == 0 ? 1 : 0)) * (NT * BM);
#pragma unroll
            for (int c = 0; c < L::SHARE; c += 4) {
                if (t0 + c >= left) break;
                uint32_t r[4];
                tmem_ld_32x32b_x4(taddr + t0 + c, r);
                tmem_ld_wait();
                if (GLU || !whole) {
                    *reinterpret_cast<uint4*>(mine + (t0 + c) * BM + 4 * wr) = make_uint4(r[0], r[1], r[2], r[3]);
                } else if (n < p.N) {
                    float a[4];
                    uint32_t rj[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a[j] = __uint_as_float(r[j]);
                        rj[j] = rs[c + j];
                    }
                    rows_epilogue<KIND, 4>(p, a, a, rj, mt * NT + t0 + c, n, scale, qm, amax);
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&aempty[b]);
            if (whole) {
                if constexpr (GLU) {
                    bar_all(1, ETH, true);
                    glu_quads(wt, mt * NT, left, 1, [&](int) { return sums; }, [](const float4* q) { return *q; });
                    __syncwarp();
                }
                continue;
            }
            // the barrier orders every thread's partial sums before the one
            // release, and the one acquire before every thread's reads
            const int c0 = rows_owner(w, tile * w.nkb), c1 = rows_owner(w, (tile + 1) * w.nkb - 1);
            bar_all(1, ETH, true);
            if (et == 0) {
                const bool last = atomic_add_acq_rel(&w.counters[tile], 1u) == (uint32_t)(c1 - c0);
                if (last) w.counters[tile] = 0;
                s_last = last;
            }
            bar_all(1, ETH, true);
            // the first CTA holds the tile in its last slot, the others in their first
            auto block = [&](int s) { return w.part + ((int64_t)(c0 + s) * 2 + (s == 0 ? 1 : 0)) * (NT * BM); };
            if (s_last) {
                if constexpr (GLU) {
                    glu_quads(wt, mt * NT, left, c1 - c0 + 1, block, [](const float4* q) { return __ldcg(q); });
                } else if (n < p.N) {
                    // quads of tokens, up to eight loads a thread in flight
                    constexpr int SEG = 8;
                    const int parts = c1 - c0 + 1;
                    rows_residual<L::SHARE>(p, mt * NT + t0, n, rs);
#pragma unroll
                    for (int c = 0; c < L::SHARE; c += 4) {
                        if (t0 + c >= left) break;
                        float a[4] = {};
                        uint32_t rj[4];
#pragma unroll 1
                        for (int s0 = 0; s0 < parts; s0 += SEG) {
                            float4 v[SEG];
#pragma unroll
                            for (int s = 0; s < SEG; ++s)
                                if (s0 + s < parts)
                                    v[s] = __ldcg(reinterpret_cast<const float4*>(block(s0 + s) + (t0 + c) * BM + 4 * wr));
#pragma unroll
                            for (int s = 0; s < SEG; ++s)
                                if (s0 + s < parts) {
                                    a[0] += v[s].x;
                                    a[1] += v[s].y;
                                    a[2] += v[s].z;
                                    a[3] += v[s].w;
                                }
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) rj[j] = rs[c + j];
                        rows_epilogue<KIND, 4>(p, a, a, rj, mt * NT + t0 + c, n, scale, qm, amax);
                    }
                }
            }
            __syncwarp();
        }
        if (p.Q) {
            amax = __reduce_max_sync(0xFFFFFFFFu, amax);
            if (lane == 0) atomicMax(reinterpret_cast<unsigned int*>(p.qstate), amax);
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, L::TMEM_COLS);
    }
}

// ------------------------------------------------ few rows, K over a cluster
// Few rows and few weight tiles (at most half as many as SMs): a cluster of
// `split` CTAs takes one tile, each an equal share of its K blocks, and their
// sums meet in the cluster's shared memory: each CTA writes its own to the ring
// that its loads have left, and after a cluster barrier CTA r adds every
// split-th quad of tokens from all of them, in the CTAs' order (the same sums
// on every call), and runs the epilogue on those.  So the join is spread over
// the cluster and no CTA reads partial tiles from L2, which in k_ffn_rows
// costs the last CTA to arrive 2 to 7 us; tiles of up to 256 tokens become
// worth while, which read the weights once.  No counters, no workspace.
// Same roles of the warps as in k_ffn_rows; a CTA has one tile, so one
// accumulator.
// One GB300, us, weights from DRAM, k_ffn_rows or k_ffn_pair -> this: gemm_act
// with residual 4096 -> 4096, 1 token 9.3 -> 7.2, 64 tokens 15.4 -> 8.7, 128
// tokens 15.9 -> 10.1; 14336 -> 4096, 128 tokens 24.8 -> 18.4, 256 tokens 37.5
// -> 23.2; 6000 -> 1040, 64 tokens 15.2 -> 7.2; gated block 4096 -> 2 x 4096, 64
// tokens 13.1 -> 11.8.  (Two quads of a thread at a time: 0.3 to 1.3 faster at
// split 2, 0.2 slower for single tokens; not kept.)
constexpr int kKsplitMax = 8;                     // CTAs of a portable cluster

template <int KIND, int NT>
struct KsplitLayout {
    static constexpr bool GLU = KIND == kEpiGlu;
    static constexpr int COLS = GLU ? BM / 2 : BM;                       // output columns of a tile
    static constexpr int STAGE = A_BYTES + NT * BK;
    static constexpr int STAGES = 200 * 1024 / STAGE;
    static constexpr int BAR_OFF = STAGES * STAGE;
    static constexpr int BYTES = BAR_OFF + 512 + 1024;
    static constexpr uint32_t TMEM_COLS = NT < 32 ? 32 : NT;
    static constexpr int SHARE = NT / 4;                                 // tokens an epilogue warp drains
    static_assert(NT * BM * 4 <= BAR_OFF, "the sums fit the ring");
    static_assert((2 * STAGES + 2) * 8 + 8 <= 512, "barriers");
};

template <int KIND, int NT>
__global__ void __launch_bounds__(kRowsThreads, 1)
    k_ffn_ksplit(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, FfnParams p,
                 int mtiles, int nkb, int split, uint32_t idesc)
{
    using L = KsplitLayout<KIND, NT>;
    constexpr int STAGES = L::STAGES;
    constexpr bool GLU = L::GLU;
    constexpr int BOX = L::COLS;                 // weight rows of a load (glu: gate rows, then up rows)
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t* empty = full + STAGES;
    uint64_t* afull = empty + STAGES;
    uint64_t* drain = afull + 1;
    uint32_t* holder = reinterpret_cast<uint32_t*>(drain + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(afull, 1);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(holder, L::TMEM_COLS);
        tmem_relinquish();
    }
    const int tile = (int)blockIdx.x / split, rank = (int)blockIdx.x - tile * split;
    const int wt = tile / mtiles, mt = tile - wt * mtiles;
    const int kb0 = rank * nkb / split, nk = (rank + 1) * nkb / split - kb0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // weights into L2 ahead of the wait, as in k_ffn_rows
    if (mt == 0) {
        const int cap = (int)(((int64_t)64 << 20) / ((int64_t)gridDim.x * A_BYTES));
        const int from = threadIdx.x == 0 ? 0 : threadIdx.x == 64 ? STAGES : 1 << 30;
        const int to = min(nk, threadIdx.x == 0 ? STAGES : cap);
        for (int i = from; i < to; ++i) {
            prefetch_l2_2d(&tmW, (kb0 + i) * BK, wt * BOX);
            if (GLU) prefetch_l2_2d(&tmW, (kb0 + i) * BK, p.N + wt * BOX);
        }
    }
    pdl_enter();
    const uint32_t tmem_base = *holder;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_bounded_err(bar, parity, p.err); };
    // epilogue: thread et takes output column n of every 4 ETH / BOX-th of the
    // CTA's quads of tokens
    constexpr int ETH = 32 * kRowsEpiWarps;
    const int et = (int)threadIdx.x - 64;
    const int n = wt * BOX + (et & (BOX - 1));
    const int m0 = mt * NT, left = min(NT, p.M - m0), quads = (left + 3) / 4;
    const int q0 = rank + split * (et / BOX), qstep = split * (ETH / BOX);
    uint32_t rs[4];
    bool live = false;

    if (__any_sync(0xFFFFFFFFu, *reinterpret_cast<volatile int*>(p.err))) {
        // a wait ran out earlier: compute nothing
    } else if (warp == 0) {
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int i = 0; i < nk; ++i) {
                if (!wait(&empty[stage], phase ^ 1u)) break;
                uint8_t* sw = smem + stage * L::STAGE;
                mbar_arrive_expect_tx(&full[stage], (uint32_t)L::STAGE);
                tma_load_2d(sw, &tmW, (kb0 + i) * BK, wt * BOX, &full[stage]);
                if (GLU) tma_load_2d(sw + A_BYTES / 2, &tmW, (kb0 + i) * BK, p.N + wt * BOX, &full[stage]);
                tma_load_2d(sw + A_BYTES, &tmX, (kb0 + i) * BK, m0, &full[stage]);
                ++issued;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            pdl_trigger();                       // (the grid is one wave: see ksplit_plan)
            drain_ring<STAGES>(full, issued);    // no copy is in flight when the CTA exits, whoever gives up a wait
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool aborted = false;
            for (int i = 0; i < nk; ++i) {
                if (!wait(&full[stage], phase)) {
                    aborted = true;
                    break;
                }
                tc_fence_after();
                const uint32_t sw = smem_addr(smem + stage * L::STAGE);
                const uint64_t dw = sdesc_kmajor_sw128(sw), dx = sdesc_kmajor_sw128(sw + A_BYTES);
#pragma unroll
                for (int k = 0; k < BK / 32; ++k)
                    mma_f8f6f4(tmem_base, dw + 2 * k, dx + 2 * k, idesc, k != 0 || i != 0 ? 1u : 0u);
                mma_commit(&empty[stage]);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!aborted) mma_commit(afull);
            mma_commit(drain);                   // every MMA issued is done before the tensor memory is freed
            wait_drain(drain, 0);
        }
    } else {
        if (!GLU && q0 < quads) rows_residual<4>(p, m0 + 4 * q0, n, rs);
        live = __all_sync(0xFFFFFFFFu, wait(afull, 0));
        if (live) {
            // the loads and the products are done: the ring holds the sums now,
            // [NT / 4][128 weight rows][4 tokens]
            tc_fence_after();
            const int quarter = warp & 3, t0 = ((warp - 2) >> 2) * L::SHARE, wr = quarter * 32 + lane;
            const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)t0;
            float* sums = reinterpret_cast<float*>(smem);
            __syncwarp();                      // (as in k_ffn_rows)
            if constexpr (L::SHARE >= 16) {
#pragma unroll
                for (int c = 0; c < L::SHARE; c += 16) {
                    if (t0 + c >= left) break;
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(taddr + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<uint4*>(sums + (t0 + c + j) * BM + 4 * wr) =
                            make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
                }
            } else {
#pragma unroll
                for (int c = 0; c < L::SHARE; c += 4) {
                    if (t0 + c >= left) break;
                    uint32_t r[4];
                    tmem_ld_32x32b_x4(taddr + c, r);
                    tmem_ld_wait();
                    *reinterpret_cast<uint4*>(sums + (t0 + c) * BM + 4 * wr) = make_uint4(r[0], r[1], r[2], r[3]);
                }
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    cluster_sync_all();                          // every CTA's sums are in its shared memory
    if (live) {
        const float scale = __ldg(p.sA) * __ldg(p.sB);
        const float qm = p.Q ? p.qstate[p.qH] : 1.0f;
        const uint32_t base = smem_addr(smem) + (uint32_t)(et & (BOX - 1)) * 16u;
        uint32_t amax = 0;
        for (int i = q0; i < quads; i += qstep) {
            float g[4] = {}, up[4] = {};
            uint32_t rn[4];
            if (!GLU && i + qstep < quads) rows_residual<4>(p, m0 + 4 * (i + qstep), n, rn);
            float4 v[8], vu[8];
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (s < split) {
                    const uint32_t q = cluster_map(base + (uint32_t)i * (BM * 16), (uint32_t)s);
                    v[s] = ld_shared_cluster_v4(q);
                    if (GLU) vu[s] = ld_shared_cluster_v4(q + 64 * 16);
                }
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (s < split) {
                    g[0] += v[s].x;
                    g[1] += v[s].y;
                    g[2] += v[s].z;
                    g[3] += v[s].w;
                    if (GLU) {
                        up[0] += vu[s].x;
                        up[1] += vu[s].y;
                        up[2] += vu[s].z;
                        up[3] += vu[s].w;
                    }
                }
            if (n < p.N) rows_epilogue<KIND, 4>(p, g, up, rs, m0 + 4 * i, n, scale, qm, amax);
#pragma unroll
            for (int j = 0; j < 4; ++j) rs[j] = rn[j];
        }
        __syncwarp();
        if (p.Q) {
            amax = __reduce_max_sync(0xFFFFFFFFu, amax);
            if (lane == 0) atomicMax(reinterpret_cast<unsigned int*>(p.qstate), amax);
        }
    }
    __syncwarp();
    cluster_sync_all();                          // ... and has been read
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, L::TMEM_COLS);
    }
}

// ------------------------------------------------------------------ host
// Co-resident clusters of `size` CTAs of a kernel on the current device,
// queried once per slot and device (the entries are atomics: concurrent first
// calls store the same value).  Slots: the pair kernel's kinds, then the sizes
// of k_ffn_ksplit's clusters, whose variants all fill an SM.
constexpr int kSlotKsplit = 3;
static cudaError_t ffn_clusters(const void* kern, int slot, int size, int threads, int smem, int* clusters)
{
    static std::atomic<int> cache[kSlotKsplit + kKsplitMax + 1][64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) {
        const int c = cache[slot][dev].load(std::memory_order_relaxed);
        if (c > 0) {
            *clusters = c - 1;
            return cudaSuccess;
        }
    }
    e = smem_attr_once(kern, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) cache[slot][dev].store(n + 1, std::memory_order_relaxed);
    *clusters = n;
    return cudaSuccess;
}

// Token columns of a few-rows tile.
static int rows_nt(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }

// Which kernel takes a product, and whether the few-rows one splits K, by an
// estimate of each one's time from measurements on the GB300 (bf16 output with
// residual, or gated codes; weights from DRAM; us):
//   few rows  3.7 and 0.022 per token column (5.5 with a split), and the longest
//             CTA's bytes at 80 KB a us (what an SM takes in); a split takes an
//             equal share of the bytes and adds its join, as long as 128 KB +
//             4 KB per token column of that stream
//   pair      8.5, what a tile's epilogue adds (pair_epi: the last tile's is
//             not overlapped), and 0.27 per K block and wave of 256 x 256
//             tiles; glu 6.0 and 0.31
// Measured, few rows / pair: gemm_act N 4096, K 4096, 300 rows 21.3 / 18.3; N
// 2064, K 1040, 300 rows 8.2 / 11.0; glu F 4096, K 4096, 64 rows 13.1 / 15.1, 200
// rows 23.6 / 16.0; F 2064, K 1024, 500 rows 10.1 / 7.7; F 14336, K 4096, 16 rows
// 25.0 / 31.1.
struct RowsPlan {
    bool use = false, split = false;
    int grid = 0;
    double t = 0.0;                      // the faster one's estimate
};
static RowsPlan rows_plan(int kind, int64_t M, int64_t N, int64_t K, int ctas, bool workspace, double pair_epi)
{
    RowsPlan r;
    const int cols = kind == kFfnGlu ? BM / 2 : BM, nt = rows_nt(M);
    const int64_t tiles = (N + cols - 1) / cols * ((M + nt - 1) / nt), nkb = (K + BK - 1) / BK, work = tiles * nkb;
    if (tiles > kRowsMaxTiles || work >= ((int64_t)1 << 31)) return r;
    if (ctas > kRowsMaxCtas) ctas = kRowsMaxCtas;
    const double stage = A_BYTES + nt * BK, rate = 80e3, join = 128e3 + 4e3 * nt;
    const int64_t most = (work + 3) / 4;                   // at least four K blocks a CTA
    const int64_t g_split = ctas < most ? ctas : most, g_whole = ctas < tiles ? ctas : tiles;
    const double whole = (double)((tiles + g_whole - 1) / g_whole * nkb) * stage;
    const double share = (double)((work + g_split - 1) / g_split) * stage + join;
    r.split = workspace && share < whole;
    r.grid = (int)(r.split ? g_split : g_whole);
    const int tile_n = kind == kFfnGlu ? kFfnBH : kFfnBN;
    const int64_t pair_tiles = (M + 2 * BM - 1) / (2 * BM) * ((N + tile_n - 1) / tile_n), pairs = ctas / 2;
    const double blocks = (double)((pair_tiles + pairs - 1) / pairs * nkb);
    const double t_pair = kind == kFfnGlu ? 6.0 + 0.31 * blocks : 8.5 + pair_epi + 0.27 * blocks;
    const double t_rows = r.split ? 5.5 + share / rate : 3.7 + 0.022 * nt + whole / rate;
    r.use = t_rows < t_pair;
    r.t = r.use ? t_rows : t_pair;
    return r;
}

// Token columns and cluster size of k_ffn_ksplit, or split 0 where the others
// are faster (their estimate: t) or its clusters would not run all at once.
// Its own time, measured as above: 3.6, what lasts longest of the loads' latency
// (0.28 a K block), the bytes into an SM (130 KB a us) and out of DRAM (5.1 MB a
// us), and a tile's sums and epilogue, 0.018 a token column and 0.052 for those
// a CTA ends with.  Measured / estimated: 4096 -> 4096, one token and 4 CTAs
// 7.2 / 7.4, 2 CTAs 7.9 / 8.8; 64 tokens and 4 CTAs 8.7 / 9.0; 128 tokens, 4
// CTAs 10.1 / 10.7; 256 tokens in tiles of 256, 4 CTAs 13.4 / 14.9; 14336 -> 4096,
// 500 tokens in tiles of 256, 2 CTAs 34.5 / 35.0.
struct KsplitPlan {
    int split = 0, nt = 0;
};
static KsplitPlan ksplit_plan(int kind, int64_t M, int64_t N, int64_t K, int sms, double t)
{
    KsplitPlan r;
    const int cols = kind == kFfnGlu ? BM / 2 : BM;
    const int64_t wtiles = (N + cols - 1) / cols, nkb = (K + BK - 1) / BK;
    if (2 * wtiles > sms || nkb < 2) return r;
    const double dram = (double)K * ((kind == kFfnGlu ? 2 : 1) * N + M) / 5.1e6;
    for (int nt = M <= 16 ? 16 : M <= 32 ? 32 : 64; nt <= 256; nt *= 2) {
        const int64_t tiles = wtiles * ((M + nt - 1) / nt);
        for (int split = 2; split <= kKsplitMax && split <= nkb && tiles * split <= sms; ++split) {
            const double blocks = (double)((nkb + split - 1) / split);
            const double lat = 0.28 * blocks, in = blocks * (A_BYTES + nt * BK) / 130e3;
            const double loads = lat > in ? lat : in;
            const double own = 3.6 + (loads > dram ? loads : dram) + nt * (0.018 + 0.052 / split);
            if (own >= t) continue;
            int clusters = 0;
            if (ffn_clusters(reinterpret_cast<const void*>(k_ffn_ksplit<kEpiAct, 64>), kSlotKsplit + split, split,
                             kRowsThreads, KsplitLayout<kEpiAct, 64>::BYTES, &clusters) != cudaSuccess ||
                tiles > clusters)
                continue;
            t = own;
            r.split = split;
            r.nt = nt;
        }
        if (nt >= M) break;
    }
    return r;
}

// bytes of the split's counters and partial sums, 0 where it never applies
size_t ffn_workspace(int kind, int64_t M, int64_t N, int64_t K)
{
    const RowsPlan r = rows_plan(kind, M, N, K, 152, true, 8.0);      // the costliest epilogue
    if (!r.use || !r.split) return 0;
    return kRowsCounterBytes + (size_t)kRowsMaxCtas * 2 * rows_nt(M) * BM * sizeof(float);
}

template <int KIND, int NT>
static cudaError_t launch_rows(const FfnArgs& a, const FfnParams& p, const RowsPlan& plan, cudaStream_t st,
                               const char** why)
{
    using L = RowsLayout<KIND, NT>;
    CUtensorMap tw, tx;
    if (!make_tmap(&tw, a.B, a.K, L::GLU ? 2 * a.N : a.N, L::COLS) || !make_tmap(&tx, a.A, a.K, a.M, NT)) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    RowsParams w = {};
    w.wtiles = (int)((a.N + L::COLS - 1) / L::COLS);
    w.mtiles = (int)((a.M + NT - 1) / NT);
    w.nkb = (int)((a.K + BK - 1) / BK);
    w.split = plan.split;
    if (plan.split) {
        w.counters = static_cast<uint32_t*>(a.workspace);
        w.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kRowsCounterBytes);
    }
    auto kern = k_ffn_rows<KIND, NT>;
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(kern), L::BYTES);
    if (e != cudaSuccess) return e;
    launch_k(kern, (unsigned)plan.grid, kRowsThreads, L::BYTES, st, tw, tx, p, w,
             make_idesc(a.b_format, a.a_format, NT));
    return cudaGetLastError();
}

template <int KIND>
static cudaError_t launch_rows_nt(const FfnArgs& a, const FfnParams& p, const RowsPlan& plan, cudaStream_t st,
                                  const char** why)
{
    switch (rows_nt(a.M)) {
    case 16: return launch_rows<KIND, 16>(a, p, plan, st, why);
    case 32: return launch_rows<KIND, 32>(a, p, plan, st, why);
    default: return launch_rows<KIND, 64>(a, p, plan, st, why);
    }
}

template <int KIND, int NT>
static cudaError_t launch_ksplit(const FfnArgs& a, const FfnParams& p, int split, cudaStream_t st, const char** why)
{
    using L = KsplitLayout<KIND, NT>;
    CUtensorMap tw, tx;
    if (!make_tmap(&tw, a.B, a.K, L::GLU ? 2 * a.N : a.N, L::COLS) || !make_tmap(&tx, a.A, a.K, a.M, NT)) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    const int wtiles = (int)((a.N + L::COLS - 1) / L::COLS), mtiles = (int)((a.M + NT - 1) / NT);
    auto kern = k_ffn_ksplit<KIND, NT>;
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(kern), L::BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(wtiles * mtiles * split));
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = L::BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, tw, tx, p, mtiles, (int)((a.K + BK - 1) / BK), split,
                              make_idesc(a.b_format, a.a_format, NT));
}

template <int KIND>
static cudaError_t launch_ksplit_nt(const FfnArgs& a, const FfnParams& p, const KsplitPlan& ks, cudaStream_t st,
                                    const char** why)
{
    switch (ks.nt) {
    case 16: return launch_ksplit<KIND, 16>(a, p, ks.split, st, why);
    case 32: return launch_ksplit<KIND, 32>(a, p, ks.split, st, why);
    case 64: return launch_ksplit<KIND, 64>(a, p, ks.split, st, why);
    case 128: return launch_ksplit<KIND, 128>(a, p, ks.split, st, why);
    default: return launch_ksplit<KIND, 256>(a, p, ks.split, st, why);
    }
}

cudaError_t launch_ffn(const FfnArgs& a, cudaStream_t st, int sms, const char** why)
{
    *why = nullptr;
    if (a.M == 0 || a.N == 0) return cudaSuccess;
    FfnParams p = {};
    p.M = (int)a.M;
    p.N = (int)a.N;
    p.K = (int)a.K;
    p.sA = a.a_scale;
    p.sB = a.b_scale;
    p.act = a.act;
    p.bias = a.bias;
    p.res = a.residual;
    p.res_f32 = a.res_dtype == kF32;
    p.D = a.D;
    p.d_f32 = a.d_dtype == kF32;
    p.Z = static_cast<__nv_bfloat16*>(a.Z);
    p.Q = a.q_out;
    p.qfmt = a.q_format;
    p.qstate = a.q_state;
    p.qH = a.q_history_len;
    p.gu = static_cast<const __nv_bfloat16*>(a.gu);
    cudaError_t e = device_error_word(&p.err);
    if (e != cudaSuccess) return e;
    const bool glu = a.kind == kFfnGlu, bwd = a.kind == kFfnGluBwd;
    if (!bwd) {
        const double epi = glu ? 0.0
                               : (a.act != kActNone ? 1.5 : 0.0) + (a.residual ? (p.res_f32 ? 3.5 : 1.0) : 0.0) +
                                     (a.D && p.d_f32 ? 1.5 : 0.0) + (a.Z ? 1.0 : 0.0);
        const RowsPlan plan = rows_plan(a.kind, a.M, a.N, a.K, sms, a.workspace != nullptr, epi);
        const KsplitPlan ks = ksplit_plan(a.kind, a.M, a.N, a.K, sms, plan.t);
        if (ks.split)
            return glu ? launch_ksplit_nt<kEpiGlu>(a, p, ks, st, why) : launch_ksplit_nt<kEpiAct>(a, p, ks, st, why);
        if (plan.use)
            return glu ? launch_rows_nt<kEpiGlu>(a, p, plan, st, why) : launch_rows_nt<kEpiAct>(a, p, plan, st, why);
    }
    CUtensorMap ta, tb;
    const bool ok_b = bwd ? make_tmap(&tb, a.B, a.N, a.K, BK) : make_tmap(&tb, a.B, a.K, glu ? 2 * a.N : a.N, kFfnBH);
    if (!make_tmap(&ta, a.A, a.K, a.M, BM) || !ok_b) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    using Kern = decltype(&k_ffn_pair<kEpiAct>);
    static const Kern kerns[3] = {k_ffn_pair<kEpiAct>, k_ffn_pair<kEpiGlu>, k_ffn_pair<kEpiGluBwd>};
    Kern kern = kerns[a.kind];
    int clusters = 0;
    static_assert((int)FfnSmem<kEpiAct>::BYTES == (int)FfnSmem<kEpiGluBwd>::BYTES, "one size for both");
    const int threads = bwd ? kFfnThreads<kEpiGluBwd> : kFfnThreads<kEpiAct>;
    const int smem = glu ? FfnSmem<kEpiGlu>::BYTES : FfnSmem<kEpiAct>::BYTES;
    e = ffn_clusters(reinterpret_cast<const void*>(kern), a.kind, 2, threads, smem, &clusters);
    if (e != cudaSuccess) {
        *why = "cluster occupancy query failed";
        return e;
    }
    if (clusters < 1) {
        *why = "no CTA pair of this kernel fits on the device";
        return cudaErrorNotSupported;
    }
    const int tile_n = glu ? kFfnBH : kFfnBN;
    TileSched sched{(int)((a.M + 2 * BM - 1) / (2 * BM)), (int)((a.N + tile_n - 1) / tile_n), 8};
    const int64_t tiles = (int64_t)sched.num_m * sched.num_n;
    const int grid = 2 * (int)(tiles < clusters ? tiles : clusters);
    sched.group = raster_group(a.K, 2 * BM, kFfnBN, grid / 2);
    uint32_t idesc = make_idesc(a.a_format, a.b_format, kFfnBN);
    idesc = (idesc & ~(0x1Fu << 24)) | ((uint32_t)((2 * BM) >> 4) << 24);   // M = 256 over the pair
    if (bwd) idesc |= 1u << 16;                                              // B MN-major
    // outputs stored in bulk; a map that the epilogue does not use is a copy of A's
    CUtensorMap o[3] = {ta, ta, ta};
    bool ok = true;
    if (bwd) {
        ok = make_tmap_codes(&o[0], a.q_out, a.M, a.N, 2 * a.N) && make_tmap_codes(&o[1], a.q_out + a.N, a.M, a.N, 2 * a.N);
    } else if (glu) {
        __nv_bfloat16* z = p.Z;
        if (z) ok = make_tmap_out(&o[0], z, a.M, a.N, true, 2 * a.N) && make_tmap_out(&o[1], z + a.N, a.M, a.N, true, 2 * a.N);
    } else {
        if (p.Z) ok = make_tmap_out(&o[0], p.Z, a.M, a.N, true);
        if (p.D) ok = ok && make_tmap_out(&o[1], p.D, a.M, a.N, a.d_dtype == kBF16);
        if (p.Q) ok = ok && make_tmap_codes(&o[2], p.Q, a.M, a.N);
    }
    if (!ok) {
        *why = "cuTensorMapEncodeTiled failed (output)";
        return cudaErrorInvalidValue;
    }
    launch_k(kern, grid, threads, (size_t)smem, st, ta, tb, p, idesc, sched, o[0], o[1], o[2]);
    return cudaGetLastError();
}

}  // namespace fp8sq
