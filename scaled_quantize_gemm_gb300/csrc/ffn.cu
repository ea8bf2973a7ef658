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
// All three run on CTA pairs (tcgen05 .cta_group::2, M = 256, N = 256): the
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
    const void* res;         // [M][N] or null
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

constexpr int kFfnStages = 6;
constexpr int kFfnEpiWarps = 8;                  // two per TMEM lane quarter
constexpr int kFfnThreads = 32 * (2 + kFfnEpiWarps);
constexpr int kFfnBN = 256, kFfnBH = 128;
using FfnSmem = Smem<kFfnBH, kFfnStages, 2>;

// ------------------------------------------------------------------ epilogue pieces
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store32_bf16(__nv_bfloat16* d, int left, const float (&v)[32])
{
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (8 * c + 8 <= left)
            *reinterpret_cast<uint4*>(d + 8 * c) =
                make_uint4(pack_bf16(v[8 * c], v[8 * c + 1]), pack_bf16(v[8 * c + 2], v[8 * c + 3]),
                           pack_bf16(v[8 * c + 4], v[8 * c + 5]), pack_bf16(v[8 * c + 6], v[8 * c + 7]));
}
__device__ __forceinline__ void store32_f32(float* d, int left, const float (&v)[32])
{
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (4 * c + 4 <= left)
            *reinterpret_cast<float4*>(d + 4 * c) = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
__device__ __forceinline__ void store32_codes(uint8_t* q, int left, const float (&v)[32], float m, int fmt)
{
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = __fmul_rn(v[4 * j], m), b = __fmul_rn(v[4 * j + 1], m);
        const float c = __fmul_rn(v[4 * j + 2], m), d = __fmul_rn(v[4 * j + 3], m);
        w[j] = fmt == kE4M3 ? (cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16))
                            : (cvt_e5m2x2(a, b) | (cvt_e5m2x2(c, d) << 16));
    }
    if (16 <= left) *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
    if (32 <= left) *reinterpret_cast<uint4*>(q + 16) = make_uint4(w[4], w[5], w[6], w[7]);
}
// the largest |v| as fp32 bits, a NaN above everything
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ void max32(uint32_t& amax, const float (&v)[32], int left)
{
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (j < left) amax = max(amax, abs_bits(v[j]));
}
__device__ __forceinline__ void load32_bf16(const __nv_bfloat16* s, int left, float (&v)[32])
{
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (8 * c + 8 <= left) w = __ldg(reinterpret_cast<const uint4*>(s + 8 * c));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[8 * c + 2 * j] = __uint_as_float(u[j] << 16);
            v[8 * c + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
    }
}

// ------------------------------------------------------------------ kernel
template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFfnThreads, 1)
    k_ffn_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, FfnParams p,
               uint32_t idesc, TileSched sched)
{
    pdl_enter();
    constexpr int BN = kFfnBN, BH = kFfnBH, STAGES = kFfnStages;
    constexpr bool b_mn = KIND == kEpiGluBwd;          // Wd [K][F]: MN-major
    using L = FfnSmem;
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
    const uint32_t rank = cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        s_skip = rank == 0 ? *reinterpret_cast<volatile int*>(p.err) : 0;
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&afull[b], 1);
            mbar_init(&aempty[b], 2 * kFfnEpiWarps);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    __syncthreads();
    cluster_sync_all();
    int skip = s_skip;
    if (rank != 0) skip = (int)ld_shared_cluster_u32(cluster_map(smem_addr(&s_skip), 0));
    cluster_sync_all();
    if (skip) return;
    if (warp == 1) {
        tmem_alloc_pair(holder, TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *holder;

    const int num_tiles = sched.num_m * sched.num_n;
    const int nkb = (p.K + BK - 1) / BK;
    const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_bounded_err_cluster(bar, parity, p.err); };

    if (warp == 0) {
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
            if (!aborted) {
                for (int i = 0; i < STAGES; ++i) {     // every stage's last release has landed
                    if (!wait(&empty[stage], phase ^ 1u)) break;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            } else if (rank == 0) {
                // the pair's copies still in flight complete on the leader's barriers
                int n = issued < STAGES ? issued : STAGES;
                int s = stage;
                uint32_t ph = phase;
                for (int i = 0; i < n; ++i) {
                    if (--s < 0) {
                        s = STAGES - 1;
                        ph ^= 1u;
                    }
                    wait_drain(&full[s], ph);
                }
            }
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
            if (!aborted) {
                for (int j = 0; j < 2; ++j) {           // both accumulators' last releases have landed
                    const int l2 = lt + j;
                    if (!wait(&aempty[l2 & 1], ((uint32_t)(l2 >> 1) & 1u) ^ 1u)) break;
                }
            } else {
                mma_pair_commit(drain, 1);              // completes once every issued MMA is done
                wait_drain(drain, 0);
            }
        }
    } else {
        const int quarter = warp & 3;       // the TMEM lane quarter this warp may read
        const int part = (warp - 2) >> 2;   // column half
        const float scale = __ldg(p.sA) * __ldg(p.sB);
        const float qm = p.Q ? p.qstate[p.qH] : 1.0f;
        uint32_t amax = 0;
        const uint32_t aempty0 = cluster_map(smem_addr(aempty), 0);
        int lt = 0;
        for (int t = cid; t < num_tiles; t += ncl, ++lt) {
            const int b = lt & 1;
            const uint32_t u = (uint32_t)(lt >> 1);
            const bool ok = wait(&afull[b], u & 1u);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
            int mb, nb;
            sched.coords(t, mb, nb);
            const int row = mb * 2 * BM + (int)rank * BM + quarter * 32 + lane;
            const bool live = row < p.M;
            const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(b * BN);
            if constexpr (KIND == kEpiGlu) {
#pragma unroll 1
                for (int c = part * (BH / 2); c < (part + 1) * (BH / 2); c += 32) {
                    uint32_t rg[32], ru[32];
                    tmem_ld_32x32b_x32(taddr + (uint32_t)c, rg);
                    tmem_ld_32x32b_x32(taddr + (uint32_t)(BH + c), ru);
                    tmem_ld_wait();
                    const int col = nb * BH + c, left = p.N - col;
                    float g[32], v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        g[j] = __uint_as_float(rg[j]) * scale;
                        v[j] = __uint_as_float(ru[j]) * scale;
                    }
                    if (live && left > 0) {
                        if (p.Z) {
                            __nv_bfloat16* z = p.Z + (int64_t)row * 2 * p.N + col;
                            store32_bf16(z, left, g);
                            store32_bf16(z + p.N, left, v);
                        }
                        act_dispatch(p.act, [&](auto tag) {
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                const float2 h = __fmul2_rn(make_float2(v[j], v[j + 1]),
                                                            act_f2<decltype(tag)::act>(make_float2(g[j], g[j + 1])));
                                v[j] = h.x;
                                v[j + 1] = h.y;
                            }
                        });
                        if (p.D) store32_bf16(static_cast<__nv_bfloat16*>(p.D) + (int64_t)row * p.N + col, left, v);
                        if (p.Q) {
                            max32(amax, v, left);
                            store32_codes(p.Q + (int64_t)row * p.N + col, left, v, qm, p.qfmt);
                        }
                    }
                    __syncwarp();
                }
            } else {
#pragma unroll 1
                for (int c = part * BH; c < (part + 1) * BH; c += 32) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(taddr + (uint32_t)c, r);
                    tmem_ld_wait();
                    const int col = nb * BN + c, left = p.N - col;
                    if (live && left > 0) {
                        float v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]) * scale;
                        if constexpr (KIND == kEpiAct) {
                            if (p.bias) {
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    if (j < left) v[j] += __ldg(p.bias + col + j);
                            }
                            if (p.Z) store32_bf16(p.Z + (int64_t)row * p.N + col, left, v);
                            act_dispatch(p.act, [&](auto tag) {
#pragma unroll
                                for (int j = 0; j < 32; j += 2) {
                                    const float2 y = act_f2<decltype(tag)::act>(make_float2(v[j], v[j + 1]));
                                    v[j] = y.x;
                                    v[j + 1] = y.y;
                                }
                            });
                            if (p.res) {
                                if (p.res_f32) {
                                    const float* s = static_cast<const float*>(p.res) + (int64_t)row * p.N + col;
#pragma unroll
                                    for (int j = 0; j < 32; j += 4)
                                        if (j + 4 <= left) {
                                            const float4 w = __ldg(reinterpret_cast<const float4*>(s + j));
                                            v[j] += w.x;
                                            v[j + 1] += w.y;
                                            v[j + 2] += w.z;
                                            v[j + 3] += w.w;
                                        }
                                } else {
                                    float s[32];
                                    load32_bf16(static_cast<const __nv_bfloat16*>(p.res) + (int64_t)row * p.N + col, left, s);
#pragma unroll
                                    for (int j = 0; j < 32; ++j) v[j] += s[j];
                                }
                            }
                            if (p.D) {
                                if (p.d_f32) store32_f32(static_cast<float*>(p.D) + (int64_t)row * p.N + col, left, v);
                                else store32_bf16(static_cast<__nv_bfloat16*>(p.D) + (int64_t)row * p.N + col, left, v);
                            }
                            if (p.Q) {
                                max32(amax, v, left);
                                store32_codes(p.Q + (int64_t)row * p.N + col, left, v, qm, p.qfmt);
                            }
                        } else {
                            float g[32], w[32];
                            const __nv_bfloat16* s = p.gu + (int64_t)row * 2 * p.N + col;
                            load32_bf16(s, left, g);
                            load32_bf16(s + p.N, left, w);
                            act_dispatch(p.act, [&](auto tag) {
#pragma unroll
                                for (int j = 0; j < 32; j += 2) {
                                    float2 f, d;
                                    act_fd2<decltype(tag)::act>(make_float2(g[j], g[j + 1]), f, d);
                                    const float2 dh = make_float2(v[j], v[j + 1]);
                                    const float2 dg = __fmul2_rn(__fmul2_rn(dh, make_float2(w[j], w[j + 1])), d);
                                    const float2 du = __fmul2_rn(dh, f);
                                    g[j] = dg.x;
                                    g[j + 1] = dg.y;
                                    w[j] = du.x;
                                    w[j + 1] = du.y;
                                }
                            });
                            max32(amax, g, left);
                            max32(amax, w, left);
                            uint8_t* q = p.Q + (int64_t)row * 2 * p.N + col;
                            store32_codes(q, left, g, qm, p.qfmt);
                            store32_codes(q + p.N, left, w, qm, p.qfmt);
                        }
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(aempty0 + 8u * b);
        }
        if (p.Q) {
            amax = __reduce_max_sync(0xFFFFFFFFu, amax);
            if (lane == 0) atomicMax(reinterpret_cast<unsigned int*>(p.qstate), amax);
        }
    }
    __syncthreads();
    cluster_sync_all();                        // nothing is pending into either CTA any more
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// ================================================================== few rows
// Up to 64 rows (serving: single tokens and small batches): the time is the
// weights' bytes, so the roles are swapped -- 128 weight rows are the M of
// the MMA and the tokens, padded to NT, its N -- and the K loop is split over
// all SMs.  The work is the list of (weight tile, 128-wide K block) pairs in
// tile order; CTA i of G takes the i-th G-th of it, so every SM streams the
// same number of bytes whatever the sizes, and a tile's K range belongs to
// one or a few neighbouring CTAs.  A CTA that holds all of a tile's K blocks
// finishes it from tensor memory; otherwise each writes its fp32 partial sums
// to the workspace and the last one to arrive (a counter per tile, which it
// sets back to 0) adds them in CTA order, so the result does not depend on
// the order of arrival, and runs the epilogue.  No CTA waits for another.
// glu: a stage holds the gate and the up rows of 128 features, accumulated in
// two column ranges of the same lanes, so a thread holds both.
//   warp 0 producer, warp 1 MMA, warps 2-5 epilogue (TMEM lane = weight row)
constexpr int kRowsThreads = 192;
constexpr int kRowsMaxM = 64;
constexpr int kRowsMaxCtas = 192;                 // partial slots in the workspace
constexpr int kRowsMaxTiles = 16384;              // counters in the workspace
constexpr size_t kRowsCounterBytes = kRowsMaxTiles * sizeof(uint32_t);

template <int KIND, int NT>
struct RowsLayout {
    static constexpr int NW = KIND == kEpiGlu ? 2 : 1;                  // weight tiles per stage
    static constexpr int STAGE = NW * A_BYTES + NT * BK;
    static constexpr int STAGES = (200 * 1024) / STAGE;
    static constexpr int BAR_OFF = STAGES * STAGE;
    static constexpr int BYTES = BAR_OFF + 512 + 1024;
    static constexpr int ACC = NW * NT;                                  // columns of one accumulator
    static constexpr uint32_t TMEM_COLS = 2 * ACC < 32 ? 32 : 2 * ACC;
    static_assert((2 * STAGES + 5) * 8 + 8 <= 512, "barriers");
};

struct RowsParams {
    int tiles, nkb, split;
    uint32_t* counters;
    float* part;              // [CTA][2][NW * NT][128]
};

// first work item of CTA i
__device__ __forceinline__ int rows_start(const RowsParams& w, int i)
{
    const int64_t g = gridDim.x;
    if (!w.split) return (int)((int64_t)i * w.tiles / g) * w.nkb;
    return (int)((int64_t)i * ((int64_t)w.tiles * w.nkb) / g);
}
// the CTA that holds work item u (split work)
__device__ __forceinline__ int rows_owner(const RowsParams& w, int u)
{
    return (int)((((int64_t)u + 1) * gridDim.x - 1) / ((int64_t)w.tiles * w.nkb));
}

template <int KIND, int NT>
__global__ void __launch_bounds__(kRowsThreads, 1)
    k_ffn_rows(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, FfnParams p,
               RowsParams w, uint32_t idesc)
{
    pdl_enter();
    using L = RowsLayout<KIND, NT>;
    constexpr int STAGES = L::STAGES, NW = L::NW, ACC = L::ACC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t* empty = full + STAGES;
    uint64_t* afull = empty + STAGES;
    uint64_t* aempty = afull + 2;
    uint64_t* drain = aempty + 2;
    uint32_t* holder = reinterpret_cast<uint32_t*>(drain + 1);
    __shared__ int s_skip;
    __shared__ int s_last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        s_skip = *reinterpret_cast<volatile int*>(p.err);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&afull[b], 1);
            mbar_init(&aempty[b], 4);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        prefetch_tmap(&tmW);
        prefetch_tmap(&tmX);
    }
    __syncthreads();
    if (s_skip) return;
    if (warp == 1) {
        tmem_alloc(holder, L::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *holder;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_bounded_err(bar, parity, p.err); };
    const int u0 = rows_start(w, blockIdx.x), u1 = rows_start(w, blockIdx.x + 1);

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool aborted = false;
            int tile = u0 / w.nkb, kb = u0 - tile * w.nkb;
            for (int u = u0; u < u1; ++u) {
                if (!wait(&empty[stage], phase ^ 1u)) {
                    aborted = true;
                    break;
                }
                uint8_t* sw = smem + stage * L::STAGE;
                mbar_arrive_expect_tx(&full[stage], (uint32_t)L::STAGE);
                tma_load_2d(sw, &tmW, kb * BK, tile * BM, &full[stage]);
                if (NW == 2) tma_load_2d(sw + A_BYTES, &tmW, kb * BK, p.N + tile * BM, &full[stage]);
                tma_load_2d(sw + NW * A_BYTES, &tmX, kb * BK, 0, &full[stage]);
                ++issued;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++kb == w.nkb) {
                    kb = 0;
                    ++tile;
                }
            }
            if (aborted) {
                // wait for the copies still in flight before the CTA can exit
                int n = issued < STAGES ? issued : STAGES;
                int s = stage;
                uint32_t ph = phase;
                for (int i = 0; i < n; ++i) {
                    if (--s < 0) {
                        s = STAGES - 1;
                        ph ^= 1u;
                    }
                    wait_drain(&full[s], ph);
                }
            }
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
                const uint32_t d = tmem_base + (uint32_t)(b * ACC);
                for (uint32_t first = 0; u < end; ++u) {
                    if (!wait(&full[stage], phase)) {
                        aborted = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sw = smem_addr(smem + stage * L::STAGE);
                    const uint64_t dx = sdesc_kmajor_sw128(sw + NW * A_BYTES);
#pragma unroll
                    for (int h = 0; h < NW; ++h) {
                        const uint64_t dw = sdesc_kmajor_sw128(sw + h * A_BYTES);
#pragma unroll
                        for (int k = 0; k < BK / 32; ++k)
                            mma_f8f6f4(d + h * NT, dw + 2 * k, dx + 2 * k, idesc, k != 0 ? 1u : first);
                    }
                    first = 1;
                    mma_commit(&empty[stage]);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!aborted) mma_commit(&afull[b]);
            }
            if (aborted) {
                mma_commit(drain);
                wait_drain(drain, 0);
            }
        }
    } else {
        const int quarter = warp & 3;
        const int wr = quarter * 32 + lane;                 // weight row within the tile
        const float scale = __ldg(p.sA) * __ldg(p.sB);
        const float qm = p.Q ? p.qstate[p.qH] : 1.0f;
        uint32_t amax = 0;
        int seg = 0;
        for (int u = u0; u < u1; ++seg) {
            const int b = seg & 1;
            const int tile = u / w.nkb, kb0 = u - tile * w.nkb;
            const int end = min(u1, (tile + 1) * w.nkb);
            const bool whole = kb0 == 0 && end == (tile + 1) * w.nkb;
            u = end;
            if (!bar_all(1, 128, wait(&afull[b], (uint32_t)(seg >> 1) & 1u))) break;
            tc_fence_after();
            float acc[ACC];
            {
                uint32_t r[ACC];
                const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(b * ACC);
#pragma unroll
                for (int c = 0; c < ACC; c += 16) tmem_ld_32x32b_x16(taddr + c, r + c);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < ACC; ++c) acc[c] = __uint_as_float(r[c]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&aempty[b]);
            if (!whole) {
                float* mine = w.part + ((int64_t)blockIdx.x * 2 + (kb0 == 0 ? 1 : 0)) * (ACC * 128) + wr;
#pragma unroll
                for (int c = 0; c < ACC; ++c)
                    if (c % NT < p.M) __stcg(mine + c * 128, acc[c]);
                const int c0 = rows_owner(w, tile * w.nkb), c1 = rows_owner(w, (tile + 1) * w.nkb - 1);
                __threadfence();
                bar_all(1, 128, true);
                if (threadIdx.x == 64) {
                    const uint32_t n = (uint32_t)(c1 - c0);
                    const bool last = atomicAdd(&w.counters[tile], 1u) == n;
                    if (last) w.counters[tile] = 0;
                    s_last = last;
                }
                bar_all(1, 128, true);
                if (!s_last) continue;
                __threadfence();
                for (int c = c0; c <= c1; ++c) {
                    const float* src = w.part + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * (ACC * 128) + wr;
#pragma unroll
                    for (int j = 0; j < ACC; ++j) {
                        if (j % NT < p.M) {
                            const float v = __ldcg(src + j * 128);
                            acc[j] = c == c0 ? v : acc[j] + v;
                        }
                    }
                }
            }
            const int n = tile * BM + wr;
            if (n < p.N) {
                if constexpr (KIND == kEpiAct) {
                    const float bias = p.bias ? __ldg(p.bias + n) : 0.0f;
#pragma unroll
                    for (int m = 0; m < NT; ++m)
                        if (m < p.M) {
                            acc[m] = acc[m] * scale;
                            if (p.bias) acc[m] += bias;
                            if (p.Z) p.Z[(int64_t)m * p.N + n] = __float2bfloat16_rn(acc[m]);
                        }
                    act_dispatch(p.act, [&](auto tag) {
#pragma unroll
                        for (int m = 0; m < NT; m += 2)
                            if (m < p.M) {
                                const float2 y = act_f2<decltype(tag)::act>(make_float2(acc[m], m + 1 < p.M ? acc[m + 1] : 0.0f));
                                acc[m] = y.x;
                                acc[m + 1] = y.y;
                            }
                    });
#pragma unroll
                    for (int m = 0; m < NT; ++m)
                        if (m < p.M) {
                            const int64_t o = (int64_t)m * p.N + n;
                            if (p.res) acc[m] += p.res_f32 ? __ldg(static_cast<const float*>(p.res) + o)
                                                           : __bfloat162float(static_cast<const __nv_bfloat16*>(p.res)[o]);
                            if (p.D) {
                                if (p.d_f32) static_cast<float*>(p.D)[o] = acc[m];
                                else static_cast<__nv_bfloat16*>(p.D)[o] = __float2bfloat16_rn(acc[m]);
                            }
                        }
                } else {
#pragma unroll
                    for (int m = 0; m < NT; ++m)
                        if (m < p.M) {
                            acc[m] *= scale;
                            acc[NT + m] *= scale;
                            if (p.Z) {
                                __nv_bfloat16* z = p.Z + (int64_t)m * 2 * p.N + n;
                                z[0] = __float2bfloat16_rn(acc[m]);
                                z[p.N] = __float2bfloat16_rn(acc[NT + m]);
                            }
                        }
                    act_dispatch(p.act, [&](auto tag) {
#pragma unroll
                        for (int m = 0; m < NT; m += 2)
                            if (m < p.M) {
                                const bool two = m + 1 < p.M;
                                const float2 h = __fmul2_rn(
                                    make_float2(acc[NT + m], two ? acc[NT + m + 1] : 0.0f),
                                    act_f2<decltype(tag)::act>(make_float2(acc[m], two ? acc[m + 1] : 0.0f)));
                                acc[m] = h.x;
                                acc[m + 1] = h.y;
                            }
                    });
                    if (p.D) {
#pragma unroll
                        for (int m = 0; m < NT; ++m)
                            if (m < p.M)
                                static_cast<__nv_bfloat16*>(p.D)[(int64_t)m * p.N + n] = __float2bfloat16_rn(acc[m]);
                    }
                }
                if (p.Q) {
#pragma unroll
                    for (int m = 0; m < NT; ++m)
                        if (m < p.M) {
                            amax = max(amax, abs_bits(acc[m]));
                            const float v = __fmul_rn(acc[m], qm);
                            p.Q[(int64_t)m * p.N + n] =
                                (uint8_t)(p.qfmt == kE4M3 ? cvt_e4m3x2(v, 0.0f) : cvt_e5m2x2(v, 0.0f));
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

// ------------------------------------------------------------------ host
// Co-resident CTA pairs of a kernel on the current device, queried once per
// kernel and device (the entries are atomics: concurrent first calls store
// the same value).
static cudaError_t ffn_clusters(const void* kern, int kind, int* clusters)
{
    static std::atomic<int> cache[3][64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) {
        const int c = cache[kind][dev].load(std::memory_order_relaxed);
        if (c > 0) {
            *clusters = c;
            return cudaSuccess;
        }
    }
    e = smem_attr_once(kern, FfnSmem::BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(kFfnThreads, 1, 1);
    cfg.dynamicSmemBytes = FfnSmem::BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && n > 0) cache[kind][dev].store(n, std::memory_order_relaxed);
    *clusters = n;
    return cudaSuccess;
}

static int rows_nt(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }

// the split of few rows over K applies: bytes of its counters and partial sums
size_t ffn_workspace(int kind, int64_t M, int64_t N, int64_t K)
{
    (void)K;
    if (M > kRowsMaxM || (N + BM - 1) / BM > kRowsMaxTiles) return 0;
    const int acc = (kind == kFfnGlu ? 2 : 1) * rows_nt(M);
    return kRowsCounterBytes + (size_t)kRowsMaxCtas * 2 * acc * 128 * sizeof(float);
}

template <int KIND, int NT>
static cudaError_t launch_rows(const FfnArgs& a, const FfnParams& p, cudaStream_t st, int sms, const char** why)
{
    using L = RowsLayout<KIND, NT>;
    CUtensorMap tw, tx;
    if (!make_tmap(&tw, a.B, a.K, L::NW * a.N, BM) || !make_tmap(&tx, a.A, a.K, a.M, NT)) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    RowsParams w = {};
    w.tiles = (int)((a.N + BM - 1) / BM);
    w.nkb = (int)((a.K + BK - 1) / BK);
    const int64_t work = (int64_t)w.tiles * w.nkb;
    w.split = a.workspace != nullptr;
    int64_t grid = sms < kRowsMaxCtas ? sms : kRowsMaxCtas;
    if (w.split) {
        w.counters = static_cast<uint32_t*>(a.workspace);
        w.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kRowsCounterBytes);
        // at least four K blocks a CTA: below that the join costs more than the split saves
        const int64_t most = (work + 3) / 4;
        grid = grid < most ? grid : most;
    } else {
        grid = grid < w.tiles ? grid : w.tiles;
    }
    auto kern = k_ffn_rows<KIND, NT>;
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(kern), L::BYTES);
    if (e != cudaSuccess) return e;
    launch_k(kern, (unsigned)grid, kRowsThreads, L::BYTES, st, tw, tx, p, w, make_idesc(a.b_format, a.a_format, NT));
    return cudaGetLastError();
}

template <int KIND>
static cudaError_t launch_rows_nt(const FfnArgs& a, const FfnParams& p, cudaStream_t st, int sms, const char** why)
{
    switch (rows_nt(a.M)) {
    case 16: return launch_rows<KIND, 16>(a, p, st, sms, why);
    case 32: return launch_rows<KIND, 32>(a, p, st, sms, why);
    default: return launch_rows<KIND, 64>(a, p, st, sms, why);
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
    if (!bwd && ffn_workspace(a.kind, a.M, a.N, a.K) != 0 && (int64_t)((a.N + BM - 1) / BM) * ((a.K + BK - 1) / BK) < ((int64_t)1 << 31))
        return glu ? launch_rows_nt<kEpiGlu>(a, p, st, sms, why) : launch_rows_nt<kEpiAct>(a, p, st, sms, why);
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
    e = ffn_clusters(reinterpret_cast<const void*>(kern), a.kind, &clusters);
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
    launch_k(kern, grid, kFfnThreads, FfnSmem::BYTES, st, ta, tb, p, idesc, sched);
    return cudaGetLastError();
}

}  // namespace fp8sq
