// ffn_rows.cuh -- products of few rows, K split over all SMs: the feed-forward
// sublayer's (ffn.cu) and the experts' (experts.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act.cuh"
#include "ffn_pair.cuh"
#include "gemm_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fp8sq {

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
    int wtiles, mtiles, nkb, split;      // tile = weight tile x mtiles + token tile (experts: see RowsTile)
    uint32_t* counters;
    float* part;                         // [CTA][2][NT / 4][128 weight rows][4 tokens]
};

// Experts: the sorted rows in blocks of NT = 32, each of one expert; a tile is
// one of an expert's weight tiles for one of its blocks, in the order of
// (expert, weight tile, block), so an expert's blocks take a weight tile one
// after another.  blocks[b] = {expert, its first block, its blocks, rows that are
// not padding in block b}.
struct RowsTile {
    int wt, mt;                          // weight tile; token tile (of NT rows from row mt NT)
    int wrow;                            // first of the expert's weight rows
    int expert, live;                    // rows of the token tile that are not padding
};
template <bool EXPERTS, typename LOAD = LoadPlan>
__device__ __forceinline__ RowsTile rows_tile(const FfnParams& p, const RowsParams& w, int tile, int nt)
{
    RowsTile x;
    if constexpr (EXPERTS) {
        const LOAD load;
        const int4 d = load(p.blocks + tile / w.wtiles);
        const int i = tile - d.y * w.wtiles, size = max(d.z, 1);
        x.wt = min(max(i / size, 0), w.wtiles - 1);          // (whatever the plan holds, all of it inside the buffers)
        x.mt = min(max(d.y + i - x.wt * size, 0), p.max_blocks - 1);
        x.expert = min(max(d.x, 0), p.E - 1);
        x.wrow = x.expert * p.wrows;
        x.live = x.mt == tile / w.wtiles ? d.w : load(p.blocks + x.mt).w;
    } else {
        x.wt = tile / w.mtiles;
        x.mt = tile - x.wt * w.mtiles;
        x.expert = x.wrow = 0;
        x.live = p.M - x.mt * nt;
    }
    return x;
}

// experts: whole tiles or equal shares, and of how many CTAs, as rows_plan decides
// it, for `rows` sorted rows in use; the CTA's work items
template <int NT, int STAGE>
__device__ __forceinline__ int rows_schedule(const FfnParams& p, RowsParams& w, int rows, int& u0, int& u1);

// first work item of CTA i of g
__device__ __forceinline__ int rows_start(const RowsParams& w, int i, int64_t g)
{
    const int tiles = w.wtiles * w.mtiles;
    if (!w.split) return (int)((int64_t)i * tiles / g) * w.nkb;
    return (int)((int64_t)i * ((int64_t)tiles * w.nkb) / g);
}
// the CTA that holds work item u (split work)
__device__ __forceinline__ int rows_owner(const RowsParams& w, int u, int64_t g)
{
    return (int)((((int64_t)u + 1) * g - 1) / ((int64_t)w.wtiles * w.mtiles * w.nkb));
}

template <int NT, int STAGE>
__device__ __forceinline__ int rows_schedule(const FfnParams& p, RowsParams& w, int rows, int& u0, int& u1)
{
    w.mtiles = min(max(rows, 0) / NT, p.max_blocks);
    const int tiles = w.wtiles * w.mtiles, work = tiles * w.nkb;
    const int g_split = min((int)gridDim.x, (work + 3) / 4), g_whole = min((int)gridDim.x, tiles);
    constexpr int JOIN = (128000 + 4000 * NT) / STAGE;                   // in K blocks
    if (w.split && work > 0)
        w.split = (work + g_split - 1) / g_split + JOIN < (tiles + g_whole - 1) / g_whole * w.nkb;
    const int ctas = w.split ? g_split : g_whole;
    u0 = u1 = 0;
    if ((int)blockIdx.x < ctas) {
        u0 = rows_start(w, blockIdx.x, ctas);
        u1 = rows_start(w, blockIdx.x + 1, ctas);
    }
    return ctas;
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
    const int live = p.M - m0;                   // tokens of the chunk inside the matrix (experts: all)
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

// EXPERTS: see RowsTile; the work is known on the device alone, after the plan.
template <int KIND, int NT, bool EXPERTS = false>
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
    int u0 = 0, u1 = 0, ctas = gridDim.x;
    if constexpr (!EXPERTS) {
        u0 = rows_start(w, blockIdx.x, ctas);
        u1 = rows_start(w, blockIdx.x + 1, ctas);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Weights into L2 while the kernel before still runs: the ring's first
    // stages by the producer, what follows (up to L2Q bytes) by an epilogue
    // thread, which has nothing to do yet.  L2 is where all SMs meet: should
    // that kernel be writing them, the loads below, after the wait, still see
    // what it wrote.
    if constexpr (EXPERTS) {
        // The plan as it stands in L2 now, as a hint: as a rule a kernel or more
        // lies between the plan's and this one, and what is fetched for a plan that
        // is not there yet is the wrong weights, no more (every tile is within the
        // weights).  Gated products of short K, behind a dispatch, are ready as soon as it
        // is, and working the hint out delays them.  A sublayer of one token, us,
        // with / without: 2 of 16 experts, 4096 -> 3584 40.0 / 41.2; 2 of 8, 4096 -> 2048 33.6 /
        // 35.2; gated K of 2304, 2048, 1024: 28.1 / 27.4, 27.8 / 27.5, 21.6 / 21.0.
        constexpr int64_t L2Q = (int64_t)64 << 20;
        const int cap = (int)(L2Q / ((int64_t)gridDim.x * A_BYTES));
        if ((!GLU || w.nkb > 20) && (threadIdx.x == 0 || threadIdx.x == 64)) {
            RowsParams hint = w;
            int h0, h1;
            rows_schedule<NT, L::STAGE>(p, hint, __ldcg(p.offsets + p.E), h0, h1);
            int i = threadIdx.x == 0 ? 0 : STAGES;
            const int to = min(h1 - h0, threadIdx.x == 0 ? STAGES : cap);
            while (i < to) {
                const int tile = (h0 + i) / hint.nkb, kb0 = h0 + i - tile * hint.nkb, n = min(to - i, hint.nkb - kb0);
                const RowsTile x = rows_tile<true, LoadPlanL2>(p, hint, tile, NT);
                const int row = x.wrow + x.wt * BOX;
                for (int k = kb0; k < kb0 + n; ++k) {
                    prefetch_l2_2d(&tmW, k * BK, row);
                    if (GLU) prefetch_l2_2d(&tmW, k * BK, p.N + row);
                }
                i += n;
            }
        }
    } else {
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
    if constexpr (EXPERTS) ctas = rows_schedule<NT, L::STAGE>(p, w, LoadPlan()(p.offsets + p.E), u0, u1);
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
            int wt = 0, mt = 0, wrow = 0;
            auto place = [&]() {
                const RowsTile x = rows_tile<EXPERTS>(p, w, tile, NT);
                wt = x.wt;
                mt = x.mt;
                wrow = x.wrow;
            };
            if (u0 < u1) place();
            for (int u = u0; u < u1; ++u) {
                if (!wait(&empty[stage], phase ^ 1u)) break;
                uint8_t* sw = smem + stage * L::STAGE;
                mbar_arrive_expect_tx(&full[stage], (uint32_t)L::STAGE);
                tma_load_2d(sw, &tmW, kb * BK, wrow + wt * BOX, &full[stage]);
                if (GLU) tma_load_2d(sw + A_BYTES / 2, &tmW, kb * BK, wrow + p.N + wt * BOX, &full[stage]);
                tma_load_2d(sw + A_BYTES, &tmX, kb * BK, mt * NT, &full[stage]);
                ++issued;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++kb == w.nkb) {
                    kb = 0;
                    if constexpr (EXPERTS) {
                        ++tile;
                        if (u + 1 < u1) place();
                    } else if (++mt == w.mtiles) {
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
        float scale = __ldg(p.sA) * __ldg(p.sB);
        const float qm = p.Q ? p.qstate[p.qH] : 1.0f;
        constexpr int ETH = 32 * kRowsEpiWarps;
        const int et = threadIdx.x - 64;
        float* sums = reinterpret_cast<float*>(smem + L::SUM_OFF);
        uint32_t amax = 0;
        int seg = 0;
        // glu: tokens 4 i .. 4 i + 3 of feature et % 64 from the sums of `parts`
        // blocks; the block s is at src(s)
        auto glu_quads = [&](int wt, int m_tile, int left, int real, int parts, auto src, auto load) {
            const int f = et & 63, n = wt * 64 + f;
#pragma unroll 1
            for (int i = et >> 6; 4 * i < left && i < NT / 4; i += ETH / 64) {
                constexpr int SEG = 6;
                float g[4] = {}, up[4] = {};
#pragma unroll 1
                for (int s0 = 0; s0 < parts && (!EXPERTS || 4 * i < real); s0 += SEG) {
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
            const RowsTile x = rows_tile<EXPERTS>(p, w, tile, NT);
            const int wt = x.wt, mt = x.mt;
            if constexpr (EXPERTS) scale = __ldg(p.sA) * __ldg(p.sB + x.expert);
            const int end = min(u1, (tile + 1) * w.nkb);
            const bool whole = kb0 == 0 && end == (tile + 1) * w.nkb;
            u = end;
            const int n = wt * BOX + wr;                    // gemm_act: the lane's output column
            const int t0 = part * L::SHARE;                 // this warp's first token in the tile
            // tokens of the tile inside the matrix; experts: all of them, but the
            // sums of those that fill up the block are zero and never written
            const int left = EXPERTS ? NT : p.M - mt * NT, real = EXPERTS ? x.live : left;
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
                if (t0 + c >= (EXPERTS && !(!GLU && whole) ? real : left)) break;
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
                    glu_quads(wt, mt * NT, left, real, 1, [&](int) { return sums; }, [](const float4* q) { return *q; });
                    __syncwarp();
                }
                continue;
            }
            // the barrier orders every thread's partial sums before the one
            // release, and the one acquire before every thread's reads
            const int c0 = rows_owner(w, tile * w.nkb, ctas), c1 = rows_owner(w, (tile + 1) * w.nkb - 1, ctas);
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
                    glu_quads(wt, mt * NT, left, real, c1 - c0 + 1, block, [](const float4* q) { return __ldcg(q); });
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
                        for (int s0 = 0; s0 < parts && (!EXPERTS || t0 + c < real); s0 += SEG) {
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

}  // namespace fp8sq
