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
#include "ffn_pair.cuh"
#include "ffn_rows.cuh"
#include "gemm_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fp8sq {

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
    const int threads = bwd ? kFfnThreads<kEpiGluBwd> : kFfnThreads<kEpiAct>;
    const int smem = glu ? FfnSmem<kEpiGlu>::BYTES : bwd ? FfnSmem<kEpiGluBwd>::BYTES : FfnSmem<kEpiAct>::BYTES;
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
        ok = make_tmap_codes64(&o[0], a.q_out, a.M, a.N, 2 * a.N) && make_tmap_codes64(&o[1], a.q_out + a.N, a.M, a.N, 2 * a.N);
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
