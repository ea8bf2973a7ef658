// experts.cu -- the experts' products of a mixture-of-experts sublayer, on rows
// sorted by expert (experts_rows.cu): the gated product, the plain product with
// the weights stored either way (down projection, data gradient), the gated
// backward pass and the weight gradients, on the CTA pairs of ffn_pair.cuh.
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ffn_pair.cuh"
#include "ffn_rows.cuh"
#include "gemm_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fp8sq {

// Co-resident pairs of a kernel on the current device, asked once per device.
template <int KIND, int GROUP>
static cudaError_t expert_pairs(int smem, int* pairs)
{
    static std::atomic<int> cache[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) {
        const int c = cache[dev].load(std::memory_order_relaxed);
        if (c > 0) {
            *pairs = c - 1;
            return cudaSuccess;
        }
    }
    const void* kern = reinterpret_cast<const void*>(k_ffn_pair<KIND, GROUP>);
    e = smem_attr_once(kern, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kFfnThreads<KIND>);
    cfg.dynamicSmemBytes = (size_t)smem;
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
    if (dev >= 0 && dev < 64) cache[dev].store(n + 1, std::memory_order_relaxed);
    *pairs = n;
    return cudaSuccess;
}

template <int KIND, int GROUP, bool PAIR = true>
static cudaError_t launch_pair(const ExpertGemmArgs& a, const FfnParams& p, cudaStream_t st, int sms, const char** why)
{
    constexpr bool GLU = KIND == kEpiGlu;
    const int64_t R = a.layout.rows;
    CUtensorMap ta, tb;
    bool ok;
    if constexpr (GROUP == kWgrad) ok = make_tmap(&ta, a.A, a.M, R, BK) && make_tmap(&tb, a.B, a.N, R, BK);
    else if constexpr (GROUP == kRowsMn) ok = make_tmap(&ta, a.A, a.K, R, BM) && make_tmap(&tb, a.B, a.N, a.E * a.K, BK);
    else ok = make_tmap(&ta, a.A, a.K, R, BM) && make_tmap(&tb, a.B, a.K, a.E * (GLU ? 2 * a.N : a.N), kFfnBH);
    if (!ok) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    constexpr int smem = FfnSmem<KIND, GROUP, PAIR>::BYTES;
    auto kern = k_ffn_pair<KIND, GROUP, PAIR>;
    int groups = sms;                        // CTA pairs, or CTAs
    if constexpr (PAIR) {
        const cudaError_t e = expert_pairs<KIND, GROUP>(smem, &groups);
        if (e != cudaSuccess) {
            *why = "cluster occupancy query failed";
            return e;
        }
        if (groups < 1) {
            *why = "no CTA pair of this kernel fits on the device";
            return cudaErrorNotSupported;
        }
    } else {
        const cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(kern), smem);
        if (e != cudaSuccess) return e;
    }
    // the tiles in use are known on the device alone: at most this many
    constexpr int tile_n = GLU ? kFfnBH : kFfnBN;
    TileSched sched{(int)((a.M + 2 * BM - 1) / (2 * BM)), (int)((a.N + tile_n - 1) / tile_n), 8};
    const int64_t most = (GROUP == kWgrad ? (int64_t)a.E * sched.num_m : (PAIR ? 1 : 2) * a.layout.max_tiles) * sched.num_n;
    uint32_t idesc = make_idesc(a.a_format, a.b_format, kFfnBN);
    if (PAIR) idesc = (idesc & ~(0x1Fu << 24)) | ((uint32_t)((2 * BM) >> 4) << 24);   // M = 256 over the pair
    if (GROUP == kWgrad) idesc |= 1u << 15;                                  // A MN-major
    if (GROUP >= kRowsMn) idesc |= 1u << 16;                                 // B MN-major
    // outputs stored in bulk; a map that the epilogue does not use is a copy of A's
    CUtensorMap o[3] = {ta, ta, ta};
    if constexpr (KIND == kEpiGluBwd) {
        ok = make_tmap_codes64(&o[0], a.q_out, R, a.N, 2 * a.N) && make_tmap_codes64(&o[1], a.q_out + a.N, R, a.N, 2 * a.N);
    } else if constexpr (GLU) {
        __nv_bfloat16* z = p.Z;
        if (z) ok = make_tmap_out(&o[0], z, R, a.N, true, 2 * a.N) && make_tmap_out(&o[1], z + a.N, R, a.N, true, 2 * a.N);
    } else {
        ok = make_tmap_lines(&o[1], p.D, GROUP == kWgrad ? a.E * a.M : R, a.N, a.d_dtype == kBF16);
    }
    if (GROUP != kWgrad) ok = ok && make_tmap(&o[2], a.A, a.K, R, 32);       // A in boxes of 32 rows (pair_rows)
    if (!ok) {
        *why = "cuTensorMapEncodeTiled failed (output)";
        return cudaErrorInvalidValue;
    }
    launch_k(kern, (unsigned)((PAIR ? 2 : 1) * (most < groups ? most : groups)), kFfnThreads<KIND>, (size_t)smem, st, ta, tb, p, idesc,
             sched, o[0], o[1], o[2]);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ which kernel
// The routing is known on the device alone, so the rules go by its sizes: n = T k
// assignments make a = n / active rows for each of active = min(E, n) experts, and
// `tiles` of 256 weight rows (glu: 128 of the gate and of the up projection).
// Figures: one GB300, us, weights from DRAM.
//
// One CTA a tile of 128 rows up to a = 20, 40 where an SM gets three tiles at most, 64
// where it gets one; from there on CTA pairs and 256 rows, whose operands cost less traffic.
// One CTA / pairs: 896 tiles (4096 -> 2 x 1792), a = 16 145 / 153, 32 161 / 155; 288 (2304 ->
// 2 x 1040), a = 40 32.7 / 33.9, 48 36.5 / 34.3; 152 (2048 -> 2 x 9728), a = 24 17.1 / 19.7, 64 17.4 / 20.2;
// 160 (2048 -> 2 x 10240), a = 40 23.6 / 23.6.
struct ExpertSizes {
    int64_t n, active, tiles;
    ExpertSizes(int64_t T, int k, int E, int64_t N)
        : n(T * k), active(E < n ? E : n), tiles(active * ((N + kFfnBN - 1) / kFfnBN))
    {
    }
};
static bool expert_single_ctas(const ExpertSizes& s, int sms)
{
    return s.n <= (s.tiles <= sms ? 64 : s.tiles <= 3 * sms ? 40 : 20) * s.active;
}
// k_ffn_rows where those tiles do not go round, or where single tokens stream long
// gated weights in one or two of them an SM: it shares the bytes out evenly, but reads
// a weight tile again (from L2) for every 32 rows of an expert, and stores column by
// column.  N: weight rows of an expert (glu: 2F).  Few rows / one CTA a tile: one
// token, 56 tiles (4096 -> 2 x 3584) 17.6 / 20.0, 112 (-> 2 x 1792) 27.0 / 26.0, plain 128 (1792 ->
// 4096) 18.1 / 15.3; 208 tiles (-> 2 x 3328), K = 1536 20.0 / 19.2, 2048 23.5 / 23.8, 2816 29.9 / 31.2,
// 4096 40.0 / 42.5; 448 (4096 -> 2 x 3584), a = 2 67.5 / 68.1, 8 77.2 / 76.3.
constexpr int kExpertNT = 32;
static bool expert_few_rows(int64_t T, int k, int E, int64_t N, int64_t K, bool glu, int sms)
{
    const ExpertLayout l = expert_layout(T, k, E);
    const int64_t wtiles = (N + BM - 1) / BM, nkb = (K + BK - 1) / BK, most = l.rows / kExpertNT * wtiles;
    if (most > kRowsMaxTiles || most * nkb >= ((int64_t)1 << 31) || sms > kRowsMaxCtas) return false;
    const ExpertSizes s(T, k, E, N);
    if (!expert_single_ctas(s, sms) || nkb < 8) return false;
    return s.tiles <= 64 || (glu && nkb > 20 && s.n <= 3 * s.active && s.tiles > sms && s.tiles <= 2 * sms);
}

size_t expert_workspace(int64_t T, int k, int E, int64_t N, int64_t K)
{
    // by the wider rule, the gated product's, on a GB300's 152 SMs (where the device has another number and
    // k_ffn_rows comes without a workspace, it takes whole tiles)
    if (!expert_few_rows(T, k, E, N, K, true, 152)) return 0;
    return kRowsCounterBytes + (size_t)kRowsMaxCtas * 2 * kExpertNT * BM * sizeof(float);
}

template <int KIND>
static cudaError_t launch_few_rows(const ExpertGemmArgs& a, FfnParams p, cudaStream_t st, int sms, const char** why)
{
    using L = RowsLayout<KIND, kExpertNT>;
    const int64_t wrows = L::GLU ? 2 * a.N : a.N;
    CUtensorMap tw, tx;
    if (!make_tmap(&tw, a.B, a.K, a.E * wrows, L::COLS) || !make_tmap(&tx, a.A, a.K, a.layout.rows, kExpertNT)) {
        *why = "cuTensorMapEncodeTiled failed";
        return cudaErrorInvalidValue;
    }
    p.blocks = reinterpret_cast<const int4*>(a.plan + a.layout.blocks_at);
    p.max_blocks = (int)(a.layout.rows / kExpertPad);
    p.wrows = (int)wrows;
    RowsParams w = {};
    w.wtiles = (int)((a.N + L::COLS - 1) / L::COLS);
    w.nkb = (int)((a.K + BK - 1) / BK);
    w.split = a.workspace != nullptr;
    if (a.workspace) {
        w.counters = static_cast<uint32_t*>(a.workspace);
        w.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kRowsCounterBytes);
    }
    auto kern = k_ffn_rows<KIND, kExpertNT, true>;
    const cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(kern), L::BYTES);
    if (e != cudaSuccess) return e;
    launch_k(kern, (unsigned)sms, kRowsThreads, L::BYTES, st, tw, tx, p, w, make_idesc(a.b_format, a.a_format, kExpertNT));
    return cudaGetLastError();
}

cudaError_t launch_expert_gemm(const ExpertGemmArgs& a, cudaStream_t st, int sms, const char** why)
{
    *why = nullptr;
    if (a.N == 0 || (a.kind == kExpertWgrad ? a.M == 0 : a.layout.rows == 0)) return cudaSuccess;
    FfnParams p = {};
    p.M = (int)(a.kind == kExpertWgrad ? a.M : a.layout.rows);
    p.N = (int)a.N;
    p.K = (int)a.K;
    p.sA = a.a_scale;
    p.sB = a.b_scale;
    p.act = a.act;
    p.D = a.D;
    p.d_f32 = a.d_dtype == kF32;
    p.Z = static_cast<__nv_bfloat16*>(a.Z);
    p.Q = a.q_out;
    p.qfmt = a.q_format;
    p.qstate = a.q_state;
    p.qH = a.q_history_len;
    p.gu = static_cast<const __nv_bfloat16*>(a.gu);
    p.E = a.E;
    p.offsets = a.plan;
    p.ntiles = a.plan + 2 * a.E + 1;
    p.tiles = reinterpret_cast<const int4*>(a.plan + a.layout.tiles_at);
    p.max_tiles = (int)a.layout.max_tiles;
    p.rows = (int)a.layout.rows;
    const cudaError_t e = device_error_word(&p.err);
    if (e != cudaSuccess) return e;
    static_assert(kExpertNT == kExpertPad, "a token tile is one of the plan's blocks");
    if ((a.kind == kExpertGlu || (a.kind == kExpertGemm && !a.b_mn)) &&
        expert_few_rows(a.T, a.k, a.E, a.kind == kExpertGlu ? 2 * a.N : a.N, a.K, a.kind == kExpertGlu, sms))
        return a.kind == kExpertGlu ? launch_few_rows<kEpiGlu>(a, p, st, sms, why) : launch_few_rows<kEpiAct>(a, p, st, sms, why);
    const bool single = expert_single_ctas(ExpertSizes(a.T, a.k, a.E, a.kind == kExpertGlu ? 2 * a.N : a.N), sms);
    switch (a.kind) {
    case kExpertGlu:
        return single ? launch_pair<kEpiGlu, kRows, false>(a, p, st, sms, why) : launch_pair<kEpiGlu, kRows>(a, p, st, sms, why);
    case kExpertGluBwd: return launch_pair<kEpiGluBwd, kRowsMn>(a, p, st, sms, why);
    case kExpertWgrad: return launch_pair<kEpiAct, kWgrad>(a, p, st, sms, why);
    default:
        if (a.b_mn) return launch_pair<kEpiAct, kRowsMn>(a, p, st, sms, why);
        return single ? launch_pair<kEpiAct, kRows, false>(a, p, st, sms, why) : launch_pair<kEpiAct, kRows>(a, p, st, sms, why);
    }
}

}  // namespace fp8sq
