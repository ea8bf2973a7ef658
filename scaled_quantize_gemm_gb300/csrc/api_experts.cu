// api_experts.cu -- the extern "C" entry points of RMSNorm and of a sublayer of
// experts (include/fp8sq.h, section 5d).  Every argument is checked on the host
// before anything is enqueued.
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/fp8sq.h"
#include "api_checks.h"
#include "internal.h"

namespace {

using fp8sq::ExpertLayout;

const int64_t kMaxRow = (int64_t)1 << 23;     // columns of the rows that are moved (a grid dimension counts their chunks)

bool valid_routing(int64_t T, int k, int E)
{
    return T >= 0 && T < kMaxDim && k >= 1 && k <= fp8sq::kExpertSlots && E >= 1 && E <= fp8sq::kExpertMax;
}
// the routing's sizes and its plan (every row and plan index fits 31 bits)
int check_routing(const char* fn, const int32_t* plan, int64_t T, int k, int E, ExpertLayout* l)
{
    if (T < 0 || k < 1 || E < 1) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad number of tokens, slots or experts", fn);
    if (!valid_routing(T, k, E))
        return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: at most %d slots a token and %d experts", fn, fp8sq::kExpertSlots, fp8sq::kExpertMax);
    *l = fp8sq::expert_layout(T, k, E);
    if (l->ints >= kMaxDim || l->rows >= kMaxDim - 256) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: routing too large", fn);
    if (!plan) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null plan", fn);
    if (!aligned(plan, 16)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: plan must be 16-byte aligned", fn);
    return FP8SQ_OK;
}
fp8sq::ExpertRowsArgs rows_args(const int32_t* plan, int64_t T, int k, int E, const ExpertLayout& l, int64_t K)
{
    fp8sq::ExpertRowsArgs a;
    a.T = T;
    a.K = K;
    a.k = k;
    a.E = E;
    a.layout = l;
    a.plan = plan;
    return a;
}
// operands and sizes of a product over sorted rows
int check_product(const char* fn, const uint8_t* A, int a_format, const float* a_scale, const uint8_t* B, int b_format,
                  const float* b_scales, int act, int64_t T, int E, int64_t N, int64_t K, bool b_mn, int64_t b_rows)
{
    int r = check_operands(fn, A, a_format, a_scale, B, b_format, b_scales, act, T, N, K, 16);
    if (r) return r;
    if (b_mn && K % 32) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: weights read MN-major need K %% 32 == 0", fn);
    if ((int64_t)E * b_rows >= kMaxDim) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: too many rows of weights", fn);
    return FP8SQ_OK;
}
int check_workspace(const char* fn, const void* ws, size_t bytes, size_t need)
{
    if (!ws) return FP8SQ_OK;
    if (!aligned(ws, 256)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: workspace must be 256-byte aligned", fn);
    if (bytes < need) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: workspace of %zu bytes, needs %zu", fn, bytes, need);
    return FP8SQ_OK;
}
int launch_product(const fp8sq::ExpertGemmArgs& a, void* stream, int sms, const char* what)
{
    const char* why = nullptr;
    const cudaError_t e = fp8sq::launch_expert_gemm(a, static_cast<cudaStream_t>(stream), sms, &why);
    return cuda_status(e, what, why);
}

}  // namespace

extern "C" {

FP8SQ_API int fp8_rmsnorm_fwd(const void* x, const void* residual, int dtype, const float* gamma, float eps, int64_t M,
                              int64_t K, void* sum_out, void* y, float* rstd_out, uint8_t* q_out, int q_format,
                              int q_gran, float* q_state, int q_history_len, void* scales_out, void* stream)
{
    const char* fn = "fp8_rmsnorm_fwd";
    if (M < 0 || K < 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: negative size", fn);
    if (M >= kMaxDim || K >= kMaxDim) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: dimension too large", fn);
    if (!valid_dtype(dtype)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (K == 0 && M != 0) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: a row needs at least one element", fn);
    if ((!x || !gamma) && M != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null x or gamma", fn);
    if (!y && !q_out && M != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: neither y nor codes asked for", fn);
    if ((residual != nullptr) != (sum_out != nullptr) && M != 0)
        return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: residual and sum_out come together", fn);
    if (!(eps >= 0.0f)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: eps must not be negative", fn);
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(sum_out, 16) || !aligned(gamma, 16))
        return api_fail(FP8SQ_ERR_MISALIGNED, "%s: x, residual, sum, y, gamma must be 16-byte aligned", fn);
    if (!aligned(rstd_out, 4)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: rstd must be 4-byte aligned", fn);
    const uint64_t n = (uint64_t)M * (uint64_t)K;
    uint64_t scale_bytes = 0;
    int sms, r;
    if (q_out && q_gran != FP8SQ_TENSOR) {
        const bool f32 = q_gran == FP8SQ_TILE_1x128, rows = q_gran == FP8SQ_MX32;
        const bool tiled = q_gran == FP8SQ_TILE_1x128_POW2 || q_gran == FP8SQ_MX32_TILED || q_gran == FP8SQ_MX32_FLOOR_TILED;
        if (!f32 && !rows && !tiled) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: no such scaling unit of a row", fn);
        if (!valid_format(q_format)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad output format", fn);
        if (!scales_out && M != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: these codes need scales_out", fn);
        if (K % (rows ? 32 : 128)) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: K %% %d != 0", fn, rows ? 32 : 128);
        if (tiled && M % 128) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: the tiled scales need M %% 128 == 0", fn);
        if (!aligned(q_out, 16) || !aligned(scales_out, tiled ? 16 : f32 ? 4 : 1))
            return api_fail(FP8SQ_ERR_MISALIGNED, "%s: codes need 16-byte, scales 4-byte (tiled 16-byte) alignment", fn);
        scale_bytes = n / 32;        // 4 bytes for 128 values, or 1 for 32
    } else if ((r = check_cast(fn, q_out, q_format, q_state, q_history_len))) {
        return r;
    }
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t bytes = n * size_of(dtype);
    if ((r = check_overlap(fn, {{"x", x, bytes, false}, {"residual", residual, bytes, false},
                                {"gamma", gamma, 4 * (uint64_t)K, false}, {"sum_out", sum_out, bytes, true},
                                {"y", y, bytes, true}, {"rstd_out", rstd_out, 4 * (uint64_t)M, true},
                                {"q_out", q_out, n, true}, {"scales_out", scales_out, scale_bytes, true}},
                           sum_out, {residual, x})))
        return r;
    fp8sq::LnArgs a;
    a.M = M;
    a.K = K;
    a.dtype = dtype;
    a.x = x;
    a.residual = residual;
    a.sum = sum_out;
    a.gamma = gamma;
    a.eps = eps;
    a.y = y;
    a.rstd = rstd_out;
    a.q = q_out;
    a.q_format = q_format;
    a.q_gran = q_gran;
    a.q_state = q_state;
    a.q_history_len = q_history_len;
    a.q_scales = scales_out;
    return cuda_status(fp8sq::launch_rmsnorm_fwd(a, static_cast<cudaStream_t>(stream), sms), "fp8_rmsnorm_fwd launch");
}

FP8SQ_API size_t fp8_rmsnorm_bwd_workspace_bytes(int64_t M, int64_t K)
{
    return M > 0 && K > 0 && M < kMaxDim && K < kMaxDim ? fp8sq::rmsnorm_bwd_workspace(M, K) : 0;
}

FP8SQ_API int fp8_rmsnorm_bwd(const void* dy, const void* x, const void* dres, int dtype, const float* gamma,
                              const float* rstd, int64_t M, int64_t K, void* dx, float* dgamma, void* workspace,
                              size_t ws_bytes, void* stream)
{
    const char* fn = "fp8_rmsnorm_bwd";
    if (M < 0 || K < 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: negative size", fn);
    if (M >= kMaxDim || K >= kMaxDim) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: dimension too large", fn);
    if (!valid_dtype(dtype)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (K == 0 && M != 0) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: a row needs at least one element", fn);
    if ((!dy || !x || !gamma || !rstd || !dx) && M != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!dgamma && K != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null dgamma", fn);
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dres, 16) || !aligned(dx, 16) || !aligned(gamma, 16))
        return api_fail(FP8SQ_ERR_MISALIGNED, "%s: dy, x, dres, dx, gamma must be 16-byte aligned", fn);
    if (!aligned(rstd, 4) || !aligned(dgamma, 4)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: rstd, dgamma must be 4-byte aligned", fn);
    const size_t need = fp8_rmsnorm_bwd_workspace_bytes(M, K);
    if (need && !workspace) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null workspace", fn);
    if (ws_bytes < need) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: workspace of %zu bytes, needs %zu", fn, ws_bytes, need);
    if (!aligned(workspace, 16)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: workspace must be 16-byte aligned", fn);
    int sms, r;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t bytes = (uint64_t)M * (uint64_t)K * size_of(dtype), col = 4 * (uint64_t)K;
    if ((r = check_overlap(fn, {{"dy", dy, bytes, false}, {"x", x, bytes, false}, {"dres", dres, bytes, false},
                                {"gamma", gamma, col, false}, {"rstd", rstd, 4 * (uint64_t)M, false}, {"dx", dx, bytes, true},
                                {"dgamma", dgamma, col, true}, {"workspace", workspace, need, true}})))
        return r;
    fp8sq::LnArgs a;
    a.M = M;
    a.K = K;
    a.dtype = dtype;
    a.dy = dy;
    a.x = x;
    a.dres = dres;
    a.gamma = gamma;
    a.rstd = const_cast<float*>(rstd);
    a.dx = dx;
    a.dgamma = dgamma;
    a.workspace = workspace;
    return cuda_status(fp8sq::launch_rmsnorm_bwd(a, static_cast<cudaStream_t>(stream), sms), "fp8_rmsnorm_bwd launch");
}

FP8SQ_API int64_t fp8_expert_rows(int64_t T, int k, int E) { return valid_routing(T, k, E) ? fp8sq::expert_layout(T, k, E).rows : 0; }

FP8SQ_API int64_t fp8_expert_plan_ints(int64_t T, int k, int E)
{
    return valid_routing(T, k, E) ? fp8sq::expert_layout(T, k, E).ints : 0;
}

FP8SQ_API int fp8_expert_plan(const int32_t* ids, int64_t T, int k, int E, int32_t* plan, void* stream)
{
    const char* fn = "fp8_expert_plan";
    ExpertLayout l;
    int r = check_routing(fn, plan, T, k, E, &l);
    if (r) return r;
    if (!ids && T != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null ids", fn);
    if (!aligned(ids, 4)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: ids must be 4-byte aligned", fn);
    int sms;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    if ((r = check_overlap(fn, {{"ids", ids, 4 * (uint64_t)T * (uint64_t)k, false}, {"plan", plan, 4 * (uint64_t)l.ints, true}})))
        return r;
    fp8sq::ExpertRowsArgs a = rows_args(plan, T, k, E, l, 0);
    a.ids = ids;
    a.plan_out = plan;
    return cuda_status(fp8sq::launch_expert_plan(a, static_cast<cudaStream_t>(stream)), "fp8_expert_plan launch");
}

FP8SQ_API int fp8_expert_dispatch(const void* x, int elem_bytes, int64_t K, const int32_t* plan, int64_t T, int k, int E,
                                  void* out, void* stream)
{
    const char* fn = "fp8_expert_dispatch";
    ExpertLayout l;
    int r = check_routing(fn, plan, T, k, E, &l);
    if (r) return r;
    if (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: elements of 1, 2 or 4 bytes", fn);
    if (K < 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: negative size", fn);
    if (K >= kMaxRow) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: rows of at most %d elements", fn, (int)kMaxRow - 1);
    if ((!x || !out) && T * K != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null x or out", fn);
    if (!aligned(x, 16) || !aligned(out, 16)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: x, out must be 16-byte aligned", fn);
    int sms;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t row = (uint64_t)K * (uint64_t)elem_bytes;
    if ((r = check_overlap(fn, {{"x", x, (uint64_t)T * row, false}, {"plan", plan, 4 * (uint64_t)l.ints, false},
                                {"out", out, (uint64_t)l.rows * row, true}})))
        return r;
    if (T == 0 || K == 0) return FP8SQ_OK;
    fp8sq::ExpertRowsArgs a = rows_args(plan, T, k, E, l, K);
    a.x = x;
    a.size = elem_bytes;
    a.rows_out = out;
    return cuda_status(fp8sq::launch_expert_dispatch(a, static_cast<cudaStream_t>(stream), sms), "fp8_expert_dispatch launch");
}

FP8SQ_API int fp8_expert_combine(const void* rows, int dtype, int64_t K, const float* weights, const void* residual,
                                 const int32_t* plan, int64_t T, int k, int E, void* y, void* stream)
{
    const char* fn = "fp8_expert_combine";
    ExpertLayout l;
    int r = check_routing(fn, plan, T, k, E, &l);
    if (r) return r;
    if (!valid_dtype(dtype)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (K < 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: negative size", fn);
    if (K >= kMaxRow) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: rows of at most %d elements", fn, (int)kMaxRow - 1);
    if ((!rows || !y) && T * K != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null rows or y", fn);
    if (!aligned(rows, 16) || !aligned(residual, 16) || !aligned(y, 16) || !aligned(weights, 4))
        return api_fail(FP8SQ_ERR_MISALIGNED, "%s: rows, residual, y need 16-byte, weights 4-byte alignment", fn);
    int sms;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t row = (uint64_t)K * size_of(dtype), tk = 4 * (uint64_t)T * (uint64_t)k;
    if ((r = check_overlap(fn, {{"rows", rows, (uint64_t)l.rows * row, false}, {"weights", weights, tk, false},
                                {"residual", residual, (uint64_t)T * row, false}, {"plan", plan, 4 * (uint64_t)l.ints, false},
                                {"y", y, (uint64_t)T * row, true}},
                           y, {residual})))
        return r;
    if (T == 0 || K == 0) return FP8SQ_OK;
    fp8sq::ExpertRowsArgs a = rows_args(plan, T, k, E, l, K);
    a.dtype = dtype;
    a.rows = rows;
    a.weights = weights;
    a.residual = residual;
    a.y = y;
    return cuda_status(fp8sq::launch_expert_combine(a, static_cast<cudaStream_t>(stream), sms), "fp8_expert_combine launch");
}

FP8SQ_API int fp8_expert_combine_bwd(const void* dy, int dtype, int64_t K, const void* rows, const float* weights,
                                     const int32_t* plan, int64_t T, int k, int E, float* dweights, void* drows,
                                     uint8_t* q_out, int q_format, float* q_state, int q_history_len, void* stream)
{
    const char* fn = "fp8_expert_combine_bwd";
    ExpertLayout l;
    int r = check_routing(fn, plan, T, k, E, &l);
    if (r) return r;
    if (!valid_dtype(dtype)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (K < 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: negative size", fn);
    if (K >= kMaxRow) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: rows of at most %d elements", fn, (int)kMaxRow - 1);
    if ((!dy || !weights) && T * K != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null dy or weights", fn);
    if (!dweights && !drows && !q_out && T * K != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: no output asked for", fn);
    if (dweights && !rows && T * K != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: dweights needs the rows", fn);
    if (!aligned(dy, 16) || !aligned(rows, 16) || !aligned(drows, 16) || !aligned(weights, 4) || !aligned(dweights, 4))
        return api_fail(FP8SQ_ERR_MISALIGNED, "%s: dy, rows, drows need 16-byte, the weights 4-byte alignment", fn);
    if ((r = check_cast(fn, q_out, q_format, q_state, q_history_len))) return r;
    int sms;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t row = (uint64_t)K * size_of(dtype), tk = 4 * (uint64_t)T * (uint64_t)k, R = (uint64_t)l.rows;
    if ((r = check_overlap(fn, {{"dy", dy, (uint64_t)T * row, false}, {"rows", rows, R * row, false},
                                {"weights", weights, tk, false}, {"plan", plan, 4 * (uint64_t)l.ints, false},
                                {"dweights", dweights, tk, true}, {"drows", drows, R * row, true},
                                {"q_out", q_out, R * (uint64_t)K, true}})))
        return r;
    if (T == 0) return FP8SQ_OK;
    fp8sq::ExpertRowsArgs a = rows_args(plan, T, k, E, l, K);
    a.dtype = dtype;
    a.dy = dy;
    a.rows = rows;
    a.weights = weights;
    a.dweights = dweights;
    a.drows = drows;
    a.q = q_out;
    a.q_format = q_format;
    a.q_state = q_state;
    a.q_history_len = q_history_len;
    return cuda_status(fp8sq::launch_expert_combine_bwd(a, static_cast<cudaStream_t>(stream), sms), "fp8_expert_combine_bwd launch");
}

FP8SQ_API size_t fp8_expert_workspace_bytes(int64_t T, int k, int E, int64_t N, int64_t K)
{
    return valid_routing(T, k, E) && T > 0 && N > 0 && K > 0 && N < kMaxDim && K < kMaxDim ? fp8sq::expert_workspace(T, k, E, N, K)
                                                                                        : 0;
}

FP8SQ_API int fp8_expert_glu_fwd(const uint8_t* A, int a_format, const float* a_scale, const uint8_t* W, int w_format,
                                 const float* w_scales, const int32_t* plan, int64_t T, int k, int E, int64_t F, int64_t K,
                                 int act, void* gu_out, void* h_out, uint8_t* q_out, int q_format, float* q_state,
                                 int q_history_len, void* workspace, size_t ws_bytes, void* stream)
{
    const char* fn = "fp8_expert_glu_fwd";
    ExpertLayout l;
    int r = check_routing(fn, plan, T, k, E, &l);
    if (r) return r;
    if ((r = check_product(fn, A, a_format, a_scale, W, w_format, w_scales, act, T, E, F, K, false, 2 * F))) return r;
    if (!h_out && !q_out && T * F != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: no output asked for", fn);
    if (!aligned(h_out, 16) || !aligned(gu_out, 16)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: h, gu must be 16-byte aligned", fn);
    if ((r = check_cast(fn, q_out, q_format, q_state, q_history_len))) return r;
    const size_t need = fp8_expert_workspace_bytes(T, k, E, 2 * F, K);
    if ((r = check_workspace(fn, workspace, ws_bytes, need))) return r;
    int sms;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t n = (uint64_t)l.rows * (uint64_t)F;
    if ((r = check_overlap(fn, {{"A", A, (uint64_t)l.rows * (uint64_t)K, false}, {"W", W, 2 * (uint64_t)E * (uint64_t)F * (uint64_t)K, false},
                                {"a_scale", a_scale, 4, false}, {"w_scales", w_scales, 4 * (uint64_t)E, false},
                                {"plan", plan, 4 * (uint64_t)l.ints, false}, {"gu_out", gu_out, 4 * n, true},
                                {"h_out", h_out, 2 * n, true}, {"q_out", q_out, n, true},
                                {"workspace", workspace, need, true}})))
        return r;
    fp8sq::ExpertGemmArgs a;
    a.kind = fp8sq::kExpertGlu;
    a.T = T;
    a.k = k;
    a.E = E;
    a.layout = l;
    a.plan = plan;
    a.N = F;
    a.K = K;
    a.A = A;
    a.B = W;
    a.a_format = a_format;
    a.b_format = w_format;
    a.a_scale = a_scale;
    a.b_scale = w_scales;
    a.act = act;
    a.D = h_out;
    a.Z = gu_out;
    a.q_out = q_out;
    a.q_format = q_format;
    a.q_state = q_state;
    a.q_history_len = q_history_len;
    a.workspace = need ? workspace : nullptr;
    return launch_product(a, stream, sms, "fp8_expert_glu_fwd launch");
}

FP8SQ_API int fp8_expert_gemm(const uint8_t* A, int a_format, const float* a_scale, const uint8_t* B, int b_format,
                              const float* b_scales, int b_major, const int32_t* plan, int64_t T, int k, int E, int64_t N,
                              int64_t K, void* D, int d_dtype, void* workspace, size_t ws_bytes, void* stream)
{
    const char* fn = "fp8_expert_gemm";
    ExpertLayout l;
    int r = check_routing(fn, plan, T, k, E, &l);
    if (r) return r;
    if (b_major != FP8SQ_K_MAJOR && b_major != FP8SQ_MN_MAJOR) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad operand major", fn);
    const bool mn = b_major == FP8SQ_MN_MAJOR;
    if ((r = check_product(fn, A, a_format, a_scale, B, b_format, b_scales, 0, T, E, N, K, mn, mn ? K : N))) return r;
    if (!valid_dtype(d_dtype)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (!D && T * N != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null D", fn);
    if (!aligned(D, 16)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: D must be 16-byte aligned", fn);
    const size_t need = mn ? 0 : fp8_expert_workspace_bytes(T, k, E, N, K);
    if ((r = check_workspace(fn, workspace, ws_bytes, need))) return r;
    int sms;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    if ((r = check_overlap(fn, {{"A", A, (uint64_t)l.rows * (uint64_t)K, false}, {"B", B, (uint64_t)E * (uint64_t)N * (uint64_t)K, false},
                                {"a_scale", a_scale, 4, false}, {"b_scales", b_scales, 4 * (uint64_t)E, false},
                                {"plan", plan, 4 * (uint64_t)l.ints, false},
                                {"D", D, (uint64_t)l.rows * (uint64_t)N * size_of(d_dtype), true},
                                {"workspace", workspace, need, true}})))
        return r;
    fp8sq::ExpertGemmArgs a;
    a.kind = fp8sq::kExpertGemm;
    a.T = T;
    a.k = k;
    a.E = E;
    a.layout = l;
    a.plan = plan;
    a.N = N;
    a.K = K;
    a.b_mn = mn;
    a.A = A;
    a.B = B;
    a.a_format = a_format;
    a.b_format = b_format;
    a.a_scale = a_scale;
    a.b_scale = b_scales;
    a.D = D;
    a.d_dtype = d_dtype;
    a.workspace = need ? workspace : nullptr;
    return launch_product(a, stream, sms, "fp8_expert_gemm launch");
}

FP8SQ_API int fp8_expert_glu_bwd(const uint8_t* dY, int dy_format, const float* dy_scale, const uint8_t* Wd, int w_format,
                                 const float* w_scales, const int32_t* plan, int64_t T, int k, int E, int64_t F, int64_t K,
                                 const void* gu, int act, uint8_t* q_dgu, int q_format, float* q_state, int q_history_len,
                                 void* stream)
{
    const char* fn = "fp8_expert_glu_bwd";
    ExpertLayout l;
    int r = check_routing(fn, plan, T, k, E, &l);
    if (r) return r;
    if ((r = check_product(fn, dY, dy_format, dy_scale, Wd, w_format, w_scales, act, T, E, F, K, true, K))) return r;
    if ((!gu || !q_dgu) && T * F != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null gu or codes", fn);
    if (!aligned(gu, 16)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: gu must be 16-byte aligned", fn);
    if ((r = check_cast(fn, q_dgu, q_format, q_state, q_history_len))) return r;
    int sms;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t n = (uint64_t)l.rows * (uint64_t)F;
    if ((r = check_overlap(fn, {{"dY", dY, (uint64_t)l.rows * (uint64_t)K, false}, {"Wd", Wd, (uint64_t)E * (uint64_t)F * (uint64_t)K, false},
                                {"dy_scale", dy_scale, 4, false}, {"w_scales", w_scales, 4 * (uint64_t)E, false},
                                {"plan", plan, 4 * (uint64_t)l.ints, false}, {"gu", gu, 4 * n, false}, {"q_dgu", q_dgu, 2 * n, true}})))
        return r;
    fp8sq::ExpertGemmArgs a;
    a.kind = fp8sq::kExpertGluBwd;
    a.T = T;
    a.k = k;
    a.E = E;
    a.layout = l;
    a.plan = plan;
    a.N = F;
    a.K = K;
    a.A = dY;
    a.B = Wd;
    a.a_format = dy_format;
    a.b_format = w_format;
    a.a_scale = dy_scale;
    a.b_scale = w_scales;
    a.act = act;
    a.gu = gu;
    a.q_out = q_dgu;
    a.q_format = q_format;
    a.q_state = q_state;
    a.q_history_len = q_history_len;
    return launch_product(a, stream, sms, "fp8_expert_glu_bwd launch");
}

FP8SQ_API int fp8_expert_wgrad(const uint8_t* A, int a_format, const float* a_scale, const uint8_t* B, int b_format,
                               const float* b_scale, const int32_t* plan, int64_t T, int k, int E, int64_t M, int64_t N,
                               void* D, int d_dtype, void* stream)
{
    const char* fn = "fp8_expert_wgrad";
    ExpertLayout l;
    int r = check_routing(fn, plan, T, k, E, &l);
    if (r) return r;
    if (!valid_format(a_format) || !valid_format(b_format)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad operand format", fn);
    if (!valid_dtype(d_dtype)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (M < 0 || N < 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: negative size", fn);
    if (M >= kMaxDim || N >= kMaxDim || (int64_t)E * M >= kMaxDim) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: dimension too large", fn);
    if (M % 32 || N % 16) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: needs M %% 32 == 0 and N %% 16 == 0", fn);
    if ((!A || !B || !a_scale || !b_scale) && T != 0 && M != 0 && N != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null operand or scale", fn);
    if (!D && M * N != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null D", fn);
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(D, 16)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: A, B, D must be 16-byte aligned", fn);
    if (!aligned(a_scale, 4) || !aligned(b_scale, 4)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: scales must be 4-byte aligned", fn);
    int sms;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t R = (uint64_t)l.rows, out = (uint64_t)E * (uint64_t)M * (uint64_t)N * size_of(d_dtype);
    if ((r = check_overlap(fn, {{"A", A, R * (uint64_t)M, false}, {"B", B, R * (uint64_t)N, false}, {"a_scale", a_scale, 4, false},
                                {"b_scale", b_scale, 4, false}, {"plan", plan, 4 * (uint64_t)l.ints, false}, {"D", D, out, true}})))
        return r;
    if (T == 0 && out != 0) return cuda_status(cudaMemsetAsync(D, 0, out, static_cast<cudaStream_t>(stream)), "fp8_expert_wgrad");
    fp8sq::ExpertGemmArgs a;
    a.kind = fp8sq::kExpertWgrad;
    a.T = T;
    a.k = k;
    a.E = E;
    a.layout = l;
    a.plan = plan;
    a.M = M;
    a.N = N;
    a.A = A;
    a.B = B;
    a.a_format = a_format;
    a.b_format = b_format;
    a.a_scale = a_scale;
    a.b_scale = b_scale;
    a.D = D;
    a.d_dtype = d_dtype;
    return launch_product(a, stream, sms, "fp8_expert_wgrad launch");
}

}  // extern "C"
