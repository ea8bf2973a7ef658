// api_ffn.cu -- the extern "C" entry points of the feed-forward sublayer's
// operators (include/fp8sq.h, section 5c).  Every argument is checked on the
// host before anything is enqueued.
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/fp8sq.h"
#include "api_checks.h"
#include "internal.h"

extern "C" {

FP8SQ_API int fp8_layernorm_fwd(const void* x, const void* residual, int dtype, const float* gamma, const float* beta,
                                float eps, int64_t M, int64_t K, void* sum_out, void* y, float* mu_out, float* rstd_out,
                                uint8_t* q_out, int q_format, float* q_state, int q_history_len, void* stream)
{
    const char* fn = "fp8_layernorm_fwd";
    if (M < 0 || K < 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: negative size", fn);
    if (M >= kMaxDim || K >= kMaxDim) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: dimension too large", fn);
    if (!valid_dtype(dtype)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (K == 0 && M != 0) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: a row needs at least one element", fn);
    if ((!x || !gamma) && M != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null x or gamma", fn);
    if (!y && !q_out && M != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: neither y nor codes asked for", fn);
    if ((residual != nullptr) != (sum_out != nullptr) && M != 0)
        return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: residual and sum_out come together", fn);
    if (!(eps >= 0.0f)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: eps must not be negative", fn);
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(sum_out, 16) || !aligned(gamma, 16) ||
        !aligned(beta, 16))
        return api_fail(FP8SQ_ERR_MISALIGNED, "%s: x, residual, sum, y, gamma, beta must be 16-byte aligned", fn);
    if (!aligned(mu_out, 4) || !aligned(rstd_out, 4)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: mu, rstd must be 4-byte aligned", fn);
    int sms, r;
    if ((r = check_cast(fn, q_out, q_format, q_state, q_history_len))) return r;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t n = (uint64_t)M * (uint64_t)K, bytes = n * size_of(dtype), row = 4 * (uint64_t)M, col = 4 * (uint64_t)K;
    if ((r = check_overlap(fn, {{"x", x, bytes, false}, {"residual", residual, bytes, false}, {"gamma", gamma, col, false},
                                {"beta", beta, col, false}, {"sum_out", sum_out, bytes, true}, {"y", y, bytes, true},
                                {"mu_out", mu_out, row, true}, {"rstd_out", rstd_out, row, true}, {"q_out", q_out, n, true}},
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
    a.beta = beta;
    a.eps = eps;
    a.y = y;
    a.mu = mu_out;
    a.rstd = rstd_out;
    a.q = q_out;
    a.q_format = q_format;
    a.q_state = q_state;
    a.q_history_len = q_history_len;
    return cuda_status(fp8sq::launch_layernorm_fwd(a, static_cast<cudaStream_t>(stream), sms), "fp8_layernorm_fwd launch");
}

FP8SQ_API size_t fp8_layernorm_bwd_workspace_bytes(int64_t M, int64_t K)
{
    return M > 0 && K > 0 && M < kMaxDim && K < kMaxDim ? fp8sq::layernorm_bwd_workspace(M, K) : 0;
}

FP8SQ_API int fp8_layernorm_bwd(const void* dy, const void* x, const void* dres, int dtype, const float* gamma,
                                const float* mu, const float* rstd, int64_t M, int64_t K, void* dx, float* dgamma,
                                float* dbeta, void* workspace, size_t ws_bytes, void* stream)
{
    const char* fn = "fp8_layernorm_bwd";
    if (M < 0 || K < 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: negative size", fn);
    if (M >= kMaxDim || K >= kMaxDim) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: dimension too large", fn);
    if (!valid_dtype(dtype)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (K == 0 && M != 0) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: a row needs at least one element", fn);
    if ((!dy || !x || !gamma || !mu || !rstd || !dx) && M != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null pointer", fn);
    if ((!dgamma || !dbeta) && K != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null dgamma or dbeta", fn);
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dres, 16) || !aligned(dx, 16) || !aligned(gamma, 16))
        return api_fail(FP8SQ_ERR_MISALIGNED, "%s: dy, x, dres, dx, gamma must be 16-byte aligned", fn);
    if (!aligned(mu, 4) || !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(dbeta, 4))
        return api_fail(FP8SQ_ERR_MISALIGNED, "%s: mu, rstd, dgamma, dbeta must be 4-byte aligned", fn);
    const size_t need = fp8_layernorm_bwd_workspace_bytes(M, K);
    if (need && !workspace) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null workspace", fn);
    if (ws_bytes < need) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: workspace of %zu bytes, needs %zu", fn, ws_bytes, need);
    if (!aligned(workspace, 16)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: workspace must be 16-byte aligned", fn);
    int sms, r;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t bytes = (uint64_t)M * (uint64_t)K * size_of(dtype), row = 4 * (uint64_t)M, col = 4 * (uint64_t)K;
    if ((r = check_overlap(fn, {{"dy", dy, bytes, false}, {"x", x, bytes, false}, {"dres", dres, bytes, false},
                                {"gamma", gamma, col, false}, {"mu", mu, row, false}, {"rstd", rstd, row, false},
                                {"dx", dx, bytes, true}, {"dgamma", dgamma, col, true}, {"dbeta", dbeta, col, true},
                                {"workspace", workspace, need, true}})))
        return r;
    fp8sq::LnArgs a;
    a.M = M;
    a.K = K;
    a.dtype = dtype;
    a.dy = dy;
    a.x = x;
    a.dres = dres;
    a.gamma = gamma;
    a.mu = const_cast<float*>(mu);
    a.rstd = const_cast<float*>(rstd);
    a.dx = dx;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.workspace = workspace;
    return cuda_status(fp8sq::launch_layernorm_bwd(a, static_cast<cudaStream_t>(stream), sms), "fp8_layernorm_bwd launch");
}

FP8SQ_API size_t fp8_gemm_act_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    return M > 0 && N > 0 && K > 0 && M < kMaxDim && N < kMaxDim / 2 && K < kMaxDim
               ? fp8sq::ffn_workspace(fp8sq::kFfnAct, M, N, K) : 0;
}

FP8SQ_API size_t fp8_glu_fwd_workspace_bytes(int64_t M, int64_t F, int64_t K)
{
    return M > 0 && F > 0 && K > 0 && M < kMaxDim && F < kMaxDim / 2 && K < kMaxDim
               ? fp8sq::ffn_workspace(fp8sq::kFfnGlu, M, F, K) : 0;
}

FP8SQ_API int fp8_gemm_act(const uint8_t* A, int a_format, const float* a_scale, const uint8_t* B, int b_format,
                           const float* b_scale, int64_t M, int64_t N, int64_t K, int act, const float* bias,
                           const void* residual, int res_dtype, void* z_out, void* D, int d_dtype, uint8_t* q_out,
                           int q_format, float* q_state, int q_history_len, void* workspace, size_t ws_bytes,
                           void* stream)
{
    const char* fn = "fp8_gemm_act";
    int r = check_operands(fn, A, a_format, a_scale, B, b_format, b_scale, act, M, N, K, q_out ? 16 : 8);
    if (r) return r;
    if (!valid_dtype(d_dtype) || !valid_dtype(res_dtype)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad dtype", fn);
    if (!D && !q_out && !z_out && M * N != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: no output asked for", fn);
    if (!aligned(D, 16) || !aligned(z_out, 16) || !aligned(residual, 16) || !aligned(bias, 16))
        return api_fail(FP8SQ_ERR_MISALIGNED, "%s: D, z, residual, bias must be 16-byte aligned", fn);
    if ((r = check_cast(fn, q_out, q_format, q_state, q_history_len))) return r;
    if (workspace && !aligned(workspace, 256)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: workspace must be 256-byte aligned", fn);
    const size_t need = fp8_gemm_act_workspace_bytes(M, N, K);
    if (workspace && ws_bytes < need) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: workspace of %zu bytes, needs %zu", fn, ws_bytes, need);
    int sms;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t n = (uint64_t)M * (uint64_t)N;
    if ((r = check_overlap(fn, {{"A", A, (uint64_t)M * (uint64_t)K, false}, {"B", B, (uint64_t)N * (uint64_t)K, false},
                                {"a_scale", a_scale, 4, false}, {"b_scale", b_scale, 4, false},
                                {"bias", bias, 4 * (uint64_t)N, false}, {"residual", residual, n * size_of(res_dtype), false},
                                {"z_out", z_out, 2 * n, true}, {"D", D, n * size_of(d_dtype), true}, {"q_out", q_out, n, true},
                                {"workspace", workspace, need, true}},
                           D, {residual})))
        return r;
    fp8sq::FfnArgs a;
    a.kind = fp8sq::kFfnAct;
    a.M = M;
    a.N = N;
    a.K = K;
    a.A = A;
    a.B = B;
    a.a_format = a_format;
    a.b_format = b_format;
    a.a_scale = a_scale;
    a.b_scale = b_scale;
    a.act = act;
    a.bias = bias;
    a.residual = residual;
    a.res_dtype = res_dtype;
    a.D = D;
    a.d_dtype = d_dtype;
    a.Z = z_out;
    a.q_out = q_out;
    a.q_format = q_format;
    a.q_state = q_state;
    a.q_history_len = q_history_len;
    a.workspace = need ? workspace : nullptr;
    const char* why = nullptr;
    const cudaError_t e = fp8sq::launch_ffn(a, static_cast<cudaStream_t>(stream), sms, &why);
    return cuda_status(e, "fp8_gemm_act launch", why);
}

FP8SQ_API int fp8_glu_fwd(const uint8_t* A, int a_format, const float* a_scale, const uint8_t* W, int w_format,
                          const float* w_scale, int64_t M, int64_t F, int64_t K, int act, void* gu_out, void* h_out,
                          uint8_t* q_out, int q_format, float* q_state, int q_history_len, void* workspace,
                          size_t ws_bytes, void* stream)
{
    const char* fn = "fp8_glu_fwd";
    int r = check_operands(fn, A, a_format, a_scale, W, w_format, w_scale, act, M, F, K, 16);
    if (r) return r;
    if (!h_out && !q_out && M * F != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: no output asked for", fn);
    if (!aligned(h_out, 16) || !aligned(gu_out, 16)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: h, gu must be 16-byte aligned", fn);
    if ((r = check_cast(fn, q_out, q_format, q_state, q_history_len))) return r;
    if (workspace && !aligned(workspace, 256)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: workspace must be 256-byte aligned", fn);
    const size_t need = fp8_glu_fwd_workspace_bytes(M, F, K);
    if (workspace && ws_bytes < need) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: workspace of %zu bytes, needs %zu", fn, ws_bytes, need);
    int sms;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t n = (uint64_t)M * (uint64_t)F;
    if ((r = check_overlap(fn, {{"A", A, (uint64_t)M * (uint64_t)K, false}, {"W", W, 2 * (uint64_t)F * (uint64_t)K, false},
                                {"a_scale", a_scale, 4, false}, {"w_scale", w_scale, 4, false},
                                {"gu_out", gu_out, 4 * n, true}, {"h_out", h_out, 2 * n, true}, {"q_out", q_out, n, true},
                                {"workspace", workspace, need, true}})))
        return r;
    fp8sq::FfnArgs a;
    a.kind = fp8sq::kFfnGlu;
    a.M = M;
    a.N = F;
    a.K = K;
    a.A = A;
    a.B = W;
    a.a_format = a_format;
    a.b_format = w_format;
    a.a_scale = a_scale;
    a.b_scale = w_scale;
    a.act = act;
    a.D = h_out;
    a.Z = gu_out;
    a.q_out = q_out;
    a.q_format = q_format;
    a.q_state = q_state;
    a.q_history_len = q_history_len;
    a.workspace = need ? workspace : nullptr;
    const char* why = nullptr;
    const cudaError_t e = fp8sq::launch_ffn(a, static_cast<cudaStream_t>(stream), sms, &why);
    return cuda_status(e, "fp8_glu_fwd launch", why);
}

FP8SQ_API int fp8_glu_bwd(const uint8_t* dY, int dy_format, const float* dy_scale, const uint8_t* Wd, int w_format,
                          const float* w_scale, int64_t M, int64_t F, int64_t K, const void* gu, int act,
                          uint8_t* q_dgu, int q_format, float* q_state, int q_history_len, void* stream)
{
    const char* fn = "fp8_glu_bwd";
    int r = check_operands(fn, dY, dy_format, dy_scale, Wd, w_format, w_scale, act, M, F, K, 16);
    if (r) return r;
    if ((!gu || !q_dgu) && M * F != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null gu or codes", fn);
    if (!aligned(gu, 16)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: gu must be 16-byte aligned", fn);
    if ((r = check_cast(fn, q_dgu, q_format, q_state, q_history_len))) return r;
    int sms;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t n = (uint64_t)M * (uint64_t)F;
    if ((r = check_overlap(fn, {{"dY", dY, (uint64_t)M * (uint64_t)K, false}, {"Wd", Wd, (uint64_t)K * (uint64_t)F, false},
                                {"dy_scale", dy_scale, 4, false}, {"w_scale", w_scale, 4, false}, {"gu", gu, 4 * n, false},
                                {"q_dgu", q_dgu, 2 * n, true}})))
        return r;
    fp8sq::FfnArgs a;
    a.kind = fp8sq::kFfnGluBwd;
    a.M = M;
    a.N = F;
    a.K = K;
    a.A = dY;
    a.B = Wd;
    a.a_format = dy_format;
    a.b_format = w_format;
    a.a_scale = dy_scale;
    a.b_scale = w_scale;
    a.act = act;
    a.gu = gu;
    a.q_out = q_dgu;
    a.q_format = q_format;
    a.q_state = q_state;
    a.q_history_len = q_history_len;
    const char* why = nullptr;
    const cudaError_t e = fp8sq::launch_ffn(a, static_cast<cudaStream_t>(stream), sms, &why);
    return cuda_status(e, "fp8_glu_bwd launch", why);
}

FP8SQ_API size_t fp8_act_bwd_workspace_bytes(int64_t M, int64_t N)
{
    return M > 0 && N > 0 && M < kMaxDim && N < kMaxDim ? fp8sq::act_bwd_workspace(M, N) : 0;
}

FP8SQ_API int fp8_act_bwd(const void* dy, const void* z, int64_t M, int64_t N, int act, float* dbias, void* dz_out,
                          uint8_t* q_out, int q_format, float* q_state, int q_history_len, void* workspace,
                          size_t ws_bytes, void* stream)
{
    const char* fn = "fp8_act_bwd";
    int r = check_dims(fn, M, N, 1);
    if (r) return r;
    if (!valid_act(act)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad activation", fn);
    if ((!dy || !z) && M * N != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null dy or z", fn);
    if (!dz_out && !q_out && !dbias && M * N != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: no output asked for", fn);
    if (!aligned(dy, 16) || !aligned(z, 16) || !aligned(dz_out, 16) || !aligned(dbias, 4))
        return api_fail(FP8SQ_ERR_MISALIGNED, "%s: dy, z, dz need 16-byte, dbias 4-byte alignment", fn);
    if ((r = check_cast(fn, q_out, q_format, q_state, q_history_len))) return r;
    const size_t need = dbias ? fp8_act_bwd_workspace_bytes(M, N) : 0;
    if (need && !workspace) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: dbias needs a workspace", fn);
    if (ws_bytes < need) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: workspace of %zu bytes, needs %zu", fn, ws_bytes, need);
    if (!aligned(workspace, 16)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: workspace must be 16-byte aligned", fn);
    int sms;
    if ((r = fp8sq::api_check_device(&sms))) return r;
    const uint64_t n = (uint64_t)M * (uint64_t)N;
    if ((r = check_overlap(fn, {{"dy", dy, 2 * n, false}, {"z", z, 2 * n, false}, {"dbias", dbias, 4 * (uint64_t)N, true},
                                {"dz_out", dz_out, 2 * n, true}, {"q_out", q_out, n, true},
                                {"workspace", workspace, need, true}})))
        return r;
    fp8sq::ActBwdArgs a;
    a.M = M;
    a.N = N;
    a.dy = dy;
    a.z = z;
    a.act = act;
    a.dbias = dbias;
    a.dz = dz_out;
    a.q = q_out;
    a.q_format = q_format;
    a.q_state = q_state;
    a.q_history_len = q_history_len;
    a.workspace = workspace;
    return cuda_status(fp8sq::launch_act_bwd(a, static_cast<cudaStream_t>(stream), sms), "fp8_act_bwd launch");
}

}  // extern "C"
