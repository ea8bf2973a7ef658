// rmsnorm.cu -- RMSNorm forward and backward (norm.cuh): rstd = 1 / sqrt(sum(s^2)
// / K + eps), y = s rstd gamma of s = x + residual, with FP8 codes of the fp32 y
// under a delayed state or with the scale of each 128 or 32 columns of a row.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "norm.cuh"
#include "ptx.cuh"

namespace fp8sq {

namespace {

// Rows beyond what a CTA holds in registers: one row a CTA at a time, its
// elements read again after the sum (from L2 as a rule).  A warp takes 128
// columns at a time, a lane four of them, so a unit's lanes are neighbours.
template <typename T>
__global__ void __launch_bounds__(256) k_rms_fwd_any(const T* x, const T* res, const float* __restrict__ gamma,
                                                     float eps, int64_t R, int64_t K, T* sum, T* __restrict__ y,
                                                     float* __restrict__ rstd, LnCast cast, int unit_cols)
{
    pdl_enter();
    __shared__ float red[8];
    const bool delayed = cast.q && unit_cols == 0;
    const float m = delayed ? cast.state[cast.H] : 1.0f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float amax = 0.0f;
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const T* xr = x + r * K;
        float s = 0.0f;
        // (the columns that the same thread reads again below)
        auto columns = [&](auto&& f) {
            for (int64_t c0 = 128 * warp; c0 < K; c0 += 8 * 128) f(c0 + 4 * lane);
        };
        columns([&](int64_t c) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < K) {
                    float v = to_f(xr[c + j]);
                    if (res) {
                        const T w = from_f<T>(v + to_f(res[r * K + c + j]));
                        sum[r * K + c + j] = w;
                        v = to_f(w);
                    }
                    s = fmaf(v, v, s);
                }
        });
        if (res) xr = sum + r * K;      // each thread reads back its own columns
        const float rs = 1.0f / sqrtf(cta_sum(s, red) / (float)K + eps);
        if (threadIdx.x == 0 && rstd) rstd[r] = rs;
        columns([&](int64_t c) {
            float v[4];
            uint32_t a = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = c + j < K ? to_f(xr[c + j]) * rs * gamma[c + j] : 0.0f;
                if (y && c + j < K) y[r * K + c + j] = from_f<T>(v[j]);
                a = max(a, __float_as_uint(v[j]) & 0x7FFFFFFFu);
            }
            if (!cast.q) return;
            float mult = m;
            if (delayed) {
                amax = max_nan(amax, __uint_as_float(a));
            } else {
                for (int o = unit_cols / 8; o >= 1; o >>= 1) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
                mult = unit_cols == 128 ? unit_scale<32>(a, cast, r, (int)c, (int)K, c < K)
                                        : unit_scale<8>(a, cast, r, (int)c, (int)K, c < K);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < K) cast.q[r * K + c + j] = code1(__fmul_rn(v[j], mult), cast.fmt);
        });
    }
    if (delayed) record_amax(amax, cast.state);
}

template <typename T>
cudaError_t rms_fwd(LnArgs a, cudaStream_t st, int sms)
{
    const int unit = !a.q || a.q_gran == kTensor ? 0 : a.q_gran == kTile || a.q_gran == kTilePow2 ? 128 : 32;
    a.q_unit = a.q_gran == kTilePow2  ? kUnitPow2
               : a.q_gran == kMX      ? kUnitMx
               : a.q_gran == kMXTiled ? kUnitMxTiled
               : a.q_gran == kMXFloor ? kUnitMxFloor
                                      : kUnitF32;
    a.beta = nullptr;
    if (a.K <= 1024 * kLnCols) {
        constexpr int WIDE = 16 / (int)sizeof(T);
        if (unit == 128) return ln_fwd_rows<T, WIDE, kCodes128, true>(a, st, sms);      // (K % 128 == 0)
        if (unit == 32) return ln_fwd_rows<T, WIDE, kCodes32, true>(a, st, sms);
        return a.q ? ln_fwd_vec<T, kCodesDelayed, true>(a, st, sms) : ln_fwd_vec<T, kNoCodes, true>(a, st, sms);
    }
    const int64_t cap = (int64_t)sms * 8;
    launch_k(k_rms_fwd_any<T>, (unsigned)(a.M < cap ? a.M : cap), 256, 0, st, static_cast<const T*>(a.x),
             static_cast<const T*>(a.residual), a.gamma, a.eps, a.M, a.K, static_cast<T*>(a.sum), static_cast<T*>(a.y),
             a.rstd, LnCast{a.q, a.q_format, a.q_history_len, a.q_state, a.q_unit, a.q_scales}, unit);
    return cudaGetLastError();
}

}  // namespace

size_t rmsnorm_bwd_workspace(int64_t M, int64_t K) { return (size_t)parts_for(M) * (size_t)K * sizeof(float); }

cudaError_t launch_rmsnorm_fwd(const LnArgs& a, cudaStream_t st, int sms)
{
    if (a.M == 0 || a.K == 0) return cudaSuccess;
    return a.dtype == kBF16 ? rms_fwd<__nv_bfloat16>(a, st, sms) : rms_fwd<float>(a, st, sms);
}

cudaError_t launch_rmsnorm_bwd(const LnArgs& a, cudaStream_t st, int sms)
{
    if (a.K == 0) return cudaSuccess;
    return a.dtype == kBF16 ? ln_bwd<__nv_bfloat16, true>(a, st, sms) : ln_bwd<float, true>(a, st, sms);
}

}  // namespace fp8sq
