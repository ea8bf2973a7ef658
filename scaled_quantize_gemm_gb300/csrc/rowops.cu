// rowops.cu -- row-wise and elementwise operators around the FP8 linear:
// LayerNorm forward and backward, and the backward pass of an activation with
// its bias gradient and FP8 cast.  All arithmetic and every sum is fp32.
//
// Column sums (dgamma, dbeta, dbias) run in two stages: a CTA sums the rows it
// owns in registers and writes one partial row per sum to the workspace, then
// k_col_reduce adds the partials in index order, so a result does not depend
// on the order in which CTAs run.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace fp8sq {

namespace {

constexpr int kMaxParts = 608;      // partial rows of a column sum

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// sum over a 256-thread CTA, the same bits in every thread
__device__ __forceinline__ float cta_sum(float v, float* red)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return ((red[0] + red[1]) + (red[2] + red[3])) + ((red[4] + red[5]) + (red[6] + red[7]));
}

// ------------------------------------------------------------------ any row length
template <typename T>
__global__ void __launch_bounds__(256) k_ln_fwd_any(const T* x, const T* __restrict__ res,
                                                    const float* __restrict__ gamma, const float* __restrict__ beta,
                                                    float eps, int64_t R, int64_t K, T* sum, T* __restrict__ y,
                                                    float* __restrict__ mu, float* __restrict__ rstd)
{
    pdl_enter();
    __shared__ float red[8];
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const T* xr = x + r * K;
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < K; c += 256) {
            float v = to_f(xr[c]);
            if (res) {
                const T w = from_f<T>(v + to_f(res[r * K + c]));
                sum[r * K + c] = w;
                v = to_f(w);
            }
            s += v;
        }
        if (res) xr = sum + r * K;      // each thread reads back its own columns
        const float mean = cta_sum(s, red) / (float)K;
        s = 0.0f;
        for (int64_t c = threadIdx.x; c < K; c += 256) {
            const float d = to_f(xr[c]) - mean;
            s = fmaf(d, d, s);
        }
        const float rs = 1.0f / sqrtf(cta_sum(s, red) / (float)K + eps);
        if (threadIdx.x == 0) {
            if (mu) mu[r] = mean;
            if (rstd) rstd[r] = rs;
        }
        for (int64_t c = threadIdx.x; c < K; c += 256)
            y[r * K + c] = from_f<T>(fmaf((to_f(xr[c]) - mean) * rs, gamma[c], beta ? beta[c] : 0.0f));
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_ln_bwd_dx_any(const T* __restrict__ dy, const T* __restrict__ x,
                                                       const T* __restrict__ dres, const float* __restrict__ gamma,
                                                       const float* __restrict__ mu, const float* __restrict__ rstd,
                                                       int64_t R, int64_t K, T* __restrict__ dx)
{
    pdl_enter();
    __shared__ float red[8];
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const float mean = mu[r], rs = rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < K; c += 256) {
            const float w = to_f(dy[r * K + c]) * gamma[c];
            s1 += w;
            s2 = fmaf(w, (to_f(x[r * K + c]) - mean) * rs, s2);
        }
        const float c1 = cta_sum(s1, red) / (float)K, c2 = cta_sum(s2, red) / (float)K;
        for (int64_t c = threadIdx.x; c < K; c += 256) {
            const float w = to_f(dy[r * K + c]) * gamma[c];
            float v = rs * (w - c1 - (to_f(x[r * K + c]) - mean) * rs * c2);
            if (dres) v += to_f(dres[r * K + c]);
            dx[r * K + c] = from_f<T>(v);
        }
    }
}

// partial dgamma (row 2 p) and dbeta (row 2 p + 1) of the rows of part p
template <typename T>
__global__ void __launch_bounds__(256) k_ln_bwd_gb_any(const T* __restrict__ dy, const T* __restrict__ x,
                                                       const float* __restrict__ mu, const float* __restrict__ rstd,
                                                       int64_t R, int64_t K, float* __restrict__ part)
{
    pdl_enter();
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= K) return;
    float g = 0.0f, b = 0.0f;
    for (int64_t r = blockIdx.y; r < R; r += gridDim.y) {
        const float d = to_f(dy[r * K + c]);
        g = fmaf(d, (to_f(x[r * K + c]) - mu[r]) * rstd[r], g);
        b += d;
    }
    part[(2 * (int64_t)blockIdx.y) * K + c] = g;
    part[(2 * (int64_t)blockIdx.y + 1) * K + c] = b;
}

// out0[c] = sum over p of part[p][c] for c < n0, out1[c - n0] for the rest
// (rows of n columns); a CTA takes 32 columns, eight warps an eighth of the
// parts each, added in a fixed order
__global__ void __launch_bounds__(256) k_col_reduce(const float* __restrict__ part, int parts, int64_t n,
                                                    float* __restrict__ out0, int64_t n0, float* __restrict__ out1)
{
    pdl_enter();
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float a = 0.0f;
    if (c < n)
        for (int p = w; p < parts; p += 8) a += part[(int64_t)p * n + c];
    s[w][lane] = a;
    __syncthreads();
    if (w == 0 && c < n) {
        const float v = ((s[0][lane] + s[1][lane]) + (s[2][lane] + s[3][lane])) +
                        ((s[4][lane] + s[5][lane]) + (s[6][lane] + s[7][lane]));
        if (c < n0) out0[c] = v;
        else out1[c - n0] = v;
    }
}

// dz = dy act'(z): codes and / or bf16, and the partial column sums
__global__ void __launch_bounds__(256) k_act_bwd_any(const __nv_bfloat16* __restrict__ dy,
                                                     const __nv_bfloat16* __restrict__ z, int act, int64_t R, int64_t N,
                                                     __nv_bfloat16* __restrict__ dz, uint8_t* __restrict__ q, int fmt,
                                                     float* qstate, int H, float* __restrict__ part)
{
    pdl_enter();
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const float m = q ? qstate[H] : 1.0f;
    float sum = 0.0f;
    uint32_t amax = 0;
    if (c < N)
        act_dispatch(act, [&](auto tag) {
            for (int64_t r = blockIdx.y; r < R; r += gridDim.y) {
                float f, d;
                act_fd<decltype(tag)::act>(to_f(z[r * N + c]), f, d);
                d = __fmul_rn(d, to_f(dy[r * N + c]));   // dz itself is summed, whatever else is stored
                sum += d;
                if (dz) dz[r * N + c] = __float2bfloat16_rn(d);
                if (q) {
                    amax = max(amax, __float_as_uint(d) & 0x7FFFFFFFu);
                    const float v = __fmul_rn(d, m);
                    q[r * N + c] = (uint8_t)(fmt == kE4M3 ? cvt_e4m3x2(v, 0.0f) : cvt_e5m2x2(v, 0.0f));
                }
            }
        });
    if (part && c < N) part[(int64_t)blockIdx.y * N + c] = sum;
    if (q) {
        amax = __reduce_max_sync(0xFFFFFFFFu, amax);
        if ((threadIdx.x & 31) == 0) atomicMax(reinterpret_cast<unsigned int*>(qstate), amax);
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t parts_for(int64_t rows) { return rows < kMaxParts ? rows : kMaxParts; }

template <typename T>
cudaError_t ln_fwd(const LnArgs& a, cudaStream_t st, int sms)
{
    const int64_t cap = (int64_t)sms * 8;
    launch_k(k_ln_fwd_any<T>, (unsigned)(a.M < cap ? a.M : cap), 256, 0, st, static_cast<const T*>(a.x),
             static_cast<const T*>(a.residual), a.gamma, a.beta, a.eps, a.M, a.K, static_cast<T*>(a.sum),
             static_cast<T*>(a.y), a.mu, a.rstd);
    return cudaGetLastError();
}

template <typename T>
cudaError_t ln_bwd(const LnArgs& a, cudaStream_t st, int sms)
{
    float* part = static_cast<float*>(a.workspace);
    int parts = 0;
    if (a.M > 0) {
        const int64_t cap = (int64_t)sms * 8;
        launch_k(k_ln_bwd_dx_any<T>, (unsigned)(a.M < cap ? a.M : cap), 256, 0, st, static_cast<const T*>(a.dy),
                 static_cast<const T*>(a.x), static_cast<const T*>(a.dres), a.gamma, (const float*)a.mu,
                 (const float*)a.rstd, a.M, a.K, static_cast<T*>(a.dx));
        parts = (int)parts_for(a.M);
        launch_k(k_ln_bwd_gb_any<T>, dim3((unsigned)cdiv(a.K, 256), parts), 256, 0, st, static_cast<const T*>(a.dy),
                 static_cast<const T*>(a.x), (const float*)a.mu, (const float*)a.rstd, a.M, a.K, part);
    }
    launch_k(k_col_reduce, (unsigned)cdiv(2 * a.K, 32), 256, 0, st, (const float*)part, parts, 2 * a.K, a.dgamma, a.K,
             a.dbeta);
    return cudaGetLastError();
}

}  // namespace

size_t layernorm_bwd_workspace(int64_t M, int64_t K) { return (size_t)parts_for(M) * 2 * (size_t)K * sizeof(float); }
size_t act_bwd_workspace(int64_t M, int64_t N) { return (size_t)parts_for(M) * (size_t)N * sizeof(float); }

cudaError_t launch_layernorm_fwd(const LnArgs& a, cudaStream_t st, int sms)
{
    if (a.M == 0 || a.K == 0) return cudaSuccess;
    return a.dtype == kBF16 ? ln_fwd<__nv_bfloat16>(a, st, sms) : ln_fwd<float>(a, st, sms);
}

cudaError_t launch_layernorm_bwd(const LnArgs& a, cudaStream_t st, int sms)
{
    if (a.K == 0) return cudaSuccess;
    return a.dtype == kBF16 ? ln_bwd<__nv_bfloat16>(a, st, sms) : ln_bwd<float>(a, st, sms);
}

cudaError_t launch_act_bwd(const ActBwdArgs& a, cudaStream_t st, int sms)
{
    (void)sms;
    if (a.N == 0) return cudaSuccess;
    float* part = a.dbias ? static_cast<float*>(a.workspace) : nullptr;
    const int parts = (int)parts_for(a.M);
    if (a.M > 0)
        launch_k(k_act_bwd_any, dim3((unsigned)cdiv(a.N, 256), parts), 256, 0, st,
                 static_cast<const __nv_bfloat16*>(a.dy), static_cast<const __nv_bfloat16*>(a.z), a.act, a.M, a.N,
                 static_cast<__nv_bfloat16*>(a.dz), a.q, a.q_format, a.q_state, a.q_history_len, part);
    if (a.dbias)
        launch_k(k_col_reduce, (unsigned)cdiv(a.N, 32), 256, 0, st, (const float*)part, parts, a.N, a.dbias, a.N,
                 (float*)nullptr);
    return cudaGetLastError();
}

}  // namespace fp8sq
