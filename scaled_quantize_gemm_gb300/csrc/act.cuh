// act.cuh -- activations and their derivatives in fp32, for the epilogues and
// the elementwise backward pass.  Two elements at a time: the multiplies and
// adds are packed f32x2 instructions, half the issue slots of two scalar ones
// (the elementwise backward pass is bound by issue slots next to DRAM).
//
//   relu       max(x, 0)                       derivative 1 for x > 0, else 0
//   gelu       x Phi(x), Phi the normal distribution function
//   gelu_tanh  (x / 2) (1 + tanh t), t = sqrt(2 / pi) (x + 0.044715 x^3)
//   silu       x / (1 + exp(-x))
// (1 + tanh t) / 2 is the logistic function of 2 t, so gelu_tanh and silu are
// both x s(u), s(u) = 1 / (1 + exp(-u)), with derivative s + x s (1 - s) u'.
// s takes the hardware exponential and reciprocal: a few units of 2^-24
// beside the argument's own rounding, far below half a step of any stored
// type but fp32, and 1 - s is formed from exp(-u) itself, so it keeps its
// relative precision where s is near 1.
// Phi on the negative side is exp(-y^2 / 2) f(y), y = -x >= 0, with f(y) = t P(t),
// t = 1 / (1 + p y): the form of formula 7.1.26 in Abramowitz and Stegun, Handbook
// of Mathematical Functions (1964), whose five coefficients bound the absolute
// error only (off by 2e-4 of Phi at -3.5, 4e-3 at -6).  P here is of degree 7,
// fitted in this project to f for 0 <= y <= 14 with the largest relative error
// made least (2^-23.4): Phi keeps its relative precision down the tail, as far
// as the argument's own rounding lets it (a unit of x is x^2 of Phi).  The
// exponential is the one the derivative's density needs.  A NaN goes through
// every form.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace fp8sq {

enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

template <int ACT>
struct ActTag {
    static constexpr int act = ACT;
};

// calls f with the compile-time tag of the run-time activation (the branch is
// uniform over the grid)
template <typename F>
__device__ __forceinline__ void act_dispatch(int act, F&& f)
{
    switch (act) {
    case kActRelu: f(ActTag<kActRelu>{}); break;
    case kActGelu: f(ActTag<kActGelu>{}); break;
    case kActGeluTanh: f(ActTag<kActGeluTanh>{}); break;
    case kActSilu: f(ActTag<kActSilu>{}); break;
    default: f(ActTag<kActNone>{}); break;
    }
}

__device__ __forceinline__ float2 f2(float v) { return make_float2(v, v); }
__device__ __forceinline__ float ex2_approx(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_approx(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float2 ex2_2(float2 v) { return make_float2(ex2_approx(v.x), ex2_approx(v.y)); }
__device__ __forceinline__ float2 rcp_2(float2 v) { return make_float2(rcp_approx(v.x), rcp_approx(v.y)); }
// bounds that a NaN passes through
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float2 max2_nan(float2 a, float b) { return make_float2(max_nan(a.x, b), max_nan(a.y, b)); }
__device__ __forceinline__ float2 min2_nan(float2 a, float b) { return make_float2(min_nan(a.x, b), min_nan(a.y, b)); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluA = 1.5957691216057308f;          // 2 sqrt(2 / pi): u = A x (1 + B x^2)
constexpr float kGeluB = 0.044715f;
constexpr float kPhiP = 0.3046f;                       // t = 1 / (1 + p y)
constexpr float kPhi0 = 1.214777827e-01f, kPhi1 = 1.223474219e-01f, kPhi2 = 1.030266806e-01f, kPhi3 = 1.220214441e-01f,
                kPhi4 = -4.002013057e-02f, kPhi5 = 1.882975101e-01f, kPhi6 = -1.539151371e-01f, kPhi7 = 3.676445782e-02f;

// exp(-u(x)) of the two sigmoid forms (2 to the scaled argument)
template <int ACT>
__device__ __forceinline__ float2 act_exp(float2 x, float2 xx)
{
    if constexpr (ACT == kActSilu) return ex2_2(__fmul2_rn(x, f2(-kLog2e)));
    else return ex2_2(__fmul2_rn(x, __ffma2_rn(xx, f2(-kLog2e * kGeluA * kGeluB), f2(-kLog2e * kGeluA))));
}

// Phi(x) and exp(-x^2 / 2)
__device__ __forceinline__ float2 normal_cdf(float2 x, float2& ex)
{
    const float2 ax = make_float2(fabsf(x.x), fabsf(x.y));
    ex = ex2_2(__fmul2_rn(__fmul2_rn(x, x), f2(-0.5f * kLog2e)));
    const float2 t = rcp_2(__ffma2_rn(ax, f2(kPhiP), f2(1.0f)));
    float2 p = __ffma2_rn(t, f2(kPhi7), f2(kPhi6));
    p = __ffma2_rn(p, t, f2(kPhi5));
    p = __ffma2_rn(p, t, f2(kPhi4));
    p = __ffma2_rn(p, t, f2(kPhi3));
    p = __ffma2_rn(p, t, f2(kPhi2));
    p = __ffma2_rn(p, t, f2(kPhi1));
    p = __ffma2_rn(p, t, f2(kPhi0));
    p = __fmul2_rn(__fmul2_rn(p, t), ex);              // Phi(-|x|)
    return make_float2(x.x > 0.0f ? 1.0f - p.x : p.x, x.y > 0.0f ? 1.0f - p.y : p.y);
}

template <int ACT>
__device__ __forceinline__ float2 act_f2(float2 x)
{
    if constexpr (ACT == kActNone) return x;
    else if constexpr (ACT == kActRelu) return max2_nan(x, 0.0f);
    else if constexpr (ACT == kActGelu) {
        float2 ex;
        return __fmul2_rn(x, normal_cdf(x, ex));
    } else {
        // exp(-u) = inf (u far below 0) gives x * 0 = -0, the limit
        const float2 e = act_exp<ACT>(x, __fmul2_rn(x, x));
        return __fmul2_rn(x, rcp_2(__fadd2_rn(e, f2(1.0f))));
    }
}

// f = act(x), d = act'(x)
template <int ACT>
__device__ __forceinline__ void act_fd2(float2 x, float2& f, float2& d)
{
    if constexpr (ACT == kActNone) {
        f = x;
        d = f2(1.0f);
    } else if constexpr (ACT == kActRelu) {
        f = max2_nan(x, 0.0f);
        d = make_float2(x.x > 0.0f ? 1.0f : (x.x != x.x ? x.x : 0.0f), x.y > 0.0f ? 1.0f : (x.y != x.y ? x.y : 0.0f));
    } else if constexpr (ACT == kActGelu) {
        float2 ex;
        const float2 phi = normal_cdf(x, ex);
        f = __fmul2_rn(x, phi);
        // |x| <= 40 in the second term (0 there): x exp(-x^2 / 2) stays finite
        const float2 xc = min2_nan(max2_nan(x, -40.0f), 40.0f);
        d = __ffma2_rn(__fmul2_rn(xc, f2(0.3989422804014327f)), ex, phi);
    } else {
        // At |x| = C the value on the negative side and the derivative's
        // distance from 0 or 1 are below 2^-115: x is held there, so that
        // exp(-u) stays finite and u', which grows as x^2, meets no 0 * inf.
        constexpr float C = ACT == kActSilu ? 86.0f : 9.95f;
        const float2 xn = max2_nan(x, -C);
        const float2 xc = min2_nan(xn, C);
        const float2 xx = __fmul2_rn(xc, xc);
        const float2 e = act_exp<ACT>(xc, xx);
        const float2 s = rcp_2(__fadd2_rn(e, f2(1.0f)));
        f = __fmul2_rn(xn, s);
        float2 t = __fmul2_rn(__fmul2_rn(xc, s), __fmul2_rn(e, s));        // x s (1 - s)
        if constexpr (ACT == kActSilu) d = __fadd2_rn(t, s);
        else d = __ffma2_rn(t, __ffma2_rn(xx, f2(3.0f * kGeluA * kGeluB), f2(kGeluA)), s);
    }
}

}  // namespace fp8sq
