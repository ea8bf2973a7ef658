// act.cuh -- activations and their derivatives in fp32, for the epilogues and
// the elementwise backward pass.
//
//   relu       max(x, 0)                       derivative 1 for x > 0, else 0
//   gelu       x Phi(x), Phi = (1 + erf(x / sqrt 2)) / 2
//   gelu_tanh  (x / 2) (1 + tanh t), t = sqrt(2 / pi) (x + 0.044715 x^3)
//   silu       x / (1 + exp(-x))
// (1 + tanh t) / 2 is the logistic function of 2 t, so gelu_tanh and silu are
// both x s(u), s(u) = 1 / (1 + exp(-u)), with derivative s + x s (1 - s) u'.
// s takes the hardware exponential and reciprocal: a few units of 2^-24
// beside the argument's own rounding, far below half a step of any stored
// type but fp32, and 1 - s is formed from exp(-u) itself, so it keeps its
// relative precision where s is near 1.  A NaN goes through every form.
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

constexpr float kGeluA = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// logistic argument u(x) of the two sigmoid forms
template <int ACT>
__device__ __forceinline__ float act_u(float x)
{
    if constexpr (ACT == kActSilu) return x;
    else return kGeluA * x * fmaf(kGeluB * x, x, 1.0f);
}

template <int ACT>
__device__ __forceinline__ float act_f(float x)
{
    if constexpr (ACT == kActNone) return x;
    else if constexpr (ACT == kActRelu) return x > 0.0f ? x : (x != x ? x : 0.0f);
    else if constexpr (ACT == kActGelu) return 0.5f * x * (1.0f + erff(x * 0.70710678118654752f));
    // exp(-u) = inf (u below -88) gives x / inf = -0, the limit
    else return __fdividef(x, 1.0f + __expf(-act_u<ACT>(x)));
}

// f = act(x), d = act'(x)
template <int ACT>
__device__ __forceinline__ void act_fd(float x, float& f, float& d)
{
    if constexpr (ACT == kActNone) {
        f = x;
        d = 1.0f;
    } else if constexpr (ACT == kActRelu) {
        f = act_f<ACT>(x);
        d = x > 0.0f ? 1.0f : (x != x ? x : 0.0f);
    } else if constexpr (ACT == kActGelu) {
        const float phi = 0.5f * (1.0f + erff(x * 0.70710678118654752f));
        f = x * phi;
        d = fmaf(x * 0.3989422804014327f, __expf(-0.5f * x * x), phi);
    } else {
        // below u = -87 the value and the derivative are under 2^-118: taken as
        // 0 before u' can overflow against them (u' only grows as x^2)
        const float u = act_u<ACT>(x);
        const float e = __expf(-u);
        const float s = u < -87.0f ? 0.0f : __fdividef(1.0f, 1.0f + e);
        const float xs = x * s;
        f = xs;
        float up;
        if constexpr (ACT == kActSilu) up = 1.0f;
        else up = kGeluA * fmaf(3.0f * kGeluB * x, x, 1.0f);
        // 1 - s = e s; for large u e is 0 and the derivative s = 1
        d = e == 0.0f || s == 0.0f ? s : fmaf(xs * (e * s), up, s);
    }
}

}  // namespace fp8sq
