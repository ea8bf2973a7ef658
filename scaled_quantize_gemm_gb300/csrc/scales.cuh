// scales.cuh -- the FP8 formats' ranges, the rules that turn a unit's amax into
// its scale, and the tiled layout of E8M0 scales.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

namespace fp8sq {

template <int FMT>
struct Fmt;
template <>
struct Fmt<kE4M3> {
    static constexpr float fmax = 448.0f;
    static constexpr int emax = 8;
};
template <>
struct Fmt<kE5M2> {
    static constexpr float fmax = 57344.0f;
    static constexpr int emax = 15;
};

// ------------------------------------------------------------------ scale rules
// current scaling: m = fmax/amax, s = amax/fmax; amax 0 or non-finite -> 1, 1
template <int FMT>
__device__ __forceinline__ void current_scale(uint32_t amax_bits, float& m, float& s)
{
    float a = __uint_as_float(amax_bits);
    if (amax_bits != 0u && amax_bits < 0x7F800000u) {
        m = __fdiv_rn(Fmt<FMT>::fmax, a);
        s = __fdiv_rn(a, Fmt<FMT>::fmax);
    } else {
        m = 1.0f;
        s = 1.0f;
    }
}

// MX: E8M0 code of the smallest 2^e with amax <= fmax * 2^e, and m = 2^-e
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax_bits, float& m)
{
    if (amax_bits >= 0x7F800000u) { m = 1.0f; return 0xFFu; }
    if (amax_bits == 0u) { m = 1.0f; return 127u; }
    int E;
    uint32_t frac;
    uint32_t ef = amax_bits >> 23;
    if (ef == 0u) {                      // subnormal: normalise
        uint32_t mant = amax_bits & 0x7FFFFFu;
        int p = 31 - __clz(mant);        // leading one position, 0..22
        E = p - 149;
        frac = (mant << (23 - p)) & 0x7FFFFFu;
    } else {
        E = (int)ef - 127;
        frac = amax_bits & 0x7FFFFFu;
    }
    int e = E - Fmt<FMT>::emax + (frac > 0x600000u ? 1 : 0);   // 1.f > 1.75
    e = max(-127, min(127, e));
    m = (e <= 126) ? __uint_as_float((uint32_t)(127 - e) << 23) : __uint_as_float(0x00400000u);
    return (uint32_t)(e + 127);
}

// MX by the OCP floor rule: e = floor(log2 amax) - emax (can clip)
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_floor(uint32_t amax_bits, float& m)
{
    if (amax_bits >= 0x7F800000u) { m = 1.0f; return 0xFFu; }
    if (amax_bits == 0u) { m = 1.0f; return 127u; }
    uint32_t ef = amax_bits >> 23;
    const int E = (ef == 0u) ? (31 - __clz(amax_bits & 0x7FFFFFu)) - 149 : (int)ef - 127;
    int e = E - Fmt<FMT>::emax;
    e = max(-127, min(127, e));
    m = (e <= 126) ? __uint_as_float((uint32_t)(127 - e) << 23) : __uint_as_float(0x00400000u);
    return (uint32_t)(e + 127);
}

// MX scales: the canonical layout is u8 [rows][cols/32]; the tiled layout
// (TILED = true) is the one the block-scaled GEMM copies straight into tensor
// memory: 512-byte chunks of 128 rows x 4 consecutive 32-blocks, chunk
// (r/128, t/4) at ((r/128) * (cols/128) + t/4) * 512, inside it
// (r % 32) * 16 + ((r / 32) % 4) * 4 + t % 4.
__device__ __forceinline__ int64_t mx_tiled_offset(int64_t r, int64_t t, int64_t cols)
{
    return ((r >> 7) * (cols >> 7) + (t >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (t & 3);
}

}  // namespace fp8sq
