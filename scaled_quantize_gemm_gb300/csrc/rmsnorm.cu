// rmsnorm.cu -- RMSNorm forward and backward: rstd = 1 / sqrt(sum(s^2) / K + eps),
// y = s rstd gamma of s = x + residual, with FP8 codes of the fp32 y under a
// delayed state or with the scale of each 128 or 32 columns of a row.  The
// backward pass, and rows that 16 bytes do not divide, are forms of LayerNorm's
// kernels (norm.cuh).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act.cuh"
#include "internal.h"
#include "norm.cuh"
#include "ptx.cuh"
#include "scales.cuh"

namespace fp8sq {

namespace {

enum { kNoCodes = 0, kCodesDelayed = 1, kCodes128 = 2, kCodes32 = 3 };
// how a unit's scale is stored: fp32 [R][K / 128]; E8M0 in the tiled layout, a
// 128-column unit's code in all of its four 32-blocks; E8M0 [R][K / 32]; E8M0
// tiled; the same by the floor rule
enum { kUnitF32 = 0, kUnitPow2 = 1, kUnitMx = 2, kUnitMxTiled = 3, kUnitMxFloor = 4 };
struct RmsCast {
    uint8_t* q;
    int fmt, H;
    float* state;
    int unit;
    void* scales;
};

// mx_scale and mx_scale_floor without their branches.  The exponent that the
// format's largest value 1.75 2^emax leaves is floor(log2 a) - emax, one more
// where a's significand is above 1.75 (add: 2^23 - 1 less that fraction; 0 by the
// floor rule); subnormal maxima end at the lowest code either way.
__device__ __forceinline__ uint32_t e8m0_scale(uint32_t a, uint32_t add, int emax, float& m)
{
    const int code = max((int)((a + add) >> 23) - emax, 0);
    const bool plain = a != 0u && a < 0x7F800000u;
    m = plain ? __uint_as_float((uint32_t)(254 - code) << 23) : 1.0f;
    return plain ? (uint32_t)code : a == 0u ? 127u : 0xFFu;
}
__device__ __forceinline__ void store_e8m0(const RmsCast& cast, uint32_t code, int64_t r, int c, int K)
{
    uint8_t* sc = static_cast<uint8_t*>(cast.scales);
    if (cast.unit == kUnitMx) sc[r * (K / 32) + c / 32] = (uint8_t)code;
    else if (cast.unit == kUnitPow2) *reinterpret_cast<uint32_t*>(sc + mx_tiled_offset(r, c / 32, K)) = code * 0x01010101u;
    else sc[mx_tiled_offset(r, c / 32, K)] = (uint8_t)code;
}
__device__ __forceinline__ float format_max(int fmt) { return fmt == kE4M3 ? Fmt<kE4M3>::fmax : Fmt<kE5M2>::fmax; }
__device__ __forceinline__ uint32_t e8m0_of(const RmsCast& cast, uint32_t a, float& m)
{
    return e8m0_scale(a, cast.unit == kUnitMxFloor ? 0u : 0x1FFFFFu, cast.fmt == kE4M3 ? Fmt<kE4M3>::emax : Fmt<kE5M2>::emax, m);
}
// fp32 units: the step a / fmax or the multiplier fmax / a (as current_scale)
__device__ __forceinline__ float f32_scale(uint32_t a, int fmt, bool step)
{
    const float fm = format_max(fmt), v = __uint_as_float(a);
    return a != 0u && a < 0x7F800000u ? __fdiv_rn(step ? v : fm, step ? fm : v) : 1.0f;
}

// ------------------------------------------------------------------ rows of 16-byte vectors
// A CTA takes one row at a time and holds it in registers as stored (16 columns
// a thread) from the sum to the output, six CTAs of 256 threads an SM, so x and
// the residual are read once.  Next to DRAM the issue slots bound it, so the
// arithmetic is in packed f32x2 instructions, the squares of bf16 are the mixed
// fma (no widening), and a unit's scale costs little: the lanes that hold a unit
// are neighbours (its amax is log2(G) shuffles), each lane works out one of the
// thread's units' scales (fp32: one of their multipliers and steps) and they
// trade them.  One GB300, 16384 x 4096 bf16, us (the bytes at the copy rate): y with
// residual 91 (79), codes in 1x128 tiles with residual 75.6 (69.7; as one more form
// of LayerNorm's kernel 79.2), codes in MX blocks without 49 (30; 64); 4096 x 4096
// fp32 tiles with residual 37.2 (32.3; 38.9).
template <typename T>
struct RmsVec;
template <>
struct RmsVec<__nv_bfloat16> {
    static constexpr int VEC = 8;
    static __device__ __forceinline__ float2 pair(const uint4& w, int j)         // columns 2 j, 2 j + 1
    {
        const uint32_t v = j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w;
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
    static __device__ __forceinline__ void add_square(const uint4& w, float2& acc)
    {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
                "fma.rn.f32.bf16 %0, lo, lo, %0;\n\tfma.rn.f32.bf16 %1, hi, hi, %1;\n\t}"
                : "+f"(acc.x), "+f"(acc.y)
                : "r"(v[j]));
    }
    static __device__ __forceinline__ uint4 pack(const float2 (&v)[4])
    {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[j].x, v[j].y);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct RmsVec<float> {
    static constexpr int VEC = 4;
    static __device__ __forceinline__ float2 pair(const uint4& w, int j)
    {
        return j == 0 ? make_float2(__uint_as_float(w.x), __uint_as_float(w.y))
                      : make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ void add_square(const uint4& w, float2& acc)
    {
#pragma unroll
        for (int j = 0; j < 2; ++j) acc = __ffma2_rn(pair(w, j), pair(w, j), acc);
    }
    static __device__ __forceinline__ uint4 pack(const float2 (&v)[2])
    {
        return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
    }
};
template <int PAIRS>
__device__ __forceinline__ void store_codes(uint8_t* q, const float2 (&v)[PAIRS], float m, int fmt)
{
    uint32_t w[PAIRS / 2];
    auto all = [&](auto cvt) {
#pragma unroll
        for (int j = 0; j < PAIRS / 2; ++j) {
            const float2 a = __fmul2_rn(v[2 * j], f2(m)), b = __fmul2_rn(v[2 * j + 1], f2(m));
            w[j] = cvt(a.x, a.y) | (cvt(b.x, b.y) << 16);
        }
    };
    if (fmt == kE4M3) all([](float a, float b) { return cvt_e4m3x2(a, b); });
    else all([](float a, float b) { return cvt_e5m2x2(a, b); });
    if constexpr (PAIRS == 4) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(q) = w[0];
}

// x, res and sum are not declared free of aliases: sum may be res or x itself (a
// thread reads both where it writes, and before).
template <typename T, int MAXT, int MINB, int CODES>
__global__ void __launch_bounds__(MAXT, MINB)
    k_rms_fwd(const T* x, const T* res, const float* __restrict__ gamma, float eps, int64_t R, int K, T* sum,
              T* __restrict__ y, float* __restrict__ rstd, RmsCast cast)
{
    using V = RmsVec<T>;
    constexpr int VEC = V::VEC, NV = kLnCols / VEC, PAIRS = VEC / 2;
    __shared__ float red[2][32];
    const int t = threadIdx.x, nt = blockDim.x, warp = t >> 5, lane = t & 31, warps = nt >> 5;
    const int span = pow2_span(warps);
    if (t < 32) red[0][t] = red[1][t] = 0.0f;
    __syncthreads();
    pdl_trigger();
    pdl_enter();
    const float m = CODES == kCodesDelayed ? cast.state[cast.H] : 1.0f;
    float amax = 0.0f;
    int par = 0;
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const int64_t base = r * K;
        uint4 raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + t) * VEC;
            raw[i] = c < K ? *reinterpret_cast<const uint4*>(x + base + c) : make_uint4(0, 0, 0, 0);
        }
        if (res) {
            uint4 rr[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * nt + t) * VEC;
                rr[i] = c < K ? *reinterpret_cast<const uint4*>(res + base + c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * nt + t) * VEC;
                float2 v[PAIRS];
#pragma unroll
                for (int j = 0; j < PAIRS; ++j) v[j] = __fadd2_rn(V::pair(raw[i], j), V::pair(rr[i], j));
                raw[i] = V::pack(v);                    // the sum as stored
                if (c < K) *reinterpret_cast<uint4*>(sum + base + c) = raw[i];
            }
        }
        float2 sq = f2(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) V::add_square(raw[i], sq);
        float s = warp_sum(sq.x + sq.y);
        if (warps > 1) {
            // one barrier a row: the rows take the two buffers in turn
            if (lane == 0) red[par][warp] = s;
            __syncthreads();
            s = block_total(red[par], span);
            par ^= 1;
        }
        const float rs = __frsqrt_rn(__fdiv_rn(s, (float)K) + eps);
        if (t == 0 && rstd) rstd[r] = rs;
        float2 v[NV][PAIRS];
        [[maybe_unused]] uint32_t a[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + t) * VEC;
            float g[VEC] = {}, top = 0.0f;
            if (c < K) load_param<VEC>(gamma, c, g);
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                v[i][j] = __fmul2_rn(__fmul2_rn(V::pair(raw[i], j), f2(rs)), make_float2(g[2 * j], g[2 * j + 1]));
                if constexpr (CODES != kNoCodes) top = max3_nan(top, fabsf(v[i][j].x), fabsf(v[i][j].y));
            }
            if (c < K && (CODES == kNoCodes || y)) *reinterpret_cast<uint4*>(y + base + c) = V::pack(v[i]);
            if constexpr (CODES == kCodesDelayed) {
                if (c < K) {
                    amax = max_nan(amax, top);
                    store_codes(cast.q + base + c, v[i], m, cast.fmt);
                }
            }
            if constexpr (CODES >= kCodes128) a[i] = __float_as_uint(top);       // not negative: ordered, a NaN above all
        }
        if constexpr (CODES >= kCodes128) {
            constexpr int G = (CODES == kCodes128 ? 128 : 32) / VEC;             // lanes of a unit
            static_assert(G >= NV && (CODES == kCodes32 || G >= 2 * NV), "a lane for each unit's scale");
#pragma unroll
            for (int o = G / 2; o >= 1; o >>= 1)
#pragma unroll
                for (int i = 0; i < NV; ++i) a[i] = max(a[i], __shfl_xor_sync(0xFFFFFFFFu, a[i], o));
            const int l = lane & (G - 1), first = lane & ~(G - 1);
            const bool f32 = CODES == kCodes128 && cast.unit == kUnitF32;
            const int mine = f32 ? (l >> 1) % NV : l % NV, cm = (mine * nt + t) * VEC;    // the unit whose scale this lane takes
            uint32_t am = a[0];
#pragma unroll
            for (int i = 1; i < NV; ++i) am = mine == i ? a[i] : am;
            float mult;
            if (f32) {
                mult = f32_scale(am, cast.fmt, l & 1);
                if ((l & 1) && l < 2 * NV && cm < K) static_cast<float*>(cast.scales)[r * (K / 128) + cm / 128] = mult;
            } else {
                const uint32_t code = e8m0_of(cast, am, mult);
                if (l < NV && cm < K) store_e8m0(cast, code, r, cm, K);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float mi = __shfl_sync(0xFFFFFFFFu, mult, first + (f32 ? 2 * i : i));
                const int c = (i * nt + t) * VEC;
                if (c < K) store_codes(cast.q + base + c, v[i], mi, cast.fmt);
            }
        }
    }
    if constexpr (CODES == kCodesDelayed) record_amax(amax, cast.state);
}

// ------------------------------------------------------------------ long rows
// Rows beyond what a CTA holds in registers: one row a CTA at a time, its
// elements read again after the sum (from L2 as a rule).  A warp takes 128
// columns at a time, a lane four of them, so a unit's lanes are neighbours.
template <typename T>
__global__ void __launch_bounds__(256) k_rms_fwd_any(const T* x, const T* res, const float* __restrict__ gamma,
                                                     float eps, int64_t R, int64_t K, T* sum, T* __restrict__ y,
                                                     float* __restrict__ rstd, RmsCast cast, int unit_cols)
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
        const float rs = __frsqrt_rn(__fdiv_rn(cta_sum(s, red), (float)K) + eps);
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
                const bool first = c < K && (lane & (unit_cols / 4 - 1)) == 0;
                if (cast.unit == kUnitF32) {
                    mult = f32_scale(a, cast.fmt, false);
                    if (first) static_cast<float*>(cast.scales)[r * (K / 128) + c / 128] = f32_scale(a, cast.fmt, true);
                } else {
                    const uint32_t code = e8m0_of(cast, a, mult);
                    if (first) store_e8m0(cast, code, r, (int)c, (int)K);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < K) cast.q[r * K + c + j] = code1(__fmul_rn(v[j], mult), cast.fmt);
        });
    }
    if (delayed) record_amax(amax, cast.state);
}

template <typename T, int MAXT, int MINB, int CODES>
cudaError_t rms_fwd_cta(const LnArgs& a, const RmsCast& cast, cudaStream_t st, int sms, int threads)
{
    auto kern = k_rms_fwd<T, MAXT, MINB, CODES>;
    const int64_t cap = resident(reinterpret_cast<const void*>(kern), threads, 0, sms);
    launch_k(kern, (unsigned)(a.M < cap ? a.M : cap), threads, 0, st, static_cast<const T*>(a.x),
             static_cast<const T*>(a.residual), a.gamma, a.eps, a.M, (int)a.K, static_cast<T*>(a.sum), static_cast<T*>(a.y),
             a.rstd, cast);
    return cudaGetLastError();
}
template <typename T, int CODES>
cudaError_t rms_fwd_rows(const LnArgs& a, const RmsCast& cast, cudaStream_t st, int sms)
{
    const int threads = 32 * (int)cdiv(a.K, 32 * kLnCols);
    if (threads <= 256) return rms_fwd_cta<T, 256, 6, CODES>(a, cast, st, sms, threads);
    if (threads <= 512) return rms_fwd_cta<T, 512, 3, CODES>(a, cast, st, sms, threads);
    if (threads <= 768) return rms_fwd_cta<T, 768, 2, CODES>(a, cast, st, sms, threads);
    return rms_fwd_cta<T, 1024, 1, CODES>(a, cast, st, sms, threads);
}

template <typename T>
cudaError_t rms_fwd(const LnArgs& a, cudaStream_t st, int sms)
{
    const int unit = !a.q || a.q_gran == kTensor ? 0 : a.q_gran == kTile || a.q_gran == kTilePow2 ? 128 : 32;
    const int store = a.q_gran == kTilePow2  ? kUnitPow2
                      : a.q_gran == kMX      ? kUnitMx
                      : a.q_gran == kMXTiled ? kUnitMxTiled
                      : a.q_gran == kMXFloor ? kUnitMxFloor
                                             : kUnitF32;
    const RmsCast cast{a.q, a.q_format, a.q_history_len, a.q_state, store, a.q_scales};
    if (a.K <= 1024 * kLnCols) {
        if (unit == 128) return rms_fwd_rows<T, kCodes128>(a, cast, st, sms);       // (K % 128 == 0)
        if (unit == 32) return rms_fwd_rows<T, kCodes32>(a, cast, st, sms);
        if (a.K % (16 / (int)sizeof(T)) == 0)
            return a.q ? rms_fwd_rows<T, kCodesDelayed>(a, cast, st, sms) : rms_fwd_rows<T, kNoCodes>(a, cast, st, sms);
        return a.q ? ln_fwd_vec<T, true, true>(a, st, sms) : ln_fwd_vec<T, false, true>(a, st, sms);
    }
    const int64_t cap = (int64_t)sms * 8;
    launch_k(k_rms_fwd_any<T>, (unsigned)(a.M < cap ? a.M : cap), 256, 0, st, static_cast<const T*>(a.x),
             static_cast<const T*>(a.residual), a.gamma, a.eps, a.M, a.K, static_cast<T*>(a.sum), static_cast<T*>(a.y),
             a.rstd, cast, unit);
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
