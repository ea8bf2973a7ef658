// rowvec.cuh -- pieces shared by the row-wise kernels: elements and vectors of a
// row as fp32, sums over a warp or a CTA, single codes, the recorded amax.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "internal.h"
#include "ptx.cuh"

namespace fp8sq {

namespace {

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

__device__ __forceinline__ uint8_t code1(float v, int fmt)
{
    return (uint8_t)(fmt == kE4M3 ? cvt_e4m3x2(v, 0.0f) : cvt_e5m2x2(v, 0.0f));
}
// a warp's largest |value| into a state's newest amax: not negative, so ordered
// as integers, a NaN above everything
__device__ __forceinline__ void record_amax(float amax, float* state)
{
    const uint32_t a = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax));
    if ((threadIdx.x & 31) == 0) atomicMax(reinterpret_cast<unsigned int*>(state), a);
}

// ------------------------------------------------------------------ vectors
// VEC consecutive elements of T as floats.  ALIGNED vectors are 16, 8, 4 or 2
// bytes: the widest that divides a row.
template <int BYTES>
struct RawVec;
template <>
struct RawVec<16> { using type = uint4; };
template <>
struct RawVec<8> { using type = uint2; };
template <>
struct RawVec<4> { using type = uint32_t; };
template <>
struct RawVec<2> { using type = uint16_t; };

template <typename T, int VEC>
struct Pack {
    using Raw = typename RawVec<sizeof(T) * VEC>::type;
    static constexpr bool PAIRS = sizeof(T) == 2 && VEC % 2 == 0;    // bf16 pairs in 32-bit words
    static __device__ __forceinline__ void to_floats(const Raw& raw, float (&v)[VEC])
    {
        if constexpr (PAIRS) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
            for (int j = 0; j < VEC; j += 2) {
                v[j] = __uint_as_float(w[j / 2] << 16);
                v[j + 1] = __uint_as_float(w[j / 2] & 0xFFFF0000u);
            }
        } else {
            const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = to_f(e[j]);
        }
    }
    static __device__ __forceinline__ Raw from_floats(const float (&v)[VEC])
    {
        Raw raw;
        if constexpr (PAIRS) {
            __nv_bfloat162* w = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
            for (int j = 0; j < VEC; j += 2) w[j / 2] = __floats2bfloat162_rn(v[j], v[j + 1]);
        } else {
            T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
            for (int j = 0; j < VEC; ++j) e[j] = from_f<T>(v[j]);
        }
        return raw;
    }
};
// fp32 parameters of VEC consecutive columns
template <int VEC>
__device__ __forceinline__ void load_param(const float* __restrict__ p, int c, float (&v)[VEC])
{
    if constexpr (VEC == 2) {
        const float2 w = __ldg(reinterpret_cast<const float2*>(p + c));
        v[0] = w.x;
        v[1] = w.y;
    } else if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
            const float4 w = __ldg(reinterpret_cast<const float4*>(p + c + j));
            v[j] = w.x;
            v[j + 1] = w.y;
            v[j + 2] = w.z;
            v[j + 3] = w.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = __ldg(p + c + j);
    }
}
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// CTAs of a kernel that are resident at once.  The answers are kept: the query
// took over a microsecond of every call.
int resident(const void* kern, int threads, int smem, int sms)
{
    struct Entry {
        const void* kern;
        int threads, smem, dev, per_sm;
    };
    static std::mutex mu;
    static Entry known[256];
    static int n = 0;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < n; ++i)
        if (known[i].kern == kern && known[i].threads == threads && known[i].smem == smem && known[i].dev == dev)
            return known[i].per_sm * sms;
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem) != cudaSuccess || per_sm < 1) {
        cudaGetLastError();
        return sms;
    }
    if (n < 256) known[n++] = {kern, threads, smem, dev, per_sm};
    return per_sm * sms;
}

}  // namespace

}  // namespace fp8sq
