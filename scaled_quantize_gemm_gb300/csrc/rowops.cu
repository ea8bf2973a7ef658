// rowops.cu -- row-wise and elementwise operators around the FP8 linear:
// LayerNorm forward and backward (norm.cuh), and the backward pass of an
// activation with its bias gradient and FP8 cast.  All arithmetic and every sum
// is fp32.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act.cuh"
#include "internal.h"
#include "norm.cuh"
#include "ptx.cuh"

namespace fp8sq {

namespace {

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
                float2 f2_, d2;
                act_fd2<decltype(tag)::act>(f2(to_f(z[r * N + c])), f2_, d2);
                float d = __fmul_rn(d2.x, to_f(dy[r * N + c]));   // dz itself is summed, whatever else is stored
                sum += d;
                if (dz) dz[r * N + c] = __float2bfloat16_rn(d);
                if (q) {
                    amax = max(amax, __float_as_uint(d) & 0x7FFFFFFFu);
                    const float v = __fmul_rn(d, m);
                    q[r * N + c] = code1(v, fmt);
                }
            }
        });
    if (part && c < N) part[(int64_t)blockIdx.y * N + c] = sum;
    if (q) {
        amax = __reduce_max_sync(0xFFFFFFFFu, amax);
        if ((threadIdx.x & 31) == 0) atomicMax(reinterpret_cast<unsigned int*>(qstate), amax);
    }
}

// ------------------------------------------------------------------ activation backward
// Rows of a multiple of 8 elements: a warp takes 256 columns (8 a lane) and
// the CTA's eight warps every eighth row of its slab, the loads two of its rows
// ahead; the eight warps' column sums are added through shared memory in warp
// order.  DRAM-bound next to the issue slots and the two hardware functions an
// element: 16384 x 14336, gelu_tanh, codes and dbias: 200 us, 5.9 TB/s.  Five
// CTAs an SM: four 206, six 251 (spills); loads three rows ahead 284 (spills);
// without the run-time tests of a bf16 dz (ONLYQ) 5 us less.
constexpr int kActCols = 256;
template <int ACT, bool ONLYQ>
__device__ __forceinline__ void act_bwd_rows(const __nv_bfloat16* __restrict__ dy, const __nv_bfloat16* __restrict__ z,
                                             int64_t r0, int64_t r1, int64_t N, int64_t c, __nv_bfloat16* __restrict__ dz,
                                             uint8_t* __restrict__ q, int fmt, float m, float2 (&sum)[4], float& amax)
{
    // the loads run two of the warp's rows ahead of the arithmetic
    constexpr int AHEAD = 2;
    uint4 zn[AHEAD], dn[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (r0 + 8 * i < r1) {
            zn[i] = __ldcs(reinterpret_cast<const uint4*>(z + (r0 + 8 * i) * N + c));
            dn[i] = __ldcs(reinterpret_cast<const uint4*>(dy + (r0 + 8 * i) * N + c));
        }
    for (int64_t r = r0; r < r1; r += 8) {
        const uint4 zr = zn[0], dr = dn[0];
#pragma unroll
        for (int i = 0; i + 1 < AHEAD; ++i) {
            zn[i] = zn[i + 1];
            dn[i] = dn[i + 1];
        }
        if (r + 8 * AHEAD < r1) {
            zn[AHEAD - 1] = __ldcs(reinterpret_cast<const uint4*>(z + (r + 8 * AHEAD) * N + c));
            dn[AHEAD - 1] = __ldcs(reinterpret_cast<const uint4*>(dy + (r + 8 * AHEAD) * N + c));
        }
        const uint32_t zw[4] = {zr.x, zr.y, zr.z, zr.w}, dw[4] = {dr.x, dr.y, dr.z, dr.w};
        float2 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 f, d;
            act_fd2<ACT>(make_float2(__uint_as_float(zw[j] << 16), __uint_as_float(zw[j] & 0xFFFF0000u)), f, d);
            v[j] = __fmul2_rn(d, make_float2(__uint_as_float(dw[j] << 16), __uint_as_float(dw[j] & 0xFFFF0000u)));
            sum[j] = __fadd2_rn(sum[j], v[j]);
        }
        if (!ONLYQ && dz) {
            float w[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[2 * j] = v[j].x;
                w[2 * j + 1] = v[j].y;
            }
            *reinterpret_cast<uint4*>(dz + r * N + c) = Pack<__nv_bfloat16, 8>::from_floats(w);
        }
        if (ONLYQ || q) {
            uint32_t w[2];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                amax = max3_nan(amax, fabsf(v[j].x), fabsf(v[j].y));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 a = __fmul2_rn(v[2 * j], f2(m)), b = __fmul2_rn(v[2 * j + 1], f2(m));
                w[j] = fmt == kE4M3 ? (cvt_e4m3x2(a.x, a.y) | (cvt_e4m3x2(b.x, b.y) << 16))
                                    : (cvt_e5m2x2(a.x, a.y) | (cvt_e5m2x2(b.x, b.y) << 16));
            }
            *reinterpret_cast<uint2*>(q + r * N + c) = make_uint2(w[0], w[1]);
        }
    }
}

__global__ void __launch_bounds__(256, 5) k_act_bwd(const __nv_bfloat16* __restrict__ dy,
                                                    const __nv_bfloat16* __restrict__ z, int act, int64_t R, int64_t N,
                                                    int64_t slab, __nv_bfloat16* __restrict__ dz,
                                                    uint8_t* __restrict__ q, int fmt, float* qstate, int H,
                                                    float* __restrict__ part)
{
    pdl_enter();
    __shared__ float2 cols[8][4][32];
    __shared__ uint32_t red[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * kActCols + 8 * lane;
    const int64_t r0 = (int64_t)blockIdx.y * slab;
    const int64_t r1 = r0 + slab < R ? r0 + slab : R;
    const float m = q ? qstate[H] : 1.0f;
    float2 sum[4] = {};
    float amax_f = 0.0f;
    if (c < N)
        act_dispatch(act, [&](auto tag) {
            if (q && !dz) act_bwd_rows<decltype(tag)::act, true>(dy, z, r0 + warp, r1, N, c, dz, q, fmt, m, sum, amax_f);
            else act_bwd_rows<decltype(tag)::act, false>(dy, z, r0 + warp, r1, N, c, dz, q, fmt, m, sum, amax_f);
        });
    if (part) {
#pragma unroll
        for (int j = 0; j < 4; ++j) cols[warp][j][lane] = sum[j];
    }
    uint32_t amax = __float_as_uint(amax_f);     // not negative: ordered as integers, a NaN above all
    if (q) {
        amax = __reduce_max_sync(0xFFFFFFFFu, amax);
        if (lane == 0) red[warp] = amax;
    }
    __syncthreads();
    if (part && warp < 4 && c < N) {         // warp j adds pair j of every lane's columns
        float2 s = cols[0][warp][lane];
#pragma unroll
        for (int w = 1; w < 8; ++w) s = __fadd2_rn(s, cols[w][warp][lane]);
        *reinterpret_cast<float2*>(part + (int64_t)blockIdx.y * N + c + 2 * warp) = s;
    }
    if (q && threadIdx.x == 0) {
#pragma unroll
        for (int w = 0; w < 8; ++w) amax = max(amax, red[w]);
        atomicMax(reinterpret_cast<unsigned int*>(qstate), amax);
    }
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
    return a.dtype == kBF16 ? ln_bwd<__nv_bfloat16, false>(a, st, sms) : ln_bwd<float, false>(a, st, sms);
}

cudaError_t launch_act_bwd(const ActBwdArgs& a, cudaStream_t st, int sms)
{
    if (a.N == 0) return cudaSuccess;
    float* part = a.dbias ? static_cast<float*>(a.workspace) : nullptr;
    int parts = 0;
    if (a.M > 0 && a.N % 8 == 0) {
        // slabs of rows: about four waves of CTAs, at least 8 rows each
        const int64_t blocks = cdiv(a.N, kActCols);
        int64_t slabs = 4 * (int64_t)resident(reinterpret_cast<const void*>(k_act_bwd), 256, 0, sms) / blocks;
        const int64_t most = cdiv(a.M, 8) < kMaxParts ? cdiv(a.M, 8) : kMaxParts;
        slabs = slabs < 1 ? 1 : slabs < most ? slabs : most;
        const int64_t slab = cdiv(cdiv(a.M, slabs), 8) * 8;
        parts = (int)cdiv(a.M, slab);
        launch_k(k_act_bwd, dim3((unsigned)blocks, parts), 256, 0, st, static_cast<const __nv_bfloat16*>(a.dy),
                 static_cast<const __nv_bfloat16*>(a.z), a.act, a.M, a.N, slab, static_cast<__nv_bfloat16*>(a.dz), a.q,
                 a.q_format, a.q_state, a.q_history_len, part);
    } else if (a.M > 0) {
        parts = (int)parts_for(a.M);
        launch_k(k_act_bwd_any, dim3((unsigned)cdiv(a.N, 256), parts), 256, 0, st,
                 static_cast<const __nv_bfloat16*>(a.dy), static_cast<const __nv_bfloat16*>(a.z), a.act, a.M, a.N,
                 static_cast<__nv_bfloat16*>(a.dz), a.q, a.q_format, a.q_state, a.q_history_len, part);
    }
    if (a.dbias)
        launch_k(k_col_reduce, (unsigned)cdiv(a.N, 32), 1024, 0, st, (const float*)part, parts, a.N, a.dbias, a.N,
                 (float*)nullptr);
    return cudaGetLastError();
}

}  // namespace fp8sq
