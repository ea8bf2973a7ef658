// norm.cuh -- LayerNorm and RMSNorm, forward and backward, and the second stage
// of column sums.  All arithmetic and every sum is fp32.  RMS selects the norm
// without a mean: rstd = 1 / sqrt(sum(x^2) / K + eps), y = x rstd gamma.
//
// Column sums (dgamma, dbeta, dbias) run in two stages: a CTA sums the rows it
// owns in registers and writes one partial row per sum to the workspace, then
// k_col_reduce adds the partials in index order, so a result does not depend
// on the order in which CTAs run.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace fp8sq {

namespace {

constexpr int kMaxParts = 608;      // partial rows of a column sum

int64_t parts_for(int64_t rows) { return rows < kMaxParts ? rows : kMaxParts; }

// ------------------------------------------------------------------ any row length
template <typename T>
__global__ void __launch_bounds__(256) k_ln_fwd_any(const T* x, const T* res, const float* __restrict__ gamma,
                                                    const float* __restrict__ beta, float eps, int64_t R, int64_t K,
                                                    T* sum, T* __restrict__ y, float* __restrict__ mu,
                                                    float* __restrict__ rstd, uint8_t* __restrict__ q, int fmt,
                                                    float* qstate, int H)
{
    pdl_enter();
    __shared__ float red[8];
    const float m = q ? qstate[H] : 1.0f;
    float amax = 0.0f;
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
        for (int64_t c = threadIdx.x; c < K; c += 256) {
            const float v = fmaf((to_f(xr[c]) - mean) * rs, gamma[c], beta ? beta[c] : 0.0f);
            if (y) y[r * K + c] = from_f<T>(v);
            if (q) {
                amax = max_nan(amax, fabsf(v));
                q[r * K + c] = code1(__fmul_rn(v, m), fmt);
            }
        }
    }
    if (q) record_amax(amax, qstate);
}

template <typename T, bool RMS>
__global__ void __launch_bounds__(256) k_ln_bwd_dx_any(const T* __restrict__ dy, const T* __restrict__ x,
                                                       const T* __restrict__ dres, const float* __restrict__ gamma,
                                                       const float* __restrict__ mu, const float* __restrict__ rstd,
                                                       int64_t R, int64_t K, T* __restrict__ dx)
{
    pdl_enter();
    __shared__ float red[8];
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const float mean = RMS ? 0.0f : mu[r], rs = rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < K; c += 256) {
            const float w = to_f(dy[r * K + c]) * gamma[c];
            s1 += w;
            s2 = fmaf(w, (to_f(x[r * K + c]) - mean) * rs, s2);
        }
        const float c1 = RMS ? 0.0f : cta_sum(s1, red) / (float)K, c2 = cta_sum(s2, red) / (float)K;
        for (int64_t c = threadIdx.x; c < K; c += 256) {
            const float w = to_f(dy[r * K + c]) * gamma[c];
            float v = rs * (w - c1 - (to_f(x[r * K + c]) - mean) * rs * c2);
            if (dres) v += to_f(dres[r * K + c]);
            dx[r * K + c] = from_f<T>(v);
        }
    }
}

// partial dgamma (row 2 p) and dbeta (row 2 p + 1) of the rows of part p; RMS:
// dgamma alone (row p)
template <typename T, bool RMS>
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
        g = fmaf(d, (to_f(x[r * K + c]) - (RMS ? 0.0f : mu[r])) * rstd[r], g);
        b += d;
    }
    part[((RMS ? 1 : 2) * (int64_t)blockIdx.y) * K + c] = g;
    if (!RMS) part[(2 * (int64_t)blockIdx.y + 1) * K + c] = b;
}

// out0[c] = sum over p of part[p][c] for c < n0, out1[c - n0] for the rest
// (rows of n columns); a CTA takes 32 columns, each of its 32 warps every 32nd
// part, and the warps' sums are added in a fixed order
__global__ void __launch_bounds__(1024) k_col_reduce(const float* __restrict__ part, int parts, int64_t n,
                                                     float* __restrict__ out0, int64_t n0, float* __restrict__ out1)
{
    pdl_enter();
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float a = 0.0f;
    if (c < n) {
#pragma unroll 8
        for (int p = w; p < parts; p += 32) a += __ldcs(part + (int64_t)p * n + c);
    }
    s[w][lane] = a;
    __syncthreads();
    // warp w takes column w: its lanes hold the 32 partial sums
    const float v = warp_sum(s[lane][w]);
    const int64_t cw = (int64_t)blockIdx.x * 32 + w;
    if (lane == 0 && cw < n) {
        if (cw < n0) out0[cw] = v;
        else out1[cw - n0] = v;
    }
}

// Sum of `red`, one float a warp, zeros up to the power of two `span` >= warps:
// every lane reads one entry and log2(span) shuffles leave the same total in
// all of them.  `red` is not written again before another barrier.
__device__ __forceinline__ int pow2_span(int warps) { return warps <= 1 ? 1 : 1 << (32 - __clz(warps - 1)); }
__device__ __forceinline__ float block_total(const float* red, int span)
{
    float v = red[threadIdx.x & (span - 1)];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        if (o < span) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// Two sums at once: lanes 0-15 end with the first's total, lanes 16-31 with the
// second's (one exchange, then four shuffles instead of ten).
__device__ __forceinline__ float warp_sum2(float a, float b)
{
    const bool hi = threadIdx.x & 16;
    float v = hi ? b : a;
    v += __shfl_xor_sync(0xFFFFFFFFu, hi ? a : b, 16);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// Two sums of one float a warp each (red[0], red[1]) over up to 32 warps, in
// every lane: the halves of a warp take one each.
__device__ __forceinline__ float2 block_total2(const float (*red)[32], int span)
{
    const float* r = red[(threadIdx.x >> 4) & 1];
    float v = r[threadIdx.x & 15 & (span - 1)];
    if (span == 32) v += r[16 + (threadIdx.x & 15)];
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1)
        if (o < span) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return make_float2(__shfl_sync(0xFFFFFFFFu, v, 0), __shfl_sync(0xFFFFFFFFu, v, 16));
}

// ------------------------------------------------------------------ LayerNorm forward
// A CTA takes one row at a time and holds it in registers (16 columns a
// thread, as stored) from the sum to the output, so x and the residual are
// read once and y (and the sum) written once; no row is prefetched, the loads
// of a CTA's row overlap the reductions of the others on its SM: MINB CTAs of
// at most MAXT threads, 1536 threads (six CTAs at 4096 columns: 82 us for 16384
// rows in bf16 with residual, 96 % of the copy rate; four 93, eight 105).
constexpr int kLnCols = 16;         // columns a thread holds
// sum may be res or x itself (a thread reads both where it writes, and before),
// so none of the three is declared free of aliases.
// CODES: y also (or only) as FP8 codes under a delayed state, cast from fp32.
// RMS: no mean, one sum a row (rows of whole 16-byte vectors: rmsnorm.cu).
struct LnCast {
    uint8_t* q;
    int fmt, H;
    float* state;
};
template <typename T, int VEC, int MAXT, int MINB, bool CODES, bool RMS>
__global__ void __launch_bounds__(MAXT, MINB)
    k_ln_fwd(const T* x, const T* res, const float* __restrict__ gamma, const float* __restrict__ beta, float eps,
             int64_t R, int K, T* sum, T* __restrict__ y, float* __restrict__ mu, float* __restrict__ rstd, LnCast cast)
{
    constexpr int NV = kLnCols / VEC;
    using P = Pack<T, VEC>;
    using Raw = typename P::Raw;
    __shared__ float red[2][32];
    const int t = threadIdx.x, nt = blockDim.x, warp = t >> 5, warps = nt >> 5;
    const int span = pow2_span(warps);
    if (t < 64) red[t >> 5][t & 31] = 0.0f;
    if (nt < 64 && t < 32) red[1][t] = 0.0f;
    __syncthreads();
    pdl_trigger();
    pdl_enter();
    const float m = CODES ? cast.state[cast.H] : 1.0f;
    float amax = 0.0f;
    [[maybe_unused]] int par = 0;
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const int64_t base = r * K;
        Raw raw[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + t) * VEC;
            raw[i] = c < K ? *reinterpret_cast<const Raw*>(x + base + c) : Raw{};
        }
        if (res) {
            Raw rr[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * nt + t) * VEC;
                rr[i] = c < K ? *reinterpret_cast<const Raw*>(res + base + c) : Raw{};
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * nt + t) * VEC;
                float v[VEC], w[VEC];
                P::to_floats(raw[i], v);
                P::to_floats(rr[i], w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[j] += w[j];
                raw[i] = P::from_floats(v);             // the sum as stored
                if (c < K) *reinterpret_cast<Raw*>(sum + base + c) = raw[i];
            }
        }
        float s = 0.0f, mean = 0.0f;
        if constexpr (!RMS) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[VEC];
                P::to_floats(raw[i], v);
#pragma unroll
                for (int j = 0; j < VEC; ++j) s += v[j];
            }
            s = warp_sum(s);
            if (warps > 1) {
                if ((t & 31) == 0) red[0][warp] = s;
                __syncthreads();
                s = block_total(red[0], span);
            }
            mean = s / (float)K;
            s = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((i * nt + t) * VEC >= K) continue;
            float v[VEC];
            P::to_floats(raw[i], v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if constexpr (!RMS) v[j] -= mean;
                s = fmaf(v[j], v[j], s);
            }
        }
        s = warp_sum(s);
        if (warps > 1) {
            // (one barrier a row in RMS: the rows take the two in turn)
            float* rd = red[RMS ? par : 1];
            if ((t & 31) == 0) rd[warp] = s;
            __syncthreads();
            s = block_total(rd, span);
            if constexpr (RMS) par ^= 1;
        }
        const float rs = 1.0f / sqrtf(s / (float)K + eps);
        if (t == 0) {
            if (mu) mu[r] = mean;
            if (rstd) rstd[r] = rs;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + t) * VEC;
            if (c >= K) continue;
            float v[VEC], g[VEC], b[VEC] = {};
            P::to_floats(raw[i], v);
            load_param<VEC>(gamma, c, g);
            if constexpr (RMS) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[j] = v[j] * rs * g[j];
            } else {
                if (beta) load_param<VEC>(beta, c, b);
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[j] = fmaf((v[j] - mean) * rs, g[j], b[j]);
            }
            if (!CODES || y) *reinterpret_cast<Raw*>(y + base + c) = P::from_floats(v);
            if constexpr (CODES) {
                uint8_t* q = cast.q + base + c;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    amax = max_nan(amax, fabsf(v[j]));
                    v[j] = __fmul_rn(v[j], m);
                }
                if constexpr (VEC >= 2) {
                    uint16_t h[VEC / 2];
#pragma unroll
                    for (int j = 0; j < VEC; j += 2)
                        h[j / 2] = (uint16_t)(cast.fmt == kE4M3 ? cvt_e4m3x2(v[j], v[j + 1]) : cvt_e5m2x2(v[j], v[j + 1]));
                    if constexpr (VEC == 8)
                        *reinterpret_cast<uint2*>(q) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
                    else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(q) = h[0] | (uint32_t)h[1] << 16;
                    else *reinterpret_cast<uint16_t*>(q) = h[0];
                } else {
                    *q = code1(v[0], cast.fmt);
                }
            }
        }
    }
    if constexpr (CODES) record_amax(amax, cast.state);
}

// ------------------------------------------------------------------ LayerNorm backward
// A group of threads takes a row at a time and each thread the same C columns
// of every row, so dgamma and dbeta accumulate in its registers; a CTA holds
// one group, or several for short rows, whose sums meet in shared memory at the
// end, and writes one partial row to the workspace.  x, dy and dres of the next
// STAGES - 1 rows are in flight while a row is worked on, and a row costs one
// barrier of its group, for its two sums.  Rows of whole 16-byte vectors: a
// thread copies (cp.async) exactly the elements that it will read, so the ring
// needs no barrier.  Other rows (BULK): one thread copies each whole, with the
// 16-byte blocks it begins and ends in, and a stage is free again after the
// next row's barrier (16-byte copies whatever the rows' alignment; one element
// or vector at a time by cp.async, and 8 columns a thread: 2051 x 1535 fp32 17.0
// -> 12.8 us, 3000 x 5001 bf16 80.5 -> 36.8, 1198 x 9849 bf16 148 -> 42, 3000 x 5002
// 39.7 -> 31.8).
// The time goes with the instructions a row costs beside its elements (ncu at
// 16384 x 4096 with 8 columns a thread: 40 instructions an element, issue slots
// 59 % busy, DRAM 53 %), so a thread takes 16 columns: 119 -> 93 us.  KEEP holds
// the row's normalised values and dy gamma in registers across the barrier
// (rows of up to 12288; longer ones read the ring again).
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bar_group(int id, int threads)
{
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
constexpr int kLnGroups = 8;        // groups of a CTA, at most
// room of a row in the ring with the 16-byte blocks it begins and ends in
__host__ __device__ constexpr int ln_row_bytes(int K, int size) { return (K * size + 30) & ~15; }

// RMS: no mean, one sum a row and no dbeta, and a CTA takes neighbouring rows
// (every gridDim.x-th row, as LayerNorm has it, 16384 x 4096 bf16 with dres 102
// us, 8192 x 8192 116; neighbours 85.6 and 86.3; LayerNorm itself 85.4 and 89.2
// against 89.2 and 92.0).
template <typename T, int VEC, int C, int STAGES, int MAXT, int MINB, bool KEEP, bool GROUPED, bool RMS>
__global__ void __launch_bounds__(MAXT, MINB)
    k_ln_bwd(const T* __restrict__ dy, const T* __restrict__ x, const T* __restrict__ dres,
             const float* __restrict__ gamma, const float* __restrict__ mu, const float* __restrict__ rstd, int64_t R,
             int K, int group_threads, T* __restrict__ dx, float* __restrict__ part, int* err)
{
    constexpr int NV = C / VEC;
    constexpr bool BULK = VEC * sizeof(T) < 16;
    using P = Pack<T, VEC>;
    using Raw = typename P::Raw;
    extern __shared__ __align__(16) uint8_t ln_ring[];
    constexpr int RG = GROUPED ? kLnGroups : 1;
    __shared__ float red[RG][2][2][32];
    __shared__ uint64_t full[RG][STAGES];               // BULK: a stage's rows have arrived
    const int nt = GROUPED ? group_threads : blockDim.x, g = GROUPED ? threadIdx.x / nt : 0, t = threadIdx.x - g * nt;
    const int groups = GROUPED ? blockDim.x / nt : 1, warp = t >> 5, warps = nt >> 5;
    const int span = pow2_span(warps);
    for (int i = threadIdx.x; i < RG * 128; i += blockDim.x) (&red[0][0][0][0])[i] = 0.0f;
    if (BULK && threadIdx.x == 0) {
        for (int i = 0; i < RG * STAGES; ++i) mbar_init(&full[0][0] + i, 1);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_enter();
    const int narr = dres ? 3 : 2;
    // the CTA's rows: every gridDim.x-th, or (RMS) a run of neighbours
    const int64_t per = (R + gridDim.x - 1) / gridDim.x;
    const int64_t from = RMS ? blockIdx.x * per : (int64_t)blockIdx.x * groups;
    const int64_t end = RMS && from + per < R ? from + per : R;
    // [stage][array][vector i][thread]
    Raw* ring = reinterpret_cast<Raw*>(ln_ring) + threadIdx.x;
    auto slot = [&](int st, int arr, int i) -> Raw* { return ring + ((st * narr + arr) * NV + i) * blockDim.x; };
    // BULK: [group][stage][array][row_bytes], a row with the 16-byte blocks it
    // begins and ends in; of the last rows only the blocks inside the array,
    // the elements after those one by one
    const int row_bytes = ln_row_bytes(K, sizeof(T));
    const int64_t whole = (R * K * (int)sizeof(T)) & ~(int64_t)15;
    auto row = [&](int st, int arr) { return ln_ring + ((g * STAGES + st) * narr + arr) * row_bytes; };
    auto stage = [&](int st, int64_t r) {
        if constexpr (BULK) {
            if (t == 0 && r < end) {
                const int64_t from = r * K * (int)sizeof(T), a0 = from & ~(int64_t)15;
                int64_t a1 = (from + K * (int)sizeof(T) + 15) & ~(int64_t)15;
                if (a1 > whole) a1 = whole;
                const uint32_t n = a1 > a0 ? (uint32_t)(a1 - a0) : 0u;
                int c = (int)((a0 + n - from) / (int)sizeof(T));
                for (c = c > 0 ? c : 0; c < K; ++c) {
                    const int to = (int)(from - a0) + c * (int)sizeof(T);
                    *reinterpret_cast<T*>(row(st, 0) + to) = x[r * K + c];
                    *reinterpret_cast<T*>(row(st, 1) + to) = dy[r * K + c];
                    if (dres) *reinterpret_cast<T*>(row(st, 2) + to) = dres[r * K + c];
                }
                mbar_arrive_expect_tx(&full[g][st], n * narr);
                if (n) {
                    bulk_load_1d(row(st, 0), reinterpret_cast<const char*>(x) + a0, n, &full[g][st]);
                    bulk_load_1d(row(st, 1), reinterpret_cast<const char*>(dy) + a0, n, &full[g][st]);
                    if (dres) bulk_load_1d(row(st, 2), reinterpret_cast<const char*>(dres) + a0, n, &full[g][st]);
                }
            }
        } else {
            if (r < end) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (i * nt + t) * VEC;
                    if (c < K) {
                        const int64_t at = r * K + c;
                        cp_async16(slot(st, 0, i), x + at);
                        cp_async16(slot(st, 1, i), dy + at);
                        if (dres) cp_async16(slot(st, 2, i), dres + at);
                    }
                }
            }
            cp_async_commit();
        }
    };
    // BULK: the thread's columns are t, t + nt, ...: the first `own` of C are in the row
    const int own = K / VEC > t ? (K / VEC - t + nt - 1) / nt : 0;
    // columns past K hold zeros in every array, so they add nothing
    auto fetch = [&](int st, int arr, int64_t r, float2 (&v)[C / 2]) {
        float f[NV][VEC];
        if constexpr (BULK) {
            const int64_t from = r * K * (int)sizeof(T);
            const uint8_t* p = row(st, arr) + ((int)from & 15) + t * (int)sizeof(Raw);
            const int hop = nt * (int)sizeof(Raw);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                Raw raw{};
                if (i < own) raw = *reinterpret_cast<const Raw*>(p);
                p += hop;
                P::to_floats(raw, f[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * nt + t) * VEC;
                P::to_floats(c < K ? *slot(st, arr, i) : Raw{}, f[i]);
            }
        }
#pragma unroll
        for (int j = 0; j < C / 2; ++j)
            v[j] = make_float2(f[(2 * j) / VEC][(2 * j) % VEC], f[(2 * j + 1) / VEC][(2 * j + 1) % VEC]);
    };
    auto params = [&](float2 (&v)[C / 2]) {
        float f[NV][VEC] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * nt + t) * VEC < K) load_param<VEC>(gamma, (i * nt + t) * VEC, f[i]);
#pragma unroll
        for (int j = 0; j < C / 2; ++j)
            v[j] = make_float2(f[(2 * j) / VEC][(2 * j) % VEC], f[(2 * j + 1) / VEC][(2 * j + 1) % VEC]);
    };
    constexpr bool GREG = KEEP && MAXT <= 512;      // gamma in registers as well
    float2 ag[C / 2] = {}, ab[C / 2] = {}, gam[C / 2];
    if constexpr (GREG) params(gam);
    const int64_t first = from + g, step = (RMS ? 1 : (int64_t)gridDim.x) * groups;
    constexpr int AHEAD = BULK && STAGES == 1 ? 1 : STAGES - 1;          // rows in flight before the first
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) stage(s, first + s * step);
    int st = 0, par = 0;
    uint32_t phase = 0;
    const float inv = 1.0f / (float)K;
    float mean = 0.0f, rs = 0.0f;
    if (first < end) {
        if constexpr (!RMS) mean = __ldg(mu + first);
        rs = __ldg(rstd + first);
    }
    for (int64_t r = first; r < end; r += step) {
        int ahead = st + STAGES - 1;
        if (ahead >= STAGES) ahead -= STAGES;
        if constexpr (!BULK) stage(ahead, r + (STAGES - 1) * step);
        const int64_t rn = r + step < end ? r + step : r;
        const float mean_n = RMS ? 0.0f : __ldg(mu + rn), rs_n = __ldg(rstd + rn);
        if constexpr (BULK) {
            // (an error word that is set already does not end the wait for the copies)
            if (!wait_bounded_err(&full[g][st], phase, err)) wait_drain(&full[g][st], phase);
        } else {
            cp_async_wait<STAGES - 1>();
        }
        float2 xh[C / 2], w[C / 2];
        auto load_row = [&]() {
            fetch(st, 0, r, xh);
            fetch(st, 1, r, w);
            if constexpr (!GREG) params(gam);
#pragma unroll
            for (int j = 0; j < C / 2; ++j)
                xh[j] = RMS ? __fmul2_rn(xh[j], f2(rs)) : __fmul2_rn(__fadd2_rn(xh[j], f2(-mean)), f2(rs));
        };
        load_row();
        float2 t1 = f2(0.0f), t2 = f2(0.0f);
#pragma unroll
        for (int j = 0; j < C / 2; ++j) {
            ag[j] = __ffma2_rn(w[j], xh[j], ag[j]);
            if constexpr (!RMS) ab[j] = __fadd2_rn(ab[j], w[j]);
            w[j] = __fmul2_rn(w[j], gam[j]);
            if constexpr (!RMS) t1 = __fadd2_rn(t1, w[j]);
            t2 = __ffma2_rn(w[j], xh[j], t2);
        }
        const float s = RMS ? warp_sum(t2.x + t2.y) : warp_sum2(t1.x + t1.y, t2.x + t2.y);
        float2 c12;
        if (warps > 1) {
            if ((t & 15) == 0) red[g][par][(t >> 4) & 1][warp] = s;      // (RMS: the same sum twice)
            if constexpr (GROUPED) bar_group(1 + g, nt);
            else __syncthreads();
            c12 = RMS ? make_float2(0.0f, block_total(red[g][par][0], span)) : block_total2(red[g][par], span);
        } else if (RMS) {
            c12 = make_float2(0.0f, s);
            if (BULK) __syncwarp();             // (shuffles order no memory)
        } else {
            c12 = make_float2(__shfl_sync(0xFFFFFFFFu, s, 0), __shfl_sync(0xFFFFFFFFu, s, 16));
            if (BULK) __syncwarp();             // (shuffles order no memory)
        }
        // the group is past its reads of the row before, whose stage is free
        if constexpr (BULK && STAGES > 1) stage(ahead, r + (STAGES - 1) * step);
        const float c1 = c12.x * inv, c2 = c12.y * inv;
        if constexpr (!KEEP) {
            load_row();
#pragma unroll
            for (int j = 0; j < C / 2; ++j) w[j] = __fmul2_rn(w[j], gam[j]);
        }
#pragma unroll
        for (int j = 0; j < C / 2; ++j)
            w[j] = __fmul2_rn(__ffma2_rn(xh[j], f2(-c2), RMS ? w[j] : __fadd2_rn(w[j], f2(-c1))), f2(rs));
        if (dres) {
            fetch(st, 2, r, xh);
#pragma unroll
            for (int j = 0; j < C / 2; ++j) w[j] = __fadd2_rn(w[j], xh[j]);
        }
        if constexpr (BULK) {
            T* o = dx + r * K + t * VEC;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int e = i * VEC + j;
                    v[j] = (e & 1) ? w[e / 2].y : w[e / 2].x;
                }
                if (i < own) *reinterpret_cast<Raw*>(o) = P::from_floats(v);
                o += nt * VEC;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * nt + t) * VEC;
                float v[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int e = i * VEC + j;
                    v[j] = (e & 1) ? w[e / 2].y : w[e / 2].x;
                }
                if (c < K) *reinterpret_cast<Raw*>(dx + r * K + c) = P::from_floats(v);
            }
        }
        if constexpr (BULK && STAGES == 1) {
            __syncthreads();
            stage(0, r + step);
        }
        mean = mean_n;
        rs = rs_n;
        par ^= 1;
        if (++st == STAGES) {
            st = 0;
            phase ^= 1u;
        }
    }
    if constexpr (GROUPED) {
        // the groups' sums, added in group order by the first (the ring is idle)
        float2* sums = reinterpret_cast<float2*>(ln_ring);
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int j = 0; j < C / 2; ++j) {
            sums[(2 * j) * blockDim.x + threadIdx.x] = ag[j];
            if constexpr (!RMS) sums[(2 * j + 1) * blockDim.x + threadIdx.x] = ab[j];
        }
        __syncthreads();
        if (g > 0) return;
        for (int o = 1; o < groups; ++o) {
#pragma unroll
            for (int j = 0; j < C / 2; ++j) {
                ag[j] = __fadd2_rn(ag[j], sums[(2 * j) * blockDim.x + o * nt + t]);
                if constexpr (!RMS) ab[j] = __fadd2_rn(ab[j], sums[(2 * j + 1) * blockDim.x + o * nt + t]);
            }
        }
    }
    float* pg = part + (int64_t)blockIdx.x * (RMS ? 1 : 2) * K;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * nt + t) * VEC;
        if (c >= K) continue;
        // (sixteen-byte stores: with single floats, 32 bytes apart in a warp,
        // 16384 x 4096 took 92 us instead of 84 and 512 x 4096 16 instead of 8)
        if constexpr (VEC % 4 == 0) {
#pragma unroll
            for (int j = 0; j < VEC; j += 4) {
                const int e = (i * VEC + j) / 2;
                *reinterpret_cast<float4*>(pg + c + j) = make_float4(ag[e].x, ag[e].y, ag[e + 1].x, ag[e + 1].y);
                if constexpr (!RMS) *reinterpret_cast<float4*>(pg + K + c + j) = make_float4(ab[e].x, ab[e].y, ab[e + 1].x, ab[e + 1].y);
            }
        } else if constexpr (VEC == 2) {
            *reinterpret_cast<float2*>(pg + c) = ag[i];
            if constexpr (!RMS) *reinterpret_cast<float2*>(pg + K + c) = ab[i];
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int e = i * VEC + j;
                pg[c + j] = (e & 1) ? ag[e / 2].y : ag[e / 2].x;
                if constexpr (!RMS) pg[K + c + j] = (e & 1) ? ab[e / 2].y : ab[e / 2].x;
            }
        }
    }
}

template <typename T, int VEC, int MAXT, int MINB, bool CODES, bool RMS>
cudaError_t ln_fwd_cta(const LnArgs& a, cudaStream_t st, int sms, int threads)
{
    auto kern = k_ln_fwd<T, VEC, MAXT, MINB, CODES, RMS>;
    const int64_t cap = resident(reinterpret_cast<const void*>(kern), threads, 0, sms);
    launch_k(kern, (unsigned)(a.M < cap ? a.M : cap), threads, 0, st, static_cast<const T*>(a.x),
             static_cast<const T*>(a.residual), a.gamma, a.beta, a.eps, a.M, (int)a.K, static_cast<T*>(a.sum),
             static_cast<T*>(a.y), a.mu, a.rstd, LnCast{a.q, a.q_format, a.q_history_len, a.q_state});
    return cudaGetLastError();
}

template <typename T, int VEC, bool CODES, bool RMS>
cudaError_t ln_fwd_rows(const LnArgs& a, cudaStream_t st, int sms)
{
    const int threads = 32 * (int)cdiv(a.K, 32 * kLnCols);
    if (threads <= 256) return ln_fwd_cta<T, VEC, 256, 6, CODES, RMS>(a, st, sms, threads);
    if (threads <= 512) return ln_fwd_cta<T, VEC, 512, 3, CODES, RMS>(a, st, sms, threads);
    if (threads <= 768) return ln_fwd_cta<T, VEC, 768, 2, CODES, RMS>(a, st, sms, threads);
    return ln_fwd_cta<T, VEC, 1024, 1, CODES, RMS>(a, st, sms, threads);
}

template <typename T, bool CODES, bool RMS>
cudaError_t ln_fwd_vec(const LnArgs& a, cudaStream_t st, int sms)
{
    constexpr int WIDE = 16 / (int)sizeof(T);        // the widest vector of 16, 8 or 4 bytes that divides a row
    if (a.K % WIDE == 0) return ln_fwd_rows<T, WIDE, CODES, RMS>(a, st, sms);
    if (a.K % (WIDE / 2) == 0) return ln_fwd_rows<T, WIDE / 2, CODES, RMS>(a, st, sms);
    if (a.K % (WIDE / 4) == 0) return ln_fwd_rows<T, WIDE / 4, CODES, RMS>(a, st, sms);
    return ln_fwd_rows<T, 1, CODES, RMS>(a, st, sms);
}

template <typename T>
cudaError_t ln_fwd(const LnArgs& a, cudaStream_t st, int sms)
{
    if (a.K <= 1024 * kLnCols)
        return a.q ? ln_fwd_vec<T, true, false>(a, st, sms) : ln_fwd_vec<T, false, false>(a, st, sms);
    const int64_t cap = (int64_t)sms * 8;
    launch_k(k_ln_fwd_any<T>, (unsigned)(a.M < cap ? a.M : cap), 256, 0, st, static_cast<const T*>(a.x),
             static_cast<const T*>(a.residual), a.gamma, a.beta, a.eps, a.M, a.K, static_cast<T*>(a.sum),
             static_cast<T*>(a.y), a.mu, a.rstd, a.q, a.q_format, a.q_state, a.q_history_len);
    return cudaGetLastError();
}

constexpr int kLnRoom = 227 * 1024 - 6 * 1024;      // shared memory of a LayerNorm ring (beside the reduction's)

template <typename T, int VEC, int C, int STAGES, int MAXT, int MINB, bool KEEP, bool GROUPED, bool RMS>
cudaError_t ln_bwd_rows(const LnArgs& a, cudaStream_t st, int sms, int group, int groups, int smem, int* parts)
{
    auto kern = k_ln_bwd<T, VEC, C, STAGES, MAXT, MINB, KEEP, GROUPED, RMS>;
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(kern), kLnRoom);
    if (e != cudaSuccess) return e;
    int* err = nullptr;
    if (VEC * sizeof(T) < 16 && (e = device_error_word(&err)) != cudaSuccess) return e;
    const int threads = group * groups;
    int64_t cap = resident(reinterpret_cast<const void*>(kern), threads, smem, sms);
    const int64_t most = parts_for(cdiv(a.M, groups));
    cap = cap < most ? cap : most;
    *parts = (int)cap;
    launch_k(kern, (unsigned)cap, threads, smem, st, static_cast<const T*>(a.dy), static_cast<const T*>(a.x),
             static_cast<const T*>(a.dres), a.gamma, (const float*)a.mu, (const float*)a.rstd, a.M, (int)a.K, group,
             static_cast<T*>(a.dx), static_cast<float*>(a.workspace), err);
    return cudaGetLastError();
}

// Three stages of the ring where they fit, else two or one.  Rows take the widest
// vector of 16, 8, 4 or 2 bytes that divides them.  Short rows share a
// CTA of MAXT threads where there are rows for all of its groups on every SM.
template <typename T, int VEC, int C, int MAXT, int MINB, bool KEEP, bool RMS>
cudaError_t ln_bwd_cols(const LnArgs& a, cudaStream_t st, int sms, int* parts)
{
    const int group = 32 * (int)cdiv(a.K, 32 * C);
    int groups = MAXT <= 256 ? MAXT / group : 1;
    groups = groups < kLnGroups ? groups : kLnGroups;
    while (groups > 1 && a.M < (int64_t)groups * sms) --groups;
    const int row = VEC * sizeof(T) < 16 ? ln_row_bytes((int)a.K, sizeof(T)) : group * C * (int)sizeof(T);
    const int stage = groups * row * (a.dres ? 3 : 2);
    if constexpr (MAXT <= 256) {
        const int sums = group * groups * C * (int)sizeof(float2), ring = 3 * stage;
        if (groups > 1)
            return ln_bwd_rows<T, VEC, C, 3, MAXT, MINB, KEEP, true, RMS>(
                a, st, sms, group, groups, ring > sums ? ring : sums, parts);
    }
    // (two CTAs with two stages each before one with three: 2048 x 4096 fp32 35.1 -> 27.5 us)
    const bool two = MINB >= 2 && 6 * stage > kLnRoom && 4 * stage <= kLnRoom;
    if (3 * stage <= kLnRoom && !two) return ln_bwd_rows<T, VEC, C, 3, MAXT, MINB, KEEP, false, RMS>(a, st, sms, group, 1, 3 * stage, parts);
    if (2 * stage <= kLnRoom) return ln_bwd_rows<T, VEC, C, 2, MAXT, MINB, KEEP, false, RMS>(a, st, sms, group, 1, 2 * stage, parts);
    return ln_bwd_rows<T, VEC, C, 1, MAXT, MINB, KEEP, false, RMS>(a, st, sms, group, 1, stage, parts);
}

template <typename T, int VEC, bool RMS>
cudaError_t ln_bwd_vec(const LnArgs& a, cudaStream_t st, int sms, int* parts)
{
    if (a.K <= 256 * 16) return ln_bwd_cols<T, VEC, 16, 256, 2, true, RMS>(a, st, sms, parts);
    if (a.K <= 512 * 16) return ln_bwd_cols<T, VEC, 16, 512, 1, true, RMS>(a, st, sms, parts);
    if (a.K <= 768 * 16) return ln_bwd_cols<T, VEC, 16, 768, 1, true, RMS>(a, st, sms, parts);
    return ln_bwd_cols<T, VEC, 16, 1024, 1, false, RMS>(a, st, sms, parts);
}

template <typename T, bool RMS>
cudaError_t ln_bwd(const LnArgs& a, cudaStream_t st, int sms)
{
    constexpr int WIDE = 16 / (int)sizeof(T);
    float* part = static_cast<float*>(a.workspace);
    int parts = 0;
    if (a.M > 0) {
        cudaError_t e = cudaSuccess;
        if (a.K <= 1024 * kLnCols) {
            e = a.K % WIDE == 0         ? ln_bwd_vec<T, WIDE, RMS>(a, st, sms, &parts)
                : a.K % (WIDE / 2) == 0 ? ln_bwd_vec<T, WIDE / 2, RMS>(a, st, sms, &parts)
                : a.K % (WIDE / 4) == 0 ? ln_bwd_vec<T, WIDE / 4, RMS>(a, st, sms, &parts)
                                        : ln_bwd_vec<T, 1, RMS>(a, st, sms, &parts);
            if (e != cudaSuccess) return e;
        } else {
            const int64_t cap = (int64_t)sms * 8;
            launch_k(k_ln_bwd_dx_any<T, RMS>, (unsigned)(a.M < cap ? a.M : cap), 256, 0, st, static_cast<const T*>(a.dy),
                     static_cast<const T*>(a.x), static_cast<const T*>(a.dres), a.gamma, (const float*)a.mu,
                     (const float*)a.rstd, a.M, a.K, static_cast<T*>(a.dx));
            parts = (int)parts_for(a.M);
            launch_k(k_ln_bwd_gb_any<T, RMS>, dim3((unsigned)cdiv(a.K, 256), parts), 256, 0, st,
                     static_cast<const T*>(a.dy), static_cast<const T*>(a.x), (const float*)a.mu,
                     (const float*)a.rstd, a.M, a.K, part);
        }
    }
    const int64_t n = (RMS ? 1 : 2) * a.K;
    launch_k(k_col_reduce, (unsigned)cdiv(n, 32), 1024, 0, st, (const float*)part, parts, n, a.dgamma, a.K, a.dbeta);
    return cudaGetLastError();
}

}  // namespace

}  // namespace fp8sq
