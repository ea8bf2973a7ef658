// experts_rows.cu -- rows sorted by expert and back, for experts' products.
//
//   plan         a stable counting sort of the assignments ids[T][k]: expert e's
//                rows are [offsets[e], offsets[e] + counts[e]) of the sorted
//                buffers, in the order of (token, slot), and its segment ends on
//                a multiple of 32 rows
//   dispatch     rows[row_of[t][j]] = x[t]; the rest of a segment is zero
//   combine      y[t] = residual[t] + sum over j of w[t][j] rows[row_of[t][j]]
//   combine_bwd  drows[row_of[t][j]] = w[t][j] dy[t] (FP8 codes and / or as
//                stored), dw[t][j] = <dy[t], rows[row_of[t][j]]>
//
// All are bound by memory: a token's row is read once and written (or summed
// from) its k places, whole rows at a time.  No atomics on data: every sum runs
// in the order of the slots, so the same call gives the same bits.
// What they read is no constant of their run: they may be resident while the kernel
// that writes it still runs, so inputs are not declared __restrict__ (nor read with
// __ldg) and the loads stay behind the wait in pdl_enter (see ld_in).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "act.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace fp8sq {

namespace {

// ------------------------------------------------------------------ plan
// One cluster of up to kSortCtas CTAs, each warp a contiguous share of the
// assignments: counts per warp and expert in shared memory, a sum over the warps of
// a CTA, over the CTAs through distributed shared memory and over the experts (padded
// to 32), after which each assignment gets its row.  The lanes of a warp that hold
// the same expert find each other by one vote a bit of its number, eight rounds of 32
// side by side, so the order within an expert is that of the assignments.  One
// launch for any size; bound by the latency of its few steps.  One GB300, us (with
// match_any, and found twice instead of kept): 8 slots 4.2 (3.8), 512 slots of 64 experts 5.1
// (4.8), 65536 of 16 8.4 (8.5), 131072 of 256 19.6 (34), 262144 of 1024 42 (65).
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortBatch = 8;       // loads of ids in flight per lane
constexpr int kSortCtas = 8;        // of the cluster, where one CTA is not enough

struct SortArgs {
    const int32_t* ids;
    int64_t n;                      // assignments
    int E;
    int32_t* plan;
    int tiles_at, blocks_at, row_of_at;
};

__global__ void __launch_bounds__(kSortThreads, 1) k_expert_plan(SortArgs a, int ctas)
{
    extern __shared__ int32_t sort_smem[];
    const int E = a.E;
    int32_t* hist = sort_smem;                          // [warp][E]
    int32_t* total = hist + kSortWarps * E;             // [E], read by the other CTAs of the cluster
    int32_t* base = total + E;                          // [E] first row of this CTA's share of an expert
    int32_t* first_tile = base + E;                     // [E]
    int32_t* first_row = first_tile + E;                // [E]
    int32_t* count = first_row + E;                     // [E] over the cluster
    __shared__ int32_t scan[2][kSortWarps];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int rank = blockIdx.x;
    for (int e = lane; e < E; e += 32) hist[warp * E + e] = 0;
    pdl_enter();
    pdl_trigger();                      // (the next kernel's launch runs under this one)
    const int64_t warps = (int64_t)ctas * kSortWarps;
    const int64_t per = ((a.n + warps - 1) / warps + 31) & ~(int64_t)31;
    const int64_t from = ((int64_t)rank * kSortWarps + warp) * per, to = from + per < a.n ? from + per : a.n;
    const uint32_t below = (1u << lane) - 1u;
    int32_t* mine = hist + warp * E;
    const int bits = 32 - __clz(E - 1);                 // of an expert's number (0 for one expert)
    // A batch of ids from index i on: the expert of each (or -1) and its rank among
    // the warp's so far, whose counts go up.
    int32_t id[kSortBatch], rank_of[kSortBatch];
    auto batch = [&](int64_t i) {
#pragma unroll
        for (int b = 0; b < kSortBatch; ++b) {
            const int64_t at = i + 32 * b + lane;
            id[b] = at < to ? a.ids[at] : -1;
        }
        uint32_t same[kSortBatch];
#pragma unroll
        for (int b = 0; b < kSortBatch; ++b) {
            if ((uint32_t)id[b] >= (uint32_t)E) id[b] = -1;
            same[b] = __ballot_sync(0xFFFFFFFFu, id[b] >= 0);           // (those without an expert need no mates)
        }
        for (int bit = 0; bit < bits; ++bit)
#pragma unroll
            for (int b = 0; b < kSortBatch; ++b) {
                if (i + 32 * b >= to) break;
                const bool on = (id[b] >> bit) & 1;
                const uint32_t v = __ballot_sync(0xFFFFFFFFu, on);
                same[b] &= on ? v : ~v;
            }
#pragma unroll
        for (int b = 0; b < kSortBatch; ++b) {
            if (i + 32 * b >= to) break;
            const int32_t seen = id[b] >= 0 ? mine[id[b]] : 0;
            rank_of[b] = seen + __popc(same[b] & below);
            __syncwarp();
            if (id[b] >= 0 && (same[b] & below) == 0) mine[id[b]] = seen + __popc(same[b]);
            __syncwarp();
        }
    };
    __syncwarp();
    // a warp's only batch stays in registers; of several the ranks wait in row_of
    int32_t* row_of = a.plan + a.row_of_at;
    const bool several = per > 32 * kSortBatch;
    for (int64_t i = from; i < to; i += 32 * kSortBatch) {
        batch(i);
        if (several) {
#pragma unroll
            for (int b = 0; b < kSortBatch; ++b)
                if (i + 32 * b + lane < to) row_of[i + 32 * b + lane] = rank_of[b];
        }
    }
    __syncthreads();
    for (int e = t; e < E; e += kSortThreads) {
        int32_t run = 0;
        for (int w = 0; w < kSortWarps; w += 8) {
            int32_t c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = hist[(w + i) * E + e];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                hist[(w + i) * E + e] = run;
                run += c[i];
            }
        }
        total[e] = run;
    }
    if (ctas > 1) cluster_sync_all();
    else __syncthreads();
    // thread e: the expert's counts over the cluster, then the padded rows and
    // the tiles of the experts before it
    static_assert(kExpertMax <= kSortThreads, "an expert a thread");
    int32_t all = 0, before = 0;
    if (t < E) {
        if (ctas > 1) {
            const uint32_t at = smem_addr(total + t);
            int32_t v[kSortCtas];
#pragma unroll
            for (int r = 0; r < kSortCtas; ++r) v[r] = (int32_t)ld_shared_cluster_u32(cluster_map(at, (uint32_t)r));
#pragma unroll
            for (int r = 0; r < kSortCtas; ++r) {
                if (r < rank) before += v[r];
                all += v[r];
            }
        } else {
            all = total[t];
        }
    }
    const int32_t padded = (all + kExpertPad - 1) & ~(kExpertPad - 1);
    const int32_t ntiles = (padded + kExpertTile - 1) / kExpertTile;
    int32_t rs = padded, ts = ntiles;                   // inclusive sums over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t r = __shfl_up_sync(0xFFFFFFFFu, rs, o), q = __shfl_up_sync(0xFFFFFFFFu, ts, o);
        if (lane >= o) {
            rs += r;
            ts += q;
        }
    }
    if (lane == 31) {
        scan[0][warp] = rs;
        scan[1][warp] = ts;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        rs += scan[0][w];
        ts += scan[1][w];
    }
    if (t < E) {
        base[t] = rs - padded + before;
        first_tile[t] = ts - ntiles;
        first_row[t] = rs - padded;
        count[t] = all;
        if (rank == 0) {
            a.plan[t] = rs - padded;
            a.plan[E + 1 + t] = all;
            if (t == E - 1) {
                a.plan[E] = rs;
                a.plan[2 * E + 1] = ts;
            }
        }
    }
    if (ctas > 1) cluster_sync_all();                   // the totals have been read: a CTA may end
    else __syncthreads();
    for (int64_t i = from; i < to; i += 32 * kSortBatch) {
        if (several) {
#pragma unroll
            for (int b = 0; b < kSortBatch; ++b) {
                const int64_t at = i + 32 * b + lane;
                if (at >= to) continue;
                id[b] = a.ids[at];
                if ((uint32_t)id[b] >= (uint32_t)E) id[b] = -1;
                rank_of[b] = row_of[at];
            }
        }
#pragma unroll
        for (int b = 0; b < kSortBatch; ++b) {
            const int64_t at = i + 32 * b + lane;
            if (at < to) row_of[at] = id[b] >= 0 ? base[id[b]] + mine[id[b]] + rank_of[b] : -1;
        }
    }
    // row tiles of the products, in groups of neighbours of one expert, and blocks
    int4* tiles = reinterpret_cast<int4*>(a.plan + a.tiles_at);
    int4* blocks = reinterpret_cast<int4*>(a.plan + a.blocks_at);
    for (int e = rank + ctas * warp; e < E; e += ctas * kSortWarps) {
        const int32_t begin = first_row[e], n = count[e], end = begin + ((n + kExpertPad - 1) & ~(kExpertPad - 1));
        const int32_t m = (end - begin + kExpertTile - 1) / kExpertTile, t0 = first_tile[e];
        for (int32_t i = lane; i < m; i += 32) {
            const int32_t g = i / kExpertGroup * kExpertGroup, left = m - g;
            const int32_t size = left < kExpertGroup ? left : kExpertGroup;
            tiles[t0 + i] = make_int4(t0 + g, e << 8 | size, begin + g * kExpertTile, end);
        }
        const int32_t b0 = begin / kExpertPad, nb = (end - begin) / kExpertPad, last = n - (nb - 1) * kExpertPad;
        for (int32_t i = lane; i < nb; i += 32) blocks[b0 + i] = make_int4(e, b0, nb, i + 1 < nb ? kExpertPad : last);
    }
}

// ------------------------------------------------------------------ dispatch
// The rows of expert `e` that fill up its segment: columns [c0, c0 + span) of
// each, zeroed by the CTA's threads.
struct Segments {
    const int32_t* plan;
    int E;
    int64_t rows;                   // of the sorted buffers; nothing is touched past them
    // (at most kExpertPad - 1 of them, inside the buffers, whatever the plan holds)
    __device__ __forceinline__ int64_t pad_end(int e) const
    {
        const int64_t end = plan[e + 1];
        return end < rows ? end : rows;
    }
    __device__ __forceinline__ int64_t pad_begin(int e) const
    {
        const int64_t begin = (int64_t)plan[e] + plan[E + 1 + e], least = pad_end(e) - (kExpertPad - 1);
        return max(max(begin, least), (int64_t)0);
    }
};

// Loads of what a kernel reads and does not write: ordinary ones, that the compiler may
// move past the kernel's stores, but not ahead of the wait, behind which alone their
// pointer is known (behind_wait).  As plain C++ loads, in order with the stores, us: combine
// of 16384 tokens of one row of 4096 bf16 68.5 instead of 57.5, of 8192 of two of 2048 fp32 45.2
// instead of 40.4, its backward pass of 16384 of one 76.7 instead of 73.4.
template <typename T>
__device__ __forceinline__ const T* behind_wait(const T* p)
{
    asm volatile("" : "+l"(p) : : "memory");
    return p;
}
__device__ __forceinline__ uint4 ld_in(const uint4* p)
{
    uint4 v;
    asm("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld_in(const uint2* p)
{
    uint2 v;
    asm("ld.global.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld_in(const uint32_t* p)
{
    uint32_t v;
    asm("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint16_t ld_in(const uint16_t* p)
{
    uint16_t v;
    asm("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint8_t ld_in(const uint8_t* p)
{
    uint32_t v;
    asm("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return (uint8_t)v;
}
__device__ __forceinline__ int32_t ld_in(const int32_t* p) { return (int32_t)ld_in(reinterpret_cast<const uint32_t*>(p)); }
__device__ __forceinline__ float ld_in(const float* p) { return __uint_as_float(ld_in(reinterpret_cast<const uint32_t*>(p))); }

constexpr int kMoveThreads = 256;

// CTAs of a column (blockIdx.y: a chunk of kMoveThreads vectors of the rows) take
// the tokens in turn: one load, k stores a thread, the next token's load on its way
// while this one is stored.  Before them the experts' padding (at most 31 rows
// each), shared out likewise.
template <typename V>
__global__ void __launch_bounds__(kMoveThreads) k_expert_dispatch(const V* x, const int32_t* row_of,
                                                                  Segments seg, int64_t T, int k, int64_t vecs,
                                                                  V* __restrict__ out)
{
    pdl_enter();
    pdl_trigger();                      // (resident as a whole: the next kernel prepares under this one)
    x = behind_wait(x);
    row_of = behind_wait(row_of);
    const int64_t c = (int64_t)blockIdx.y * kMoveThreads + threadIdx.x;
    if (c >= vecs) return;
    int64_t t = blockIdx.x;
    V next{};
    if (t < T) next = ld_in(x + t * vecs + c);
    for (int e = blockIdx.x; e < seg.E; e += gridDim.x) {
        const int64_t end = seg.pad_end(e);
        for (int64_t r = seg.pad_begin(e); r < end; ++r) out[r * vecs + c] = V{};
    }
    for (; t < T; t += gridDim.x) {
        const V v = next;
        if (t + gridDim.x < T) next = ld_in(x + (t + gridDim.x) * vecs + c);
        const int32_t* to = row_of + t * k;
#pragma unroll 4
        for (int j = 0; j < k; ++j) {
            const int32_t r = ld_in(to + j);
            if (r >= 0 && r < seg.rows) out[r * vecs + c] = v;
        }
    }
}

// ------------------------------------------------------------------ combine
// CTAs of a column (blockIdx.y: a chunk of kMoveThreads vectors) take the tokens in
// turn, FLY rows' loads in flight a thread; fp32 sums in the order of the slots, in
// packed instructions, the residual last.  y may be the residual itself.  (8192
// tokens of 4 rows of 4096 bf16 with residual, 59.5 us at the copy rate: 59.5; one element at a
// time and eight rows' registers for any k 75.)
template <typename T, int VEC, int FLY>
__global__ void __launch_bounds__(kMoveThreads, FLY <= 4 ? 6 : 4) k_expert_combine(const T* rows, const int32_t* row_of,
                                                                 const float* w, const T* res, int64_t nt,
                                                                 int k, int64_t K, int64_t R, T* y)
{
    using P = Pack<T, VEC>;
    using Raw = typename P::Raw;
    pdl_enter();
    row_of = behind_wait(row_of);
    rows = behind_wait(rows);
    const int64_t c = ((int64_t)blockIdx.y * kMoveThreads + threadIdx.x) * VEC;
    if (c >= K) return;
    for (int64_t t = blockIdx.x; t < nt; t += gridDim.x) {
        constexpr int PAIRS = (VEC + 1) / 2;
        float2 acc[PAIRS] = {};
        Raw rr{};
        if (res) rr = *reinterpret_cast<const Raw*>(res + t * K + c);
        for (int j0 = 0; j0 < k; j0 += FLY) {
            Raw raw[FLY];
            float wj[FLY];
#pragma unroll
            for (int j = 0; j < FLY; ++j) {
                int32_t r = -1;
                if (j0 + j < k) r = ld_in(row_of + t * k + j0 + j);
                wj[j] = 0.0f;
                raw[j] = Raw{};
                if ((uint32_t)r < (uint32_t)R) {
                    raw[j] = ld_in(reinterpret_cast<const Raw*>(rows + r * K + c));
                    wj[j] = w ? w[t * k + j0 + j] : 1.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < FLY; ++j) {
                float v[2 * PAIRS] = {};
                P::to_floats(raw[j], reinterpret_cast<float(&)[VEC]>(v));
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) acc[i] = __ffma2_rn(f2(wj[j]), make_float2(v[2 * i], v[2 * i + 1]), acc[i]);
            }
        }
        float out[VEC], v[2 * PAIRS] = {};
        if (res) P::to_floats(rr, reinterpret_cast<float(&)[VEC]>(v));
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            out[i] = (i & 1) ? acc[i / 2].y : acc[i / 2].x;
            if (res) out[i] += v[i];
        }
        *reinterpret_cast<Raw*>(y + t * K + c) = P::from_floats(out);
    }
}

// ------------------------------------------------------------------ combine, backward
// A CTA takes a token at a time and JB of its slots at once: dy[t] is read once for
// them (by the next ones from the SM's own cache), their dot products accumulate in
// registers.  The padding of the experts' segments comes first, shared out by
// expert.  One GB300, codes and dweights of rows of 4096 bf16, us (the bytes at the
// copy rate): 8192 tokens of 4 75.8 (69.4); 4096 of 8 73.0 (64.5), eight slots at once 84.8;
// 16384 of 1 72.9 (49.6), with the registers of four slots 81.5; the next token's rows and
// weights fetched ahead: no faster.
template <int VEC>
__device__ __forceinline__ void store_codes(uint8_t* q, const float (&v)[VEC], float m, int fmt)
{
    if constexpr (VEC == 1) {
        *q = code1(__fmul_rn(v[0], m), fmt);
    } else {
        uint16_t h[VEC / 2];
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
            const float a = __fmul_rn(v[j], m), b = __fmul_rn(v[j + 1], m);
            h[j / 2] = (uint16_t)(fmt == kE4M3 ? cvt_e4m3x2(a, b) : cvt_e5m2x2(a, b));
        }
        if constexpr (VEC == 8) *reinterpret_cast<uint2*>(q) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
        else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(q) = h[0] | (uint32_t)h[1] << 16;
        else *reinterpret_cast<uint16_t*>(q) = h[0];
    }
}
struct CombineBwdOut {
    uint8_t* q;
    int fmt, H;
    float* state;
    void* drows;
    float* dw;
};
template <typename T, int VEC, int JB>
__global__ void __launch_bounds__(256, JB <= 2 ? 6 : 4) k_expert_combine_bwd(const T* dy, const T* rows,
                                                            const int32_t* row_of, const float* w,
                                                            Segments seg, int64_t nt, int k, int64_t K, CombineBwdOut o)
{
    using P = Pack<T, VEC>;
    using Raw = typename P::Raw;
    constexpr int PAIRS = (VEC + 1) / 2;
    __shared__ float red[2][8][JB];
    pdl_enter();
    dy = behind_wait(dy);
    rows = behind_wait(rows);
    row_of = behind_wait(row_of);
    w = behind_wait(w);
    const int th = threadIdx.x, lane = th & 31, warp = th >> 5, warps = blockDim.x >> 5;
    T* drows = static_cast<T*>(o.drows);
    const float none[VEC] = {};
    for (int64_t e = blockIdx.x; e < seg.E; e += gridDim.x) {
        const int64_t end = seg.pad_end((int)e);
        for (int64_t r = seg.pad_begin((int)e); r < end; ++r)
            for (int64_t c = (int64_t)th * VEC; c < K; c += (int64_t)blockDim.x * VEC) {
                if (drows) *reinterpret_cast<Raw*>(drows + r * K + c) = Raw{};
                if (o.q) store_codes<VEC>(o.q + r * K + c, none, 0.0f, o.fmt);
            }
    }
    const float m = o.q ? o.state[o.H] : 1.0f;
    float amax = 0.0f;
    int par = 0;
    for (int64_t t = blockIdx.x; t < nt; t += gridDim.x) {
        for (int j0 = 0; j0 < k; j0 += JB) {
            int32_t at[JB];
            float wj[JB];
            float2 dot[JB] = {};
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                const int32_t r = j0 + j < k ? ld_in(row_of + t * k + j0 + j) : -1;
                at[j] = r < seg.rows ? r : -1;
                wj[j] = at[j] >= 0 ? ld_in(w + t * k + j0 + j) : 0.0f;
            }
            for (int64_t c = (int64_t)th * VEC; c < K; c += (int64_t)blockDim.x * VEC) {
                float d[2 * PAIRS] = {};
                P::to_floats(ld_in(reinterpret_cast<const Raw*>(dy + t * K + c)), reinterpret_cast<float(&)[VEC]>(d));
                Raw raw[JB];
                if (o.dw) {
#pragma unroll
                    for (int j = 0; j < JB; ++j)
                        if (at[j] >= 0) raw[j] = ld_in(reinterpret_cast<const Raw*>(rows + (int64_t)at[j] * K + c));
                }
#pragma unroll
                for (int j = 0; j < JB; ++j) {
                    if (at[j] < 0) continue;
                    float w2[2 * PAIRS] = {};
                    float(&v)[VEC] = reinterpret_cast<float(&)[VEC]>(w2);
                    if (o.dw) {
                        P::to_floats(raw[j], v);
#pragma unroll
                        for (int i = 0; i < PAIRS; ++i)
                            dot[j] = __ffma2_rn(make_float2(d[2 * i], d[2 * i + 1]), make_float2(w2[2 * i], w2[2 * i + 1]), dot[j]);
                    }
                    float top = 0.0f;
#pragma unroll
                    for (int i = 0; i < PAIRS; ++i) {
                        const float2 x = __fmul2_rn(make_float2(d[2 * i], d[2 * i + 1]), f2(wj[j]));
                        w2[2 * i] = x.x;
                        w2[2 * i + 1] = x.y;
                        top = max3_nan(top, fabsf(x.x), fabsf(x.y));
                    }
                    if (drows) *reinterpret_cast<Raw*>(drows + (int64_t)at[j] * K + c) = P::from_floats(v);
                    if (o.q) {
                        amax = max_nan(amax, top);
                        store_codes<VEC>(o.q + (int64_t)at[j] * K + c, v, m, o.fmt);
                    }
                }
            }
            if (o.dw) {
#pragma unroll
                for (int j = 0; j < JB; ++j) {
                    const float s = warp_sum(dot[j].x + dot[j].y);
                    if (lane == 0) red[par][warp][j] = s;
                }
                __syncthreads();
                if (th < JB && j0 + th < k) {
                    float s = 0.0f;
                    for (int i = 0; i < warps; ++i) s += red[par][i][th];
                    o.dw[t * k + j0 + th] = s;
                }
                par ^= 1;
            }
        }
    }
    if (o.q) record_amax(amax, o.state);
}

template <typename F>
cudaError_t with_vector(int64_t row_bytes, F&& f)
{
    if (row_bytes % 16 == 0) return f(uint4{});
    if (row_bytes % 8 == 0) return f(uint2{});
    if (row_bytes % 4 == 0) return f(uint32_t{});
    if (row_bytes % 2 == 0) return f(uint16_t{});
    return f(uint8_t{});
}

template <typename T, int VEC, int FLY>
cudaError_t combine_slots(const ExpertRowsArgs& a, cudaStream_t st, int sms)
{
    auto kern = k_expert_combine<T, VEC, FLY>;
    const int64_t chunks = cdiv(a.K, kMoveThreads * VEC);
    const int64_t cap = cdiv(resident(reinterpret_cast<const void*>(kern), kMoveThreads, 0, sms), chunks);
    launch_k(kern, dim3((unsigned)(a.T < cap ? a.T : cap), (unsigned)chunks), kMoveThreads, 0, st,
             static_cast<const T*>(a.rows), a.plan + a.layout.row_of_at, a.weights, static_cast<const T*>(a.residual), a.T,
             a.k, a.K, a.layout.rows, static_cast<T*>(a.y));
    return cudaGetLastError();
}
template <typename T, int VEC>
cudaError_t combine(const ExpertRowsArgs& a, cudaStream_t st, int sms)
{
    return a.k <= 4 ? combine_slots<T, VEC, 4>(a, st, sms) : combine_slots<T, VEC, 8>(a, st, sms);
}
template <typename T, int VEC, int JB>
cudaError_t combine_bwd_slots(const ExpertRowsArgs& a, cudaStream_t st, int sms)
{
    auto kern = k_expert_combine_bwd<T, VEC, JB>;
    const int64_t lanes = cdiv(a.K, VEC);
    const int threads = (int)(lanes >= 256 ? 256 : lanes < 1 ? 32 : (lanes + 31) & ~(int64_t)31);
    const int64_t cap = resident(reinterpret_cast<const void*>(kern), threads, 0, sms);
    const int64_t most = a.T > a.E ? a.T : a.E;
    launch_k(kern, (unsigned)(most < cap ? most : cap), threads, 0, st, static_cast<const T*>(a.dy),
             static_cast<const T*>(a.rows), a.plan + a.layout.row_of_at, a.weights, Segments{a.plan, a.E, a.layout.rows},
             a.T, a.k, a.K, CombineBwdOut{a.q, a.q_format, a.q_history_len, a.q_state, a.drows, a.dweights});
    return cudaGetLastError();
}
template <typename T, int VEC>
cudaError_t combine_bwd(const ExpertRowsArgs& a, cudaStream_t st, int sms)
{
    return a.k <= 2 ? combine_bwd_slots<T, VEC, 2>(a, st, sms) : combine_bwd_slots<T, VEC, 4>(a, st, sms);
}
// the widest vector of 16, 8, 4 or 2 bytes that divides a row
template <typename T>
cudaError_t with_elements(const ExpertRowsArgs& a, cudaStream_t st, int sms, bool bwd)
{
    constexpr int WIDE = 16 / (int)sizeof(T);
    auto go = [&](auto n) {
        constexpr int VEC = decltype(n)::value;
        return bwd ? combine_bwd<T, VEC>(a, st, sms) : combine<T, VEC>(a, st, sms);
    };
    if (a.K % WIDE == 0) return go(std::integral_constant<int, WIDE>{});
    if (a.K % (WIDE / 2) == 0) return go(std::integral_constant<int, WIDE / 2>{});
    if (a.K % (WIDE / 4) == 0) return go(std::integral_constant<int, WIDE / 4>{});
    return go(std::integral_constant<int, 1>{});
}

}  // namespace

ExpertLayout expert_layout(int64_t T, int k, int E)
{
    ExpertLayout l;
    const int64_t n = T * k, active = E < n ? E : n;
    l.rows = (n + (kExpertPad - 1) * active) & ~(int64_t)(kExpertPad - 1);
    l.max_tiles = l.rows / kExpertTile + active;
    l.tiles_at = (2 * (int64_t)E + 2 + 3) & ~(int64_t)3;
    l.blocks_at = l.tiles_at + 4 * l.max_tiles;
    l.row_of_at = l.blocks_at + 4 * (l.rows / kExpertPad);
    l.ints = l.row_of_at + n;
    return l;
}

cudaError_t launch_expert_plan(const ExpertRowsArgs& a, cudaStream_t st)
{
    const int64_t n = a.T * a.k;
    // one CTA as long as a warp has four rounds of 32 ids (or no more to gain)
    const int ctas = n <= 4 * 32 * kSortWarps ? 1 : kSortCtas;
    const int smem = (kSortWarps + 5) * a.E * (int)sizeof(int32_t);
    cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(k_expert_plan),
                                   (kSortWarps + 5) * kExpertMax * (int)sizeof(int32_t));
    if (e != cudaSuccess) return e;
    SortArgs s{a.ids, n, a.E, a.plan_out, (int)a.layout.tiles_at, (int)a.layout.blocks_at, (int)a.layout.row_of_at};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_expert_plan, s, ctas);
}

cudaError_t launch_expert_dispatch(const ExpertRowsArgs& a, cudaStream_t st, int sms)
{
    const int64_t bytes = a.K * a.size;
    return with_vector(bytes, [&](auto v) {
        using V = decltype(v);
        auto kern = k_expert_dispatch<V>;
        const int64_t vecs = bytes / (int64_t)sizeof(V), chunks = cdiv(vecs, kMoveThreads);
        const int64_t cap = resident(reinterpret_cast<const void*>(kern), kMoveThreads, 0, sms) / chunks;   // resident as a whole
        const int64_t most = a.T > a.E ? a.T : a.E, ctas = cap < 1 ? 1 : most < cap ? most : cap;
        launch_k(kern, dim3((unsigned)ctas, (unsigned)chunks), kMoveThreads, 0, st, static_cast<const V*>(a.x),
                 a.plan + a.layout.row_of_at, Segments{a.plan, a.E, a.layout.rows}, a.T, a.k, vecs,
                 static_cast<V*>(a.rows_out));
        return cudaGetLastError();
    });
}

cudaError_t launch_expert_combine(const ExpertRowsArgs& a, cudaStream_t st, int sms)
{
    return a.dtype == kBF16 ? with_elements<__nv_bfloat16>(a, st, sms, false) : with_elements<float>(a, st, sms, false);
}

cudaError_t launch_expert_combine_bwd(const ExpertRowsArgs& a, cudaStream_t st, int sms)
{
    return a.dtype == kBF16 ? with_elements<__nv_bfloat16>(a, st, sms, true) : with_elements<float>(a, st, sms, true);
}

}  // namespace fp8sq
