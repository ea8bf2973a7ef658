// api_checks.h -- argument checks shared by the entry points of the operators
// around the FP8 linear: each returns FP8SQ_OK or an error whose message is set.
#pragma once
#include <cstdint>
#include <initializer_list>
#include <cuda_runtime.h>

#include "../../include/fp8sq.h"
#include "internal.h"

namespace {

using fp8sq::api_fail;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_format(int f) { return f == FP8SQ_E4M3 || f == FP8SQ_E5M2; }
bool valid_dtype(int d) { return d == FP8SQ_BF16 || d == FP8SQ_F32; }
bool valid_act(int a) { return a >= FP8SQ_ACT_NONE && a <= FP8SQ_ACT_SILU; }
const int64_t kMaxDim = (int64_t)1 << 31;

int cuda_status(cudaError_t e, const char* what, const char* why = nullptr)
{
    if (e == cudaSuccess) return FP8SQ_OK;
    cudaGetLastError();
    return api_fail(FP8SQ_ERR_CUDA, "%s: %s", what, why ? why : cudaGetErrorString(e));
}

int check_dims(const char* fn, int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: negative size", fn);
    if (M >= kMaxDim || N >= kMaxDim / 2 || K >= kMaxDim)
        return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: dimension too large", fn);
    return FP8SQ_OK;
}

// the delayed output cast: codes, state, format and history length together
int check_cast(const char* fn, const uint8_t* q, int format, const float* state, int H)
{
    if (!q) return FP8SQ_OK;
    if (!state) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: codes need a delayed state", fn);
    if (!valid_format(format)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad output format", fn);
    if (H < 1 || H > 4096) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad history_len", fn);
    if (!aligned(q, 16) || !aligned(state, 4)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: codes need 16-byte, the state 4-byte alignment", fn);
    return FP8SQ_OK;
}

// operands shared by the three products
int check_operands(const char* fn, const uint8_t* A, int a_format, const float* a_scale, const uint8_t* B, int b_format,
                   const float* b_scale, int act, int64_t M, int64_t N, int64_t K, int64_t n_mult)
{
    int r = check_dims(fn, M, N, K);
    if (r) return r;
    if (!valid_format(a_format) || !valid_format(b_format)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad operand format", fn);
    if (!valid_act(act)) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: bad activation", fn);
    if (K == 0) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: needs K > 0", fn);
    if (K % 16) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: K %% 16 != 0", fn);
    if (N % n_mult) return api_fail(FP8SQ_ERR_UNSUPPORTED, "%s: N %% %d != 0", fn, (int)n_mult);
    if ((!A || !B || !a_scale || !b_scale) && M * N != 0) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: null operand or scale", fn);
    if (!aligned(A, 16) || !aligned(B, 16)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: A, B must be 16-byte aligned", fn);
    if (!aligned(a_scale, 4) || !aligned(b_scale, 4)) return api_fail(FP8SQ_ERR_MISALIGNED, "%s: scales must be 4-byte aligned", fn);
    return FP8SQ_OK;
}

// A buffer of `bytes` bytes that a call reads, or writes (out).
struct Span {
    const char* name;
    const void* p;
    uint64_t bytes;
    bool out;
};
// Refuses an output that overlaps another buffer of the call.  In place exactly
// (the same bytes from first to last) are the pairs where each element is read
// before it is written, by the thread that writes it: `into` over one of `over`.
int check_overlap(const char* fn, std::initializer_list<Span> spans, const void* into = nullptr,
                  std::initializer_list<const void*> over = {})
{
    for (const Span& a : spans) {
        if (!a.out || !a.p || !a.bytes) continue;
        const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p);
        for (const Span& b : spans) {
            if (&a == &b || !b.p || !b.bytes) continue;
            const uintptr_t b0 = reinterpret_cast<uintptr_t>(b.p);
            if (a0 >= b0 + b.bytes || b0 >= a0 + a.bytes) continue;
            bool in_place = false;
            if (a.p == into && a0 == b0 && a.bytes == b.bytes && !b.out)
                for (const void* o : over) in_place |= o == b.p;
            if (!in_place) return api_fail(FP8SQ_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, a.name, b.name);
        }
    }
    return FP8SQ_OK;
}
uint64_t size_of(int dtype) { return dtype == FP8SQ_F32 ? 4 : 2; }

}  // namespace
