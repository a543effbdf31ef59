// kdn_checks.h -- argument checks that the operators around the mixer share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kdn.h"
#include "kdn_errors.h"

namespace kdn {

constexpr long long kMaxElems = 1ll << 31;  // of every dense tensor
constexpr long long kMaxStride = 1ll << 30;
// the recurrence steps over a tile of rows with 32-bit byte offsets
constexpr long long kMaxRecStride = 1ll << 22;
constexpr int kMaxD = 1 << 20, kMaxTokens = 1 << 30;

// One buffer of a call: its bytes (0: not given) and what the call does to it.
struct Buf {
    const void* p;
    long long elems;
    int size;  // bytes of an element, and its alignment
    const char* name;
    bool out;
    bool required;  // when elems > 0
};

inline long long bytes_of(const Buf& b) { return b.p ? b.elems * b.size : 0; }

// NULL where a buffer is needed, misaligned pointers, outputs that overlap
template <int N>
kdn_status check_buffers(const Buf (&bufs)[N])
{
    for (const Buf& b : bufs) {
        if (b.required && b.elems > 0 && !b.p)
            return fail(KDN_ERR_INVALID_ARG, "%s must not be NULL", b.name);
        if (reinterpret_cast<uintptr_t>(b.p) % (unsigned)b.size)
            return fail(KDN_ERR_INVALID_ARG, "%s must be %d-byte aligned", b.name, b.size);
    }
    for (const Buf& o : bufs) {
        if (!o.out || !bytes_of(o))
            continue;
        const uintptr_t o0 = reinterpret_cast<uintptr_t>(o.p), o1 = o0 + bytes_of(o);
        for (const Buf& b : bufs) {
            const uintptr_t b0 = reinterpret_cast<uintptr_t>(b.p), b1 = b0 + bytes_of(b);
            if (&b != &o && o0 < b1 && b0 < o1)
                return fail(KDN_ERR_INVALID_ARG, "%s must not overlap %s", o.name, b.name);
        }
    }
    return KDN_OK;
}

inline kdn_status check_io(int io)
{
    if (io != KDN_F32 && io != KDN_BF16)
        return fail(KDN_ERR_INVALID_ARG, "io_dtype must be KDN_F32 (0) or KDN_BF16 (1), got %d", io);
    return KDN_OK;
}

// an io_dtype that may hold KDN_CLEAR_TAIL, which is taken out of it
inline kdn_status check_packed_io(int& io, bool& clear)
{
    clear = io & KDN_CLEAR_TAIL;
    io &= ~KDN_CLEAR_TAIL;
    if (io != KDN_F32 && io != KDN_BF16)
        return fail(KDN_ERR_INVALID_ARG, "io_dtype must be KDN_F32 (0) or KDN_BF16 (1), with KDN_CLEAR_TAIL (0x400) "
                    "if wanted, got %d", clear ? io | KDN_CLEAR_TAIL : io);
    return KDN_OK;
}

inline kdn_status check_width(int D)
{
    if (D < 1)
        return fail(KDN_ERR_INVALID_ARG, "need D >= 1 (got %d)", D);
    if (D > kMaxD)
        return fail(KDN_ERR_UNSUPPORTED, "D is at most 2^20, got %d", D);
    return KDN_OK;
}

// rows of D elements, stride apart: the elements from the first to the last
inline kdn_status check_rows(long long rows, int D, long long stride, const char* name, long long& span,
                      long long most = kMaxStride)
{
    if (stride < D)
        return fail(KDN_ERR_INVALID_ARG, "%s_stride must be at least D = %d, got %lld", name, D, stride);
    if (stride > most)
        return fail(KDN_ERR_UNSUPPORTED, "%s_stride is at most %lld, got %lld", name, most, stride);
    span = rows ? (rows - 1) * stride + D : 0;
    return KDN_OK;
}

// [B,T,D] and the sequences in it; N becomes B where rows are not packed
inline kdn_status check_sequence(int B, int T, int D, const int* cu, int& N)
{
    if (B < 1 || T < 0)
        return fail(KDN_ERR_INVALID_ARG, "need B >= 1, T >= 0 (got B=%d T=%d)", B, T);
    const kdn_status st = check_width(D);
    if (st != KDN_OK)
        return st;
    if (cu && B != 1)
        return fail(KDN_ERR_INVALID_ARG, "packed sequences (cu_seqlens) need B = 1, got %d", B);
    if (cu && N < 1)
        return fail(KDN_ERR_INVALID_ARG, "packed sequences need N >= 1, got %d", N);
    if (!cu)
        N = B;
    // 128-bit products: three factors below 2^31
    if ((__int128)B * T * D >= kMaxElems || (__int128)N * D >= kMaxElems)
        return fail(KDN_ERR_UNSUPPORTED, "tensor sizes must stay below 2^31 elements");
    // token numbers, and those a tile further, are ints; a row is a workgroup or more
    if ((long long)B * T > kMaxTokens || B >= 1 << 24)
        return fail(KDN_ERR_UNSUPPORTED, "B T is at most 2^30 and B below 2^24 (got B=%d T=%d)", B, T);
    return KDN_OK;
}

inline kdn_status check_workspace(const void* ws, size_t bytes, size_t need)
{
    if (!need)
        return KDN_OK;
    if (!ws || bytes < need)
        return fail(KDN_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, ws ? bytes : (size_t)0);
    if (reinterpret_cast<uintptr_t>(ws) & 15u)
        return fail(KDN_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    return KDN_OK;
}

inline kdn_status launched(hipError_t e, const char* what)
{
    return e == hipSuccess ? ok() : fail(KDN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

#define KDN_TRY(call)               \
    do {                            \
        const kdn_status st_ = call; \
        if (st_ != KDN_OK)          \
            return st_;             \
    } while (0)

inline int io_size(int io) { return io == KDN_BF16 ? 2 : 4; }

}  // namespace kdn
