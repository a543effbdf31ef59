// kdn_stream.h -- adjacent values of a row, loaded and stored at any alignment of
// their elements, and data that a call touches once.
#pragma once

#include "kdn_common.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kdn {

// N words at the alignment of an E
template <typename E, int N>
using Words = uint32_t __attribute__((ext_vector_type(N), aligned(sizeof(E))));

// N values as they are in memory.  Held as words, not as elements: the compiler
// splits a load of two elements into two, joins them again, and drops on the way
// that it was non-temporal.
template <typename E, int N>
struct Raw {
    static constexpr int kWords = (sizeof(E) * N + 3) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(E) == 4)
            return __uint_as_float(w[i]);
        else
            return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
};

// ONCE: non-temporal
template <bool ONCE, typename E, int N>
__device__ __forceinline__ Raw<E, N> load_raw(const E* p)
{
    constexpr int W = Raw<E, N>::kWords;
    Raw<E, N> r;
    if constexpr (sizeof(E) * N % 4) {
        static_assert(W == 1, "one element of two bytes");
        r.w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
        const Words<E, W>* q = reinterpret_cast<const Words<E, W>*>(p);
        Words<E, W> x;
        if constexpr (ONCE)
            x = __builtin_nontemporal_load(q);
        else
            x = *q;
#pragma unroll
        for (int i = 0; i < W; ++i)
            r.w[i] = x[i];
    }
    return r;
}

// values as they were loaded
template <typename E, int N>
__device__ __forceinline__ void store_same(E* p, const Raw<E, N>& r)
{
    constexpr int W = Raw<E, N>::kWords;
    if constexpr (sizeof(E) * N % 4) {
        *reinterpret_cast<uint16_t*>(p) = r.w[0];
    } else {
        Words<E, W> x;
#pragma unroll
        for (int i = 0; i < W; ++i)
            x[i] = r.w[i];
        *reinterpret_cast<Words<E, W>*>(p) = x;
    }
}

template <typename E, int N>
__device__ __forceinline__ void store_raw(E* p, const float (&v)[N])
{
    typedef E Values __attribute__((ext_vector_type(N), aligned(sizeof(E))));
    Values x;
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = from_f32<E>(v[i]);
    *reinterpret_cast<Values*>(p) = x;
}

// Bytes of the last-level cache.  A call too large for it loads its rows as ONCE: they
// then take no place in it from the rows being written, which leave it for HBM at their
// own pace.  What is too large is measured (us, without and with; sizes are x's, bf16):
// - The recurrence gains where all that it reads and writes is more than the cache:
//   forward 134 MB 92 and 82, 268 MB 154 and 140; forward and backward on one x of 134,
//   268, 537 MB 232 and 219, 419 and 403, 818 and 796 (fp32 of 40 MB in all 29.9 and 32.3).
//   Where rows are not whole cache lines a line is read in pieces by two workgroups, and x
//   alone has to be less than the cache (fp32 1023 channels, 134 MB, forward 95 and 86; 2047
//   channels, 537 MB, 342 and 390).
// - The convolution, whose next call may still find a smaller x there, gains where x alone
//   fills it and rows are whole cache lines: forward 268, 336, 537 MB 112 and 89, 140 and 141,
//   224 and 224; forward and backward on one x 290 and 250, 363 and 362, 581 and 586.  2040
//   channels, 286 MB: forward 144 and 119, but with the backward 367 and 434.
// - The layer norm does not: its forward takes 100 and 88 for 268 MB and its backward 151 and
//   136, but the forward 124 and 127 for 336 MB, and both on one x of 268, 336, 537 MB 252
//   and 254, 311 and 325, 490 and 513 (537 MB in rows of 128 509 and 578).
// Stores marked the same way gave less, and cost up to 12% where a row is not whole cache
// lines.
constexpr long long kLastLevelCache = 256ll << 20;
constexpr size_t kCacheLine = 128;

}  // namespace kdn
