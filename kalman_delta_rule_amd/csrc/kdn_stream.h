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
// own pace.  What is too large is measured (without and with, us): the recurrence gains
// where all that it reads and writes is more than the cache (forward 403 MB 92 and 80,
// 805 MB 175 and 161, backward 335 MB 85 and 74, 1.3 GB 311 and 291; fp32 40 MB read
// again 29.9 and 32.3); the convolution and the layer norm, whose next call may still
// find a smaller x there, where x alone fills it (convolution forward 537 MB 112 and
// 89, backward 805 MB 179 and 164; layer norm forward 537 MB 101 and 90, fp32 102 and
// 83, backward 805 MB 152 and 136; forward and backward on one x of 134 MB, marked
// from half the size on, layer norm 129 and 140, packed convolution 157 and 164).
// Stores marked the same way gave less, and cost up to 12% where a row is not whole
// cache lines.
constexpr long long kLastLevelCache = 256ll << 20;

}  // namespace kdn
