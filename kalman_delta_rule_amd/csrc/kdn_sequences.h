// kdn_sequences.h -- packed sequences, however many: those that touch a tile of tokens.
// The offsets may hold anything: what is read lies within their N sequences all the same.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kdn {

// How many of the offsets p[0], .. p[n - 1] are at most x, by THREADS threads, all of
// which call it: each looks at the last offset of its piece, and the first piece that
// goes beyond x is cut into pieces again.  (Offsets that decrease give some number from
// 0 to n.)
template <int THREADS>
__device__ __forceinline__ int count_at_most(const int* p, int n, int x)
{
    int before = 0;
    while (n > 0) {
        const uint32_t size = (uint32_t)(n - 1) / THREADS + 1, i = threadIdx.x * size;
        const bool within = i < (uint32_t)n && p[before + min(i + size, (uint32_t)n) - 1] <= x;
        const int done = (int)min((uint32_t)__syncthreads_count(within) * size, (uint32_t)n);
        before += done;
        n = min((int)size, n - done) - 1;
    }
    return before;
}

struct SequenceRange {
    int first, end;
};

// Sequences among which are all those that start or end at the tokens [t0, t0 + count).
// A few offsets a thread are looked through faster than searched (65536 tokens of 512
// channels, us, looked through and searched: convolution forward N 1000 42 and 45, N 2000
// 51 and 50, N 4096 66 and 57; recurrence backward N 2000 136 and 141, N 8192 175 and
// 163; N 65536 521 and 172, 598 and 262).
template <int THREADS>
__device__ __forceinline__ SequenceRange sequences_at(const int* cu, int N, int t0, int count)
{
    if (N <= 8 * THREADS)
        return {0, N};
    const int first = count_at_most<THREADS>(cu + 1, N, t0);  // those end at t0 or before
    return {first, first + count_at_most<THREADS>(cu + first, N - first, t0 + count - 1)};
}

}  // namespace kdn
