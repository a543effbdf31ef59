// kdn_sequences.h -- packed sequences, however many: those that touch a tile of tokens,
// and the states of empty ones.  The offsets may hold anything: what is read and written
// lies within their N sequences all the same.
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

// The states of empty sequences are looked after by the kernels' first tile of tokens,
// its runs taking turns, up to so many a run; of more by a launch of their own, 2 us at
// the least (N sequences in 1000 tokens of 2048 channels, us, turns and launch:
// recurrence, 16 runs, N 300 27.1 and 28.5, N 1000 65.6 and 39.6; convolution, 4 runs,
// N 300 32 and 17; in 65536 tokens of 512, N 65536, 11800 and 520).
constexpr int kStatesOfRun = 20;

// to[n] = from[n] (zeros where that is not given), rows of `width`, for empty sequences n:
// of cu, or all of them without.  16 sequences a wave and time, 256 columns a workgroup and
// time (rows may be wider than a grid's second axis holds workgroups).
template <typename E>
__global__ __launch_bounds__(256) void empty_states_kernel(const int* cu, int N, int width, const E* from, E* to)
{
    const int lane = threadIdx.x & 63;
    for (long long n0 = (blockIdx.x * 4ll + (threadIdx.x >> 6)) * 16; n0 < N; n0 += gridDim.x * 64ll) {
        const long long n = n0 + lane;
        const bool empty = lane < 16 && n < N && (!cu || cu[n] >= cu[n + 1]);
        for (unsigned long long left = __ballot(empty); left; left &= left - 1) {
            const size_t row = (size_t)(n0 + __builtin_ctzll(left)) * width;
            for (int c0 = blockIdx.y * 256; c0 < width; c0 += gridDim.y * 256)
                for (int c = c0 + lane; c < min(c0 + 256, width); c += 64)
                    to[row + c] = from ? from[row + c] : E(0);
        }
    }
}

template <typename E>
void launch_empty_states(const int* cu, int N, int width, const void* from, void* to, hipStream_t stream)
{
    const long long groups = ((long long)N + 63) / 64;
    const unsigned columns = ((unsigned)width + 255) / 256;
    const dim3 grid(groups < 4096 ? (unsigned)groups : 4096u, columns < 4096 ? columns : 4096u);
    empty_states_kernel<E><<<grid, 256, 0, stream>>>(cu, N, width, static_cast<const E*>(from), static_cast<E*>(to));
}

}  // namespace kdn
