// kdn_block_device.h -- device helpers that the operators around the mixer share.
#pragma once

#include "kdn_block.h"
#include "kdn_common.h"

namespace kdn {

// The sequence that token t of row b belongs to and its span [p, q) in the
// row; n = -1 where it belongs to none.  With any offsets n stays in [0, N).
struct Span {
    int n, p, q;
};
__device__ __forceinline__ Span span_of(const int* cu, int N, int b, int t, int T)
{
    if (!cu)
        return {b, 0, T};
    int lo = 0, hi = N;  // the last n with cu[n] <= t
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (cu[m] <= t)
            lo = m;
        else
            hi = m;
    }
    const int p = cu[lo], q = min(cu[lo + 1], T);
    return (p >= 0 && p <= t && t < q) ? Span{lo, p, q} : Span{-1, t, t + 1};
}

}  // namespace kdn
