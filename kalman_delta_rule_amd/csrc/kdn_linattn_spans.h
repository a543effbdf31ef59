// kdn_linattn_spans.h -- which tokens a walk of linear attention reads: the spans of a segment's
// sequences, and what a segment hands on.  Offsets may hold anything: every span that comes out
// lies in its segment and so in [0, T), and a sequence's number in [0, N).  Plain arithmetic,
// which the host can run too: `Count` finds how many of the offsets p[0], .. p[n - 1] are at most
// x (some number from 0 to n where they decrease).
#pragma once

#include <hip/hip_runtime.h>

#include "kdn_linattn.h"

namespace kdn {

#define KDN_SPANS __host__ __device__ inline __attribute__((always_inline))

KDN_SPANS int smaller(int a, int b) { return a < b ? a : b; }
KDN_SPANS int larger(int a, int b) { return a > b ? a : b; }

// Tokens [from, to) of sequence n, and whether they hold its first and last token in
// the order of the walk
struct Span {
    int n, from, to;
    bool first, last;
};

// The spans of one segment [t0, t1) of a row, in the order of the walk; with offsets, those
// that begin in a part of it.  They follow one another.
template <typename Count>
struct Spans {
    const int* cu;
    int N, t0, t1, rev, at, n;
    int u0, u1;  // the part

    // (all threads) cu[n] <= token, the last such n
    KDN_SPANS int holding(int token) const { return Count::at_most(cu, N, token) - 1; }

    KDN_SPANS void start(const LinArgs& a, int b, int begin, int end, int backwards, int part)
    {
        cu = a.cu, N = a.N, t0 = begin, t1 = end, rev = backwards;
        u0 = smaller(t1, t0 + part * a.tokens), u1 = smaller(t1, u0 + a.tokens);
        at = rev ? u1 : u0;
        n = cu ? -1 : b;
        if (cu && u0 < u1 && at != (rev ? t1 : t0)) {
            // a sequence that goes on here is the neighbour's
            const int m = holding(at - 1);
            if (m >= 0 && cu[m + 1] > at)
                at = rev ? larger(smaller(cu[m], at), u0) : smaller(cu[m + 1], u1);
        }
    }
    KDN_SPANS bool next(Span& s, int T)
    {
        if (rev ? at <= u0 : at >= u1)
            return false;
        if (!cu) {
            s = Span{n, t0, t1, rev ? t1 == T : t0 == 0, rev ? t0 == 0 : t1 == T};
            at = rev ? t0 : t1;
            return true;
        }
        // the sequence of the next token: mostly the neighbour of the last one
        const int token = rev ? at - 1 : at;
        int m = rev ? n - 1 : n + 1;
        if (n < 0 || m < 0 || m >= N || cu[m] > token || cu[m + 1] <= token)
            m = holding(token);
        if (m < 0 || cu[m + 1] <= token) {
            // behind the last sequence; backwards there may be sequences before
            if (!rev || m < 0)
                return false;
            const int e = smaller(cu[m + 1], token);
            if (e <= u0)
                return false;
            at = e;
            n = -1;
            return next_of(s, holding(e - 1));
        }
        return next_of(s, m);
    }
    KDN_SPANS bool next_of(Span& s, int m)
    {
        if (m < 0)
            return false;
        const int p = cu[m], e = cu[m + 1];
        s.n = m;
        if (rev) {
            s.to = at, s.from = larger(p, t0);
            if (s.from >= s.to || e < at)
                return false;
            s.first = e == s.to, s.last = p == s.from;
            at = s.from;
        } else {
            s.from = at, s.to = smaller(e, t1);
            if (s.to <= s.from || p > at)
                return false;
            s.first = p == s.from, s.last = e == s.to;
            at = s.to;
        }
        n = m;
        return true;
    }
};

// Which tokens of segment s the state that it hands on to the next one (in the order of the walk)
// comes from: false where the next one begins with a sequence of its own.  The last segment hands
// nothing on, whatever offsets behind it claim (its border may lie beyond T).
template <typename Count>
KDN_SPANS bool handed_on(const LinArgs& a, int b, int s, int rev, Span& x)
{
    // the border between segment s and the next one in the order of the walk
    const int border = rev ? s * a.L : (s + 1) * a.L;
    if (rev ? s == 0 : border >= a.T)
        return false;
    const int t0 = s * a.L, t1 = smaller(a.T, t0 + a.L);
    x.n = b;
    int p = 0, e = a.T;
    if (a.cu) {
        x.n = Count::at_most(a.cu, a.N, border - 1) - 1;
        if (x.n < 0)
            return false;
        p = a.cu[x.n], e = a.cu[x.n + 1];
    }
    if (p >= border || e <= border)
        return false;
    x.from = rev ? border : larger(p, t0);
    x.to = rev ? smaller(e, t1) : border;
    x.first = rev ? e <= t1 : p >= t0;
    x.last = false;
    return true;
}

}  // namespace kdn
