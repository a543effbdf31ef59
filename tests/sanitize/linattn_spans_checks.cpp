// The arithmetic of kdn_linattn_spans.h on the host: with any offsets every span lies in its
// segment, every sequence number in [0, N), and every walk ends; with valid ones the spans of all
// parts are the sequences, once each, and what is handed on is what they lack.  Exits nonzero
// after a failed expectation.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <vector>

#include "kdn_linattn_spans.h"

using namespace kdn;

static int failures = 0;

static uint64_t rng_state = 1;
static uint32_t rng()
{
    rng_state = rng_state * 6364136223846793005ull + 1442695040888963407ull;
    return (uint32_t)(rng_state >> 33);
}
static int below(int n) { return (int)(rng() % (uint32_t)n); }

static bool wild = false;  // any number that decreasing offsets may be counted as

struct Host {
    // what the kernels' 256 threads find: each looks at the last offset of its piece, and the
    // first piece that goes beyond x is cut into pieces again
    static int at_most(const int* p, int n, int x)
    {
        if (wild)
            return below(n + 1);
        int before = 0;
        while (n > 0) {
            const uint32_t size = (uint32_t)(n - 1) / 256 + 1;
            uint32_t within = 0;
            for (uint32_t t = 0; t < 256; ++t) {
                const uint32_t i = t * size, last = i + size < (uint32_t)n ? i + size : (uint32_t)n;
                within += i < (uint32_t)n && p[before + last - 1] <= x;
            }
            const uint32_t got = within * size;
            const int done = got < (uint32_t)n ? (int)got : n;
            before += done;
            n = ((int)size < n - done ? (int)size : n - done) - 1;
        }
        return before;
    }
};

static LinArgs args(int T, int S, const std::vector<int>& cu, int parts)
{
    LinArgs a{};
    a.B = 1, a.T = T, a.N = (int)cu.size() - 1, a.cu = cu.data();
    // as the launches choose: segments of a multiple of 64 tokens, the last one short
    a.L = S <= 1 ? T : ((T + S - 1) / S + 63) / 64 * 64;
    a.S = (T + a.L - 1) / a.L;
    a.parts = parts, a.tokens = (a.L + parts - 1) / parts;
    return a;
}

static void bad(const char* what, const LinArgs& a, int rev, const Span& x)
{
    if (++failures > 20)
        return;
    std::printf("FAILED %s: T %d S %d L %d parts %d rev %d span %d [%d, %d), offsets", what, a.T, a.S, a.L, a.parts, rev, x.n,
                x.from, x.to);
    for (int n = 0; n <= a.N && n < 12; ++n)
        std::printf(" %d", a.cu[n]);
    std::printf("\n");
}

static void check_inside(const LinArgs& a)
{
    for (int rev = 0; rev < 2; ++rev)
        for (int s = 0; s < a.S; ++s) {
            const int t0 = s * a.L, t1 = smaller(a.T, t0 + a.L);
            Span x{};
            if (a.S > 1 && handed_on<Host>(a, 0, s, rev, x)) {
                if (x.from < t0 || x.to > t1 || x.from >= x.to || x.n < 0 || x.n >= a.N)
                    bad("handed on", a, rev, x);
                if (rev ? s == 0 : s == a.S - 1)
                    bad("nothing follows", a, rev, x);
            }
            for (int part = 0; part < a.parts; ++part) {
                Spans<Host> spans;
                spans.start(a, 0, t0, t1, rev, part);
                for (int i = 0; spans.next(x, a.T); ++i) {
                    if (x.from < t0 || x.to > t1 || x.from >= x.to || x.n < 0 || x.n >= a.N)
                        bad("walk", a, rev, x);
                    if (i > a.T) {
                        bad("no end", a, rev, x);
                        break;
                    }
                }
            }
        }
}

static void check_whole(const LinArgs& a)
{
    check_inside(a);
    for (int rev = 0; rev < 2; ++rev) {
        std::vector<int> owner(a.T, -1);
        for (int s = 0; s < a.S; ++s) {
            const int t0 = s * a.L, t1 = smaller(a.T, t0 + a.L);
            for (int part = 0; part < a.parts; ++part) {
                Spans<Host> spans;
                spans.start(a, 0, t0, t1, rev, part);
                Span x{};
                while (spans.next(x, a.T)) {
                    const int p = a.cu[x.n], e = a.cu[x.n + 1];
                    if (x.from != larger(p, t0) || x.to != smaller(e, t1) || x.first != (rev ? x.to == e : x.from == p) ||
                        x.last != (rev ? x.from == p : x.to == e))
                        bad("a sequence's tokens", a, rev, x);
                    for (int t = x.from; t < x.to; ++t) {
                        if (owner[t] >= 0)
                            bad("twice", a, rev, x);
                        owner[t] = x.n;
                    }
                }
            }
            // the state on the border to the next segment, where a sequence goes on over it
            const int border = rev ? t0 : t1;
            int n = -1;
            for (int m = 0; m < a.N; ++m)
                if (a.cu[m] < border && a.cu[m + 1] > border)
                    n = m;
            Span x{};
            const bool some = handed_on<Host>(a, 0, s, rev, x);
            if (some != (n >= 0))
                bad("whether it is handed on", a, rev, x);
            else if (some && (x.n != n || x.from != larger(a.cu[n], t0) || x.to != smaller(a.cu[n + 1], t1) ||
                              x.first != (rev ? a.cu[n + 1] <= t1 : a.cu[n] >= t0)))
                bad("what is handed on", a, rev, x);
        }
        for (int t = 0; t < a.T; ++t) {
            int n = -1;
            for (int m = 0; m < a.N; ++m)
                if (a.cu[m] <= t && t < a.cu[m + 1])
                    n = m;
            if (owner[t] != n)
                bad("a token's sequence", a, rev, Span{owner[t], t, t + 1, false, false});
        }
    }
}

int main()
{
    // lengths that are not whole segments, offsets above T, below zero and decreasing
    for (int S : {1, 2, 8, 11})
        for (int parts : {1, 3, 64})
            for (const std::vector<int>& cu : std::vector<std::vector<int>>{
                     {0, 900, 100, 5000, 1400}, {-5, 3, -1, 70000, 2}, {1500, 0, 1500, 0, 1500}, {7, 7, 7, 7, 9},
                     {0, 5000}, {0, INT_MAX}, {INT_MIN, INT_MAX}, {-1, 1536}, {0, 1500, 1537}, {0, 1501}})
                check_inside(args(1500, S, cu, parts));
    const int any[] = {INT_MIN, -70000, -1, 0, 1, 63, 64, 65, 1 << 20, INT_MAX};
    for (int i = 0; i < 20000; ++i) {
        const int T = 1 + below(i % 4 ? 700 : 3000), N = 1 + below(i % 8 ? 9 : 600);
        std::vector<int> cu(N + 1);
        for (int& c : cu)
            c = below(4) ? below(T + 300) - 100 : any[below(10)];
        if (i % 2)
            cu[0] = 0;
        const LinArgs a = args(T, 1 + below(12), cu, 1 + below(8));
        wild = i % 3 == 0;
        check_inside(a);
        wild = false;
    }
    // valid offsets, empty sequences among them, with and without tokens behind the last one
    for (int i = 0; i < 3000; ++i) {
        const int T = 1 + below(i % 4 ? 300 : 1500), N = 1 + below(i % 8 ? 9 : 400);
        const int end = i % 3 ? T : below(T + 1);
        std::vector<int> cu(N + 1);
        for (int& c : cu)
            c = below(end + 1);
        cu[0] = 0, cu[N] = end;
        for (size_t k = 1; k < cu.size(); ++k)  // in order
            for (size_t j = k; j > 0 && cu[j - 1] > cu[j]; --j) {
                const int t = cu[j];
                cu[j] = cu[j - 1], cu[j - 1] = t;
            }
        check_whole(args(T, 1 + below(12), cu, 1 + below(8)));
    }
    if (failures) {
        std::printf("%d failures\n", failures);
        return 1;
    }
    std::printf("all checks passed\n");
    return 0;
}
