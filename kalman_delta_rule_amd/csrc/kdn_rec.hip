// kdn_rec.hip -- gated recurrence per channel, forward, backward and
// single-token step, gfx950.
//
//   h_t = alpha_t h_{t-1} + u_t         u = x, or (1 - alpha) x ("blend")
//   lam_t = dh_t + g_{t+1},  g_t = alpha_t lam_t  (g behind a sequence: dh_T)
//   dx = lam (1 - alpha if blend),  dalpha = lam (h_{t-1} - x if blend)
//
// Both recurrences are affine in what they carry: over any span of tokens
// carry -> A carry + U with A the product of the decays.  So a workgroup takes a
// tile of 128 or 256 tokens and 64 channels, each half-wave of it a run of tokens (two
// channels a lane): the run's (A, U) first, from registers; then one wave joins
// the runs in order, gets what the tile starts from, and hands every run its own
// start; then the runs are walked again, from the same registers, with their
// outputs stored.  Inputs are read once and outputs written once.
//
// Tiles of the same channels are chained through the workspace (Link): each
// publishes its (A, U), the last of 8 that of the whole group, and the last of 64
// the value behind it.  A tile's start is that value of the 64 before, with the
// (A, U) of the groups and tiles between applied in token order: always the same
// operations, so results do not depend on timing, and few steps that wait for
// one another (one in 64 tiles, about 2 us each, the time of a word from one XCD
// to the next; chained by groups of 8 alone, B1 T65536 D64 took 117 us instead of
// 37).  A word is 4 or 8 bytes, stored and loaded whole (relaxed, agent scope: it
// may cross to another XCD's L2), and is its own flag: a launch before sets them
// to all ones, which no published word is (a NaN is made canonical).
//
// Bound by HBM and by the time from load to store of the tiles that the registers
// hold at a time.  Measured (kernel time; bytes of inputs and outputs): forward B8
// T4096 D2048 bf16 77 us (5.2 TB/s), B1 T65536 172 us (4.7 TB/s); backward 134 us
// (5.0 TB/s) and 305 us (4.4 TB/s); with loads that are not marked as non-temporal 88,
// 184, 148 and 319 us.  fp32, alpha given, B4 T4096 D2048: 73 us (5.5 TB/s) and 118 us (5.7
// TB/s, part of it from the last-level cache).  Loading the next tile ahead in a workgroup that
// stays (128 registers, or 8 tokens a run) was slower, 111 us and more; a scratch
// access anywhere in the walks costs half the speed.
//
// Where a sequence starts (forward) or ends (backward) inside a span, A is kCut, and
// such a span gives U whatever it is handed: nothing, infinities and NaN included,
// passes from one sequence to another.  Within a sequence they stay to its end, as by
// the definition: a product of decays that underflows is kept above zero, where an
// infinity stays one, and a decay of zero makes it NaN.
#include "kdn.h"
#include "kdn_block.h"
#include "kdn_common.h"
#include "kdn_sequences.h"
#include "kdn_stream.h"

namespace kdn {

namespace {

constexpr int kChk = KDN_REC_CHECKPOINT;
constexpr int kGroup = 8;    // tiles of a group of the chain, groups of a block
constexpr int kBlock = kGroup * kGroup;
constexpr int kPolls = 1 << 18;  // about 1 us each

// ---- the chain through the workspace ----------------------------------------

struct Chain {
    uint32_t* tickets;          // [kQueues], kTicketWords apart
    unsigned long long* spans;   // [tiles][columns]: (A, U) of a tile
    unsigned long long* groups;  // [tiles / kGroup][columns]: (A, U) of a group
    uint32_t* starts;            // [tiles / kBlock][columns]: the value behind a block
    int tiles, columns;
    int queues;
};

constexpr int kQueues = 8;         // one for each XCD
constexpr int kTicketWords = 32;   // a cache line a counter

inline Chain chain_at(void* ws, int tiles, int columns, int queues)
{
    Chain c;
    c.tiles = tiles;
    c.columns = columns;
    c.queues = queues;
    c.tickets = static_cast<uint32_t*>(ws);
    c.spans = reinterpret_cast<unsigned long long*>(c.tickets + kQueues * kTicketWords);
    c.groups = c.spans + (size_t)tiles * columns;
    c.starts = reinterpret_cast<uint32_t*>(c.groups + (size_t)(tiles / kGroup) * columns);
    return c;
}

// 16-byte units of the workspace, and of the tickets at its front
constexpr size_t kTicketUnits = kQueues * kTicketWords / 4;
inline size_t chain_units(int tiles, int columns)
{
    const size_t words = ((size_t)tiles + tiles / kGroup) * 2 + tiles / kBlock;
    return kTicketUnits + (words * columns + 3) / 4;
}

__global__ __launch_bounds__(256) void rec_clear_kernel(uint4* ws, size_t n)
{
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n)
        ws[i] = i < kTicketUnits ? uint4{0, 0, 0, 0} : uint4{~0u, ~0u, ~0u, ~0u};
}

__device__ __forceinline__ uint32_t word_of(float v)
{
    return v != v ? 0x7FC00000u : __float_as_uint(v);
}

__device__ __forceinline__ void publish(uint32_t* p, float v)
{
    __hip_atomic_store(p, word_of(v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ void publish(unsigned long long* p, float A, float U)
{
    __hip_atomic_store(p, (unsigned long long)word_of(U) << 32 | word_of(A), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}

template <typename Word>
__device__ __forceinline__ Word peek(const Word* p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Wait for a word.  Tiles are handed out by ticket in the order of their
// dependences, so the tile that publishes it has its workgroup running already
// and waits for earlier ones only: the wait ends.  Were the workspace shared
// with another call against the rules, the bound on the polls ends it, with NaN.
template <typename Word>
__device__ __forceinline__ Word await(const Word* p, Word v)
{
    for (int k = 0; v == ~Word(0) && k < kPolls; ++k) {
        __builtin_amdgcn_s_sleep(1);
        v = peek(p);
    }
    return v;
}

// A of a span: the product of its decays, at least kLeast unless one of them is zero;
// kCut with a sequence's border in it (or with a decay that is NaN: U is then NaN too).
constexpr float kLeast = 0x1p-149f, kCut = __builtin_nanf("");

__device__ __forceinline__ float apply(float A, float U, float carry)
{
    return A != A ? U : fmaf(A, carry, U);
}

// The spans [kGroup - 1][columns] at p up to the n-th, as they are now.
__device__ __forceinline__ void peek_spans(unsigned long long (&w)[kGroup - 1],
                                           const unsigned long long* p, int n, int columns)
{
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i)
        w[i] = i < n ? peek(p + (size_t)i * columns) : 0;
}

__device__ __forceinline__ float2 span_of(unsigned long long w)
{
    return float2{__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}

// span a, then span b
__device__ __forceinline__ float2 join(float2 a, float2 b)
{
    const float A = a.x * b.x, least = fminf(fminf(fabsf(a.x), fabsf(b.x)), kLeast);
    return float2{A == 0.f ? least : A, apply(b.x, b.y, a.y)};
}

// For column `col` of this lane and tile `k` in chain order, whose span is
// `own`: the tiles before it in its group as one span.  Publishes its own span
// and, from a group's last tile, the group's.
__device__ __forceinline__ float2 chain_near(const Chain& ch, int k, int col, float2 own)
{
    const int g = k / kGroup, j = k % kGroup;
    const bool more = k + 1 < ch.tiles;
    unsigned long long* spans = ch.spans + (size_t)(k - j) * ch.columns + col;
    if (j != kGroup - 1 && more)
        publish(spans + (size_t)j * ch.columns, own.x, own.y);
    unsigned long long w[kGroup - 1];
    peek_spans(w, spans, j, ch.columns);
    float2 near{1.f, 0.f};
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i)
        if (i < j)
            near = join(near, span_of(await(spans + (size_t)i * ch.columns, w[i])));
    if (j == kGroup - 1 && g % kGroup != kGroup - 1 && more) {
        const float2 all = join(near, own);
        publish(ch.groups + (size_t)g * ch.columns + col, all.x, all.y);
    }
    return near;
}

// What the tile's group starts from.
__device__ __forceinline__ float chain_far(const Chain& ch, int k, int col)
{
    const int b = k / kBlock, g = k / kGroup, j = g % kGroup;
    const unsigned long long* groups = ch.groups + (size_t)(g - j) * ch.columns + col;
    unsigned long long w[kGroup - 1];
    peek_spans(w, groups, j, ch.columns);
    float carry = 0.f;
    if (b) {
        const uint32_t* start = ch.starts + (size_t)(b - 1) * ch.columns + col;
        carry = __uint_as_float(await(start, peek(start)));
    }
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i)
        if (i < j) {
            const float2 v = span_of(await(groups + (size_t)i * ch.columns, w[i]));
            carry = apply(v.x, v.y, carry);
        }
    return carry;
}

// From a block's last tile: the value behind it, which starts the next block.
__device__ __forceinline__ void chain_block(const Chain& ch, int k, int col, float behind)
{
    if (k % kBlock == kBlock - 1 && k + 1 < ch.tiles)
        publish(ch.starts + (size_t)(k / kBlock) * ch.columns + col, behind);
}

// A tile's part in the chain, by its first two waves, a lane a column; all
// threads call it.  In: the spans of its runs; out: those of the tile before
// each run, the span `near` of the tiles before it in the group and the value
// `far` that the group starts from.  REVERSE: the last run is the first.
template <int RUNS, int CT, bool REVERSE>
struct Link {
    float2 runs[RUNS][CT];
    float2 near[CT], own[CT];
    float far[CT];

    __device__ __forceinline__ void work(const Chain& ch, int k, int col)
    {
        const int wave = threadIdx.x >> 6, s = threadIdx.x & 63;
        if (wave == 0 && s < CT) {
            float2 t{1.f, 0.f};
#pragma unroll
            for (int i = 0; i < RUNS; ++i) {
                float2& r = runs[REVERSE ? RUNS - 1 - i : i][s];
                const float2 g = r;
                r = t;
                t = join(t, g);
            }
            own[s] = t;
            near[s] = ch.tiles > 1 ? chain_near(ch, k, col + s, t) : float2{1.f, 0.f};
        } else if (wave == 1 && s < CT) {
            far[s] = ch.tiles > 1 ? chain_far(ch, k, col + s) : 0.f;
        }
    }
    // after a barrier: what run `run` starts from in the tile's column s
    __device__ __forceinline__ float start(int run, int s) const
    {
        return apply(runs[run][s].x, runs[run][s].y, apply(near[s].x, near[s].y, far[s]));
    }
    __device__ __forceinline__ void finish(const Chain& ch, int k, int col) const
    {
        const int s = threadIdx.x;
        if (s < CT && ch.tiles > 1)
            chain_block(ch, k, col + s, apply(own[s].x, own[s].y, apply(near[s].x, near[s].y, far[s])));
    }
};

// ---- values ------------------------------------------------------------------

// V values of each of a run's L tokens: rows `stride` bytes apart from `base`, the
// run's first at row `first`, the lane's values at byte `col` of a row.  Where the
// tile reaches behind the row's end (`rows` < TILE), the last row is repeated.
template <bool ONCE, int TILE, typename E, int V, int L>
__device__ __forceinline__ void load_run(Raw<E, V> (&r)[L], const char* base, uint32_t stride,
                                         int first, uint32_t col, int rows)
{
    if (rows >= TILE) {
        const uint32_t off = first * stride + col;
#pragma unroll
        for (int i = 0; i < L; ++i)
            r[i] = load_raw<ONCE, E, V>(reinterpret_cast<const E*>(base + (size_t)i * stride + off));
    } else if (rows > 0) {
#pragma unroll
        for (int i = 0; i < L; ++i)
            r[i] = load_raw<ONCE, E, V>(reinterpret_cast<const E*>(base + min(first + i, rows - 1) * stride + col));
    }
}

// alpha and 1 - alpha.  From a pre-activation the smaller of the two is formed
// as e / (1 + e), e = exp(-|a|) <= 1, with full relative accuracy, the larger
// as one minus it, off by half a step: with alpha near one its error is
// carried through hundreds of products.
template <bool PRE>
__device__ __forceinline__ void gate_of(float a, float& alpha, float& rest)
{
    if constexpr (PRE) {
        const float e = __builtin_amdgcn_exp2f(fabsf(a) * -kLog2e);
        const float s = e * rcp(1.f + e), l = 1.f - s;
        alpha = a < 0.f ? s : l;
        rest = a < 0.f ? l : s;
    } else {
        alpha = a;
        rest = 1.f - a;
    }
}

// The sequences that start and end in a tile.  Of packed ones the offsets (which
// may be anything) are looked through for marks, a token each; otherwise the row is
// one sequence.
template <int TILE, int L, int THREADS>
struct Marks {
    int start[TILE], end[TILE];  // the sequence that starts or ends at the token, or -1

    // all threads of the workgroup
    __device__ __forceinline__ void fill(const RecArgs& a, int t0)
    {
        if (!a.cu)
            return;
        for (int i = threadIdx.x; i < TILE; i += THREADS)
            start[i] = end[i] = -1;
        __syncthreads();
        const SequenceRange near = sequences_at<THREADS>(a.cu, a.N, t0, TILE);
        for (int n = near.first + threadIdx.x; n < near.end; n += THREADS) {
            const int p = a.cu[n], q = a.cu[n + 1];
            if (p < 0 || p >= q)
                continue;
            if (p >= t0 && p - t0 < TILE)
                start[p - t0] = n;
            if (q > t0 && q - 1 - t0 < TILE)
                end[q - 1 - t0] = n;
        }
        __syncthreads();
    }
    // bits of the L tokens from `first` on, where a sequence starts or ends
    __device__ __forceinline__ uint32_t starts(const RecArgs& a, int t0, int first) const
    {
        return a.cu ? bits(start + first) : t0 + first == 0 && a.T > 0;
    }
    __device__ __forceinline__ uint32_t ends(const RecArgs& a, int t0, int first) const
    {
        const int last = a.T - 1 - t0 - first;
        return a.cu ? bits(end + first) : last >= 0 && last < L ? 1u << last : 0u;
    }
    // the sequence at a token of the tile whose bit is set
    __device__ __forceinline__ int starting(const RecArgs& a, int b, int i) const { return a.cu ? start[i] : b; }
    __device__ __forceinline__ int ending(const RecArgs& a, int b, int i) const { return a.cu ? end[i] : b; }

private:
    // of a half-wave's tokens
    __device__ __forceinline__ static uint32_t bits(const int* marks)
    {
        const int l = threadIdx.x & 31;
        const unsigned long long w = __ballot(l < L && marks[l < L ? l : 0] >= 0);
        return (uint32_t)((threadIdx.x & 32) ? w >> 32 : w);
    }
};

// values [V] of a state [N,D] at sequence n, channel c, or zeros where it is not given
template <int V>
__device__ __forceinline__ void state_at(const float* s, int n, int D, int c, float (&h)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        h[v] = s ? s[(size_t)n * D + c + v] : 0.f;
}

// tokens of the row that belong to a sequence
__device__ __forceinline__ int token_limit(const RecArgs& a)
{
    return a.cu ? min(max(a.cu[a.N], 0), a.T) : a.T;
}

// The A of a run from the product of the decays of its tokens (those before `valid`)
template <int L, int V>
__device__ __forceinline__ void close_run(float (&A)[V], const float (&al)[L][V], int valid, bool cut)
{
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (A[v] == 0.f) {
            bool zero = false;
#pragma unroll
            for (int i = 0; i < L; ++i)
                zero |= i < valid && al[i][v] == 0.f;
            A[v] = zero ? 0.f : kLeast;
        }
        if (cut)
            A[v] = kCut;
    }
}

// whether a mark is set at one of a run's tokens before `valid`
__device__ __forceinline__ bool any_before(uint32_t marks, int valid)
{
    return valid > 0 && (valid < 32 ? marks & ((1u << valid) - 1) : marks);
}

struct Tile {
    int k;   // in chain order
    int b, t0, c0;  // row, first token, first channel
    int col;        // first column of the chain
};

// The tile of this workgroup.  Chained tiles are taken by ticket, from one queue a
// XCD (workgroups are dealt to the XCDs in turn), each with its own share of
// the columns, adjacent ones, so that the pieces of a row that one XCD reads
// lie together, and its own counter.  Within a queue all tiles of a time come
// before the next time's.  A workgroup that finds its queue empty goes on to the
// next one: there are as many workgroups as tiles, so each gets one.
template <int TILE, int CT>
__device__ __forceinline__ Tile take_tile(const RecArgs& a, const Chain& ch, int ctiles, bool backward)
{
    const uint32_t per = a.B * ctiles;
    __shared__ int s_tile[3];
    if (threadIdx.x == 0) {
        uint32_t k = 0, r = blockIdx.x;
        if (ch.tiles > 1) {
            uint32_t q = blockIdx.x % ch.queues;
            for (int n = 0; n < ch.queues; ++n) {
                const uint32_t c0 = q * per / ch.queues, own = (q + 1) * per / ch.queues - c0;
                const uint32_t i = __hip_atomic_fetch_add(ch.tickets + q * kTicketWords, 1u,
                                                          __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                if (i < own * ch.tiles) {
                    k = i / own;
                    r = c0 + (i - k * own);
                    break;
                }
                q = q + 1 == (uint32_t)ch.queues ? 0 : q + 1;
            }
        }
        const uint32_t b = r / ctiles;
        s_tile[0] = k;
        s_tile[1] = b;
        s_tile[2] = r - b * ctiles;
    }
    __syncthreads();
    // the same for the whole wave: addresses from here on are scalar
    Tile t;
    t.k = __builtin_amdgcn_readfirstlane(s_tile[0]);
    t.b = __builtin_amdgcn_readfirstlane(s_tile[1]);
    const int ct = __builtin_amdgcn_readfirstlane(s_tile[2]);
    t.c0 = ct * CT;
    t.col = (t.b * ctiles + ct) * CT;
    t.t0 = (backward ? ch.tiles - 1 - t.k : t.k) * TILE;
    return t;
}

// ---- forward -------------------------------------------------------------------

// Half-waves of 16 tokens: eight, or sixteen where the columns are few.  A longer tile
// halves the chain, a shorter one leaves more workgroups out of step, one loading
// while another waits (D 2048 bf16, loads not marked, eight and sixteen: B8 T4096 94 and 101 us, B32
// T1024 99 and 110; B4 T4096 50 and 51; B2 T32768 177 and 164; B1 T65536 198 and 176;
// D 64, B1 T65536 37 and 23).
constexpr int kFwdRun = 16, kManyColumnTiles = 192;
int fwd_runs(long long column_tiles) { return column_tiles >= kManyColumnTiles ? 8 : 16; }

template <typename IO, bool PRE, bool BLEND, int V, int RUNS, bool ONCE>
__global__ __launch_bounds__(RUNS * 32, 4) void rec_fwd_kernel(RecArgs a, Chain ch, int ctiles)
{
    typedef typename std::conditional<PRE, IO, float>::type GT;
    constexpr int L = kFwdRun, TILE = L * RUNS, CT = 32 * V;
    __shared__ Marks<TILE, L, RUNS * 32> marks;
    __shared__ Link<RUNS, CT, false> link;

    const Tile tile = take_tile<TILE, CT>(a, ch, ctiles, false);
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    // lanes behind the last channel repeat the last ones
    const int c = min(tile.c0 + lane * V, a.D - V);
    const int first = run * L;  // of the run, in the tile
    const size_t row0 = (size_t)tile.b * a.T + tile.t0;

    Raw<GT, V> ra[L];
    Raw<IO, V> rx[L];
    const int rows = a.T - tile.t0;
    load_run<ONCE, TILE, GT, V, L>(ra, static_cast<const char*>(a.a) + row0 * a.as * sizeof(GT),
                       (uint32_t)a.as * sizeof(GT), first, c * sizeof(GT), rows);
    load_run<ONCE, TILE, IO, V, L>(rx, static_cast<const char*>(a.x) + row0 * a.xs * sizeof(IO),
                       (uint32_t)a.xs * sizeof(IO), first, c * sizeof(IO), rows);

    marks.fill(a, tile.t0);
    const int valid = token_limit(a) - (tile.t0 + first);  // tokens of the run, if positive
    const uint32_t start = marks.starts(a, tile.t0, first), end = marks.ends(a, tile.t0, first);
    const bool plain = __all(valid >= L && !start && !end);

    float al[L][V], u[L][V];
#pragma unroll
    for (int i = 0; i < L; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float rest;
            gate_of<PRE>(ra[i].get(v), al[i][v], rest);
            const float x = rx[i].get(v);
            u[i][v] = BLEND ? rest * x : x;
        }

    float A[V], U[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        A[v] = 1.f, U[v] = 0.f;
    if (plain) {
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                U[v] = fmaf(al[i][v], U[v], u[i][v]);
                A[v] *= al[i][v];
            }
    } else {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (i >= valid)
                continue;
            if (start >> i & 1)
                state_at<V>(a.h0, marks.starting(a, tile.b, first + i), a.D, c, U);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                U[v] = fmaf(al[i][v], U[v], u[i][v]);
                A[v] *= al[i][v];
            }
        }
    }
    close_run<L, V>(A, al, valid, any_before(start, valid));
#pragma unroll
    for (int v = 0; v < V; ++v)
        link.runs[run][lane * V + v] = float2{A[v], U[v]};
    __syncthreads();
    link.work(ch, tile.k, tile.col);
    __syncthreads();
    link.finish(ch, tile.k, tile.col);

    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        h[v] = link.start(run, lane * V + v);
    if (a.ckpt && (tile.t0 + first) % kChk == 0 && (valid > 0 || (a.clear && first < rows))) {
        const int blocks = (a.T + kChk - 1) / kChk;
        float* p = a.ckpt + ((size_t)tile.b * blocks + (tile.t0 + first) / kChk) * a.D + c;
        if (start & 1)
            state_at<V>(a.h0, marks.starting(a, tile.b, first), a.D, c, h);
#pragma unroll
        for (int v = 0; v < V; ++v)
            p[v] = valid > 0 ? h[v] : 0.f;
    }
    char* ph = static_cast<char*>(a.h) + row0 * a.D * sizeof(IO);
    const uint32_t sh = (uint32_t)a.D * sizeof(IO);
    const uint32_t oh = first * sh + c * (uint32_t)sizeof(IO);
    constexpr float zeros[V] = {};
    if (plain) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[v] = fmaf(al[i][v], h[v], u[i][v]);
            store_raw<IO, V>(reinterpret_cast<IO*>(ph + (size_t)i * sh + oh), h);
        }
    } else {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            IO* out = reinterpret_cast<IO*>(ph + (size_t)i * sh + oh);
            if (i >= valid) {
                if (a.clear && first + i < rows)
                    store_raw<IO, V>(out, zeros);
                continue;
            }
            if (start >> i & 1)
                state_at<V>(a.h0, marks.starting(a, tile.b, first + i), a.D, c, h);
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[v] = fmaf(al[i][v], h[v], u[i][v]);
            if ((end >> i & 1) && a.h_T) {
                float* p = a.h_T + (size_t)marks.ending(a, tile.b, first + i) * a.D + c;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    p[v] = h[v];
            }
            store_raw<IO, V>(out, h);
        }
    }

    // empty sequences keep their state
    if (tile.k == 0 && a.h_T && (!a.cu || a.N <= kStatesOfRun * RUNS)) {
        for (int n = a.cu ? run : tile.b; n < (a.cu ? a.N : tile.b + 1); n += RUNS) {
            if (a.cu ? a.cu[n] < a.cu[n + 1] : a.T > 0 || run > 0)
                continue;
#pragma unroll
            for (int v = 0; v < V; ++v)
                a.h_T[(size_t)n * a.D + c + v] = a.h0 ? a.h0[(size_t)n * a.D + c + v] : 0.f;
        }
    }
}

// ---- backward ------------------------------------------------------------------

// Sixteen half-waves of 8 tokens: the inputs, the decays and the states of 16 would not
// fit the registers of two workgroups a CU (with eight of them, B1 T65536 D2048
// bf16 353 us against 312).  The states before the runs come from the forward's
// checkpoints, so only the adjoint is chained, in reverse.
constexpr int kBwdRun = 8, kBwdRuns = 16;

template <typename IO, bool PRE, bool BLEND, int V, bool ONCE>
__global__ __launch_bounds__(kBwdRuns * 32, 4) void rec_bwd_kernel(RecArgs a, Chain ch, int ctiles)
{
    typedef typename std::conditional<PRE, IO, float>::type GT;
    constexpr int L = kBwdRun, RUNS = kBwdRuns, TILE = L * RUNS, CT = 32 * V;
    constexpr int PER = kChk / L;  // runs of a checkpoint
    __shared__ Marks<TILE, L, RUNS * 32> marks;
    __shared__ float2 spans[RUNS][CT];
    __shared__ Link<RUNS, CT, true> link;

    const Tile tile = take_tile<TILE, CT>(a, ch, ctiles, true);
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int c = min(tile.c0 + lane * V, a.D - V);
    const int first = run * L;
    const size_t row0 = (size_t)tile.b * a.T + tile.t0;

    Raw<GT, V> ra[L];
    Raw<IO, V> rx[L], rd[L];
    const int rows = a.T - tile.t0;
    load_run<ONCE, TILE, GT, V, L>(ra, static_cast<const char*>(a.a) + row0 * a.as * sizeof(GT),
                       (uint32_t)a.as * sizeof(GT), first, c * sizeof(GT), rows);
    load_run<ONCE, TILE, IO, V, L>(rx, static_cast<const char*>(a.x) + row0 * a.xs * sizeof(IO),
                       (uint32_t)a.xs * sizeof(IO), first, c * sizeof(IO), rows);
    load_run<ONCE, TILE, IO, V, L>(rd, static_cast<const char*>(a.dh) + row0 * a.D * sizeof(IO),
                       (uint32_t)a.D * sizeof(IO), first, c * sizeof(IO), rows);

    marks.fill(a, tile.t0);
    const int valid = token_limit(a) - (tile.t0 + first);
    const uint32_t start = marks.starts(a, tile.t0, first), end = marks.ends(a, tile.t0, first);
    const bool plain = __all(valid >= L && !start && !end);

    float al[L][V], rest[L][V];
#pragma unroll
    for (int i = 0; i < L; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v)
            gate_of<PRE>(ra[i].get(v), al[i][v], rest[i][v]);

    float A[V], U[V], RU[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        A[v] = 1.f, U[v] = RU[v] = 0.f;
    if (plain) {
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float x = rx[i].get(v);
                U[v] = fmaf(al[i][v], U[v], BLEND ? rest[i][v] * x : x);
                A[v] *= al[i][v];
            }
#pragma unroll
        for (int i = L - 1; i >= 0; --i)
#pragma unroll
            for (int v = 0; v < V; ++v)
                RU[v] = al[i][v] * (rd[i].get(v) + RU[v]);
    } else {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (i >= valid)
                continue;
            if (start >> i & 1)
                state_at<V>(a.h0, marks.starting(a, tile.b, first + i), a.D, c, U);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float x = rx[i].get(v);
                U[v] = fmaf(al[i][v], U[v], BLEND ? rest[i][v] * x : x);
                A[v] *= al[i][v];
            }
        }
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            if (i >= valid)
                continue;
            if (end >> i & 1)
                state_at<V>(a.dh_T, marks.ending(a, tile.b, first + i), a.D, c, RU);
#pragma unroll
            for (int v = 0; v < V; ++v)
                RU[v] = al[i][v] * (rd[i].get(v) + RU[v]);
        }
    }
    close_run<L, V>(A, al, valid, false);
    const bool starts = any_before(start, valid), ends = any_before(end, valid);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        spans[run][lane * V + v] = float2{starts ? kCut : A[v], U[v]};
        link.runs[run][lane * V + v] = float2{ends ? kCut : A[v], RU[v]};
    }
    __syncthreads();

    link.work(ch, tile.k, tile.col);

    // the states again, meanwhile: from the checkpoint over the runs between, then of
    // each token only what its gradients take, h_{t-1}, or h_{t-1} - x_t
    float h[V], part[L][V], g[V];
    const int blocks = (a.T + kChk - 1) / kChk, blk = min((tile.t0 + first) / kChk, blocks - 1);
#pragma unroll
    for (int v = 0; v < V; ++v)
        h[v] = valid > 0 ? a.ckpt[((size_t)tile.b * blocks + blk) * a.D + c + v] : 0.f;
    for (int r = run / PER * PER; r < run; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = apply(spans[r][lane * V + v].x, spans[r][lane * V + v].y, h[v]);
    auto forward = [&](int i) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float x = rx[i].get(v);
            part[i][v] = BLEND ? h[v] - x : h[v];
            h[v] = fmaf(al[i][v], h[v], BLEND ? rest[i][v] * x : x);
        }
    };
    if (plain) {
#pragma unroll
        for (int i = 0; i < L; ++i)
            forward(i);
    } else {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (start >> i & 1)
                state_at<V>(a.h0, marks.starting(a, tile.b, first + i), a.D, c, h);
            forward(i);
        }
    }
    __syncthreads();
    link.finish(ch, tile.k, tile.col);

#pragma unroll
    for (int v = 0; v < V; ++v)
        g[v] = link.start(run, lane * V + v);
    char* px = static_cast<char*>(a.dx) + row0 * a.D * sizeof(IO);
    char* pa = static_cast<char*>(a.da) + row0 * a.D * sizeof(GT);
    const uint32_t sx = (uint32_t)a.D * sizeof(IO), sa = (uint32_t)a.D * sizeof(GT);
    const uint32_t ox = first * sx + c * (uint32_t)sizeof(IO), oa = first * sa + c * (uint32_t)sizeof(GT);
    auto store = [&](int i, const float(&dx)[V], const float(&da)[V]) {
        store_raw<IO, V>(reinterpret_cast<IO*>(px + (size_t)i * sx + ox), dx);
        store_raw<GT, V>(reinterpret_cast<GT*>(pa + (size_t)i * sa + oa), da);
    };
    auto reverse = [&](int i) {
        float dx[V], da[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float lam = rd[i].get(v) + g[v];
            dx[v] = BLEND ? lam * rest[i][v] : lam;
            g[v] = al[i][v] * lam;
            // dalpha times alpha (1 - alpha), of the factors at hand
            da[v] = PRE ? g[v] * rest[i][v] * part[i][v] : lam * part[i][v];
        }
        store(i, dx, da);
    };
    constexpr float zeros[V] = {};
    if (plain) {
#pragma unroll
        for (int i = L - 1; i >= 0; --i)
            reverse(i);
    } else {
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            if (i >= valid) {
                if (a.clear && first + i < rows)
                    store(i, zeros, zeros);
                continue;
            }
            if (end >> i & 1)
                state_at<V>(a.dh_T, marks.ending(a, tile.b, first + i), a.D, c, g);
            reverse(i);
            if ((start >> i & 1) && a.dh0) {
                float* p = a.dh0 + (size_t)marks.starting(a, tile.b, first + i) * a.D + c;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    p[v] = g[v];
            }
        }
    }

    if (tile.k == 0 && a.dh0 && (!a.cu || a.N <= kStatesOfRun * RUNS)) {
        for (int n = a.cu ? run : tile.b; n < (a.cu ? a.N : tile.b + 1); n += RUNS) {
            if (a.cu ? a.cu[n] < a.cu[n + 1] : a.T > 0 || run > 0)
                continue;
#pragma unroll
            for (int v = 0; v < V; ++v)
                a.dh0[(size_t)n * a.D + c + v] = a.dh_T ? a.dh_T[(size_t)n * a.D + c + v] : 0.f;
        }
    }
}

// ---- one token ---------------------------------------------------------------------

// Four channels a thread (at a row's end those left, one by one: the state is
// updated in place, so no two threads may have the same channel).
constexpr int kStepVec = 4;

template <typename IO, bool PRE>
__global__ __launch_bounds__(256) void rec_step_kernel(RecArgs a)
{
    typedef typename std::conditional<PRE, IO, float>::type GT;
    constexpr int VE = kStepVec;
    const int c0 = (blockIdx.y * 256 + threadIdx.x) * VE, b = blockIdx.x;
    auto step = [&](auto ve, int c) {
        constexpr int N = decltype(ve)::value;
        float* st = a.h_T + (size_t)b * a.D + c;
        const auto ra = load_raw<false, GT, N>(static_cast<const GT*>(a.a) + (size_t)b * a.as + c);
        const auto rx = load_raw<false, IO, N>(static_cast<const IO*>(a.x) + (size_t)b * a.xs + c);
        const auto rs = load_raw<false, float, N>(st);
        float h[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float alpha, rest;
            gate_of<PRE>(ra.get(j), alpha, rest);
            const float x = rx.get(j);
            h[j] = fmaf(alpha, rs.get(j), a.blend ? rest * x : x);
        }
        store_raw<float, N>(st, h);
        store_raw<IO, N>(static_cast<IO*>(a.h) + (size_t)b * a.D + c, h);
    };
    if (c0 + VE <= a.D) {
        step(std::integral_constant<int, VE>{}, c0);
    } else {
        for (int c = c0; c < a.D; ++c)
            step(std::integral_constant<int, 1>{}, c);
    }
}

// The tiles of a call: of channels and of tokens.
struct Tiling {
    int ctiles, runs, tiles;  // runs: the forward's
};
Tiling tiling(int B, int T, int D, bool backward)
{
    const int ct = D == 1 ? 32 : 64;
    Tiling t;
    t.ctiles = (D + ct - 1) / ct;
    t.runs = fwd_runs((long long)B * t.ctiles);
    const int tokens = backward ? kBwdRun * kBwdRuns : kFwdRun * t.runs;
    t.tiles = T > tokens ? (int)(((long long)T + tokens - 1) / tokens) : 1;
    return t;
}

template <typename IO, bool PRE, bool BLEND, int V>
hipError_t launch(const RecArgs& a, bool backward, hipStream_t stream)
{
    const Tiling t = tiling(a.B, a.T, a.D, backward);
    const int columns = a.B * t.ctiles * 32 * V;
    // with fewer columns than XCDs some would have none of their own
    const Chain ch = chain_at(a.ws, t.tiles, columns, a.B * t.ctiles < kQueues ? 1 : kQueues);
    if (t.tiles > 1) {
        const size_t n = chain_units(t.tiles, columns);
        rec_clear_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(static_cast<uint4*>(a.ws), n);
    }
    const unsigned grid = (unsigned)t.tiles * a.B * t.ctiles;
    auto run = [&](auto once) {
        constexpr bool ONCE = decltype(once)::value;
        if (backward)
            rec_bwd_kernel<IO, PRE, BLEND, V, ONCE><<<grid, kBwdRuns * 32, 0, stream>>>(a, ch, t.ctiles);
        else if (t.runs == 8)
            rec_fwd_kernel<IO, PRE, BLEND, V, 8, ONCE><<<grid, 8 * 32, 0, stream>>>(a, ch, t.ctiles);
        else
            rec_fwd_kernel<IO, PRE, BLEND, V, 16, ONCE><<<grid, 16 * 32, 0, stream>>>(a, ch, t.ctiles);
    };
    const long long io = sizeof(IO), gate = PRE ? io : 4, values = (long long)a.B * a.T * a.D;
    const bool lines = (a.D * io | a.xs * io | a.as * gate) % kCacheLine == 0;
    if (V > 1 && values * (backward ? 3 * io + 2 * gate : 2 * io + gate) > kLastLevelCache &&
        (lines || values * io < kLastLevelCache))
        run(std::integral_constant<bool, (V > 1)>{});
    else
        run(std::false_type{});
    float* states = backward ? a.dh0 : a.h_T;
    if (states && a.cu && a.N > kStatesOfRun * (backward ? kBwdRuns : t.runs))
        launch_empty_states<float>(a.cu, a.N, a.D, backward ? a.dh_T : a.h0, states, stream);
    return hipGetLastError();
}

template <typename IO>
hipError_t launch_io(const RecArgs& a, bool backward, hipStream_t stream)
{
    // one channel alone is half a lane's pair
    if (a.D == 1)
        return a.preact ? (a.blend ? launch<IO, true, true, 1>(a, backward, stream)
                                   : launch<IO, true, false, 1>(a, backward, stream))
                        : (a.blend ? launch<IO, false, true, 1>(a, backward, stream)
                                   : launch<IO, false, false, 1>(a, backward, stream));
    return a.preact ? (a.blend ? launch<IO, true, true, 2>(a, backward, stream)
                               : launch<IO, true, false, 2>(a, backward, stream))
                    : (a.blend ? launch<IO, false, true, 2>(a, backward, stream)
                               : launch<IO, false, false, 2>(a, backward, stream));
}

}  // namespace

size_t rec_workspace_bytes(int B, int T, int D, bool backward)
{
    const Tiling t = tiling(B, T, D, backward);
    return t.tiles == 1 ? 0 : chain_units(t.tiles, B * t.ctiles * (D == 1 ? 32 : 64)) * 16;
}

unsigned long long rec_threads(int B, int T, int D, bool backward)
{
    const Tiling t = tiling(B, T, D, backward);
    return (unsigned long long)t.tiles * B * t.ctiles * 32 * (backward ? kBwdRuns : t.runs);
}

hipError_t launch_rec_fwd(const RecArgs& a, bool bf, hipStream_t stream)
{
    return bf ? launch_io<bf16>(a, false, stream) : launch_io<float>(a, false, stream);
}

hipError_t launch_rec_bwd(const RecArgs& a, bool bf, hipStream_t stream)
{
    return bf ? launch_io<bf16>(a, true, stream) : launch_io<float>(a, true, stream);
}

hipError_t launch_rec_step(const RecArgs& a, bool bf, hipStream_t stream)
{
    const dim3 grid(a.B, (a.D + 256 * kStepVec - 1) / (256 * kStepVec));
    if (bf)
        a.preact ? rec_step_kernel<bf16, true><<<grid, 256, 0, stream>>>(a)
                 : rec_step_kernel<bf16, false><<<grid, 256, 0, stream>>>(a);
    else
        a.preact ? rec_step_kernel<float, true><<<grid, 256, 0, stream>>>(a)
                 : rec_step_kernel<float, false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace kdn
