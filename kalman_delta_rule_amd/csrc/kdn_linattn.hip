// kdn_linattn.hip -- linear attention with a decay for each head, gfx950.
//
//   S_t = g S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
//
// Every pass over a sequence is one walk with a state X [kd x vd] and inputs
// q, k [kd], v [vd] a token, in the order of the walk:
//
//   y_i = of_x g^(i + 1 - late) X^T q_i + of_p sum_{j <= i} g^(i - j) (q_i k_j) v_j
//   X  <- g^C X + of_u sum_j g^(C - 1 - j + late) k_j v_j^T          (chunks of C tokens)
//
//   forward   y = o:  q, k, v; state S
//   backward  y = dq: do, v, k forwards, state S^T
//             y = dv: k, q, do backwards, state dL/dS, with late = 1: a state behind a
//                     token has decayed once more before it meets that token's k
//             y = dk: v, do, q backwards, state (dL/dS)^T, late = 1
//
// A workgroup of four waves has one head and 64 columns of v and X.  A wave keeps X of
// its 16 columns in matrix accumulators for the whole walk: they are at once the operand
// of q X.  q k^T is formed transposed, so that
// a lane's four values are adjacent in a row of the decayed product, which goes through
// LDS to all waves.  The token's decay is put on v, in registers, not on k.
//
// bf16: the products' operands are bf16, sums and states fp32.  q, k, v are exact.  What
// is rounded to an operand once: the decayed q k (2^-8 of each term of a y that is
// itself rounded to 2^-8) and X where y is formed from it (the same).  X itself is summed
// from v's decayed values as two bf16 parts (2^-16 of each term), since states are fp32
// outputs.  fp32: matrix instructions with fp32 operands throughout.
#include "kdn_common.h"
#include "kdn_linattn.h"
#include "kdn_sequences.h"
#include "kdn_stream.h"

#include <type_traits>

// the steps of a walk are lambdas; called out of line they would put the state into memory
#define KDN_INLINE __attribute__((always_inline))

namespace kdn {

namespace {

constexpr int kThreads = 256, kCols = 64;  // columns of v a workgroup

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// A matrix in LDS, rows of W elements without a gap.  Its 16-byte blocks are exchanged
// within a row by a number that goes by the row, so that all banks are busy in each of
// the ways it is read: one block of 16 rows, and
// - bf16, read transposed: pieces of 4 to 16 bytes of 4 adjacent rows;
// - fp32, read by columns: 4 blocks of rows that lie 4 apart.
// (256 bytes are all banks: of rows of 128 or 64 bytes, two or four lie side by side.)
// The number's bits are bits of the row, so a place ROW rows and BLOCK blocks further, in
// bits that the place itself has not set, is an exclusive or and an offset away.
template <typename IO, int W>
struct Lds {
    static constexpr int VE = 16 / sizeof(IO), BLOCKS = W / VE, BYTES = W * sizeof(IO);
    static_assert(BLOCKS == 4 || BLOCKS == 8 || BLOCKS % 16 == 0, "rows of 64, 128 or whole 256 bytes");
    static __device__ __forceinline__ constexpr int turn(int row)
    {
        if constexpr (sizeof(IO) == 4)
            return BLOCKS == 8 ? (row >> 1 & 1) | (row >> 1 & 6) : (row >> 2 & 3) << 2 | (row & 3);
        else
            return BLOCKS == 4   ? row >> 2 & 3
                   : BLOCKS == 8 ? (row >> 1 & 1) << 2 | (row >> 2 & 3)
                                 : (row & 3) << 2 | (row >> 2 & 3);
    }
    // bytes from the matrix's front, which is a multiple of 256
    static __device__ __forceinline__ uint32_t at(int row, int block)
    {
        return row * BYTES + ((block ^ turn(row)) << 4);
    }
    static __device__ __forceinline__ uint32_t further(uint32_t place, int row, int block)
    {
        return (place ^ (uint32_t)((turn(row) ^ (block & 15)) << 4)) + row * BYTES + (block >> 4) * 256;
    }
};

template <typename V>
__device__ __forceinline__ V lds_read(uint32_t at)
{
    return *(const __attribute__((address_space(3))) V*)(size_t)at;
}
template <typename V>
__device__ __forceinline__ void lds_write(uint32_t at, const V& v)
{
    *(__attribute__((address_space(3))) V*)(size_t)at = v;
}

// Operands of one step of a 16 x 16 product, and how they are read.  A lane (g, c) =
// (lane / 16, lane % 16) holds VE adjacent k for row c of an operand, VE g the first.  The
// state's accumulators are such an operand: of the two tiles of 16 rows that a step of 32
// takes in bf16, the first stands for rows 8 g .. 8 g + 3 of the step, the second for
// 8 g + 4 .. 8 g + 7 (an accumulator's lane holds rows 4 g .. 4 g + 3 of its tile).
template <typename IO>
struct Op;

template <>
struct Op<bf16> {
    typedef bf16x8 frag;
    static constexpr int K = 32;  // of a step
    static constexpr int VE = 8;  // elements of 16 bytes
    // row of the state that tile t's row 4 g + e stands for
    static __device__ __forceinline__ int state_row(int t, int g, int e) { return 32 * (t / 2) + 8 * g + 4 * (t % 2) + e; }
    // From a matrix whose columns hold the k, [k][row]: the transposing read gives lane j of
    // 16 element j % 4 of the 8 bytes that lanes 4 e + j / 4 address, e = 0 .. 3.  Place of the
    // first piece; the operand's rows are four pieces of 4 columns, `apart` elements apart.
    template <int W>
    static __device__ __forceinline__ uint32_t cols_at(int col, int apart, int lane)
    {
        const int at = col + apart * (lane & 3);
        return Lds<bf16, W>::at(8 * (lane >> 4) + ((lane >> 2) & 3), at / 8) + at % 8 * 2;
    }
    template <int W>
    static __device__ __forceinline__ frag cols(uint32_t place, int step, int block)
    {
        const auto a = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4*)(size_t)Lds<bf16, W>::further(place, 32 * step, block)));
        const auto b = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4*)(size_t)Lds<bf16, W>::further(place, 32 * step + 4, block)));
        return frag{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
    // rows of the state's tile t, from [k][row]
    template <int W>
    static __device__ __forceinline__ frag state_cols(uint32_t place, int step, int t)
    {
        return cols<W>(place + 8 * (t % 2), step, 4 * (t / 2));
    }
    static constexpr int kApart = 8;  // of cols_at for them
    static __device__ __forceinline__ void mma(f32x4& acc, const frag& a, const frag& b)
    {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
    }
};

template <>
struct Op<float> {
    typedef f32x4 frag;
    static constexpr int K = 16, VE = 4, kApart = 4;
    static __device__ __forceinline__ int state_row(int t, int g, int e) { return 16 * t + 4 * g + e; }
    template <int W>
    static __device__ __forceinline__ uint32_t cols_at(int col, int, int lane)
    {
        const int at = col + (lane & 15);
        return Lds<float, W>::at(4 * (lane >> 4), at / 4) + at % 4 * 4;
    }
    template <int W>
    static __device__ __forceinline__ frag cols(uint32_t place, int step, int block)
    {
        frag x;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[e] = lds_read<float>(Lds<float, W>::further(place, 16 * step + e, block));
        return x;
    }
    template <int W>
    static __device__ __forceinline__ frag state_cols(uint32_t place, int step, int t)
    {
        return cols<W>(place, step, 4 * t);
    }
    static __device__ __forceinline__ void mma(f32x4& acc, const frag& a, const frag& b)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], acc, 0, 0, 0);
    }
};

// From a matrix whose rows hold the k, [row][k]: place of row c's first piece, and the
// operand of 16 rows from `row` on.
template <typename IO, int W>
__device__ __forceinline__ uint32_t rows_at(int lane)
{
    return Lds<IO, W>::at(lane & 15, lane >> 4);
}
template <typename IO, int W>
__device__ __forceinline__ typename Op<IO>::frag rows(uint32_t place, int row, int step)
{
    return lds_read<typename Op<IO>::frag>(Lds<IO, W>::further(place, row, 4 * step));
}

// g^n, n >= 0.  The exponent's product is formed in 64 bits: its rounding would show
// in powers of a decay near one.
struct Decay {
    double log;
    __device__ __forceinline__ float power(int n) const { return n > 0 ? expf((float)(n * log)) : 1.f; }
};

// Elements of 16 bytes, as in memory.
template <typename IO>
struct Piece {
    static constexpr int VE = Op<IO>::VE;
    typedef uint32_t four __attribute__((ext_vector_type(4)));
    four w;
    // its first n elements, at any alignment of an element
    __device__ __forceinline__ void store(IO* p, int n) const
    {
        if (n >= VE) {
            typedef Words<IO, 4> W;
            *reinterpret_cast<W*>(p) = w;
            return;
        }
        IO e[VE];
        __builtin_memcpy(e, &w, 16);
#pragma unroll
        for (int j = 0; j < VE; ++j)
            if (j < n)
                p[j] = e[j];
    }
};

// A tile of C tokens by W columns, of which `width` are there: 16 bytes a thread and turn,
// always of the same columns.  Loads go through a buffer descriptor that ends behind the
// tile's last element: rows and columns that are not there read as zero without a branch.
template <typename IO, int C, int W>
struct Tile {
    static constexpr int VE = Op<IO>::VE, PER = W / VE, ROWS = kThreads / PER, NP = C / ROWS;
    static_assert(kThreads % PER == 0 && C % ROWS == 0, "whole turns of the threads");
    static __device__ __forceinline__ int row(int i) { return i * ROWS + (int)threadIdx.x / PER; }
    static __device__ __forceinline__ int col() { return (int)threadIdx.x % PER * VE; }
    // rows p, p + ts, .. or, backwards, from the last to p
    static __device__ __forceinline__ void load(Piece<IO> (&x)[NP], const IO* p, int ts, int len, int width, bool back)
    {
        constexpr int E = sizeof(IO);
        const int end = ((len - 1) * ts + width) * E;
        const bool odd = E == 2 && ((reinterpret_cast<uintptr_t>(p) & 3) || (ts & 1));
        // a word that ends half a word behind the last element is read whole where words are
        // aligned (it lies in one page); elsewhere it is out of range
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<IO*>(p), (short)0, odd ? end : (end + 3) & ~3, 0x00020000);
        int at = ((back ? len - 1 - row(0) : row(0)) * ts + col()) * E;
        const int step = (back ? -ROWS : ROWS) * ts * E;
        if (col() >= width)
            at = (int)0x80000000u;  // out of range, and so are steps of it: a tile spans less than 2^30 bytes
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            x[i].w = __builtin_bit_cast(typename Piece<IO>::four, __builtin_amdgcn_raw_buffer_load_b128(
                rsrc, (uint32_t)at + (uint32_t)(i * step), 0u, 0));
        }
        if (odd && ((width - 1) % VE) % 2 == 0) {
            const int last = back ? 0 : len - 1;
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (row(i) == last && col() == (width - 1) / VE * VE) {
                    const uint32_t e = *reinterpret_cast<const uint16_t*>(p + (ptrdiff_t)(len - 1) * ts + width - 1);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[i].w[j] = j == (width - 1) % VE / 2 ? e : x[i].w[j];
                }
        }
    }
    // place of this thread's first piece
    static __device__ __forceinline__ uint32_t place() { return Lds<IO, W>::at(row(0), col() / VE); }
    static __device__ __forceinline__ uint32_t place(uint32_t first, int i) { return Lds<IO, W>::further(first, i * ROWS, 0); }
    static __device__ __forceinline__ void put(Piece<IO> (&x)[NP], uint32_t first, int width)
    {
        // elements of a piece behind the row's end: the next head's, or the next token's
        if (width % VE) {
            constexpr int EW = VE / 4;  // elements of a word
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = width - col() - j * EW;
                const uint32_t mask = n >= EW ? ~0u : n <= 0 ? 0u : 0xFFFFu;
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    x[i].w[j] &= mask;
            }
        }
#pragma unroll
        for (int i = 0; i < NP; ++i)
            lds_write(place(first, i), x[i].w);
    }
};

// Tokens [from, to) of sequence n, and whether they hold its first and last token in
// the order of the walk
struct Span {
    int n, from, to;
    bool first, last;
};

// The spans of one segment [t0, t1) of a row, in the order of the walk.  Offsets may hold
// anything: spans lie in the segment and follow one another.
struct Spans {
    const int* cu;
    int N, t0, t1, rev, at, n;

    // (all threads) cu[n] <= token, the last such n
    __device__ __forceinline__ int holding(int token) const { return count_at_most<kThreads>(cu, N, token) - 1; }

    __device__ __forceinline__ void start(const LinArgs& a, int b, int begin, int end, int backwards)
    {
        cu = a.cu, N = a.N, t0 = begin, t1 = end, rev = backwards;
        at = rev ? t1 : t0;
        n = -1;
        if (!cu)
            n = b;
    }
    __device__ __forceinline__ bool next(Span& s, int T)
    {
        if (rev ? at <= t0 : at >= t1)
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
            const int e = min(cu[m + 1], token);
            if (e <= t0)
                return false;
            at = e;
            n = -1;
            return next_of(s, holding(e - 1));
        }
        return next_of(s, m);
    }
    __device__ __forceinline__ bool next_of(Span& s, int m)
    {
        if (m < 0)
            return false;
        const int p = cu[m], e = cu[m + 1];
        s.n = m;
        if (rev) {
            s.to = at, s.from = max(p, t0);
            if (s.from >= s.to || e < at)
                return false;
            s.first = e == s.to, s.last = p == s.from;
            at = s.from;
        } else {
            s.from = at, s.to = min(e, t1);
            if (s.to <= s.from || p > at)
                return false;
            s.first = p == s.from, s.last = e == s.to;
            at = s.to;
        }
        n = m;
        return true;
    }
};

// Which tokens of the segment before (in the order of the walk) the state handed on to
// segment s comes from: false where s begins with a sequence of its own.
__device__ __forceinline__ bool handed_on(const LinArgs& a, int b, int s, int rev, Span& x)
{
    // the border between segment s and the next one in the order of the walk
    const int border = rev ? s * a.L : (s + 1) * a.L;
    const int t0 = s * a.L, t1 = min(a.T, t0 + a.L);
    x.n = b;
    int p = 0, e = a.T;
    if (a.cu) {
        x.n = count_at_most<kThreads>(a.cu, a.N, border - 1) - 1;
        if (x.n < 0)
            return false;
        p = a.cu[x.n], e = a.cu[x.n + 1];
    }
    if (p >= border || e <= border)
        return false;
    x.from = rev ? border : max(p, t0);
    x.to = rev ? min(e, t1) : border;
    x.first = rev ? e <= t1 : p >= t0;
    x.last = false;
    return true;
}

template <typename IO, int KD, int C>
struct Walk {
    typedef Op<IO> O;
    typedef typename O::frag frag;
    typedef Tile<IO, C, KD> TK;
    typedef Tile<IO, C, kCols> TV;
    static constexpr int NT = C / 16, ST = KD / 16, KS = KD / O::K, CS = C / O::K, FE = O::K / 4;
    static constexpr bool BF = sizeof(IO) == 2;
    static constexpr int E = sizeof(IO), kTileK = C * KD * E, kTileV = C * kCols * E, kTileP = C * C * E;  // bytes
    static constexpr int kLds = 2 * kTileK + kTileV + kTileP + C * 4;
};

// STATE: the states that segments hand on, nothing else
template <typename IO, int KD, int C, bool STATE>
__global__ __launch_bounds__(kThreads, 2) void linattn_kernel(LinArgs a)
{
    typedef Walk<IO, KD, C> W;
    typedef typename W::O O;
    typedef typename W::frag frag;
    typedef typename W::TK TK;
    typedef typename W::TV TV;
    typedef Lds<IO, kCols> LV;
    typedef Lds<IO, C> LP;
    typedef Lds<IO, KD> LK;
    constexpr int NT = W::NT, ST = W::ST, KS = W::KS, CS = W::CS, FE = W::FE;
    constexpr bool BF = W::BF;
    __shared__ __attribute__((aligned(256))) char lds[W::kLds];
    const uint32_t Qs = (uint32_t)(size_t)(__attribute__((address_space(3))) char*)lds;
    const uint32_t Ks = Qs + W::kTileK, Vs = Ks + W::kTileK, Ps = Vs + W::kTileV,
                   Ws = Ps + W::kTileP;  // of_u g^(len - 1 - j + rev), of each token of a chunk of `len`

    const LinRole& r = a.role[blockIdx.y];
    // slices of one head follow one another on one XCD (workgroups go round the eight)
    const int slices = (r.vd + kCols - 1) / kCols;
    const int index = blockIdx.x / 8, unit = index / slices * 8 + (int)(blockIdx.x & 7), slice = index % slices;
    if (unit >= a.B * a.H * a.S)
        return;
    const int h = unit % a.H, s = unit / a.H % a.S, b = unit / a.H / a.S;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, c = lane & 15;
    const int col0 = slice * kCols, width = min(r.vd - col0, kCols);  // of v
    const int mine = 16 * wave + c, mycol = col0 + mine;
    const int rev = r.rev, dir = rev ? -1 : 1;

    const long long row0 = (long long)b * a.T;
    const IO* q = static_cast<const IO*>(r.q.p) + (long long)(h / r.q.div) * r.q.hs;
    const IO* k = static_cast<const IO*>(r.k.p) + (long long)(h / r.k.div) * r.k.hs;
    const IO* v = static_cast<const IO*>(r.v.p) + (long long)(h / r.v.div) * r.v.hs + col0;

    const Decay decay{log((double)a.decay[h])};
    // decays of q k^T: lane (g, c) holds rows j = 4 g + e of column i = c of a 16 x 16
    // block; those below the diagonal block are 16 further each
    float on[4], below[4], front[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        on[e] = c >= 4 * g + e ? r.of_p * decay.power(c - 4 * g - e) : 0.f;
        below[e] = r.of_p * decay.power(16 + c - 4 * g - e);
        front[e] = r.of_x * decay.power(4 * g + e + 1 - rev);
    }
    const float g16 = decay.power(16);
    int held = -1;  // tokens of the chunk that Ws is for
    float whole = 0.f;

    f32x4 X[ST];
    const size_t dense = (size_t)r.kd * r.vd;
    // elements that are not there are out of the descriptor's range: read as zero, not written
    auto state = [&](const float* p, int rs, int cs, auto each) KDN_INLINE {
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p), (short)0, (int)dense * 4, 0x00020000);
        int at = mycol < r.vd ? mycol * cs * 4 : 1 << 30;
        asm volatile("" : "+v"(at));  // formed here, not held over the walk
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = O::state_row(t, g, e);
                each(rsrc, i < r.kd ? at + i * rs * 4 : 1 << 30, t, e);
            }
    };
    auto state_in = [&](const float* p, int rs, int cs) KDN_INLINE {
        if (!p) {
#pragma unroll
            for (int t = 0; t < ST; ++t)
                X[t] = zero4();
            return;
        }
        state(p, rs, cs, [&](auto rsrc, int at, int t, int e) KDN_INLINE {
            X[t][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsrc, at, 0, 0));
        });
    };
    auto state_out = [&](float* p, int rs, int cs) KDN_INLINE {
        state(p, rs, cs, [&](auto rsrc, int at, int t, int e) KDN_INLINE {
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(X[t][e]), rsrc, at, 0, 0);
        });
    };
    auto handed = [&](int seg) KDN_INLINE { return r.seg + (((size_t)b * a.S + seg) * a.H + h) * dense; };

    // blocks of the decayed product above the diagonal that a step of K tokens covers
    if constexpr (!STATE) {
        for (int i = threadIdx.x * 4; i < W::kTileP; i += kThreads * 4)
            lds_write(Ps + i, 0);
    }

    // places in LDS, of a lane or a thread, in the first row or tile that it touches
    uint32_t kput = Ks + TK::place(), vput = Vs + TV::place();
    uint32_t qrow = Qs + rows_at<IO, KD>(lane), kcol = Ks + O::template cols_at<KD>(0, O::kApart, lane);
    uint32_t vcol = Vs + O::template cols_at<kCols>(16 * wave, 4, lane);
    uint32_t prow = Ps + rows_at<IO, C>(lane);
    // C = 64: a wave forms q k^T for 16 tokens' k and every q behind; C = 32: for one block of q
    const int jt = NT == 4 ? wave : wave & 1;
    uint32_t pput = Ps + LP::at(c, (16 * jt + 4 * g) / O::VE) + 4 * g % O::VE * W::E;
    uint32_t yput = Vs + LV::at(4 * g, mine / O::VE) + mine % O::VE * W::E;

    Piece<IO> nq[STATE ? 1 : TK::NP], nk[TK::NP], nv[TV::NP];
    // the chunk of `len` tokens whose first (in the order of the walk) is `token`
    auto fetch = [&](int token, int len) KDN_INLINE {
        const long long at = row0 + (rev ? token - len + 1 : token);
        if constexpr (!STATE)
            TK::load(nq, q + at * r.q.ts, (int)r.q.ts, len, r.kd, rev);
        TK::load(nk, k + at * r.k.ts, (int)r.k.ts, len, r.kd, rev);
        TV::load(nv, v + at * r.v.ts, (int)r.v.ts, len, width, rev);
    };
    // y of a chunk, which stands in Vs: each thread stores the pieces whose places it fills
    // with v next
    const int apart = a.H * r.vd;  // elements from a token's y to the next one's
    auto lowest = [&](int token, int len) { return ((row0 + (rev ? token - len + 1 : token)) * a.H + h) * r.vd + col0; };
    auto store = [&](int token, int len) KDN_INLINE {
        IO* y = static_cast<IO*>(r.out) + lowest(token, len);
        const int n = width - TV::col();
#pragma unroll
        for (int i = 0; i < TV::NP; ++i) {
            const int row = TV::row(i);
            if (row < len && n > 0) {
                Piece<IO> x;
                x.w = lds_read<typename Piece<IO>::four>(TV::place(vput, i));
                x.store(y + (rev ? len - 1 - row : row) * apart + TV::col(), n);
            }
        }
    };

    auto walk = [&](const Span& span) KDN_INLINE {
        int token = rev ? span.to - 1 : span.from, left = span.to - span.from;
        fetch(token, min(left, C));
        for (bool first = true; left > 0; first = false) {
            const int len = min(left, C);
            // places a few bits away are formed again in every chunk: held over the walk, they
            // would take the registers of the products
            for (uint32_t* p : {&kput, &vput, &qrow, &kcol, &vcol, &prow, &pput, &yput})
                asm volatile("" : "+v"(*p));
            __syncthreads();  // the last chunk's reads are done, its y is whole
            if constexpr (!STATE) {
                if (!first && !r.out_f32)
                    store(token - dir * C, C);
                TK::put(nq, kput - W::kTileK, r.kd);
            }
            TK::put(nk, kput, r.kd);
            TV::put(nv, vput, width);
            if (len != held) {
                held = len;
                whole = decay.power(len);
                if (threadIdx.x < C)
                    lds_write(Ws + 4 * threadIdx.x, r.of_u * decay.power(len - 1 - (int)threadIdx.x + rev));
            }
            __syncthreads();
            if (left > C)
                fetch(token + dir * C, min(left - C, C));
            frag fv[CS];
#pragma unroll
            for (int s = 0; s < CS; ++s)
                fv[s] = O::template cols<kCols>(vcol, s, 0);
            f32x4 acc[NT];
            if constexpr (!STATE) {
                frag fx[KS];
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    if constexpr (BF) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            fx[s][e] = static_cast<bf16>(X[2 * s + e / 4][e % 4]);
                    } else {
                        fx[s] = X[s];
                    }
                }
                const uint32_t krow = qrow + W::kTileK + 16 * jt * LK::BYTES;
                frag fk[BF ? KS : 1];
                if constexpr (BF) {
#pragma unroll
                    for (int s = 0; s < KS; ++s)
                        fk[s] = rows<IO, KD>(krow, 0, s);
                }
                float far = 1.f;
#pragma unroll
                for (int it = 0; it < NT; ++it) {
                    const bool mixed = it >= jt && (NT == 4 || it == wave >> 1);
                    f32x4 p = zero4();
                    acc[it] = zero4();
                    if constexpr (BF) {
                        frag fq[KS];
#pragma unroll
                        for (int s = 0; s < KS; ++s)
                            fq[s] = rows<IO, KD>(qrow, 16 * it, s);
#pragma unroll
                        for (int s = 0; s < KS; ++s)
                            O::mma(acc[it], fq[s], fx[s]);
                        if (mixed) {
#pragma unroll
                            for (int s = 0; s < KS; ++s)
                                O::mma(p, fk[s], fq[s]);
                        }
                    } else {
#pragma unroll
                        for (int s = 0; s < KS; ++s) {
                            const frag fq = rows<IO, KD>(qrow, 16 * it, s);
                            O::mma(acc[it], fq, fx[s]);
                            if (mixed)
                                O::mma(p, rows<IO, KD>(krow, 0, s), fq);
                        }
                    }
                    if (mixed) {
                        typedef IO Four __attribute__((ext_vector_type(4)));
                        Four out;
                        if (it == jt) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)  // a choice, not a product: k may be infinite
                                out[e] = from_f32<IO>(c >= 4 * g + e ? p[e] * on[e] : 0.f);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                out[e] = from_f32<IO>(p[e] * (below[e] * far));
                            far *= g16;
                        }
                        lds_write(LP::further(pput, 16 * it, 0), out);
                    }
                }
                float tile = 1.f;
#pragma unroll
                for (int it = 0; it < NT; ++it) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[it][e] *= front[e] * tile;
                    tile *= g16;
                }
            }
            // v's decayed values, in two parts where they are rounded; any that is not finite
            frag hi[CS], lo[BF ? CS : 1];
            float wrong = 0.f;
#pragma unroll
            for (int s = 0; s < CS; ++s) {
                f32x4 weight[FE / 4];
#pragma unroll
                for (int e = 0; e < FE / 4; ++e)
                    weight[e] = lds_read<f32x4>(Ws + 4 * (s * O::K + FE * g + 4 * e));
#pragma unroll
                for (int e = 0; e < FE; ++e) {
                    const float x = to_f32(fv[s][e]), y = x * weight[e / 4][e % 4];
                    wrong = fmaf(x, 0.f, wrong);
                    hi[s][e] = from_f32<IO>(y);
                    if constexpr (BF) {
                        lo[s][e] = static_cast<bf16>(y - to_f32(hi[s][e]));
                    }
                }
            }
            const bool bad = __ballot(wrong != 0.f);
            if constexpr (BF) {
                if (bad) {  // the second part of an infinity is none, not a NaN
#pragma unroll
                    for (int s = 0; s < CS; ++s)
#pragma unroll
                        for (int e = 0; e < FE; ++e)
                            if (lo[s][e] != lo[s][e])
                                lo[s][e] = bf16(0.f);
                }
            }
            if constexpr (!STATE) {
                __syncthreads();  // Ps is whole
                if (bad) {
                    // zeros of Ps times what is not finite: those are left out of the products,
                    // and added where they belong
#pragma unroll
                    for (int s = 0; s < CS; ++s)
#pragma unroll
                        for (int e = 0; e < FE; ++e) {
                            const float x = to_f32(fv[s][e]);
                            fv[s][e] = from_f32<IO>(x - x == 0.f ? x : 0.f);
                        }
                }
#pragma unroll
                for (int it = 0; it < NT; ++it)
#pragma unroll
                    for (int s = 0; s < CS; ++s)
                        if (s * O::K < 16 * (it + 1))
                            O::mma(acc[it], rows<IO, C>(prow, 16 * it, s), fv[s]);
                if (bad) {
                    for (int j = 0; j < len; ++j) {
                        const float x = to_f32(lds_read<IO>(Vs + LV::at(j, mine / O::VE) + mine % O::VE * W::E));
                        if (x - x == 0.f)
                            continue;
#pragma unroll
                        for (int it = 0; it < NT; ++it)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int i = 16 * it + 4 * g + e;
                                if (i >= j)
                                    acc[it][e] = fmaf(
                                        to_f32(lds_read<IO>(Ps + LP::at(i, j / O::VE) + j % O::VE * W::E)), x,
                                        acc[it][e]);
                            }
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < ST; ++t) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    X[t][e] *= whole;
#pragma unroll
                for (int s = 0; s < CS; ++s) {
                    const frag fk = O::template state_cols<KD>(kcol, s, t);
                    O::mma(X[t], fk, hi[s]);
                    if constexpr (BF)
                        O::mma(X[t], fk, lo[s]);
                }
            }
            if constexpr (!STATE) {
                if (r.out_f32) {
                    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
                        static_cast<float*>(r.out) + lowest(token, len), (short)0, ((len - 1) * apart + width) * 4, 0x00020000);
                    int at = mine < width ? ((rev ? len - 1 - 4 * g : 4 * g) * apart + mine) * 4 : (int)0x80000000u;
                    asm volatile("" : "+v"(at));
#pragma unroll
                    for (int it = 0; it < NT; ++it)
#pragma unroll
                        for (int e = 0; e < 4; ++e)  // tokens that are not there: out of range
                            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[it][e]), rsrc,
                                                                  (uint32_t)at + (uint32_t)(dir * (16 * it + e) * apart * 4), 0, 0);
                } else {
                    // this wave's columns of Vs are its own: y takes v's place
#pragma unroll
                    for (int it = 0; it < NT; ++it)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            lds_write(LV::further(yput, 16 * it + e, 0), from_f32<IO>(acc[it][e]));
                }
            }
            if (!STATE && left <= C && !r.out_f32) {
                __syncthreads();
                store(token, len);
            }
            token += dir * C;
            left -= len;
        }
    };

    if constexpr (STATE) {
        Span span;
        if (handed_on(a, b, s, rev, span)) {
            state_in(nullptr, 0, 0);
            walk(span);
            state_out(handed(s), r.vd, 1);
        }
    } else {
        const int t0 = s * a.L, t1 = min(a.T, t0 + a.L);
        Spans spans;
        Span span;
        spans.start(a, b, t0, t1, rev);
        while (spans.next(span, a.T)) {
            const size_t n = ((size_t)span.n * a.H + h) * dense;
            // (offsets that begin below zero claim a segment before the first one)
            if (span.first || (rev ? s + 1 >= a.S : s == 0))
                state_in(r.X0 ? r.X0 + n : nullptr, r.rs, r.cs);
            else
                state_in(handed(rev ? s + 1 : s - 1), r.vd, 1);
            walk(span);
            if (span.last && r.XT)
                state_out(r.XT + n, r.rs, r.cs);
        }
        if (a.cu && a.clear && !r.out_f32) {
            IO* y = static_cast<IO*>(r.out);
            for (int t = max(t0, max(a.cu[a.N], 0)); t < t1; ++t)
                if ((int)threadIdx.x < width)
                    y[((row0 + t) * a.H + h) * r.vd + col0 + threadIdx.x] = IO(0.f);
        }
    }
}

// The states handed on, one segment after another: what a segment adds, and what it got,
// decayed over its tokens.  A thread has one element of one head's state.
__global__ __launch_bounds__(kThreads) void linattn_join_kernel(LinArgs a)
{
    const LinRole& r = a.role[blockIdx.z];
    const int h = blockIdx.y % a.H, b = blockIdx.y / a.H;
    const size_t dense = (size_t)r.kd * r.vd, i = (size_t)blockIdx.x * kThreads + threadIdx.x;
    const Decay decay{log((double)a.decay[h])};
    float x = 0.f;
    for (int m = 0; m + 1 < a.S; ++m) {
        const int s = r.rev ? a.S - 1 - m : m;
        Span span;
        if (!handed_on(a, b, s, r.rev, span) || i >= dense)
            continue;
        if (span.first)
            x = r.X0 ? r.X0[((size_t)span.n * a.H + h) * dense + (i / r.vd) * r.rs + (i % r.vd) * r.cs] : 0.f;
        float* p = r.seg + (((size_t)b * a.S + s) * a.H + h) * dense + i;
        x = fmaf(decay.power(span.to - span.from), x, *p);
        *p = x;
    }
}

// y [tokens, Hk, d] = the sum over each group's heads of x [tokens, H, d] (fp32)
template <typename IO>
__global__ __launch_bounds__(256) void linattn_group_kernel(LinArgs a, const float* x, IO* y, int G, int d)
{
    const int Hk = a.H / G;
    const long long n = (long long)a.B * a.T * Hk * d;
    const int end = a.cu ? a.cu[a.N] : 0;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const long long token = i / (Hk * d);
        const int at = (int)(i % (Hk * d)), hk = at / d, j = at % d;
        if (a.cu && token >= end) {
            if (a.clear)
                y[i] = IO(0.f);
            continue;
        }
        float s = 0.f;
        for (int m = 0; m < G; ++m)
            s += x[(token * a.H + hk * G + m) * d + j];
        y[i] = from_f32<IO>(s);
    }
}

// ---- single tokens -------------------------------------------------------------------

// One token: a workgroup has one head and 64 columns of the state, a thread four columns
// of every 16th row; rows are joined through LDS.
template <typename IO>
__global__ __launch_bounds__(256) void linattn_step_kernel(LinStepArgs a)
{
    __shared__ float part[16][kCols];
    const int slices = (a.dv + kCols - 1) / kCols;
    const int slice = blockIdx.x % slices, unit = blockIdx.x / slices, h = unit % a.H, b = unit / a.H;
    const int rg = threadIdx.x >> 4, c = 4 * (threadIdx.x & 15), col = slice * kCols + c, n = min(a.dv - col, 4);
    const IO* q = static_cast<const IO*>(a.q) + (long long)b * a.qs + (long long)(h / a.G) * a.qh;
    const IO* k = static_cast<const IO*>(a.k) + (long long)b * a.ks + (long long)(h / a.G) * a.kh;
    const IO* v = static_cast<const IO*>(a.v) + (long long)b * a.vs + (long long)h * a.vh;
    float* S = a.S + (size_t)unit * a.dk * a.dv;
    const float g = a.decay[h];
    float vv[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        vv[e] = e < n ? to_f32(v[col + e]) : 0.f;
    if (n > 0) {
        for (int i = rg; i < a.dk; i += 16) {
            const float kk = to_f32(k[i]), qq = to_f32(q[i]);
            float* p = S + (size_t)i * a.dv + col;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n) {
                    const float x = fmaf(g, p[e], kk * vv[e]);
                    p[e] = x;
                    o[e] = fmaf(qq, x, o[e]);
                }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        part[rg][c + e] = o[e];
    __syncthreads();
    const int out = slice * kCols + threadIdx.x;
    if (threadIdx.x < kCols && out < a.dv) {
        float s = 0.f;
#pragma unroll
        for (int m = 0; m < 16; ++m)
            s += part[m][threadIdx.x];
        static_cast<IO*>(a.o)[(size_t)unit * a.dv + out] = from_f32<IO>(s * a.scale);
    }
}

// ---- host ------------------------------------------------------------------------------

int padded(int kd) { return kd <= 32 ? 32 : kd <= 64 ? 64 : kd <= 128 ? 128 : 256; }

template <typename IO, int KD, bool STATE>
void launch_walk(const LinArgs& a, int roles, hipStream_t stream)
{
    constexpr int C = sizeof(IO) == 2 && KD <= 128 ? 64 : 32;
    const int slices = (a.role[0].vd + kCols - 1) / kCols;
    const unsigned units = ((unsigned)a.B * a.H * a.S + 7) / 8 * 8;
    linattn_kernel<IO, KD, C, STATE><<<dim3(units * slices, roles), kThreads, 0, stream>>>(a);
}

template <typename IO>
void launch_walks(const LinArgs& a, int roles, hipStream_t stream)
{
    const int kd = padded(a.role[0].kd);
    auto run = [&](auto state) {
        constexpr bool S = decltype(state)::value;
        if (kd == 32)
            launch_walk<IO, 32, S>(a, roles, stream);
        else if (kd == 64)
            launch_walk<IO, 64, S>(a, roles, stream);
        else if (kd == 128)
            launch_walk<IO, 128, S>(a, roles, stream);
        else
            launch_walk<IO, 256, S>(a, roles, stream);
    };
    if (a.S > 1) {
        run(std::true_type{});
        const size_t dense = (size_t)a.role[0].kd * a.role[0].vd;
        linattn_join_kernel<<<dim3((unsigned)((dense + kThreads - 1) / kThreads), a.B * a.H, roles), kThreads, 0,
                              stream>>>(a);
    }
    run(std::false_type{});
}

// Tokens of a segment: a multiple of 64
int segments(int B, int T, int H, int slices, int& L)
{
    const long long groups = (long long)B * H * slices;
    const long long want = (512 + groups - 1) / groups, most = T / 512;
    const long long S = want < most ? want : most;
    L = S <= 1 ? (T > 0 ? T : 1) : (int)(((T + S - 1) / S + 63) / 64 * 64);
    return T > 0 ? (T + L - 1) / L : 1;
}

int slices_of(int vd) { return (vd + kCols - 1) / kCols; }

size_t aligned16(size_t n) { return (n + 15) / 16 * 16; }

template <typename IO>
hipError_t linattn_fwd(const LinArgs& a, hipStream_t stream)
{
    if (a.T > 0)
        launch_walks<IO>(a, 1, stream);
    return hipGetLastError();
}

}  // namespace

size_t linattn_fwd_workspace_bytes(int B, int T, int H, int dk, int dv)
{
    int L;
    const int S = segments(B, T, H, slices_of(dv), L);
    return S > 1 ? sizeof(float) * B * S * H * dk * dv : 0;
}

static size_t bwd_segments_bytes(int B, int T, int H, int dk, int dv, int& S, int& L)
{
    S = segments(B, T, H, slices_of(dk) * 2 + slices_of(dv), L);
    return S > 1 ? sizeof(float) * B * S * H * dk * dv : 0;
}

size_t linattn_bwd_workspace_bytes(int B, int T, int H, int Hk, int dk, int dv)
{
    int S, L;
    const size_t seg = bwd_segments_bytes(B, T, H, dk, dv, S, L);
    return 3 * seg + (Hk != H ? 2 * aligned16(sizeof(float) * B * T * H * dk) : 0);
}

// the states of sequences without tokens
static void empty_states(const LinArgs& a, const float* from, float* to, hipStream_t stream)
{
    if (to && (a.cu || a.T == 0))
        launch_empty_states<float>(a.cu, a.N, a.H * a.role[0].kd * a.role[0].vd, from, to, stream);
}

hipError_t launch_linattn_fwd(const LinCall& c, bool bf, hipStream_t stream)
{
    LinArgs a{};
    a.B = c.B, a.T = c.T, a.H = c.H, a.N = c.N, a.cu = c.cu, a.decay = c.decay, a.clear = c.clear;
    a.S = segments(c.B, c.T, c.H, slices_of(c.dv), a.L);
    LinRole& r = a.role[0];
    r.q = c.q, r.k = c.k, r.v = c.v;
    r.out = c.o, r.X0 = c.S0, r.XT = c.S_T, r.seg = static_cast<float*>(c.ws);
    r.kd = c.dk, r.vd = c.dv, r.rs = c.dv, r.cs = 1;
    r.of_p = r.of_x = c.scale, r.of_u = 1.f;
    empty_states(a, c.S0, c.S_T, stream);
    return bf ? linattn_fwd<bf16>(a, stream) : linattn_fwd<float>(a, stream);
}

template <typename IO>
static hipError_t linattn_bwd(const LinCall& c, hipStream_t stream)
{
    LinArgs a{};
    a.B = c.B, a.T = c.T, a.H = c.H, a.N = c.N, a.cu = c.cu, a.decay = c.decay, a.clear = c.clear;
    const int G = c.H / c.Hk;
    const size_t seg = bwd_segments_bytes(c.B, c.T, c.H, c.dk, c.dv, a.S, a.L) / sizeof(float);
    float* ws = static_cast<float*>(c.ws);
    const size_t whole = aligned16(sizeof(float) * c.B * c.T * c.H * c.dk) / sizeof(float);
    float* gq = ws + 3 * seg;
    float* gk = gq + whole;

    LinRole dq{}, dk{}, dv{};
    dq.q = c.d_o, dq.k = c.v, dq.v = c.k;
    dq.out = G > 1 ? gq : c.dq, dq.out_f32 = G > 1;
    dq.X0 = c.S0, dq.kd = c.dv, dq.vd = c.dk, dq.rs = 1, dq.cs = c.dv;
    dq.of_p = dq.of_x = c.scale, dq.of_u = 1.f, dq.seg = ws;
    dk.q = c.v, dk.k = c.d_o, dk.v = c.q;
    dk.out = G > 1 ? gk : c.dk_out, dk.out_f32 = G > 1;
    dk.X0 = c.dS_T, dk.kd = c.dv, dk.vd = c.dk, dk.rs = 1, dk.cs = c.dv;
    dk.of_p = dk.of_u = c.scale, dk.of_x = 1.f, dk.rev = 1, dk.seg = ws + seg;
    dv.q = c.k, dv.k = c.q, dv.v = c.d_o;
    dv.out = c.dv_out, dv.X0 = c.dS_T, dv.XT = c.dS0;
    dv.kd = c.dk, dv.vd = c.dv, dv.rs = c.dv, dv.cs = 1;
    dv.of_p = dv.of_u = c.scale, dv.of_x = 1.f, dv.rev = 1, dv.seg = ws + 2 * seg;

    a.role[0] = dv;
    empty_states(a, c.dS_T, c.dS0, stream);
    if (c.T == 0)
        return hipGetLastError();
    if (c.dk == c.dv) {
        a.role[1] = dq, a.role[2] = dk;
        launch_walks<IO>(a, 3, stream);
    } else {
        launch_walks<IO>(a, 1, stream);
        a.role[0] = dq, a.role[1] = dk;
        launch_walks<IO>(a, 2, stream);
    }
    if (G > 1) {
        const long long n = (long long)c.B * c.T * c.Hk * c.dk;
        const unsigned groups = (unsigned)((n + 255) / 256 < 8192 ? (n + 255) / 256 : 8192);
        linattn_group_kernel<IO><<<groups, 256, 0, stream>>>(a, gq, static_cast<IO*>(c.dq), G, c.dk);
        linattn_group_kernel<IO><<<groups, 256, 0, stream>>>(a, gk, static_cast<IO*>(c.dk_out), G, c.dk);
    }
    return hipGetLastError();
}

hipError_t launch_linattn_bwd(const LinCall& c, bool bf, hipStream_t stream)
{
    return bf ? linattn_bwd<bf16>(c, stream) : linattn_bwd<float>(c, stream);
}

hipError_t launch_linattn_step(const LinStepArgs& a, bool bf, hipStream_t stream)
{
    const unsigned groups = (unsigned)a.B * a.H * slices_of(a.dv);
    if (bf)
        linattn_step_kernel<bf16><<<groups, 256, 0, stream>>>(a);
    else
        linattn_step_kernel<float><<<groups, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace kdn
