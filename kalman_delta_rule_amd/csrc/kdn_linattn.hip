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
// bf16: the products' operands are bf16, sums and states fp32.  q, k, v are exact.  Every
// other operand is two bf16 parts (2^-16 of each term), so that a y is off by its own rounding
// alone: the decayed q k, X where y is formed from it, and v's decayed values that X is summed
// from.  (With one part of the first two y was 2.3e-3 off in the 2-norm, instead of 1.7e-3.
// Their second parts take vector instructions, which bound a walk at one workgroup a compute
// unit: B8 T4096, 16 heads of 128, forward 147 us with one part, 177 with two; B16 T2048, at
// two workgroups, 138 and 146; backward of the first 355 and 418, of 65536 tokens 893 and
// 1010; B2 T2048, 16 heads of 256, backward 143 and 202.)
// Where X is an fp32 output v has a third part (2^-24), for the tokens before its last that
// still have an eighth of their weight in it; of the others the two parts' error is as small.
// It costs 6% at two workgroups a compute unit (B16 T2048 forward 146 us without a state out,
// 155 with), 15 to 20% at one, where the slowest decay's walk sets the time (B8 T4096 177 and
// 205), so walks that hand no state out do not form it, and are kernels of their own: the
// branch alone cost them 2%.
// fp32: matrix instructions with fp32 operands throughout.
#include "kdn_common.h"
#include "kdn_linattn.h"
#include "kdn_linattn_spans.h"
#include "kdn_sequences.h"
#include "kdn_stream.h"

#include <type_traits>

// the steps of a walk are lambdas; called out of line they would put the state into memory
#define KDN_INLINE __attribute__((always_inline))

namespace kdn {

namespace {

constexpr int kThreads = 256, kCols = 64;  // columns of v a workgroup

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// A matrix in LDS, rows of W elements without a gap.  Its 16-byte blocks are exchanged
// within a row by a number that goes by the row, so that neighbours lie in banks of their
// own in each of the ways it is read (8 x 4096 tokens of 16 heads, forward: 205 us, with padded
// rows 221; and copies straight into LDS, which rows without gaps allow, 153): one block of 16
// rows, and
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
            return (row >> 1 & 2) | (row >> 3 & 1) | (BLOCKS == 4 ? 0 : BLOCKS == 8 ? row << 1 & 4 : row << 2 & 12);
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

__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// two values in a word as bf16, and they as fp32.  (The word is made opaque: values taken
// from it one by one would be rounded one by one too.)
__device__ __forceinline__ uint32_t two_bf16(float a, float b)
{
    typedef float two __attribute__((ext_vector_type(2)));
    typedef bf16 out __attribute__((ext_vector_type(2)));
    uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(two{a, b}, out));
    asm volatile("" : "+v"(w));
    return w;
}
__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// What is left of two values whose words as bf16 `near` is, as bf16.  An infinity leaves a
// NaN, which the larger of two drops: some finite value, which no sum with an infinity shows.
__device__ __forceinline__ uint32_t rest_bf16(float a, float b, uint32_t near)
{
    typedef float two __attribute__((ext_vector_type(2)));
    typedef bf16 out __attribute__((ext_vector_type(2)));
    const two rest{fmaxf(a - low_bf16(near), -0x1p120f), fmaxf(b - high_bf16(near), -0x1p120f)};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, out));
}

// What this wave copies into LDS, loads and stores has arrived, but for the last N asked
// for.  (The compiler has to know: it would otherwise wait for loads of before the walk
// inside it, and so for the copies.)
template <int N>
__device__ __forceinline__ void arrived()
{
    __builtin_amdgcn_s_waitcnt(0x0F70 | N);  // vmcnt
    asm volatile("" ::: "memory");
}

// A tile of C tokens by W columns of which `width` are there, 16 bytes a thread and turn.
// It is copied from memory straight into LDS, through a buffer descriptor that ends behind
// the tile's last element: what is not there arrives as zeros.  A wave's 1024 bytes follow
// one another in LDS, so blocks change places in the addresses that are read.
template <typename IO, int C, int W>
struct Tile {
    typedef Lds<IO, W> L;
    static constexpr int VE = Op<IO>::VE, E = sizeof(IO), PER = W / VE, ROWS = kThreads / PER, NP = C / ROWS;
    static_assert(kThreads % PER == 0 && C % ROWS == 0, "whole turns of the threads");
    static __device__ __forceinline__ int row(int i) { return i * ROWS + (int)threadIdx.x / PER; }
    static __device__ __forceinline__ int block(int i) { return (int)threadIdx.x % PER ^ L::turn(row(0)) ^ L::turn(i * ROWS); }
    // Bytes of a thread's pieces from the first row's front, turns that differ in the blocks'
    // exchange apart; out of any range for columns that are not there (a tile spans less
    // than 2^30 bytes, so what is added to them leaves them out of range)
    static constexpr int KINDS = ROWS < 16 ? 16 / ROWS : 1;
    struct Places {
        uint32_t at[KINDS];
        __device__ __forceinline__ Places(int ts, int width, int dir)
        {
#pragma unroll
            for (int i = 0; i < KINDS; ++i)
                at[i] = block(i) * VE < width ? (uint32_t)(dir * row(0) * ts * E + block(i) * 16) : 0x80000000u;
        }
    };
    // Copies to LDS from rows p, p + ts, .. or (dir < 0) from the last of them to p, turn by
    // turn: a wave that asks for many at once waits for the last.
    struct Copy {
        typedef uint32_t four __attribute__((ext_vector_type(4)));
        four rsrc;
        uint32_t lds, first, step;
        __device__ __forceinline__ Copy(uint32_t to, const IO* p, int ts, int len, int width, int dir)
        {
            const uint64_t at = reinterpret_cast<uint64_t>(p);
            const uint32_t last = (uint32_t)(len - 1) * ts * E;
            // a word that ends behind the last element is read whole (it lies in one page)
            rsrc = four{(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, (last + width * E + 3) & ~3u, 0x00020000u};
            lds = to, first = dir < 0 ? last : 0, step = (uint32_t)(dir * ROWS * ts * E);
        }
        __device__ __forceinline__ void turn(const Places& from, int i) const
        {
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                         ::"s"(lds + i * (kThreads * 16)), "v"(from.at[i % KINDS] + (first + i * step)), "s"(rsrc)
                         : "memory");
        }
        // its share of `of` parts, the whole of them being all turns
        __device__ __forceinline__ void share(const Places& from, int part, int of) const
        {
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (i * of / NP == part)
                    turn(from, i);
        }
    };
    // the same where rows begin in the middle of a word, through registers: a row's last piece
    // is read so that it ends with the row, and moved.  (One load after another, without a
    // branch: what waits for one would wait for all.)
    static __device__ __forceinline__ void copy_odd(uint32_t lds, const IO* p, int ts, int len, int width, int dir)
    {
        struct __attribute__((packed, aligned(2))) Piece {
            uint32_t w[4];
        };
        const int j = (int)threadIdx.x % PER * VE;
        if (width < VE) {
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                const int i = min(row(n), len - 1);
                const IO* from = p + (ptrdiff_t)(dir < 0 ? len - 1 - i : i) * ts;
                IO x[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    x[e] = from[min(e, width - 1)];
                u32x4 w = {};
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (j + e < width && row(n) < len)
                        w[e * E / 4] |= (uint32_t) __builtin_bit_cast(uint16_t, (bf16)x[e]) << (e % 2 * 16);
                lds_write(lds + L::at(row(n), j / VE), w);
            }
            return;
        }
        Piece x[NP];
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const int i = min(row(n), len - 1);
            x[n] = *reinterpret_cast<const Piece*>(p + (ptrdiff_t)(dir < 0 ? len - 1 - i : i) * ts + min(j, width - VE));
        }
        const int over = j + VE - width, by = (VE - width % VE) * 16;  // bits (where a piece is not whole)
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            u32x4 w = {x[n].w[0], x[n].w[1], x[n].w[2], x[n].w[3]};
            if (over > 0) {
                typedef uint64_t two __attribute__((ext_vector_type(2)));
                two d = __builtin_bit_cast(two, w);
                d = by < 64 ? two{d.x >> by | d.y << (64 - by), d.y >> by} : two{d.y >> (by - 64 & 63), 0};
                w = over < VE ? __builtin_bit_cast(u32x4, d) : u32x4{};
            }
            if (row(n) >= len)
                w = u32x4{};
            lds_write(lds + L::at(row(n), j / VE), w);
        }
    }
    // row i's piece that the row ends in: what follows is the next head's, or the next token's
    static __device__ __forceinline__ void end_row(uint32_t lds, int i, int width)
    {
        typedef uint32_t four __attribute__((ext_vector_type(4)));
        const uint32_t at = lds + L::at(i, width / VE);
        four w = lds_read<four>(at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = width % VE - j * (VE / 4);
            w[j] &= n >= VE / 4 ? ~0u : n <= 0 ? 0u : 0xFFFFu;
        }
        lds_write(at, w);
    }
};

// of the spans' offsets: by all threads
struct Counted {
    static __device__ __forceinline__ int at_most(const int* p, int n, int x) { return count_at_most<kThreads>(p, n, x); }
};

// What bounds a walk (16 heads of 128 in bf16, forward, no state out).  With one workgroup a
// compute unit (B8 T4096, 180 us) the chain of a chunk's instructions: a chunk of 64 tokens
// takes 2.8 us, 2.4 with copies and stores left out, 1.9 with the arithmetic left out; the
// matrix units are busy a fifth of it.  With two (B16 T2048, 143 us) the copies: 2.2 us, 1.6
// and 2.0.  A chunk's copies are asked for while the one before is computed, and no earlier: a
// further tile of q, k and v takes the LDS of the second workgroup where there are two, and
// where there is one (it would fit: 118 KB) the copies are not what sets the time.  C = 32
// leaves room for both: with three workgroups the backward of 8 x 4096 tokens took 338 us
// instead of 350, the forward, which has one, more than with 64 (the operands that are not
// inputs in one part).  Heads of 256, and fp32, have 32, as their tiles would not fit twice.
template <typename IO, int KD, int C>
struct Walk {
    typedef Op<IO> O;
    typedef typename O::frag frag;
    typedef Tile<IO, C, KD> TK;
    typedef Tile<IO, C, kCols> TV;
    static constexpr int NT = C / 16, ST = KD / 16, KS = KD / O::K, CS = C / O::K, FE = O::K / 4;
    static constexpr bool BF = sizeof(IO) == 2;
    static constexpr int E = sizeof(IO), kTileK = C * KD * E, kTileV = C * kCols * E;  // bytes
    // The decayed product.  fp32: rows of C tokens j.  bf16: for each step of 32 tokens j the rows
    // i from there on, the 32 values of the first part beside those of the second.
    static constexpr int PW = BF ? 64 : C, kTileP = (BF && C == 64 ? 64 + 32 : C) * PW * E;
    // bytes to step s, and the rows that it leaves out
    static constexpr int step_at(int s) { return BF ? s * C * PW * E : 0; }
    static constexpr int step_row(int s) { return BF ? 32 * s : 0; }
    // q once, k and v twice, the decayed product, the tokens' decays
    static constexpr int lds(bool state) { return (state ? 2 : 3) * kTileK + 2 * kTileV + (state ? 0 : kTileP) + C * 4 + (C + 1) * 4; }
};

// STATE: the states that segments hand on, nothing else
// EDGE: rows that are not whole pieces of 16 bytes, or y's not whole words
template <typename IO, int KD, int C, bool STATE, bool EDGE, bool EXACT>
__global__ __launch_bounds__(kThreads, sizeof(IO) * KD > 512 ? 1 : 2) void linattn_kernel(LinArgs a)
{
    typedef Walk<IO, KD, C> W;
    typedef typename W::O O;
    typedef typename W::frag frag;
    typedef typename W::TK TK;
    typedef typename W::TV TV;
    typedef Lds<IO, kCols> LV;
    typedef Lds<IO, W::PW> LP;
    typedef Lds<IO, KD> LK;
    constexpr int NT = W::NT, ST = W::ST, KS = W::KS, CS = W::CS, FE = W::FE;
    constexpr bool BF = W::BF;
    __shared__ __attribute__((aligned(256))) char lds[W::lds(STATE)];
    const uint32_t Qs = (uint32_t)(size_t)(__attribute__((address_space(3))) char*)lds;
    const uint32_t Ks = Qs + (STATE ? 0 : W::kTileK), Vs = Ks + 2 * W::kTileK, Ps = Vs + 2 * W::kTileV,
                   Ws = Ps + (STATE ? 0 : W::kTileP);  // of_u g^(len - 1 - j + rev) of each token of a chunk

    // the walks over one head's tokens, and their slices, follow one another on one XCD
    // (workgroups go round the eight) and find each other's inputs in its cache
    const int index = blockIdx.x / 8, each = a.slices * a.roles, unit = index / each * 8 + (int)(blockIdx.x & 7);
    const LinRole& r = a.role[index % each / a.slices];
    const int slice = index % a.slices;
    if (unit >= a.B * a.H * a.S * a.parts || slice * kCols >= r.vd)
        return;
    const int h = unit % a.H, piece = unit / a.H % a.parts, s = unit / a.H / a.parts % a.S, b = unit / a.H / a.parts / a.S;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, c = lane & 15;
    const int col0 = slice * kCols, width = min(r.vd - col0, kCols);  // of v
    const int mine = 16 * wave + c, mycol = col0 + mine;
    const int rev = r.rev, dir = rev ? -1 : 1;

    const long long row0 = (long long)b * a.T;
    const IO* q = static_cast<const IO*>(r.q.p) + (long long)(h / r.q.div) * r.q.hs;
    const IO* k = static_cast<const IO*>(r.k.p) + (long long)(h / r.k.div) * r.k.hs;
    const IO* v = static_cast<const IO*>(r.v.p) + (long long)(h / r.v.div) * r.v.hs + col0;

    // Powers of the decay to C are formed once, a thread each, while the first copies are on
    // their way.
    // C = 64: a wave forms q k^T for 16 tokens' k (block jt) and every q; C = 32: for one block
    // of q.  Lane (g, c) holds q k^T of k's tokens j = 4 g + e of a block and q's token i = c.
    const int jt = NT == 4 ? wave : wave & 1;
    const uint32_t Ts = Ws + 4 * C;
    f32x4 pdecay[NT == 4 ? 4 : 1];
    bool ready = false;
    // tokens until a term of the state has decayed to an eighth
    int reach = 0;
    auto power = [&](int n) KDN_INLINE { return lds_read<float>(Ts + 4 * max(n, 0)); };
    auto powers = [&]() KDN_INLINE {
        if (ready)
            return;
        ready = true;
        const Decay decay{log((double)a.decay[h])};
        reach = __builtin_amdgcn_readfirstlane(decay.log < 0 ? (int)fminf(-2.1f / (float)decay.log, 2e9f) : 2000000000);
        if (threadIdx.x <= C)
            lds_write(Ts + 4 * threadIdx.x, decay.power(threadIdx.x));
        lds_barrier();
        if constexpr (!STATE) {
#pragma unroll
            for (int i = 0; i < (NT == 4 ? 4 : 1); ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    pdecay[i][e] = r.of_p * power(16 * ((NT == 4 ? i : wave >> 1) - jt) + c - 4 * g - e);
        }
    };
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

    // places in LDS of a lane, in the first row or tile that it touches
    uint32_t qrow = Qs + rows_at<IO, KD>(lane), prow = Ps + rows_at<IO, W::PW>(lane);
    const uint32_t kcol = Ks + O::template cols_at<KD>(0, O::kApart, lane);
    const uint32_t vcol = Vs + O::template cols_at<kCols>(16 * wave, 4, lane);
    const int js = BF ? jt / 2 : 0;  // the step that this wave's tokens j belong to
    uint32_t pput = Ps + W::step_at(js) - W::step_row(js) * LP::BYTES
                    + LP::at(c, (16 * (jt - 2 * js) + 4 * g) / O::VE) + 4 * g % O::VE * W::E;

    const LinTensor tq = r.q, tk = r.k, tv = r.v;
    const int kd = r.kd;
    const typename TK::Places qfrom((int)tq.ts, kd, dir), kfrom((int)tk.ts, kd, dir);
    const typename TV::Places vfrom((int)tv.ts, width, dir);
    const uint32_t part = 1024 * wave;  // of a turn's copies, this wave's
    const bool ragged = EDGE && (kd % O::VE || width % O::VE);
    const bool odd = BF && EDGE && a.odd;  // some rows begin in the middle of a word
    auto copies = [&](auto tile, uint32_t to, const IO* p, int ts, int wide, int len) KDN_INLINE {
        return typename decltype(tile)::Copy(to + part, p, ts, len, wide, dir);
    };
    // y: a lane has four adjacent columns of a token in each 16 of them
    const bool out_f32 = r.out_f32;
    const int eo = BF && !out_f32 ? 2 : 4, apart = a.H * r.vd * eo;  // bytes of an element, to the next token
    const int left_cols = width - (16 * wave + 4 * g);
    const uint32_t yfrom = left_cols > 0 ? (uint32_t)(dir * c * apart + (16 * wave + 4 * g) * eo) : 0x80000000u;
    auto store = [&](const f32x4 (&y)[NT], char* to, int len) KDN_INLINE {
        const int last = (len - 1) * apart;
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(to, (short)0, last + width * eo, 0x00020000);
        // tokens that are not there are out of range
        const uint32_t first = yfrom + (rev ? last : 0), step = dir * 16 * apart;
        typedef uint32_t two __attribute__((ext_vector_type(2)));
        typedef uint32_t four __attribute__((ext_vector_type(4)));
        if (EDGE && (width % 4 || (reinterpret_cast<uintptr_t>(r.out) & 3))) {
#pragma unroll
            for (int it = 0; it < NT; ++it)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t at = e < left_cols ? first + it * step + e * eo : 0x80000000u;
                    if (!BF || out_f32)
                        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y[it][e]), rsrc, at, 0, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b16(
                            __builtin_bit_cast(unsigned short, static_cast<bf16>(y[it][e])), rsrc, at, 0, 0);
                }
        } else if (!BF || out_f32) {
#pragma unroll
            for (int it = 0; it < NT; ++it)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(four, y[it]), rsrc, first + it * step, 0, 0);
        } else {
#pragma unroll
            for (int it = 0; it < NT; ++it)
                __builtin_amdgcn_raw_buffer_store_b64(
                    __builtin_bit_cast(two, __builtin_convertvector(y[it], bf16x4)), rsrc, first + it * step, 0, 0);
        }
    };

    auto walk = [&](const Span& span) KDN_INLINE {
        // (the same in all lanes; said so, addresses and counts are scalars)
        const int from = __builtin_amdgcn_readfirstlane(span.from), to = __builtin_amdgcn_readfirstlane(span.to);
        int left = to - from, turn = 0;
        lds_barrier();  // the last span's reads are done
        // lowest addresses of the next chunk to copy, and of the one whose y is next
        const int qts = (int)tq.ts, kts = (int)tk.ts, vts = (int)tv.ts;
        const long long low = row0 + (rev ? to - min(left, C) : from);
        const IO *qp = q + low * qts, *kp = k + low * kts, *vp = v + low * vts;
        char* yp = static_cast<char*>(r.out) + low * apart + (h * r.vd + col0) * eo;
        // the first chunk
        const int some = min(left, C);
        if (odd) {
            if constexpr (!STATE)
                TK::copy_odd(Qs, qp, qts, some, kd, dir);
            TK::copy_odd(Ks, kp, kts, some, kd, dir);
            TV::copy_odd(Vs, vp, vts, some, width, dir);
        } else {
            if constexpr (!STATE)
                copies(TK{}, Qs, qp, qts, kd, some).share(qfrom, 0, 1);
            copies(TK{}, Ks, kp, kts, kd, some).share(kfrom, 0, 1);
            copies(TV{}, Vs, vp, vts, width, some).share(vfrom, 0, 1);
        }
        powers();
        // of a state that is an output: tokens before its last that a third part is formed of
        const int near = __builtin_amdgcn_readfirstlane(EXACT && r.exact && (STATE || span.last) ? reach : -1);
        arrived<0>();
        for (; left > 0; turn ^= 1) {
            const int len = min(left, C), more = min(left - C, C);
            const uint32_t K = Ks + turn * W::kTileK, V = Vs + turn * W::kTileV;
            // the other buffers of k and v
            const uint32_t K2 = Ks + (turn ^ 1) * W::kTileK, V2 = Vs + (turn ^ 1) * W::kTileV;
            // places a few bits away are formed again in every chunk: held over the walk, they
            // would take the registers of the products
            for (uint32_t* p : {&qrow, &prow, &pput})
                asm volatile("" : "+v"(*p));
            lds_barrier();  // all waves' copies have arrived, and the last chunk's reads are done
            if (ragged || len != held) {
                const int x = threadIdx.x;
                if (x < C) {
                    if (kd % O::VE)
                        TK::end_row(K, x, kd);
                    if (!STATE && kd % O::VE)
                        TK::end_row(Qs, x, kd);
                    if (width % O::VE)
                        TV::end_row(V, x, width);
                    if (len != held)
                        lds_write(Ws + 4 * x, r.of_u * power(len - 1 - x + rev));
                }
                if (len != held)
                    whole = power(len);
                held = len;
                lds_barrier();
            }
            // the next chunk's copies, asked for between the products (none: of no tokens)
            const int on = rev ? -more : C;  // tokens to its lowest
            qp += on * qts, kp += on * kts, vp += on * vts;
            const auto k2 = copies(TK{}, K2, kp, kts, kd, more);
            const auto v2 = copies(TV{}, V2, vp, vts, width, more);
            if (odd && more > 0) {
                TK::copy_odd(K2, kp, kts, more, kd, dir);
                TV::copy_odd(V2, vp, vts, more, width, dir);
            }
            auto ahead = [&](int part, int of) KDN_INLINE {
                if (!odd && more > 0) {
                    k2.share(kfrom, part, of);
                    v2.share(vfrom, part, of);
                }
            };
            if constexpr (STATE)
                ahead(0, 1);
            frag fv[CS];
#pragma unroll
            for (int s = 0; s < CS; ++s)
                fv[s] = O::template cols<kCols>(vcol + turn * W::kTileV, s, 0);
            f32x4 acc[NT];
            if constexpr (!STATE) {
                const uint32_t krow = K + (qrow - Qs) + 16 * jt * LK::BYTES;
                // q's operands are read a group of steps ahead of their products
                constexpr int GS = KS < 4 ? KS : 4, NG = KS / GS;
                static_assert(NT == 2 || NG == 1, "p is one block's");
                frag fx[GS], fl[BF ? GS : 1];  // X as operands, in two parts where they are rounded
                frag fk[NT == 4 ? KS : 1], fq[2][GS];
                if constexpr (NT == 4) {
#pragma unroll
                    for (int s = 0; s < KS; ++s)
                        fk[s] = rows<IO, KD>(krow, 0, s);
                }
                auto read = [&](int u) KDN_INLINE {
#pragma unroll
                    for (int s = 0; s < GS; ++s)
                        fq[u % 2][s] = rows<IO, KD>(qrow, 16 * (u % NT), u / NT * GS + s);
                };
                read(0);
                f32x4 p;
#pragma unroll
                for (int u = 0; u < NT * NG; ++u) {
                    const int it = u % NT, s0 = u / NT * GS;
                    // (C = 32: two waves form a block each)
                    const bool mixed = NT == 4 || it == wave >> 1;
                    if (u + 1 < NT * NG)
                        read(u + 1);
                    ahead(u, NT * NG);
                    if (s0 == 0)
                        acc[it] = zero4();
                    if (NT == 4 || u == 0)
                        p = zero4();
                    if (it == 0) {
#pragma unroll
                        for (int s = 0; s < GS; ++s) {
                            if constexpr (BF) {
                                u32x4 high, low;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const f32x4& x = X[2 * (s0 + s) + i / 2];
                                    high[i] = two_bf16(x[i % 2 * 2], x[i % 2 * 2 + 1]);
                                    low[i] = rest_bf16(x[i % 2 * 2], x[i % 2 * 2 + 1], high[i]);
                                }
                                fx[s] = __builtin_bit_cast(frag, high);
                                fl[s] = __builtin_bit_cast(frag, low);
                            } else {
                                fx[s] = X[s0 + s];
                            }
                        }
                    }
                    // (sums by turns: a product waits for the one before of its own sum)
#pragma unroll
                    for (int s = 0; s < GS; ++s) {
                        O::mma(acc[it], fx[s], fq[u % 2][s]);
                        if constexpr (NT == 4)
                            O::mma(p, fk[s0 + s], fq[u % 2][s]);
                        if constexpr (BF)
                            O::mma(acc[it], fl[s], fq[u % 2][s]);
                    }
                    if constexpr (NT != 4) {
                        if (mixed) {
#pragma unroll
                            for (int s = 0; s < GS; ++s)
                                O::mma(p, rows<IO, KD>(krow, 0, s0 + s), fq[u % 2][s]);
                        }
                    }
                    // (the blocks that no step reads are not there)
                    if (mixed && s0 + GS == KS && (NT != 4 || it >= 2 * js)) {
                        p *= pdecay[NT == 4 ? it : 0];
#pragma unroll
                        for (int e = 0; e < 4; ++e)  // a choice, not a product with zero: k may be infinite
                            p[e] = it > jt || (it == jt && c >= 4 * g + e) ? p[e] : 0.f;
                        const uint32_t to = LP::further(pput, 16 * it, 0);
                        if constexpr (BF) {
                            typedef uint32_t two __attribute__((ext_vector_type(2)));
                            const two high{two_bf16(p[0], p[1]), two_bf16(p[2], p[3])};
                            lds_write(to, high);
                            lds_write(LP::further(to, 0, 4), two{rest_bf16(p[0], p[1], high.x), rest_bf16(p[2], p[3], high.y)});
                        } else {
                            lds_write(to, p);
                        }
                    }
                }
#pragma unroll
                for (int it = 0; it < NT; ++it)
                    acc[it] *= r.of_x * power(16 * it + c + 1 - rev);
            }
            if constexpr (!STATE) {
                lds_barrier();  // Ps is whole, q is read
                if (odd && more > 0)
                    TK::copy_odd(Qs, qp, qts, more, kd, dir);
            }
            const auto q2 = copies(TK{}, Qs, qp, qts, kd, more);
            // v's decayed values, in two parts where they are rounded
            frag hi[CS], lo[BF ? CS : 1], rest[EXACT ? CS : 1];
            f32x4 none = zero4();  // zero times v: what is not finite shows
#pragma unroll
            for (int s = 0; s < CS; ++s) {
                f32x4 weight[FE / 4];
#pragma unroll
                for (int e = 0; e < FE / 4; ++e)
                    weight[e] = lds_read<f32x4>(Ws + 4 * (s * O::K + FE * g + 4 * e));
                O::mma(none, frag{}, fv[s]);
                if (!STATE && !odd && more > 0)
                    q2.share(qfrom, s, CS);
                if constexpr (BF) {
                    u32x4 high, low, x = __builtin_bit_cast(u32x4, fv[s]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float w0 = weight[i / 2][i % 2 * 2], w1 = weight[i / 2][i % 2 * 2 + 1];
                        high[i] = two_bf16(low_bf16(x[i]) * w0, high_bf16(x[i]) * w1);
                        low[i] = two_bf16(fmaf(low_bf16(x[i]), w0, -low_bf16(high[i])),
                                          fmaf(high_bf16(x[i]), w1, -high_bf16(high[i])));
                    }
                    hi[s] = __builtin_bit_cast(frag, high);
                    lo[s] = __builtin_bit_cast(frag, low);
                    if constexpr (EXACT) {
                        u32x4 last;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float w0 = weight[i / 2][i % 2 * 2], w1 = weight[i / 2][i % 2 * 2 + 1];
                            last[i] = two_bf16(
                                fmaf(low_bf16(x[i]), w0, -low_bf16(high[i])) - low_bf16(low[i]),
                                fmaf(high_bf16(x[i]), w1, -high_bf16(high[i])) - high_bf16(low[i]));
                        }
                        rest[s] = __builtin_bit_cast(frag, last);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < FE; ++e)
                        hi[s][e] = fv[s][e] * weight[0][e];
                }
            }
            const bool exact = EXACT && left - len <= near;
            const bool bad = __ballot(none[0] != 0.f);
            if constexpr (BF) {
                if (bad) {  // the second part of an infinity is none, not a NaN
#pragma unroll
                    for (int s = 0; s < CS; ++s)
#pragma unroll
                        for (int e = 0; e < FE; ++e)
                            if (lo[s][e] != lo[s][e])
                                lo[s][e] = bf16(0.f);
                    if constexpr (EXACT) {
#pragma unroll
                        for (int s = 0; s < CS; ++s)
#pragma unroll
                            for (int e = 0; e < FE; ++e)
                                if (rest[s][e] != rest[s][e])
                                    rest[s][e] = bf16(0.f);
                    }
                }
            }
            if constexpr (!STATE) {
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
                for (int s = 0; s < CS; ++s)
#pragma unroll
                    for (int part = 0; part < (BF ? 2 : 1); ++part)
#pragma unroll
                        for (int it = 0; it < NT; ++it)
                            if (s * O::K < 16 * (it + 1))
                                O::mma(acc[it], fv[s], rows<IO, W::PW>(prow + W::step_at(s), 16 * it - W::step_row(s), BF ? part : s));
                if (bad) {
                    typedef IO Four __attribute__((ext_vector_type(4)));
                    int i = c, four = 16 * wave + 4 * g;  // of v's columns, this lane's
                    asm volatile("" : "+v"(i), "+v"(four));
#pragma unroll 1
                    for (int j = 0; j < len; ++j) {
                        const Four vj = lds_read<Four>(V + LV::at(j, four / O::VE) + four % O::VE * W::E);
                        f32x4 x;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[e] = to_f32(vj[e]);
#pragma unroll
                        for (int it = 0; it < NT; ++it) {
                            const int s = BF ? j / 32 : 0, row = max(16 * it + i - W::step_row(s), 0), col = j - W::step_row(s);
                            const uint32_t at = Ps + W::step_at(s) + LP::at(row, col / O::VE) + col % O::VE * W::E;
                            float pj = to_f32(lds_read<IO>(at));
                            if constexpr (BF)
                                pj += to_f32(lds_read<IO>(LP::further(at, 0, 4)));
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (16 * it + i >= j && x[e] - x[e] != 0.f)
                                    acc[it][e] = fmaf(pj, x[e], acc[it][e]);
                        }
                    }
                }
            }
            const uint32_t kc = kcol + turn * W::kTileK;
            frag fk[2][2][CS];
            auto read = [&](int t) KDN_INLINE {  // of tiles t, t + 1
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int s = 0; s < CS; ++s)
                        fk[t / 2 % 2][i][s] = O::template state_cols<KD>(kc, s, t + i);
            };
            auto add = [&](auto parts) KDN_INLINE {
                read(0);
#pragma unroll
                for (int t = 0; t < ST; t += 2) {
                    if (t + 2 < ST)
                        read(t + 2);
                    // A chunk's sum is formed apart, so that X is rounded once a chunk (errors of
                    // states of fp32 4e-7 -> 2.5e-7, of bf16 2.9e-7 -> 1.7e-7; up to 1% slower);
                    // walks of two parts, whose terms lose more than that, go without.
                    constexpr bool APART = !BF || EXACT;
                    f32x4 sum[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        sum[i] = APART ? zero4() : X[t + i] * whole;
#pragma unroll
                    for (int s = 0; s < CS; ++s)
#pragma unroll
                        for (int part = 0; part < parts; ++part)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                O::mma(sum[i], fk[t / 2 % 2][i][s], part == 0 ? hi[s] : part == 1 ? lo[s] : rest[EXACT ? s : 0]);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            X[t + i][e] = APART ? fmaf(X[t + i][e], whole, sum[i][e]) : sum[i][e];
                }
            };
            if constexpr (EXACT) {
                if (exact)
                    add(std::integral_constant<int, 3>{});
                else
                    add(std::integral_constant<int, 2>{});
            } else {
                add(std::integral_constant<int, BF ? 2 : 1>{});
            }
            if constexpr (!STATE) {
                store(acc, yp, len);
                yp += (rev ? -more : C) * apart;
                arrived<NT>();  // all but the stores, which follow the copies
            } else {
                arrived<0>();
            }
            left -= len;
        }
    };

    if constexpr (STATE) {
        Span span;
        const bool some = handed_on<Counted>(a, b, s, rev, span);
        if (h == 0 && slice == 0 && threadIdx.x == 0)
            r.spans[b * a.S + s] = int4{some ? span.to - span.from : 0, span.first ? span.n : -1, 0, 0};
        if (some) {
            state_in(nullptr, 0, 0);
            walk(span);
            state_out(handed(s), r.vd, 1);
        }
    } else {
        const int t0 = s * a.L, t1 = min(a.T, t0 + a.L);
        Spans<Counted> spans;
        Span span;
        spans.start(a, b, t0, t1, rev, piece);
        while (spans.next(span, a.T)) {
            const size_t n = ((size_t)__builtin_amdgcn_readfirstlane(span.n) * a.H + h) * dense;
            // (offsets that begin below zero claim a segment before the first one)
            if (span.first || (rev ? s + 1 >= a.S : s == 0))
                state_in(r.X0 ? r.X0 + n : nullptr, r.rs, r.cs);
            else
                state_in(handed(rev ? s + 1 : s - 1), r.srs, r.scs);
            walk(span);
            if (span.last && r.XT)
                state_out(r.XT + n, r.rs, r.cs);
        }
        if (a.cu && a.clear && !r.out_f32) {
            IO* y = static_cast<IO*>(r.out);
            for (int t = max(spans.u0, max(a.cu[a.N], 0)); t < spans.u1; ++t)
                if ((int)threadIdx.x < width)
                    y[((row0 + t) * a.H + h) * r.vd + col0 + threadIdx.x] = IO(0.f);
        }
    }
}

// The states handed on, one segment after another: what a segment adds, and what it got,
// decayed over its tokens.  A thread has one element of one head's state; what the next
// segments add is loaded ahead.  (65536 tokens of 16 heads, forward and backward: 13 + 11 us of
// 1467.)
__global__ __launch_bounds__(kThreads) void linattn_join_kernel(LinArgs a)
{
    const LinRole& r = a.role[blockIdx.z];
    const int h = blockIdx.y % a.H, b = blockIdx.y / a.H;
    const size_t dense = (size_t)r.kd * r.vd, i = (size_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= dense)
        return;
    const Decay decay{log((double)a.decay[h])};
    const size_t far = (size_t)a.H * dense;  // to the next segment's state
    float* seg = r.seg + ((size_t)b * a.S * a.H + h) * dense + i;
    const int n = a.S - 1;  // segments that hand on
    auto at = [&](int m) { return r.rev ? a.S - 1 - m : m; };
    constexpr int AHEAD = 8;
    float next[AHEAD], x = 0.f;
#pragma unroll
    for (int m = 0; m < AHEAD; ++m)
        next[m] = m < n ? seg[at(m) * far] : 0.f;
    for (int m0 = 0; m0 < n; m0 += AHEAD) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int m = m0 + k;
            const float added = next[k];
            if (m + AHEAD < n)
                next[k] = seg[at(m + AHEAD) * far];
            if (m >= n)
                break;
            const int4 span = r.spans[b * a.S + at(m)];  // tokens (0: nothing is handed on), sequence that begins
            if (span.x == 0)
                continue;
            if (span.y >= 0)
                x = r.X0 ? r.X0[((size_t)span.y * a.H + h) * dense + (i / r.vd) * r.rs + (i % r.vd) * r.cs] : 0.f;
            x = fmaf(decay.power(span.x), x, added);
            seg[at(m) * far] = x;
        }
    }
}

// y [tokens, Hk, d] = the sum over each group's heads of x [tokens, H, d] (fp32), of both
// tensors; VE values a thread.  Bound by HBM, which x's fp32 keeps busy: 32768 tokens of 4 x 4
// heads of 64, 54 us, 5.6 TB/s.
template <typename IO, int VE>
__global__ __launch_bounds__(256) void linattn_group_kernel(LinArgs a, LinSums sums, int G, int d)
{
    const float* x = sums.x[blockIdx.y];
    IO* y = static_cast<IO*>(sums.y[blockIdx.y]);
    const int Hk = a.H / G, row = Hk * d;
    const long long n = (long long)a.B * a.T * row / VE;
    const int end = a.cu ? a.cu[a.N] : 0;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const long long token = i * VE / row;
        const int at = (int)(i * VE - token * row), hk = at / d, j = at % d;
        float s[VE] = {};
        if (a.cu && token >= end) {
            if (!a.clear)
                continue;
        } else {
            const float* p = x + (token * a.H + hk * G) * d + j;
            for (int m = 0; m < G; ++m, p += d) {
                const Raw<float, VE> r = load_raw<false, float, VE>(p);
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    s[e] += r.get(e);
            }
        }
        store_raw<IO, VE>(y + i * VE, s);
    }
}

// ---- single tokens -------------------------------------------------------------------

// One token.  A workgroup has a head's state rows by 64 columns, a thread VE adjacent
// columns of every 16th (64th) row: bound by HBM, the state being read and written once.
// Rows are taken ROWS at a time, so that many loads are on their way; the rows' shares of o
// are joined through LDS.  256 sequences of 16 heads of 128 x 128: 102 us, 5.3 TB/s (200 with
// a value a load).
template <typename IO, int VE, int ROWS>
__global__ __launch_bounds__(256) void linattn_step_kernel(LinStepArgs a)
{
    constexpr int LANES = kCols / VE, STEP = 256 / LANES;
    __shared__ float part[STEP][kCols];
    const int slices = (a.dv + kCols - 1) / kCols;
    const int slice = blockIdx.x % slices, unit = blockIdx.x / slices, h = unit % a.H, b = unit / a.H;
    const int rg = threadIdx.x / LANES, c = VE * (threadIdx.x % LANES), col = slice * kCols + c;
    const IO* q = static_cast<const IO*>(a.q) + (long long)b * a.qs + (long long)(h / a.G) * a.qh;
    const IO* k = static_cast<const IO*>(a.k) + (long long)b * a.ks + (long long)(h / a.G) * a.kh;
    const IO* v = static_cast<const IO*>(a.v) + (long long)b * a.vs + (long long)h * a.vh;
    float* S = a.S + (size_t)unit * a.dk * a.dv + col;
    const float g = a.decay[h];
    float vv[VE], o[VE] = {};
    if (col < a.dv) {
#pragma unroll
        for (int e = 0; e < VE; ++e)
            vv[e] = to_f32(v[col + e]);
        for (int i0 = rg; i0 < a.dk; i0 += STEP * ROWS) {
            Raw<float, VE> x[ROWS];
            float kk[ROWS], qq[ROWS];
#pragma unroll
            for (int m = 0; m < ROWS; ++m) {
                const int i = min(i0 + m * STEP, a.dk - 1);
                x[m] = load_raw<false, float, VE>(S + (size_t)i * a.dv);
                kk[m] = to_f32(k[i]);
                qq[m] = to_f32(q[i]);
            }
#pragma unroll
            for (int m = 0; m < ROWS; ++m) {
                const int i = i0 + m * STEP;
                if (i >= a.dk)
                    break;
                float y[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    y[e] = fmaf(g, x[m].get(e), kk[m] * vv[e]);
                    o[e] = fmaf(qq[m], y[e], o[e]);
                }
                store_raw<float, VE>(S + (size_t)i * a.dv, y);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < VE; ++e)
        part[rg][c + e] = o[e];
    __syncthreads();
    const int out = slice * kCols + threadIdx.x;
    if (threadIdx.x < kCols && out < a.dv) {
        float s = 0.f;
#pragma unroll
        for (int m = 0; m < STEP; ++m)
            s += part[m][threadIdx.x];
        static_cast<IO*>(a.o)[(size_t)unit * a.dv + out] = from_f32<IO>(s * a.scale);
    }
}

// ---- host ------------------------------------------------------------------------------

size_t aligned16(size_t n) { return (n + 15) / 16 * 16; }

int slices_of(int vd) { return (vd + kCols - 1) / kCols; }

int padded(int kd) { return kd <= 32 ? 32 : kd <= 64 ? 64 : kd <= 128 ? 128 : 256; }

// whether copies of words reach a tensor's rows
bool in_words(const LinTensor& t)
{
    return !((reinterpret_cast<uintptr_t>(t.p) & 3) || (t.ts & 1) || (t.hs & 1));
}

template <typename IO, int KD, bool STATE>
void launch_walk(const LinArgs& a, int roles, hipStream_t stream)
{
    constexpr int C = sizeof(IO) == 2 && KD <= 128 ? 64 : 32;
    constexpr int VE = 16 / sizeof(IO);
    LinArgs b = a;
    b.roles = roles;
    bool edge = false, exact = false;
    for (int i = 0; i < roles; ++i) {
        exact = exact || a.role[i].exact;
        b.slices = b.slices > slices_of(a.role[i].vd) ? b.slices : slices_of(a.role[i].vd);
        edge = edge || a.role[i].kd % VE || a.role[i].vd % VE;
        if (sizeof(IO) == 2 && !(in_words(a.role[i].q) && in_words(a.role[i].k) && in_words(a.role[i].v)))
            b.odd = true;
        if (reinterpret_cast<uintptr_t>(a.role[i].out) & 3)
            edge = true;
    }
    // Sequences of a segment go to several workgroups where there are few: as many as let two
    // stay on a compute unit (30 sequences in 90 tokens of 6 heads, with backward: 571 us by
    // one workgroup a head, 60 so).
    const long long walks = (long long)a.B * a.H * a.S, wide = walks * b.slices * roles;
    b.parts = 1;
    if (!STATE && a.cu && wide < 512) {
        const int most = a.N < a.L ? a.N : a.L;
        b.parts = 512 / wide < most ? (int)(512 / wide) : most;
    }
    b.tokens = (a.L + b.parts - 1) / b.parts;
    const unsigned grid = ((unsigned)walks * b.parts + 7) / 8 * 8 * b.slices * roles;
    auto launch = [&](auto exactly) {
        constexpr bool EXACT = decltype(exactly)::value;
        if (edge || b.odd)
            linattn_kernel<IO, KD, C, STATE, true, EXACT><<<grid, kThreads, 0, stream>>>(b);
        else
            linattn_kernel<IO, KD, C, STATE, false, EXACT><<<grid, kThreads, 0, stream>>>(b);
    };
    if (sizeof(IO) == 2 && exact)
        launch(std::bool_constant<sizeof(IO) == 2>{});
    else
        launch(std::false_type{});
}

template <typename IO, bool STATE>
void launch_roles(const LinArgs& a, int roles, hipStream_t stream)
{
    const int kd = padded(a.role[0].kd);
    if (kd == 32)
        launch_walk<IO, 32, STATE>(a, roles, stream);
    else if (kd == 64)
        launch_walk<IO, 64, STATE>(a, roles, stream);
    else if (kd == 128)
        launch_walk<IO, 128, STATE>(a, roles, stream);
    else
        launch_walk<IO, 256, STATE>(a, roles, stream);
}

// the states that segments hand on
template <typename IO>
void launch_states(const LinArgs& a, int roles, hipStream_t stream)
{
    launch_roles<IO, true>(a, roles, stream);
    const size_t dense = (size_t)a.role[0].kd * a.role[0].vd;
    linattn_join_kernel<<<dim3((unsigned)((dense + kThreads - 1) / kThreads), a.B * a.H, roles), kThreads, 0, stream>>>(a);
}

// Segments of a row and the tokens of one, a multiple of 64, of 128 at least: one where the
// walks fill the chip, else as many as let two workgroups stay on a compute unit.  The
// backward's walks, which meet each other's inputs in the caches, take half as many again
// where segments stay long.  (us, heads of 128 in bf16.  From 256 walks on, 8 x 4096 tokens of
// 16 heads: 181 forward in one segment, 205 in two.  65536 tokens of 16 heads: 432 forward by
// 512 workgroups, 493 by 256, 467 by 1024; backward 1043 by 512, 1038 by 768, 1064 by 1024.
// 2 x 16384 tokens backward 586 by 512, 518 by 768; 2 x 2048 90 and 92.  512 tokens of 4 heads
// in fp32: 29 forward in segments, 52 in one; of 256 tokens at least, 2 x 2047 tokens of 6
// heads in fp32 take 74 instead of 62.)
int segments(int B, int T, int H, int slices, bool backward, int& L)
{
    const long long groups = (long long)B * H * slices, wanted = backward && T * groups >= 2048 * 768 ? 768 : 512;
    const long long want = groups >= 256 ? 1 : wanted / groups, most = T < 512 ? 1 : T / 128;
    const long long S = want < most ? want : most;
    L = S <= 1 ? (T > 0 ? T : 1) : (int)(((T + S - 1) / S + 63) / 64 * 64);
    return T > 0 ? (T + L - 1) / L : 1;
}

// workspace of a walk's handed states: they, and which tokens they are of
size_t handed_bytes(int B, int S, int H, int dk, int dv)
{
    return S > 1 ? aligned16(sizeof(float) * B * S * H * dk * dv) + sizeof(int4) * B * S : 0;
}

void set_handed(LinRole& r, void* ws, int B, int S, int H)
{
    r.seg = static_cast<float*>(ws);
    r.spans = reinterpret_cast<int4*>(static_cast<char*>(ws) + aligned16(sizeof(float) * B * S * H * r.kd * r.vd));
}

template <typename IO>
hipError_t linattn_fwd(const LinArgs& a, hipStream_t stream)
{
    if (a.T > 0) {
        if (a.S > 1)
            launch_states<IO>(a, 1, stream);
        launch_roles<IO, false>(a, 1, stream);
    }
    return hipGetLastError();
}

}  // namespace

size_t linattn_fwd_workspace_bytes(int B, int T, int H, int dk, int dv)
{
    int L;
    const int S = segments(B, T, H, slices_of(dv), false, L);
    return handed_bytes(B, S, H, dk, dv);
}

static size_t bwd_segments_bytes(int B, int T, int H, int dk, int dv, int& S, int& L)
{
    // walks of the same width go in one launch
    const int of_dv = slices_of(dv), of_dk = 2 * slices_of(dk);
    S = segments(B, T, H, padded(dk) == padded(dv) ? of_dv + of_dk : of_dv < of_dk ? of_dv : of_dk, true, L);
    return handed_bytes(B, S, H, dk, dv);
}

size_t linattn_bwd_workspace_bytes(int B, int T, int H, int Hk, int dk, int dv)
{
    int S, L;
    const size_t seg = bwd_segments_bytes(B, T, H, dk, dv, S, L);
    return 2 * seg + (Hk != H ? 2 * aligned16(sizeof(float) * B * T * H * dk) : 0);
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
    a.S = segments(c.B, c.T, c.H, slices_of(c.dv), false, a.L);
    LinRole& r = a.role[0];
    r.q = c.q, r.k = c.k, r.v = c.v;
    r.out = c.o, r.X0 = c.S0, r.XT = c.S_T, r.exact = c.S_T != nullptr;
    r.kd = c.dk, r.vd = c.dv, r.rs = r.srs = c.dv, r.cs = r.scs = 1;
    r.of_p = r.of_x = c.scale, r.of_u = 1.f;
    set_handed(r, c.ws, a.B, a.S, a.H);
    empty_states(a, c.S0, c.S_T, stream);
    return bf ? linattn_fwd<bf16>(a, stream) : linattn_fwd<float>(a, stream);
}

template <typename IO>
static hipError_t linattn_bwd(const LinCall& c, hipStream_t stream)
{
    LinArgs a{};
    a.B = c.B, a.T = c.T, a.H = c.H, a.N = c.N, a.cu = c.cu, a.decay = c.decay, a.clear = c.clear;
    const int G = c.H / c.Hk;
    const size_t seg = bwd_segments_bytes(c.B, c.T, c.H, c.dk, c.dv, a.S, a.L);
    char* ws = static_cast<char*>(c.ws);
    const size_t whole = aligned16(sizeof(float) * c.B * c.T * c.H * c.dk) / sizeof(float);
    float* gq = reinterpret_cast<float*>(ws + 2 * seg);
    float* gk = gq + whole;

    LinRole dq{}, dk{}, dv{};
    dq.q = c.d_o, dq.k = c.v, dq.v = c.k;
    dq.out = G > 1 ? gq : c.dq, dq.out_f32 = G > 1;
    dq.X0 = c.S0, dq.kd = c.dv, dq.vd = c.dk, dq.rs = dq.srs = 1, dq.cs = dq.scs = c.dv;
    dq.of_p = dq.of_x = c.scale, dq.of_u = 1.f;
    set_handed(dq, ws, a.B, a.S, a.H);
    dk.q = c.v, dk.k = c.d_o, dk.v = c.q;
    dk.out = G > 1 ? gk : c.dk_out, dk.out_f32 = G > 1;
    dk.X0 = c.dS_T, dk.kd = c.dv, dk.vd = c.dk, dk.rs = dk.srs = 1, dk.cs = dk.scs = c.dv;
    dk.of_p = dk.of_u = c.scale, dk.of_x = 1.f, dk.rev = 1;
    set_handed(dk, ws + seg, a.B, a.S, a.H);
    dv.q = c.k, dv.k = c.q, dv.v = c.d_o;
    dv.out = c.dv_out, dv.X0 = c.dS_T, dv.XT = c.dS0, dv.exact = c.dS0 != nullptr;
    dv.kd = c.dk, dv.vd = c.dv, dv.rs = dv.srs = c.dv, dv.cs = dv.scs = 1;
    dv.of_p = dv.of_u = c.scale, dv.of_x = 1.f, dv.rev = 1;
    set_handed(dv, ws + seg, a.B, a.S, a.H);

    a.role[0] = dv;
    empty_states(a, c.dS_T, c.dS0, stream);
    if (c.T == 0)
        return hipGetLastError();
    if (a.S > 1) {
        // the forward's states, and those that dv and (turned) dk start from
        LinRole& fwd = a.role[1];
        fwd = dv;
        fwd.q = c.q, fwd.k = c.k, fwd.v = c.v;
        fwd.X0 = c.S0, fwd.of_u = 1.f, fwd.rev = 0, fwd.exact = 0;
        set_handed(fwd, ws, a.B, a.S, a.H);
        launch_states<IO>(a, 2, stream);
    }
    if (padded(c.dk) == padded(c.dv)) {
        a.role[1] = dq, a.role[2] = dk;
        launch_roles<IO, false>(a, 3, stream);
    } else {
        launch_roles<IO, false>(a, 1, stream);
        a.role[0] = dq, a.role[1] = dk;
        launch_roles<IO, false>(a, 2, stream);
    }
    if (G > 1) {
        const LinSums sums{{gq, gk}, {c.dq, c.dk_out}};
        const bool four = c.dk % 4 == 0;
        const long long n = (long long)c.B * c.T * c.Hk * c.dk / (four ? 4 : 1), groups = (n + 255) / 256;
        const dim3 grid((unsigned)(groups < 4096 ? groups : 4096), 2);
        if (four)
            linattn_group_kernel<IO, 4><<<grid, 256, 0, stream>>>(a, sums, G, c.dk);
        else
            linattn_group_kernel<IO, 1><<<grid, 256, 0, stream>>>(a, sums, G, c.dk);
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
    auto run = [&](auto io) {
        typedef decltype(io) IO;
        if (a.dv % 4 == 0)
            linattn_step_kernel<IO, 4, 8><<<groups, 256, 0, stream>>>(a);
        else
            linattn_step_kernel<IO, 1, 8><<<groups, 256, 0, stream>>>(a);
    };
    bf ? run(bf16{}) : run(0.f);
    return hipGetLastError();
}

}  // namespace kdn
