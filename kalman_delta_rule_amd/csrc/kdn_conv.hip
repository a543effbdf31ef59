// kdn_conv.hip -- short causal convolution per channel, forward, backward and
// single-token step, gfx950.
//
//   z_t = b + sum_k w_k x_{t-(W-1)+k},  y = z or z sigmoid(z)
//   g_t = dy_t act'(z_t),  dx_t = sum_k w_k g_{t+(W-1)-k},
//   dw_k = sum_t g_t x_{t-(W-1)+k},  db = sum_t g_t
//
// The rows [B,T] are taken as one row of B T tokens with a sequence starting at
// every T-th (or where the offsets of packed sequences say).  A thread walks a run of
// consecutive tokens for VE adjacent channels with the last W - 1 inputs in
// registers, the next rows' loads issued before the present ones are used.  Each
// input is read once: a run reads the W - 1 rows before it, and the run ahead of it in
// the workgroup takes those, its own last ones, through LDS.  The backward walks
// forward too: it keeps the partial dx of the last W - 1 tokens and stores a token's
// when its last term is added, W - 1 tokens later or at its sequence's end; a run
// stores what its own tokens finish, after the W - 1 tokens before it have gone
// through to begin those sums.
//
// A run without a sequence's border in reach goes the plain way, four tokens at a
// time; the others look for a mark at every token: at a sequence's start the last
// inputs come from its state, at its end they go there.
//
// The forward is bound by HBM: 32768 x 2048 bf16 49 us (5.5 TB/s of inputs and
// outputs), 65536 x 2048 89 us (6.0 TB/s), 16384 x 2048 fp32 44 us (6.1 TB/s).  The
// backward, 95 to 103, 164 and 88 us (3.9 to 4.9 TB/s), is bound by neither HBM nor the
// vector units alone: 31 instructions a value keep those busy 69% of the time (counted),
// with three waves a SIMD to cover loads (four taps and SiLU: 152 registers a thread in
// bf16; in fp32 168, and 20 more spilled).  3 x 1021 x 333 fp32, three taps: 6 us forward,
// 9 and 4 us backward, 192 workgroups whose runs of 8 tokens are walked one token after
// another.
#include "kdn_block.h"
#include "kdn_common.h"
#include "kdn_sequences.h"
#include "kdn_stream.h"

namespace kdn {

namespace {

constexpr int kBatch = 4;  // rows loaded together (at least W - 1); a run is a multiple of it
constexpr int kMostTokens = 1024, kMostRun = 128;  // of a workgroup's tile, of a run

template <typename E, int VE>
__device__ __forceinline__ void widen(const Raw<E, VE>& r, float (&x)[VE])
{
#pragma unroll
    for (int j = 0; j < VE; ++j)
        x[j] = r.get(j);
}

// fp32 values [VE] at p, or zeros
template <typename E, int VE>
__device__ __forceinline__ void load_or_zero(const E* p, bool given, float (&x)[VE])
{
    if (given) {
        widen<E, VE>(load_raw<false, E, VE>(p), x);
    } else {
#pragma unroll
        for (int j = 0; j < VE; ++j)
            x[j] = 0.f;
    }
}

// Which tokens and channels a workgroup works on.
struct Plan {
    int lanes_log2;  // threads side by side on a row: 8 to 64
    int ctiles;      // tiles of channels
    int batches;     // of kBatch tokens in a run
    int tiles;       // tiles of tokens
};

template <int VE>
struct Place {
    int tt;                       // tile of tokens
    int lane, run, runs, length;  // length: tokens of a run
    int c;                        // first channel
    int m0, m;                    // first token of the tile, of the run (B T < 2^31)

    __device__ __forceinline__ Place(const Plan& p, int D)
    {
        tt = blockIdx.x / p.ctiles;
        const int ct = blockIdx.x - tt * p.ctiles;
        lane = threadIdx.x & ((1 << p.lanes_log2) - 1);
        run = threadIdx.x >> p.lanes_log2;
        runs = 256 >> p.lanes_log2;
        length = p.batches * kBatch;
        // lanes behind the last channel repeat the last ones
        c = min(((ct << p.lanes_log2) + lane) * VE, D - VE);
        m0 = tt * runs * length;
        m = m0 + run * length;
    }
};

// The sequences that start and end at the tokens m0 - before .. m0 + count - 1
// (-1 where none does); tokens outside all sequences have neither.
struct Marks {
    int start[kMostTokens + 8], end[kMostTokens + 8];
};

__device__ __forceinline__ void mark_tokens(Marks& k, const ConvArgs& a, int first, int count)
{
    const int M = a.B * a.T;
    if (a.cu) {
        for (int i = threadIdx.x; i < count; i += 256)
            k.start[i] = k.end[i] = -1;
        __syncthreads();
        const SequenceRange near = sequences_at<256>(a.cu, a.N, first, count);
        for (int n = near.first + threadIdx.x; n < near.end; n += 256) {
            const int p = a.cu[n], q = a.cu[n + 1];
            if (p < 0 || p >= q)
                continue;
            if (p >= first && p - first < count)
                k.start[p - first] = n;
            if (q - 1 >= first && q - 1 - first < count)
                k.end[q - 1 - first] = n;
        }
    } else {
        for (int i = threadIdx.x; i < count; i += 256) {
            const int m = first + i;
            const bool in = m >= 0 && m < M;
            const int n = in ? (int)((uint32_t)m / (uint32_t)a.T) : 0, t = m - n * a.T;
            k.start[i] = in && t == 0 ? n : -1;
            k.end[i] = in && t == a.T - 1 ? n : -1;
        }
    }
    __syncthreads();
}

// tokens from this one on belong to no sequence
__device__ __forceinline__ int token_limit(const ConvArgs& a)
{
    return a.cu ? min(max(a.cu[a.N], 0), a.T) : a.B * a.T;
}

// zeros in the rows of `out` for a run's tokens from the i-th on, where the call asks
// for them: those behind the last sequence
template <typename IO, int VE>
__device__ __forceinline__ void clear_rows(const ConvArgs& a, const Place<VE>& at, int i, IO* out)
{
    if (!a.clear)
        return;
    constexpr float zeros[VE] = {};
    const int stop = min(at.length, a.B * a.T - at.m);
    for (i = max(i, 0); i < stop; ++i)
        store_raw<IO, VE>(out + (size_t)(at.m + i) * a.D, zeros);
}

// whether any of marks [i, i + count) is set, for this thread's run (`lanes`
// threads side by side look)
__device__ __forceinline__ bool any_mark(const Marks& k, int i, int count, int lane, int lanes)
{
    bool any = false;
    for (int j = lane; j < count; j += lanes)
        any |= k.start[i + j] >= 0 || k.end[i + j] >= 0;
    return any;
}

// d act(z) / dz and act(z)
__device__ __forceinline__ float silu(float z) { return z * gate_sigmoid(z); }
__device__ __forceinline__ float silu_slope(float z)
{
    const float p = gate_sigmoid(z);
    return p * fmaf(z, 1.f - p, 1.f);
}

// The filter and the last inputs of VE channels.
template <typename IO, int VE, int W>
struct Filter {
    float w[W][VE], b[VE], win[W - 1][VE];

    __device__ __forceinline__ void init(const ConvArgs& a, int c)
    {
#pragma unroll
        for (int k = 0; k < W; ++k)
            load_or_zero<float, VE>(a.weight + (size_t)k * a.D + c, true, w[k]);
        load_or_zero<float, VE>(a.bias + c, a.bias, b);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int j = 0; j < VE; ++j)
                win[k][j] = 0.f;
    }

    __device__ __forceinline__ void from_state(const ConvArgs& a, int n, int c)
    {
        const IO* s = static_cast<const IO*>(a.state0) + (size_t)n * (W - 1) * a.D + c;
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            load_or_zero<IO, VE>(s + (size_t)k * a.D, a.state0, win[k]);
    }

    __device__ __forceinline__ void z(const float (&x)[VE], float (&out)[VE]) const
    {
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            out[j] = b[j];
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                out[j] = fmaf(w[k][j], win[k][j], out[j]);
            out[j] = fmaf(w[W - 1][j], x[j], out[j]);
        }
    }

    __device__ __forceinline__ void push(const float (&x)[VE])
    {
#pragma unroll
        for (int j = 0; j < VE; ++j) {
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k)
                win[k][j] = win[k + 1][j];
            win[W - 2][j] = x[j];
        }
    }
};

// Rows of VE channels of [tokens, `stride` apart].
template <typename IO, int VE, bool ONCE>
struct Rows {
    const IO* base;
    size_t stride;
    int last;  // token

    __device__ __forceinline__ Rows(const void* x, long long stride, int tokens, int c)
        : base(static_cast<const IO*>(x) + c), stride(stride), last(tokens - 1)
    {
    }
    __device__ __forceinline__ const IO* at(int m) const { return base + m * stride; }
    // tokens outside repeat the nearest
    __device__ __forceinline__ Raw<IO, VE> near(int m) const
    {
        return load_raw<ONCE, IO, VE>(at(min(max(m, 0), last)));
    }
};

// The rows before every run of a workgroup, which the run ahead of it ends with: read
// once, by the run behind, and handed on through LDS (slot d - 1: d tokens before
// the run, a thread its own channels).
template <typename IO, int VE, int ROWS>
struct Handed {
    struct alignas(4 * Raw<IO, VE>::kWords) Row {
        uint32_t w[Raw<IO, VE>::kWords];
    };
    Row rows[ROWS][256];

    __device__ __forceinline__ void put(int d, const Raw<IO, VE>& x)
    {
#pragma unroll
        for (int j = 0; j < Raw<IO, VE>::kWords; ++j)
            rows[d - 1][threadIdx.x].w[j] = x.w[j];
    }
    // of the run behind this thread's
    __device__ __forceinline__ Raw<IO, VE> get(int d, int lanes) const
    {
        Raw<IO, VE> x;
#pragma unroll
        for (int j = 0; j < Raw<IO, VE>::kWords; ++j)
            x.w[j] = rows[d - 1][threadIdx.x + lanes].w[j];
        return x;
    }
};

// ---- forward ------------------------------------------------------------------

template <typename IO, int VE, int W, bool SILU, bool ONCE>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a, Plan plan)
{
    __shared__ Marks marks;
    __shared__ Handed<IO, VE, W - 1> handed;
    const Place<VE> at(plan, a.D);
    const int M = a.B * a.T, lanes = 1 << plan.lanes_log2;
    Filter<IO, VE, W> f;
    f.init(a, at.c);

    if (M) {
        const Rows<IO, VE, ONCE> rows(a.x, a.xs, M, at.c);
        Raw<IO, VE> before[W - 1], next[kBatch];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            before[k] = rows.near(at.m - (W - 1) + k);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            next[i] = rows.near(at.m + i);
        mark_tokens(marks, a, at.m0 - (W - 1), at.runs * at.length + W - 1);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            handed.put(W - 1 - k, before[k]);
        __syncthreads();
        const int base = at.run * at.length;  // mark of the first token before the run
        const int limit = token_limit(a);
        // (a run at the row's front has a mark, so a plain one has tokens all around it)
        const bool plain = !__any(at.m + at.length > limit ||
                                  any_mark(marks, base, at.length + W - 1, at.lane, lanes));
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            float x[VE];
            widen<IO, VE>(before[k], x);
            if (!plain && marks.start[base + k] >= 0)
                f.from_state(a, marks.start[base + k], at.c);
            f.push(x);
        }
        if (plain) {
            const IO* ahead = rows.at(at.m + kBatch);
            IO* y = static_cast<IO*>(a.y) + (size_t)at.m * a.D + at.c;
            for (int q = 0; q < plan.batches; ++q) {
                Raw<IO, VE> now[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    now[i] = next[i];
                if (q + 1 < plan.batches) {
                    const bool ends = q + 2 == plan.batches && at.run + 1 < at.runs;
#pragma unroll
                    for (int i = 0; i < kBatch; ++i, ahead += a.xs)
                        next[i] = ends && kBatch - i < W ? handed.get(kBatch - i, lanes) : load_raw<ONCE, IO, VE>(ahead);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i, y += a.D) {
                    float x[VE], z[VE];
                    widen<IO, VE>(now[i], x);
                    f.z(x, z);
                    if constexpr (SILU) {
#pragma unroll
                        for (int j = 0; j < VE; ++j)
                            z[j] = silu(z[j]);
                    }
                    store_raw<IO, VE>(y, z);
                    f.push(x);
                }
            }
        } else {
            const int stop = min(at.length, limit - at.m);
            for (int i = 0; i < stop; ++i) {
                const int k = base + W - 1 + i;  // mark of this token
                float x[VE], z[VE];
                widen<IO, VE>(next[0], x);
#pragma unroll
                for (int r = 0; r + 1 < kBatch; ++r)
                    next[r] = next[r + 1];
                next[kBatch - 1] = rows.near(at.m + i + kBatch);
                if (marks.start[k] >= 0)
                    f.from_state(a, marks.start[k], at.c);
                f.z(x, z);
                if constexpr (SILU) {
#pragma unroll
                    for (int j = 0; j < VE; ++j)
                        z[j] = silu(z[j]);
                }
                store_raw<IO, VE>(static_cast<IO*>(a.y) + (size_t)(at.m + i) * a.D + at.c, z);
                f.push(x);
                if (marks.end[k] >= 0 && a.state_T) {
                    IO* s = static_cast<IO*>(a.state_T) + (size_t)marks.end[k] * (W - 1) * a.D + at.c;
#pragma unroll
                    for (int r = 0; r < W - 1; ++r)
                        store_raw<IO, VE>(s + (size_t)r * a.D, f.win[r]);
                }
            }
            clear_rows<IO, VE>(a, at, stop, static_cast<IO*>(a.y) + at.c);
        }
    }

    // the state of an empty sequence stays what it was
    if (at.m0 == 0 && a.state_T && (a.cu || !M) && a.N <= kStatesOfRun * at.runs) {
        for (int n = at.run; n < a.N; n += at.runs) {
            if (a.cu && a.cu[n] < a.cu[n + 1])
                continue;
            f.from_state(a, n, at.c);
            IO* s = static_cast<IO*>(a.state_T) + (size_t)n * (W - 1) * a.D + at.c;
#pragma unroll
            for (int r = 0; r < W - 1; ++r)
                store_raw<IO, VE>(s + (size_t)r * a.D, f.win[r]);
        }
    }
}

// ---- backward -----------------------------------------------------------------

template <typename IO, int VE, int W, bool SILU, bool ONCE>
__global__ __launch_bounds__(256, 3) void conv_bwd_kernel(ConvArgs a, Plan plan)
{
    __shared__ Marks marks;
    __shared__ Handed<IO, VE, 2 * (W - 1)> handed_x;
    __shared__ Handed<IO, VE, W - 1> handed_y;
    const Place<VE> at(plan, a.D);
    const int M = a.B * a.T;
    const int lanes = 1 << plan.lanes_log2;
    Filter<IO, VE, W> f;
    f.init(a, at.c);
    float dw[W][VE], db[VE], part[W][VE];  // part[k]: dx of the token W-1-k before this one, so far
#pragma unroll
    for (int j = 0; j < VE; ++j) {
        db[j] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k)
            dw[k][j] = part[k][j] = 0.f;
    }

    if (M) {
        const Rows<IO, VE, ONCE> rows(a.x, a.xs, M, at.c), grads(a.dy, a.D, M, at.c);
        Raw<IO, VE> before[W - 1], wx[W - 1], wy[W - 1], nx[kBatch], ny[kBatch];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            before[k] = rows.near(at.m - 2 * (W - 1) + k);
            wx[k] = rows.near(at.m - (W - 1) + k);
            wy[k] = grads.near(at.m - (W - 1) + k);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            nx[i] = rows.near(at.m + i);
            ny[i] = grads.near(at.m + i);
        }
        mark_tokens(marks, a, at.m0 - 2 * (W - 1), at.runs * at.length + 2 * (W - 1));
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            handed_x.put(2 * (W - 1) - k, before[k]);
            handed_x.put(W - 1 - k, wx[k]);
            handed_y.put(W - 1 - k, wy[k]);
        }
        __syncthreads();
        const int base = at.run * at.length;  // mark of the first token loaded
        const int limit = token_limit(a);
        // (with bad offsets the row's front may have no mark: nothing lies before it)
        const bool plain = !__any(at.m == 0 || at.m + at.length > limit ||
                                  any_mark(marks, base, at.length + 2 * (W - 1), at.lane, lanes));
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            float x[VE];
            widen<IO, VE>(before[k], x);
            if (!plain && marks.start[base + k] >= 0)
                f.from_state(a, marks.start[base + k], at.c);
            f.push(x);
        }
        // adds a token, of input x and output gradient dy, to the partial gradients;
        // `own`: to the sums too
        auto add = [&](const Raw<IO, VE>& rx, const Raw<IO, VE>& ry, bool own) {
            float x[VE], g[VE];
            widen<IO, VE>(rx, x);
            widen<IO, VE>(ry, g);
            if constexpr (SILU) {
                float z[VE];
                f.z(x, z);
#pragma unroll
                for (int j = 0; j < VE; ++j)
                    g[j] *= silu_slope(z[j]);
            }
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                if (own) {
                    db[j] += g[j];
#pragma unroll
                    for (int r = 0; r < W - 1; ++r)
                        dw[r][j] = fmaf(g[j], f.win[r][j], dw[r][j]);
                    dw[W - 1][j] = fmaf(g[j], x[j], dw[W - 1][j]);
                }
#pragma unroll
                for (int r = 0; r < W - 1; ++r)
                    part[r][j] = fmaf(f.w[r][j], g[j], part[r][j]);
                part[W - 1][j] = f.w[W - 1][j] * g[j];
            }
            f.push(x);
        };
        auto shift = [&] {
#pragma unroll
            for (int j = 0; j < VE; ++j)
#pragma unroll
                for (int r = 0; r < W - 1; ++r)
                    part[r][j] = part[r + 1][j];
        };
        IO* dx = static_cast<IO*>(a.dx) + at.c;
        if (plain) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                add(wx[k], wy[k], false);
                shift();
            }
            const IO *ax = rows.at(at.m + kBatch), *ay = grads.at(at.m + kBatch);
            IO* out = dx + (size_t)(at.m - (W - 1)) * a.D;
            for (int q = 0; q < plan.batches; ++q) {
                Raw<IO, VE> cx[kBatch], cy[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    cx[i] = nx[i], cy[i] = ny[i];
                if (q + 1 < plan.batches) {
                    const bool ends = q + 2 == plan.batches && at.run + 1 < at.runs;
#pragma unroll
                    for (int i = 0; i < kBatch; ++i, ax += a.xs, ay += a.D) {
                        const int d = kBatch - i;
                        nx[i] = ends && d <= 2 * (W - 1) ? handed_x.get(d <= 2 * (W - 1) ? d : 1, lanes) : load_raw<ONCE, IO, VE>(ax);
                        ny[i] = ends && d < W ? handed_y.get(d < W ? d : 1, lanes) : load_raw<ONCE, IO, VE>(ay);
                    }
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    add(cx[i], cy[i], true);
                    store_raw<IO, VE>(out, part[0]);
                    out += a.D;
                    shift();
                }
            }
        } else {
            // the sequence that started last, and where
            int seq = -1, began = -1;
            // a finished gradient: of token m, or of the state's row before `began`
            auto finish = [&](int m, const float (&v)[VE]) {
                if (m >= began) {
                    if (m >= 0)
                        store_raw<IO, VE>(dx + (size_t)m * a.D, v);
                } else if (seq >= 0 && a.dstate0) {
                    store_raw<IO, VE>(static_cast<IO*>(a.dstate0) +
                                          ((size_t)seq * (W - 1) + (m - began + W - 1)) * a.D + at.c, v);
                }
            };
            // (one row ahead: more would hold the registers of a wave's worth)
            Raw<IO, VE> x1 = wx[0], y1 = wy[0];
            const int stop = min(at.length, limit - at.m);
            for (int i = -(W - 1); i < stop; ++i) {
                const int m = at.m + i, k = base + 2 * (W - 1) + i;
                const Raw<IO, VE> cx = x1, cy = y1;
                x1 = rows.near(m + 1);
                y1 = grads.near(m + 1);
                if (m < 0)
                    continue;
                const bool own = i >= 0;
                if (marks.start[k] >= 0) {
                    f.from_state(a, marks.start[k], at.c);
                    seq = marks.start[k];
                    began = m;
                }
                add(cx, cy, own);
                if (own)
                    finish(m - (W - 1), part[0]);
                shift();
                if (marks.end[k] >= 0) {
                    // nothing follows in this sequence but its state's gradient
                    const IO* s = static_cast<const IO*>(a.dstate_T) + (size_t)marks.end[k] * (W - 1) * a.D + at.c;
#pragma unroll
                    for (int r = 0; r < W - 1; ++r) {
                        float d[VE];
                        load_or_zero<IO, VE>(s + (size_t)r * a.D, a.dstate_T, d);
#pragma unroll
                        for (int j = 0; j < VE; ++j) {
                            d[j] += part[r][j];
                            part[r][j] = 0.f;
                        }
                        if (own)
                            finish(m - (W - 2) + r, d);
                    }
                }
            }
            clear_rows<IO, VE>(a, at, stop, dx);
        }
    }

    // the gradient by the state of an empty sequence
    if (at.m0 == 0 && a.dstate0 && (a.cu || !M) && a.N <= kStatesOfRun * at.runs) {
        for (int n = at.run; n < a.N; n += at.runs) {
            if (a.cu && a.cu[n] < a.cu[n + 1])
                continue;
            const size_t o = (size_t)n * (W - 1) * a.D + at.c;
#pragma unroll
            for (int r = 0; r < W - 1; ++r) {
                float d[VE];
                load_or_zero<IO, VE>(static_cast<const IO*>(a.dstate_T) + o + (size_t)r * a.D, a.dstate_T, d);
                store_raw<IO, VE>(static_cast<IO*>(a.dstate0) + o + (size_t)r * a.D, d);
            }
        }
    }
    if (!M)
        return;

    // sums over the tile: runs within a wave, then the four waves
    __shared__ float sums[4][64 * VE];
    const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    float* out = a.ws + (size_t)at.tt * (W + 1) * a.D;
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        float s[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            s[j] = k < W ? dw[k < W ? k : 0][j] : db[j];
            for (int o = lanes; o < 64; o *= 2)
                s[j] += __shfl_xor(s[j], o);
        }
        __syncthreads();
        if (l < lanes) {
#pragma unroll
            for (int j = 0; j < VE; ++j)
                sums[wave][l * VE + j] = s[j];
        }
        __syncthreads();
        if (threadIdx.x < lanes) {
#pragma unroll
            for (int j = 0; j < VE; ++j)
                s[j] = (sums[0][l * VE + j] + sums[1][l * VE + j]) + (sums[2][l * VE + j] + sums[3][l * VE + j]);
            store_raw<float, VE>(out + (size_t)k * a.D + at.c, s);
        }
    }
}

// Adds the tiles' sums [tiles][(W+1) D]: 64 columns a workgroup, 16 shares of the
// tiles each, joined in order.
__global__ __launch_bounds__(1024) void conv_sum_kernel(ConvArgs a, int tiles)
{
    __shared__ float share[16][64];
    const int l = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + l, n = (a.W + 1) * a.D;
    float s = 0.f;
    if (c < n) {
#pragma unroll 8
        for (int g = q; g < tiles; g += 16)
            s += a.ws[(size_t)g * n + c];
    }
    share[q][l] = s;
    __syncthreads();
    if (q || c >= n)
        return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        s += share[i][l];
    if (c < a.W * a.D)
        a.dweight[c] = s;
    else if (a.dbias)
        a.dbias[c - a.W * a.D] = s;
}

// ---- one token ---------------------------------------------------------------------

// Four channels a thread (at the end of a row as many as are left, one by one: the
// state is moved on in place, so no two threads may have the same channel).  256 x
// 6144 bf16, four taps: 25 MB.
constexpr int kStepVec = 4;

template <typename IO, int W>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a)
{
    constexpr int VE = kStepVec;
    const int c0 = (blockIdx.y * 256 + threadIdx.x) * VE, b = blockIdx.x;
    auto step = [&](auto ve, int c) {
        constexpr int N = decltype(ve)::value;
        IO* st = static_cast<IO*>(a.state_T) + (size_t)b * (W - 1) * a.D + c;
        Raw<IO, N> in[W];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            in[k] = load_raw<false, IO, N>(st + (size_t)k * a.D);
        in[W - 1] = load_raw<false, IO, N>(static_cast<const IO*>(a.x) + (size_t)b * a.xs + c);
        float z[N];
        load_or_zero<float, N>(a.bias + c, a.bias, z);
#pragma unroll
        for (int k = 0; k < W; ++k) {
            float w[N], x[N];
            load_or_zero<float, N>(a.weight + (size_t)k * a.D + c, true, w);
            widen<IO, N>(in[k], x);
#pragma unroll
            for (int j = 0; j < N; ++j)
                z[j] = fmaf(w[j], x[j], z[j]);
        }
        if (a.silu) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                z[j] = silu(z[j]);
        }
        store_raw<IO, N>(static_cast<IO*>(a.y) + (size_t)b * a.D + c, z);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            store_same<IO, N>(st + (size_t)k * a.D, in[k + 1]);
    };
    if (c0 + VE <= a.D) {
        step(std::integral_constant<int, VE>{}, c0);
    } else {
        for (int c = c0; c < a.D; ++c)
            step(std::integral_constant<int, 1>{}, c);
    }
}

// ---- shapes ------------------------------------------------------------------------

// Threads side by side on a row: as many as its vectors, 8 to 64.  Runs as long as
// give each place for a workgroup on the chip four of them, 8 to 128 tokens.  A
// longer run has fewer tokens before it to go through twice and writes the
// backward's sums once for more tokens, but the workgroups at work then reach over
// more memory at a time (one, three, four and eight a place: backward of 32768 x
// 2048 bf16 122, 102, 101 and 112 us, of 4 x 4096 x 2048 fp32 122, 97, 88 and 90 us).
Plan plan_of(int M, int D, int ve, bool backward)
{
    const int wanted = 4 * 256 * (backward ? 3 : 4);  // places a compute unit, by the registers
    Plan p;
    const int vecs = (D + ve - 1) / ve;
    p.lanes_log2 = vecs <= 8 ? 3 : vecs <= 16 ? 4 : vecs <= 32 ? 5 : 6;
    p.ctiles = (vecs + (1 << p.lanes_log2) - 1) >> p.lanes_log2;
    const int runs = 256 >> p.lanes_log2, most = kMostTokens / runs < kMostRun ? kMostTokens / runs : kMostRun;
    long long length = ((long long)M / runs * p.ctiles + wanted - 1) / wanted;
    length = (length + kBatch - 1) / kBatch * kBatch;
    p.batches = (int)(length < 8 ? 8 : length > most ? most : length) / kBatch;
    const long long per = (long long)runs * p.batches * kBatch;
    p.tiles = M ? (int)((M + per - 1) / per) : 1;
    return p;
}

template <typename IO, int VE, int W, bool SILU>
void launch(const ConvArgs& a, bool backward, hipStream_t stream)
{
    const Plan p = plan_of(a.B * a.T, a.D, VE, backward);
    const unsigned grid = (unsigned)p.tiles * p.ctiles;
    auto run = [&](auto once) {
        constexpr bool ONCE = decltype(once)::value;
        if (backward)
            conv_bwd_kernel<IO, VE, W, SILU, ONCE><<<grid, 256, 0, stream>>>(a, p);
        else
            conv_fwd_kernel<IO, VE, W, SILU, ONCE><<<grid, 256, 0, stream>>>(a, p);
    };
    const size_t e = sizeof(IO), row = a.D * e, x_row = a.xs * e;
    const bool lines = (row | x_row | reinterpret_cast<uintptr_t>(a.x)) % kCacheLine == 0;
    if (VE > 1 && lines && (long long)a.B * a.T * (long long)row >= kLastLevelCache)
        run(std::integral_constant<bool, (VE > 1)>{});
    else
        run(std::false_type{});
    void* states = backward ? a.dstate0 : a.state_T;
    if (states && (a.cu || !a.T) && a.N > kStatesOfRun * (256 >> p.lanes_log2))
        launch_empty_states<IO>(a.cu, a.N, (W - 1) * a.D, backward ? a.dstate_T : a.state0, states, stream);
    if (backward)
        conv_sum_kernel<<<((a.W + 1) * a.D + 63) / 64, 1024, 0, stream>>>(a, a.T ? p.tiles : 0);
}

template <typename IO, int VE, int W>
void launch_act(const ConvArgs& a, bool backward, hipStream_t stream)
{
    a.silu ? launch<IO, VE, W, true>(a, backward, stream) : launch<IO, VE, W, false>(a, backward, stream);
}

template <typename IO, int VE>
void launch_taps(const ConvArgs& a, bool backward, hipStream_t stream)
{
    a.W == 2   ? launch_act<IO, VE, 2>(a, backward, stream)
    : a.W == 3 ? launch_act<IO, VE, 3>(a, backward, stream)
               : launch_act<IO, VE, 4>(a, backward, stream);
}

// Four channels a thread (8 bytes of bf16: eight would take the registers of twice
// the waves, 60 us against 52 at 32768 x 2048); fewer than four go one a thread.
int vector_of(int D) { return D < 4 ? 1 : 4; }

template <typename IO>
hipError_t launch_io(const ConvArgs& a, bool backward, hipStream_t stream)
{
    vector_of(a.D) == 1 ? launch_taps<IO, 1>(a, backward, stream) : launch_taps<IO, 4>(a, backward, stream);
    return hipGetLastError();
}

}  // namespace

int conv_bwd_groups(int B, int T, int D)
{
    return T ? plan_of(B * T, D, vector_of(D), true).tiles : 0;
}

hipError_t launch_conv_fwd(const ConvArgs& a, bool bf, hipStream_t stream)
{
    return bf ? launch_io<bf16>(a, false, stream) : launch_io<float>(a, false, stream);
}

hipError_t launch_conv_bwd(const ConvArgs& a, bool bf, hipStream_t stream)
{
    return bf ? launch_io<bf16>(a, true, stream) : launch_io<float>(a, true, stream);
}

template <typename IO>
static hipError_t conv_step(const ConvArgs& a, hipStream_t stream)
{
    const dim3 grid(a.B, (a.D + 256 * kStepVec - 1) / (256 * kStepVec));
    if (a.W == 2)
        conv_step_kernel<IO, 2><<<grid, 256, 0, stream>>>(a);
    else if (a.W == 3)
        conv_step_kernel<IO, 3><<<grid, 256, 0, stream>>>(a);
    else
        conv_step_kernel<IO, 4><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_conv_step(const ConvArgs& a, bool bf, hipStream_t stream)
{
    return bf ? conv_step<bf16>(a, stream) : conv_step<float>(a, stream);
}

}  // namespace kdn
