// kdn_group_norm.hip -- group norm with an activation, channels last, gfx950.
//
//   x [N, S, C], G groups of C / G channels; mean, rstd over a sample's positions and a
//   group's channels;  z = (x - mean) rstd w + b,  y = z or z sigmoid(z)
//   g = dy (times the activation's slope),  xh = (x - mean) rstd
//   dx = rstd (g w - mean(g w) - xh mean(g w xh)),  dw = sum g xh,  db = sum g
//
// Both are bound by HBM (heads of 128, 32768 x 2048 bf16 with SiLU: forward 60 us, 4.5 TB/s;
// backward 97 us, 4.2 TB/s, and 5 for the channels' sums).  Where a group of a sample (a unit) fits the registers of up to
// 1024 threads it is read once: a thread holds NV vectors of 16 bytes, always of the same
// channels of its group, so that w and b, and in the backward the channels' sums, stay in
// registers over all the units that it walks.  The variance is taken around the mean, and
// the mean is corrected by what is left around it.  Larger units are
// read twice by many workgroups, whose sums by channel are joined in between.
#include "kdn_common.h"
#include "kdn_lanes.h"
#include "kdn_layer_ops.h"
#include "kdn_stream.h"

#include <type_traits>

namespace kdn {

namespace {

__device__ __forceinline__ float silu_of(float z) { return z * gate_sigmoid(z); }
__device__ __forceinline__ float silu_slope(float z)
{
    const float p = gate_sigmoid(z);
    return p * fmaf(z, 1.f - p, 1.f);
}

// (a NaN stays one)
__device__ __forceinline__ float not_below_zero(float x) { return x < 0.f ? 0.f : x; }

// 1 / sqrt(x) within 1 ulp, denormal numbers included
__device__ __forceinline__ float rsqrt_of(float x)
{
    const bool tiny = x < 0x1p-100f;
    return __builtin_amdgcn_rsqf(tiny ? x * 0x1p100f : x) * (tiny ? 0x1p50f : 1.f);
}

// The sums of two values over the TPR threads of a unit, in all of them; `red` holds a
// slot for each wave of the workgroup.
template <int TPR>
__device__ __forceinline__ float2 unit_sum(float a, float b, float2* red)
{
    constexpr int N = TPR < 64 ? TPR : 64;
    a = lane_sum<N>(a);
    b = lane_sum<N>(b);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        __syncthreads();  // the last sum's reads are done
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = float2{a, b};
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float2 r = red[threadIdx.x / TPR * W + w];
            a += r.x;
            b += r.y;
        }
    }
    return float2{a, b};
}

// VE adjacent values, the first n of them there (WHOLE: all or none), without a branch a value.
// A vector that is not whole is read so that it ends with its last value, if VE values end there
// (back), else in halves, quarters, ..; `settle` puts its values in place once they are used,
// since what waits for one load would wait for all.  (2497 x 73 positions of 16 groups of 20,
// forward: 164 us a value at a time, 102 so.)
template <bool WHOLE, typename E, int VE>
__device__ __forceinline__ Raw<E, VE> load_part(const E* p, int n, bool back)
{
    Raw<E, VE> r{};
    if (WHOLE || back) {
        if (n)
            r = load_raw<false, E, VE>(WHOLE ? p : p - (VE - n));
    } else if (n == VE) {
        r = load_raw<false, E, VE>(p);
    } else if constexpr (VE == 8) {
        if (n & 4) {
            const auto x = load_raw<false, E, 4>(p);
            r.w[0] = x.w[0], r.w[1] = x.w[1];
        }
        if (n & 2)
            r.w[2] = load_raw<false, E, 2>(p + (n & 4)).w[0];
        if (n & 1)
            r.w[3] = load_raw<false, E, 1>(p + (n & 6)).w[0];
    } else {
        if (n & 2) {
            const auto x = load_raw<false, E, 2>(p);
            r.w[0] = x.w[0], r.w[1] = x.w[1];
        }
        if (n & 1)
            r.w[3] = load_raw<false, E, 1>(p + (n & 2)).w[0];
    }
    return r;
}
template <bool WHOLE, typename E, int VE>
__device__ __forceinline__ void settle(Raw<E, VE>& r, int n, bool back)
{
    if (WHOLE || n == VE || n == 0)
        return;
    if (back) {
        const int by = (VE - n) * (int)sizeof(E) * 8;  // under 128
        const uint64_t low = r.w[0] | (uint64_t)r.w[1] << 32, high = r.w[2] | (uint64_t)r.w[3] << 32;
        const uint64_t x = by < 64 ? low >> by | high << (64 - by) : high >> (by - 64), y = by < 64 ? high >> by : 0;
        r.w[0] = (uint32_t)x, r.w[1] = (uint32_t)(x >> 32), r.w[2] = (uint32_t)y, r.w[3] = (uint32_t)(y >> 32);
    } else if constexpr (VE == 8) {
        const uint32_t two = r.w[2], one = r.w[3], x = n & 2 ? two : one, y = n & 2 ? one : 0;
        if (n & 4)
            r.w[2] = x, r.w[3] = y;
        else
            r.w[0] = x, r.w[1] = y, r.w[2] = r.w[3] = 0;
    } else {
        if (n & 2)
            r.w[2] = r.w[3];
        else
            r.w[0] = r.w[3];
        r.w[3] = 0;
    }
}
template <typename E, int VE>
__device__ __forceinline__ void store_some(E* p, const float (&v)[VE], int n)
{
    if (n >= VE) {
        store_raw<E, VE>(p, v);
        return;
    }
    // by halves, quarters, ..
    E x[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j)
        x[j] = from_f32<E>(v[j]);
    if constexpr (VE == 8) {
        if (n & 4) {
            store_raw<E, 4>(p, {v[0], v[1], v[2], v[3]});
            p += 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = x[j + 4];
        }
    }
    if (n & 2) {
        p[0] = x[0], p[1] = x[1];
        p += 2;
        x[0] = x[2];
    }
    if (n & 1)
        p[0] = x[0];
}
// Values are taken from their words again: kept as fp32 from one pass over a unit to the
// next they would need twice the registers.
template <typename E, int VE, int NV>
__device__ __forceinline__ void anew(Raw<E, VE> (&r)[NV])
{
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < Raw<E, VE>::kWords; ++i)
            asm volatile("" : "+v"(r[v].w[i]));
}
template <int VE>
__device__ __forceinline__ void load_param(const float* p, float other, int n, float (&w)[VE])
{
#pragma unroll
    for (int j = 0; j < VE; ++j)
        w[j] = p && j < n ? p[j] : other;
}

// What a unit's threads hold, and which units they walk.
struct Held {
    int tpr, nv;  // tpr 0: too large
    int pad;      // threads side by side over a group's channels, a power of two
    int grid;     // workgroups
    int share;    // units that touch a cache line, on one XCD
};

template <typename IO, int TPR, int NV, int THREADS>
struct Part {
    static constexpr int VE = 16 / sizeof(IO), SETS = THREADS / TPR;
    int set, n, g, step;    // of units: this one's sample and group, sets of the launch
    int s0, ds, col, width; // this thread's first position, positions a turn, channels
    bool on;                // there is such a unit
    bool back;              // VE values end with a group's last

    __device__ __forceinline__ Part(const GroupNormArgs& a, const Held& held)
    {
        const int Cg = a.C / a.G;
        int block = blockIdx.x;
        if (held.share > 1 && SETS == 1) {
            // units that share cache lines on one XCD: workgroups go round the eight
            const int round = 8 * held.share, at = block / round * round;
            if (at + round <= (int)gridDim.x) {
                const int i = block - at;
                block = at + (i & 7) * held.share + (i >> 3);
            }
        }
        const int t = threadIdx.x % TPR;
        set = block * SETS + threadIdx.x / TPR;
        if constexpr (TPR >= 64)
            set = __builtin_amdgcn_readfirstlane(set);
        step = gridDim.x * SETS;
        n = set / a.G, g = set % a.G;
        on = n < a.N;
        const int piece = t & (held.pad - 1);
        s0 = t / held.pad, ds = TPR / held.pad;
        col = g * Cg + piece * VE;
        width = min(max(Cg - piece * VE, 0), VE);
        back = Cg >= VE;
    }
    // elements that there are of vector v
    __device__ __forceinline__ int there(int S, int v) const { return s0 + v * ds < S ? width : 0; }
    __device__ __forceinline__ size_t at(const GroupNormArgs& a, int v, long long stride, int sample) const
    {
        return ((size_t)sample * a.S + s0 + v * ds) * stride + col;
    }
};

// WHOLE: a group's channels are whole vectors
template <typename IO, int TPR, int NV, bool WHOLE>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void group_norm_fwd_kernel(GroupNormArgs a, Held held)
{
    constexpr int THREADS = TPR > 256 ? TPR : 256;
    typedef Part<IO, TPR, NV, THREADS> P;
    constexpr int VE = P::VE;
    __shared__ float2 red[THREADS / 64];
    P part(a, held);
    // the first mean is divided by the count, not multiplied with its reciprocal: that of
    // equal values is that value
    const float count = (float)a.S * (a.C / a.G), inv = 1.f / count;
    float w[VE], b[VE];
    load_param(a.weight ? a.weight + part.col : nullptr, 1.f, part.on ? part.width : 0, w);
    load_param(a.bias ? a.bias + part.col : nullptr, 0.f, part.on ? part.width : 0, b);
    const IO* x = static_cast<const IO*>(a.x);
    IO* y = static_cast<IO*>(a.y);
    // Small units are loaded one ahead (524288 units of 128 bf16: 60 us, 73 without).
    constexpr bool AHEAD = NV <= 2;
    const long long units = (long long)a.N * a.G;
    Raw<IO, VE> raw[NV], next[AHEAD ? NV : 1];
    auto load = [&](Raw<IO, VE>(&to)[NV], int sample) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int n = sample < a.N ? part.there(a.S, v) : 0;
            to[v] = load_part<WHOLE, IO, VE>(x + (n ? part.at(a, v, a.xs, sample) : 0), n, part.back);
        }
    };
    if constexpr (AHEAD)
        load(next, part.n);
    // all sets walk as many units; those behind the last sample hold nothing
    for (long long u = P::SETS == 1 ? part.set : blockIdx.x * (long long)P::SETS; u < units; u += part.step, part.n += part.step / a.G) {
        const bool on = part.n < a.N;
        if constexpr (AHEAD) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                raw[v] = next[v];
            if (u + part.step < units)
                load(next, part.n + part.step / a.G);
        } else {
            load(raw, part.n);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            settle<WHOLE>(raw[v], part.width, part.back);
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < VE; ++j)
                s += raw[v].get(j);
        const float near = unit_sum<TPR>(s, 0.f, red).x / count;
        if constexpr (NV > 2)
            anew(raw);
        float d1 = 0.f, d2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int n = on ? part.there(a.S, v) : 0;
            if (n == 0)
                continue;
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const float d = WHOLE || j < n ? raw[v].get(j) - near : 0.f;
                d1 += d;
                d2 = fmaf(d, d, d2);
            }
        }
        const float2 m = unit_sum<TPR>(d1, d2, red);
        if constexpr (NV > 2)
            anew(raw);
        const float off = m.x * inv, mean = near + off;
        const float rstd = rsqrt_of(not_below_zero(m.y * inv - off * off) + a.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int n = on ? part.there(a.S, v) : 0;
            if (n == 0)
                continue;
            float o[VE];
#pragma unroll
            for (int j = 0; j < VE; ++j)
                o[j] = fmaf((raw[v].get(j) - near - off) * rstd, w[j], b[j]);
            if (a.silu) {
#pragma unroll
                for (int j = 0; j < VE; ++j)
                    o[j] = silu_of(o[j]);
            }
            store_some<IO, VE>(y + part.at(a, v, a.C, part.n), o, WHOLE ? VE : n);
        }
        if (on && threadIdx.x % TPR == 0) {
            const size_t i = (size_t)part.n * a.G + part.g;
            if (a.mean)
                a.mean[i] = mean;
            if (a.rstd)
                a.rstd[i] = rstd;
        }
    }
}

// (512: the sums by channel of a workgroup are for more units, fewer slots: 32768 x 2048 bf16
// forward and backward 159 us, with 256 170)
constexpr int bwd_threads(int tpr) { return tpr > 512 ? tpr : 512; }

// Slots of sums by channel that a backward launch leaves: a workgroup's where it holds all
// groups, else one for every G units side by side.
__host__ __device__ inline int slots_of(int grid, int sets, int G) { return sets >= G ? grid : (grid * sets + G - 1) / G; }

template <typename IO, int TPR, int NV, bool WHOLE>
__global__ __launch_bounds__(bwd_threads(TPR)) void group_norm_bwd_kernel(GroupNormArgs a, Held held)
{
    constexpr int THREADS = bwd_threads(TPR);
    typedef Part<IO, TPR, NV, THREADS> P;
    constexpr int VE = P::VE, SETS = P::SETS;
    constexpr bool KEEP = NV * VE <= 16;  // g is kept, not formed again
    __shared__ float2 red[THREADS / 64];
    __shared__ float sums[THREADS * VE];
    P part(a, held);
    const float inv = 1.f / ((float)a.S * (a.C / a.G));
    float w[VE], b[VE], dw[VE] = {}, db[VE] = {};
    load_param(a.weight ? a.weight + part.col : nullptr, 1.f, part.on ? part.width : 0, w);
    load_param(a.bias ? a.bias + part.col : nullptr, 0.f, part.on ? part.width : 0, b);
    const IO* x = static_cast<const IO*>(a.x);
    const IO* dy = static_cast<const IO*>(a.dy);
    IO* dx = static_cast<IO*>(a.dx);
    const long long units = (long long)a.N * a.G;
    Raw<IO, VE> rx[NV], ry[NV];
    auto load = [&](Raw<IO, VE>(&tx)[NV], Raw<IO, VE>(&ty)[NV], int sample) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int n = sample < a.N ? part.there(a.S, v) : 0;
            tx[v] = load_part<WHOLE, IO, VE>(x + (n ? part.at(a, v, a.xs, sample) : 0), n, part.back);
            ty[v] = load_part<WHOLE, IO, VE>(dy + (n ? part.at(a, v, a.C, sample) : 0), n, part.back);
        }
    };
    for (long long u = SETS == 1 ? part.set : blockIdx.x * (long long)SETS; u < units; u += part.step, part.n += part.step / a.G) {
        const bool on = part.n < a.N;
        float kept[KEEP ? NV : 1][VE];
        load(rx, ry, part.n);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            settle<WHOLE>(rx[v], part.width, part.back);
            settle<WHOLE>(ry[v], part.width, part.back);
        }
        const size_t i = (size_t)(on ? part.n : 0) * a.G + part.g;
        const float mean = a.mean[i], rstd = a.rstd[i];
        auto slope = [&](int v, int j, float xh) {
            const float d = ry[v].get(j);
            return a.silu ? d * silu_slope(fmaf(xh, w[j], b[j])) : d;
        };
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int n = on ? part.there(a.S, v) : 0;
            if (n == 0)
                continue;
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const float xh = (rx[v].get(j) - mean) * rstd;
                const float g = WHOLE || j < n ? slope(v, j, xh) : 0.f;
                if constexpr (KEEP)
                    kept[v][j] = g;
                if (WHOLE || j < n) {
                    s1 = fmaf(g, w[j], s1);
                    s2 = fmaf(g * w[j], xh, s2);
                    dw[j] = fmaf(g, xh, dw[j]);
                    db[j] += g;
                }
            }
        }
        const float2 m = unit_sum<TPR>(s1, s2, red);
        const float m1 = m.x * inv, m2 = m.y * inv;
        if constexpr (!KEEP)
            anew(rx), anew(ry);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int n = on ? part.there(a.S, v) : 0;
            if (n == 0)
                continue;
            float o[VE];
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const float xh = (rx[v].get(j) - mean) * rstd;
                float g;
                if constexpr (KEEP)
                    g = kept[v][j];
                else
                    g = slope(v, j, xh);
                o[j] = rstd * (g * w[j] - m1 - xh * m2);
            }
            store_some<IO, VE>(dx + part.at(a, v, a.C, part.n), o, WHOLE ? VE : n);
        }
    }
    if (!a.ws)
        return;
    // threads of the same channels: lanes of a wave, then waves of a set, then sets of the
    // same group, which lie G apart
    constexpr int LANES = TPR < 64 ? TPR : 64;
    const int row = held.pad < LANES ? held.pad : LANES;  // threads whose sums are left of a part
    const int Cg = a.C / a.G, first = part.set - (int)threadIdx.x / TPR;  // the workgroup's first set
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            float s = k ? db[j] : dw[j];
            for (int o = held.pad; o < LANES; o *= 2)
                s += __shfl_xor(s, o);
            if ((int)threadIdx.x % LANES < row)
                sums[(threadIdx.x / LANES * row + threadIdx.x % LANES) * VE + j] = s;
        }
        __syncthreads();
        // of a set: TPR / LANES parts of `row` threads; part i holds pieces i row .. modulo pad
        const int groups = SETS < a.G ? SETS : a.G, cols = groups * Cg;
        for (int i = threadIdx.x; i < cols; i += THREADS) {
            const int q = i / Cg, c = i % Cg, piece = c / VE, j = c % VE;
            float s = 0.f;
            for (int set = q; set < SETS; set += a.G)
                for (int p = piece / row; p < TPR / LANES; p += held.pad / row)
                    s += sums[((set * (TPR / LANES) + p) * row + piece % row) * VE + j];
            const int id = first + q, g = id % a.G;
            const int slot = SETS >= a.G ? (int)blockIdx.x : id / a.G;
            static_cast<float*>(a.ws)[((size_t)slot * 2 + k) * a.C + g * Cg + c] = s;
        }
    }
}

// dw and db from sums [slots][2][C]: 64 columns a workgroup, 16 shares of the slots each,
// joined in order.  `units` of them side by side in G groups have written (0: all).
__global__ __launch_bounds__(1024) void group_norm_sum_kernel(GroupNormArgs a, const float* ws, int slots, int units)
{
    __shared__ float share[16][64];
    const int l = threadIdx.x & 63, q = threadIdx.x >> 6, n = 2 * a.C;
    const int c = blockIdx.x * 64 + l;
    float s = 0.f;
    if (c < n) {
        const int g = c % a.C / (a.C / a.G);
        const int end = units ? min(slots, (units - g + a.G - 1) / a.G) : slots;
#pragma unroll 8
        for (int i = q; i < end; i += 16)
            s += ws[(size_t)i * n + c];
    }
    share[q][l] = s;
    __syncthreads();
    if (q || c >= n)
        return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        s += share[i][l];
    float* out = c < a.C ? a.dweight : a.dbias;
    if (out)
        out[c < a.C ? c : c - a.C] = s;
}

// ---- large units: sums by channel of tiles of positions, joined in between -------------

struct Split {
    int lanes;          // threads side by side over channels (VE each), a power of two
    int blocks, tiles;  // of channels, of positions
    int rows;           // positions of a tile
};

// This thread's channels and positions; workgroups (sample, tile, block of channels).
template <int VE>
struct Place {
    int n, tile, c, width, s, s1, ds, lane;
    bool back;  // VE values end with a row's last
    __device__ __forceinline__ Place(const GroupNormArgs& a, const Split& p)
    {
        int i = blockIdx.x;
        const int block = i % p.blocks;
        i /= p.blocks;
        tile = i % p.tiles, n = i / p.tiles;
        lane = threadIdx.x & (p.lanes - 1);
        c = (block * p.lanes + lane) * VE;
        width = min(max(a.C - c, 0), VE);
        back = a.C >= VE;
        ds = 256 / p.lanes;
        s = tile * p.rows + threadIdx.x / p.lanes;
        s1 = min(a.S, (tile + 1) * p.rows);
    }
};

// Sums for each of VE channels over the threads that hold them, in all of these
template <int VE>
__device__ __forceinline__ void channel_sum(const Split& p, int lane, float (&a)[VE], float (*lds)[VE])
{
    __syncthreads();  // the last sum's reads are done
#pragma unroll
    for (int j = 0; j < VE; ++j)
        lds[threadIdx.x][j] = a[j];
    for (int half = 128; half >= p.lanes; half >>= 1) {
        __syncthreads();
        if ((int)threadIdx.x < half)
#pragma unroll
            for (int j = 0; j < VE; ++j)
                lds[threadIdx.x][j] += lds[threadIdx.x + half][j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VE; ++j)
        a[j] = lds[lane][j];
}

// A tile's mean and sum of squares around it, by channel.  A thread takes four positions at a
// time: their mean, and their squares around it, joined with those of the positions before
// (Chan, Golub, LeVeque 1979); the threads' are joined around the tile's mean.  Only squares
// are added, so that nothing cancels wherever single values lie.  (Sums around one of the
// values left rstd 1.3e-3 off where that one lay far from the others, 1030 x 100000 positions,
// the first at 10000, and took as long: 64 x 4096 positions of 256 channels fp32 forward 171
// us, 168 so; 2497 x 292 of 320 in groups of 20, bf16, 370 and 354.)  Values are taken from
// one of the tile's, the middle one of three: what lies far from zero keeps its digits.
// ws [N][tiles][C][2]
template <typename IO, bool WHOLE>
__global__ __launch_bounds__(256) void group_norm_stats_kernel(GroupNormArgs a, Split p, float2* ws)
{
    constexpr int VE = 16 / sizeof(IO);
    __shared__ float lds[256][VE];
    const Place<VE> at(a, p);
    const IO* x = static_cast<const IO*>(a.x) + (size_t)at.n * a.S * a.xs + at.c;
    const int s0 = at.tile * p.rows;
    float k[VE], mean[VE] = {}, squares[VE] = {}, n = 0.f;
    {
        const int last = min(a.S, s0 + p.rows) - 1;
        Raw<IO, VE> r[3];
#pragma unroll
        for (int i = 0; i < 3; ++i)
            r[i] = load_part<WHOLE, IO, VE>(x + (at.width ? (size_t)(i == 0 ? s0 : i == 1 ? (s0 + last) / 2 : last) * a.xs : 0),
                                            at.width, at.back);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            settle<WHOLE>(r[i], at.width, at.back);
#pragma unroll
        for (int j = 0; j < VE; ++j)
            k[j] = __builtin_amdgcn_fmed3f(r[0].get(j), r[1].get(j), r[2].get(j));
    }
    auto take = [&](int s, auto rows) {
        constexpr int R = decltype(rows)::value;
        Raw<IO, VE> r[R];
#pragma unroll
        for (int i = 0; i < R; ++i)
            r[i] = load_part<WHOLE, IO, VE>(x + (size_t)(s + i * at.ds) * a.xs, WHOLE ? VE : at.width, at.back);
#pragma unroll
        for (int i = 0; i < R; ++i)
            settle<WHOLE>(r[i], at.width, at.back);
        const float share = R / (n + R), both = n * share;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            float sum = 0.f, q = 0.f;
#pragma unroll
            for (int i = 0; i < R; ++i)
                sum += r[i].get(j) - k[j];
            const float here = sum * (1.f / R), apart = here - mean[j];
            if constexpr (R > 1)
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float d = r[i].get(j) - k[j] - here;
                    q = fmaf(d, d, q);
                }
            mean[j] = fmaf(apart, share, mean[j]);
            squares[j] += fmaf(apart * apart, both, q);
        }
        n += R;
    };
    if (at.width) {
        int s = at.s;
        for (; s + 3 * at.ds < at.s1; s += 4 * at.ds)
            take(s, std::integral_constant<int, 4>{});
        for (; s < at.s1; s += at.ds)
            take(s, std::integral_constant<int, 1>{});
    }
    const float count = at.s1 - s0;
    float all[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j)
        all[j] = n * mean[j];
    channel_sum<VE>(p, at.lane, all, lds);
#pragma unroll
    for (int j = 0; j < VE; ++j) {
        all[j] /= count;
        const float d = mean[j] - all[j];
        squares[j] = fmaf(n * d, d, squares[j]);
    }
    channel_sum<VE>(p, at.lane, squares, lds);
    if ((int)threadIdx.x < p.lanes)
#pragma unroll
        for (int j = 0; j < VE; ++j)
            if (j < at.width)
                ws[((size_t)at.n * p.tiles + at.tile) * a.C + at.c + j] = float2{k[j] + all[j], squares[j]};
}

// A group's statistics from its channels' in every tile.  mean, rstd [N,G] (a.mean, a.rstd
// and, for the kernel that follows, stats)
__global__ __launch_bounds__(256) void group_norm_join_kernel(GroupNormArgs a, Split p, const float2* ws, float2* stats)
{
    __shared__ float2 red[4];
    const int n = blockIdx.x / a.G, g = blockIdx.x % a.G, Cg = a.C / a.G, items = p.tiles * Cg;
    const float count = (float)a.S * Cg;
    const float2* from = ws + (size_t)n * p.tiles * a.C + g * Cg;
    auto item = [&](int i, float& positions) {
        const int tile = i / Cg;
        positions = min(a.S, (tile + 1) * p.rows) - tile * p.rows;
        return from[(size_t)tile * a.C + i % Cg];
    };
    float s = 0.f, q = 0.f, positions;
    const float first = from[0].x;  // sums around it: means far from zero cancel exactly
#pragma unroll 4
    for (int i = threadIdx.x; i < items; i += 256) {
        const float2 x = item(i, positions);
        s = fmaf(positions, x.x - first, s);
    }
    const float mean = first + unit_sum<256>(s, 0.f, red).x / count;
#pragma unroll 4
    for (int i = threadIdx.x; i < items; i += 256) {
        const float2 x = item(i, positions);
        const float d = x.x - mean;
        q += fmaf(positions * d, d, x.y);
    }
    const float rstd = rsqrt_of(unit_sum<256>(q, 0.f, red).x / count + a.eps);
    if (threadIdx.x == 0) {
        stats[blockIdx.x] = float2{mean, rstd};
        if (a.mean)
            a.mean[blockIdx.x] = mean;
        if (a.rstd)
            a.rstd[blockIdx.x] = rstd;
    }
}

template <typename IO, bool WHOLE>
__global__ __launch_bounds__(256) void group_norm_apply_kernel(GroupNormArgs a, Split p, const float2* stats)
{
    constexpr int VE = 16 / sizeof(IO);
    const Place<VE> at(a, p);
    if (!at.width)
        return;
    float w[VE], b[VE], mean[VE], rstd[VE];
    load_param(a.weight ? a.weight + at.c : nullptr, 1.f, at.width, w);
    load_param(a.bias ? a.bias + at.c : nullptr, 0.f, at.width, b);
    const int Cg = a.C / a.G;
#pragma unroll
    for (int j = 0; j < VE; ++j) {
        const float2 m = stats[(size_t)at.n * a.G + min(at.c + j, a.C - 1) / Cg];
        mean[j] = m.x, rstd[j] = m.y;
    }
    const IO* x = static_cast<const IO*>(a.x) + (size_t)at.n * a.S * a.xs + at.c;
    IO* y = static_cast<IO*>(a.y) + (size_t)at.n * a.S * a.C + at.c;
#pragma unroll 4
    for (int s = at.s; s < at.s1; s += at.ds) {
        Raw<IO, VE> r = load_part<WHOLE, IO, VE>(x + (size_t)s * a.xs, WHOLE ? VE : at.width, at.back);
        settle<WHOLE>(r, at.width, at.back);
        float o[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j)
            o[j] = fmaf((r.get(j) - mean[j]) * rstd[j], w[j], b[j]);
        if (a.silu) {
#pragma unroll
            for (int j = 0; j < VE; ++j)
                o[j] = silu_of(o[j]);
        }
        store_some<IO, VE>(y + (size_t)s * a.C, o, WHOLE ? VE : at.width);
    }
}

// The backward's first pass (APPLY false): sums of g and g xh by channel of a tile, ws
// [N][tiles][2][C]; and its second: dx, with the groups' means of g w and g w xh in `means`.
template <typename IO, bool APPLY, bool WHOLE>
__global__ __launch_bounds__(256) void group_norm_bwd_split_kernel(GroupNormArgs a, Split p, float* ws, const float2* means)
{
    constexpr int VE = 16 / sizeof(IO);
    __shared__ float lds[APPLY ? 1 : 256][VE];
    const Place<VE> at(a, p);
    float w[VE], b[VE], mean[VE], rstd[VE], m1[VE] = {}, m2[VE] = {};
    load_param(a.weight ? a.weight + at.c : nullptr, 1.f, at.width, w);
    load_param(a.bias ? a.bias + at.c : nullptr, 0.f, at.width, b);
    const int Cg = a.C / a.G;
#pragma unroll
    for (int j = 0; j < VE; ++j) {
        const size_t i = (size_t)at.n * a.G + min(at.c + j, a.C - 1) / Cg;
        mean[j] = a.mean[i], rstd[j] = a.rstd[i];
        if constexpr (APPLY)
            m1[j] = means[i].x, m2[j] = means[i].y;
    }
    const IO* x = static_cast<const IO*>(a.x) + (size_t)at.n * a.S * a.xs + at.c;
    const IO* dy = static_cast<const IO*>(a.dy) + (size_t)at.n * a.S * a.C + at.c;
    IO* dx = static_cast<IO*>(a.dx) + (size_t)at.n * a.S * a.C + at.c;
    float d1[VE] = {}, d2[VE] = {};
    if (at.width)
#pragma unroll 2
        for (int s = at.s; s < at.s1; s += at.ds) {
            Raw<IO, VE> rx = load_part<WHOLE, IO, VE>(x + (size_t)s * a.xs, WHOLE ? VE : at.width, at.back);
            Raw<IO, VE> ry = load_part<WHOLE, IO, VE>(dy + (size_t)s * a.C, WHOLE ? VE : at.width, at.back);
            settle<WHOLE>(rx, at.width, at.back);
            settle<WHOLE>(ry, at.width, at.back);
            float o[VE];
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const float xh = (rx.get(j) - mean[j]) * rstd[j], d = ry.get(j);
                const float g = a.silu ? d * silu_slope(fmaf(xh, w[j], b[j])) : d;
                if constexpr (APPLY) {
                    o[j] = rstd[j] * (g * w[j] - m1[j] - xh * m2[j]);
                } else {
                    d1[j] += g;
                    d2[j] = fmaf(g, xh, d2[j]);
                }
            }
            if constexpr (APPLY)
                store_some<IO, VE>(dx + (size_t)s * a.C, o, WHOLE ? VE : at.width);
        }
    if constexpr (!APPLY) {
        float* out = ws + ((size_t)at.n * p.tiles + at.tile) * 2 * a.C + at.c;
        channel_sum<VE>(p, at.lane, d1, lds);
        channel_sum<VE>(p, at.lane, d2, lds);
        if ((int)threadIdx.x < p.lanes)
#pragma unroll
            for (int j = 0; j < VE; ++j)
                if (j < at.width) {
                    out[j] = d2[j];
                    out[a.C + j] = d1[j];
                }
    }
}

// A group's means of g w and g w xh
__global__ __launch_bounds__(256) void group_norm_means_kernel(GroupNormArgs a, Split p, const float* ws, float2* means)
{
    __shared__ float2 red[4];
    const int n = blockIdx.x / a.G, g = blockIdx.x % a.G, Cg = a.C / a.G, items = p.tiles * Cg;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < items; i += 256) {
        const int c = g * Cg + i % Cg;
        const float* from = ws + ((size_t)n * p.tiles + i / Cg) * 2 * a.C + c;
        const float w = a.weight ? a.weight[c] : 1.f;
        s1 = fmaf(w, from[a.C], s1);
        s2 = fmaf(w, from[0], s2);
    }
    const float2 m = unit_sum<256>(s1, s2, red);
    const float inv = 1.f / ((float)a.S * Cg);
    if (threadIdx.x == 0)
        means[blockIdx.x] = float2{m.x * inv, m.y * inv};
}

// samples without positions: statistics of nothing
__global__ __launch_bounds__(256) void group_norm_none_kernel(int units, float* mean, float* rstd)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= units)
        return;
    if (mean)
        mean[i] = 0.f;
    if (rstd)
        rstd[i] = 0.f;
}

// ---- which kernels --------------------------------------------------------------------

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

int power_of_two(int n)
{
    int p = 1;
    while (p < n)
        p *= 2;
    return p;
}

int common(int a, int b) { return b ? common(b, a % b) : a; }

// The fewest threads whose registers hold a unit, up to 4 vectors each (8 of 1024, forward);
// more threads where units are few.  Larger units are split.  (bf16 with SiLU, held against
// split: units of 65536 values forward, 512 of them 41 us against 48, 32 of them 15 against
// 18, one 14.5 against 17.  The backward holds two tensors, 4 vectors of each.)
//
// Groups that are not whole vectors leave threads without one: large calls are split from as
// many positions on as the sums by channel then cost less.  (320 channels, held against split:
// 512 x 256 positions, 16 groups: forward 62 us against 60, backward 155 against 87; 256 x 256
// positions, 64 groups, 101 and 168 against 48 and 63; 1024 x 64 positions 41 and 117 against 88
// and 87; of 6 MB, 32 x 256 positions of 352 channels, 12 and 19 against 18 and 24.)
Held held_shape(int N, int S, int C, int G, bool bf, bool backward)
{
    const int VE = bf ? 8 : 4, Cg = C / G;
    const long long units = (long long)N * G;
    Held h{};
    h.pad = power_of_two(ceil_div(Cg, VE));
    const long long pieces = (long long)S * h.pad;
    const bool uneven = Cg % VE && S >= (backward ? 64 : 256) && (long long)N * S * C * (bf ? 2 : 4) >= 32 << 20;
    if (h.pad > 1024 || pieces > (backward ? 4 : 8) * 1024 || uneven)
        return h;
    const int sizes[] = {8, 16, 32, 64, 256, 1024};
    int k = 0;
    auto fits = [&](int k) { return sizes[k] >= h.pad && (long long)sizes[k] * (sizes[k] == 1024 && !backward ? 8 : 4) >= pieces; };
    while (!fits(k))
        ++k;
    while (k < 5 && sizes[k] < pieces && units * sizes[k] < 64 * 1024)
        ++k;
    h.tpr = sizes[k];
    h.nv = power_of_two(ceil_div(pieces, h.tpr));
    const int threads = backward ? bwd_threads(h.tpr) : h.tpr > 256 ? h.tpr : 256, sets = threads / h.tpr;
    const int full = ceil_div(units, sets), most = backward ? 768 : 2048;
    h.grid = full;
    if (full > most) {
        // every set keeps its group: sets of a launch are a multiple of G
        const int unit = G / common(sets, G);
        if (unit <= most)
            h.grid = most / unit * unit;
    }
    h.share = 1;
    while (h.share < 8 && Cg * (bf ? 2 : 4) * h.share < 128)
        h.share *= 2;
    return h;
}

Split split_shape(int N, int S, int C, bool bf)
{
    const int VE = bf ? 8 : 4;
    Split p{};
    p.lanes = power_of_two(ceil_div(C, VE));
    p.lanes = p.lanes < 64 ? p.lanes : 64;
    p.blocks = ceil_div(C, p.lanes * VE);
    const int at_once = 256 / p.lanes;
    const long long others = (long long)N * p.blocks;
    long long tiles = others >= 1024 ? 1 : 1024 / others;
    const int most = ceil_div(S, at_once * 4);
    tiles = tiles < most ? tiles : most;
    p.rows = ceil_div(ceil_div(S, tiles), at_once) * at_once;
    p.tiles = ceil_div(S, p.rows);
    return p;
}

// calls f(threads, vectors) with the shape as constants
template <int T, int V, typename F>
bool with(const Held& h, F f)
{
    if (h.tpr != T || h.nv != V)
        return false;
    f(std::integral_constant<int, T>{}, std::integral_constant<int, V>{});
    return true;
}
template <typename F>
void with_held(const Held& h, F f)
{
    with<8, 1>(h, f) || with<8, 2>(h, f) || with<8, 4>(h, f) || with<16, 1>(h, f) || with<16, 2>(h, f) ||
        with<16, 4>(h, f) || with<32, 1>(h, f) || with<32, 2>(h, f) || with<32, 4>(h, f) || with<64, 1>(h, f) ||
        with<64, 2>(h, f) || with<64, 4>(h, f) || with<256, 1>(h, f) || with<256, 2>(h, f) || with<256, 4>(h, f) ||
        with<1024, 1>(h, f) || with<1024, 2>(h, f) || with<1024, 4>(h, f) || with<1024, 8>(h, f);
}

// calls f with whether rows of C values are whole vectors
template <typename IO, typename F>
void with_whole(int C, F f)
{
    if (C % (16 / sizeof(IO)) == 0)
        f(std::true_type{});
    else
        f(std::false_type{});
}

template <typename IO>
hipError_t group_norm_fwd(const GroupNormArgs& a, hipStream_t stream)
{
    const Held h = held_shape(a.N, a.S, a.C, a.G, sizeof(IO) == 2, false);
    const bool whole = a.C / a.G % (16 / sizeof(IO)) == 0;
    if (h.tpr) {
        with_held(h, [&](auto t, auto v) {
            constexpr int T = decltype(t)::value, V = decltype(v)::value;
            if (whole)
                group_norm_fwd_kernel<IO, T, V, true><<<h.grid, T > 256 ? T : 256, 0, stream>>>(a, h);
            else
                group_norm_fwd_kernel<IO, T, V, false><<<h.grid, T > 256 ? T : 256, 0, stream>>>(a, h);
        });
        return hipGetLastError();
    }
    const Split p = split_shape(a.N, a.S, a.C, sizeof(IO) == 2);
    const unsigned grid = (unsigned)a.N * p.tiles * p.blocks;
    float2* ws = static_cast<float2*>(a.ws);
    float2* stats = ws + (size_t)a.N * p.tiles * a.C;
    with_whole<IO>(a.C, [&](auto w) {
        constexpr bool WHOLE = decltype(w)::value;
        group_norm_stats_kernel<IO, WHOLE><<<grid, 256, 0, stream>>>(a, p, ws);
        group_norm_join_kernel<<<(unsigned)a.N * a.G, 256, 0, stream>>>(a, p, ws, stats);
        group_norm_apply_kernel<IO, WHOLE><<<grid, 256, 0, stream>>>(a, p, stats);
    });
    return hipGetLastError();
}

template <typename IO>
hipError_t group_norm_bwd(const GroupNormArgs& args, hipStream_t stream)
{
    GroupNormArgs a = args;
    const bool sums = a.dweight || a.dbias;
    const Held h = held_shape(a.N, a.S, a.C, a.G, sizeof(IO) == 2, true);
    const bool whole = a.C / a.G % (16 / sizeof(IO)) == 0;
    float* ws = static_cast<float*>(a.ws);
    int slots = 0, units = 0;
    if (h.tpr) {
        if (!sums)
            a.ws = nullptr;
        const int sets = bwd_threads(h.tpr) / h.tpr;
        slots = a.S ? slots_of(h.grid, sets, a.G) : 0;
        units = sets >= a.G ? 0 : h.grid * sets;
        if (a.N && a.S)
            with_held(h, [&](auto t, auto v) {
                constexpr int T = decltype(t)::value, V = decltype(v)::value;
                if constexpr (V <= 4) {
                    if (whole)
                        group_norm_bwd_kernel<IO, T, V, true><<<h.grid, bwd_threads(T), 0, stream>>>(a, h);
                    else
                        group_norm_bwd_kernel<IO, T, V, false><<<h.grid, bwd_threads(T), 0, stream>>>(a, h);
                }
            });
    } else if (a.N && a.S) {
        const Split p = split_shape(a.N, a.S, a.C, sizeof(IO) == 2);
        const unsigned grid = (unsigned)a.N * p.tiles * p.blocks;
        float2* means = reinterpret_cast<float2*>(ws + (size_t)a.N * p.tiles * 2 * a.C);
        with_whole<IO>(a.C, [&](auto w) {
            constexpr bool WHOLE = decltype(w)::value;
            group_norm_bwd_split_kernel<IO, false, WHOLE><<<grid, 256, 0, stream>>>(a, p, ws, nullptr);
            group_norm_means_kernel<<<(unsigned)a.N * a.G, 256, 0, stream>>>(a, p, ws, means);
            group_norm_bwd_split_kernel<IO, true, WHOLE><<<grid, 256, 0, stream>>>(a, p, ws, means);
        });
        slots = a.N * p.tiles;
    }
    if (sums)
        group_norm_sum_kernel<<<(2 * a.C + 63) / 64, 1024, 0, stream>>>(a, ws, slots, units);
    return hipGetLastError();
}

size_t split_bytes(int N, int S, int C, int G, bool bf)
{
    const Split p = split_shape(N, S, C, bf);
    return ((size_t)N * p.tiles * C + (size_t)N * G) * sizeof(float2);
}

}  // namespace

// the larger of the two types' numbers, so that one workspace fits both
size_t group_norm_fwd_workspace_bytes(int N, int S, int C, int G)
{
    size_t most = 0;
    for (const bool bf : {false, true})
        if (N && S && !held_shape(N, S, C, G, bf, false).tpr) {
            const size_t n = split_bytes(N, S, C, G, bf);
            most = most > n ? most : n;
        }
    return most;
}

size_t group_norm_bwd_workspace_bytes(int N, int S, int C, int G)
{
    size_t most = 0;
    for (const bool bf : {false, true}) {
        if (!N || !S)
            continue;
        const Held h = held_shape(N, S, C, G, bf, true);
        const size_t n = h.tpr ? (size_t)slots_of(h.grid, bwd_threads(h.tpr) / h.tpr, G) * 2 * C * sizeof(float)
                               : split_bytes(N, S, C, G, bf);
        most = most > n ? most : n;
    }
    return most;
}

hipError_t launch_group_norm_fwd(const GroupNormArgs& a, bool bf, hipStream_t stream)
{
    if (a.N == 0)
        return hipSuccess;
    if (a.S == 0) {
        if (a.mean || a.rstd)
            group_norm_none_kernel<<<(unsigned)ceil_div((long long)a.N * a.G, 256), 256, 0, stream>>>(a.N * a.G, a.mean, a.rstd);
        return hipGetLastError();
    }
    return bf ? group_norm_fwd<bf16>(a, stream) : group_norm_fwd<float>(a, stream);
}

hipError_t launch_group_norm_bwd(const GroupNormArgs& a, bool bf, hipStream_t stream)
{
    return bf ? group_norm_bwd<bf16>(a, stream) : group_norm_bwd<float>(a, stream);
}

}  // namespace kdn
