// kdn_norm.hip -- layer norm over rows, forward and backward, gfx950.
//
//   y = (x - mean) rstd w + b
//   dx = rstd (g - mean(g) - xh mean(g xh)),  g = dy w,  xh = (x - mean) rstd
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Both are bound by HBM.  A row is held in the registers of TPR threads, NV
// vectors of 16 bytes each, from one load to the store: x is read once, and the
// variance is taken around the mean without a second read.  A workgroup walks
// many rows, with w and b (in the backward w and the sums dw and db of the
// thread's columns) in registers all along.  The backward's sums are joined over
// the workgroup at the end and written once a workgroup; a second launch adds
// those, always in the same order.
//
// Measured (kernel time; bytes of inputs and outputs): forward 524288 x 128 bf16 49 us
// (5.5 TB/s), 32768 x 2048 46 us (5.8 TB/s), 4099 x 1537 fp32 11 us (4.6 TB/s); backward
// 32768 x 2048 bf16 79 us (5.1 TB/s) and 5 us for the sums, 4099 x 1537 fp32 16 and 4 us.
// Few wide rows are further off: backward 1024 x 16384 bf16 30 and 6 us (2.8 TB/s), 256 x
// 16384 18 and 6 us, where the partial sums of up to 256 workgroups outweigh the rows.
#include "kdn_block.h"
#include "kdn_common.h"
#include "kdn_lanes.h"

namespace kdn {

namespace {

// The sums of two values over the TPR threads of a row, in all of them; `red`
// holds two slots for each wave of the workgroup.
template <int TPR>
__device__ __forceinline__ float2 row_sum(float a, float b, float2* red)
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

// VE adjacent values as they are in memory, at any alignment of an element
template <typename E, int VE>
struct __attribute__((packed, aligned(sizeof(E)))) Vec {
    E v[VE];
};

// A thread's part of a row of D: NV vectors, TPR vectors apart; n[v] values of
// vector v lie in the row (all VE, a few at the row's end, or none).
template <typename IO, int TPR, int NV>
struct Part {
    static constexpr int VE = 16 / sizeof(IO);
    int col[NV], n[NV];

    __device__ __forceinline__ Part(int D)
    {
        const int l = threadIdx.x % TPR;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            col[v] = (v * TPR + l) * VE;
            n[v] = min(max(D - col[v], 0), VE);
        }
    }

    template <typename E>
    __device__ __forceinline__ void load(const E* row, Vec<E, VE> (&x)[NV]) const
    {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (n[v] == VE) {
                x[v] = *reinterpret_cast<const Vec<E, VE>*>(row + col[v]);
            } else {
#pragma unroll
                for (int j = 0; j < VE; ++j)
                    x[v].v[j] = j < n[v] ? row[col[v] + j] : E(0.f);
            }
        }
    }

    template <typename E>
    __device__ __forceinline__ void store(E* row, int v, const float (&y)[VE]) const
    {
        if (n[v] == VE) {
            Vec<E, VE> p;
#pragma unroll
            for (int j = 0; j < VE; ++j)
                p.v[j] = from_f32<E>(y[j]);
            *reinterpret_cast<Vec<E, VE>*>(row + col[v]) = p;
        } else {
#pragma unroll
            for (int j = 0; j < VE; ++j)
                if (j < n[v])
                    row[col[v] + j] = from_f32<E>(y[j]);
        }
    }

    // a parameter [D], or `other` where it is not given
    __device__ __forceinline__ void param(const float* p, float other, float (&w)[NV][VE]) const
    {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < VE; ++j)
                w[v][j] = other;
        if (!p)
            return;
        Vec<float, VE> x[NV];
        load(p, x);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < VE; ++j)
                w[v][j] = x[v].v[j];
    }
};

// row of this thread in the workgroup's first set of rows; one for a whole wave
// where TPR fills it
template <int TPR>
__device__ __forceinline__ int row_of_thread()
{
    const int r = threadIdx.x / TPR;
    return TPR >= 64 ? __builtin_amdgcn_readfirstlane(r) : r;
}

template <typename IO, int TPR, int NV>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_fwd_kernel(NormArgs a)
{
    typedef Part<IO, TPR, NV> P;
    constexpr int VE = P::VE;
    __shared__ float2 red[TPR > 64 ? TPR / 64 : 1];
    const P part(a.D);
    const int per = blockDim.x / TPR, step = gridDim.x * per;
    const float n = a.D;  // divided by, not multiplied with 1 / n: the mean of equal values is that value
    float w[NV][VE], b[NV][VE];
    part.param(a.weight, 1.f, w);
    part.param(a.bias, 0.f, b);

    const IO* x = static_cast<const IO*>(a.x);
    int row = blockIdx.x * per + row_of_thread<TPR>();
    Vec<IO, VE> raw[NV];
    part.load(x + (size_t)min(row, a.rows - 1) * a.xs, raw);
    // every thread walks the same number of rows: rows behind the last repeat it
    for (int r0 = blockIdx.x * per; r0 < a.rows; r0 += step, row += step) {
        float d[NV][VE];
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                d[v][j] = to_f32(raw[v].v[j]);
                s += d[v][j];
            }
        if (r0 + step < a.rows)
            part.load(x + (size_t)min(row + step, a.rows - 1) * a.xs, raw);
        const float mean = row_sum<TPR>(s, 0.f, red).x / n;
        s = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                d[v][j] -= mean;
                if (j < part.n[v])
                    s = fmaf(d[v][j], d[v][j], s);
            }
        const float rstd = 1.f / sqrtf(row_sum<TPR>(s, 0.f, red).x / n + a.eps);
        if (row < a.rows) {
            IO* y = static_cast<IO*>(a.y) + (size_t)row * a.D;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float o[VE];
#pragma unroll
                for (int j = 0; j < VE; ++j)
                    o[j] = fmaf(d[v][j] * rstd, w[v][j], b[v][j]);
                part.store(y, v, o);
            }
            if (threadIdx.x % TPR == 0) {
                if (a.mean)
                    a.mean[row] = mean;
                if (a.rstd)
                    a.rstd[row] = rstd;
            }
        }
    }
}

// 1024 threads whatever a row takes: the sums of its columns are written once a
// workgroup, and few values a thread leave the registers for eight waves a SIMD,
// which cover the loads better than loading a row ahead does with fewer (32768 rows
// of 2048 bf16: 84 us; a wave a row with the next one loaded ahead 127 us, 256
// threads a workgroup 91 us, with four times the sums to write).
constexpr int kBwdThreads = 1024;

template <typename IO, int TPR, int NV>
__global__ __launch_bounds__(kBwdThreads) void norm_bwd_kernel(NormArgs a)
{
    typedef Part<IO, TPR, NV> P;
    constexpr int VE = P::VE, THREADS = kBwdThreads, WAVES = THREADS / 64;
    __shared__ float2 red[WAVES];
    const P part(a.D);
    const int per = THREADS / TPR, step = gridDim.x * per;
    const float inv = 1.f / a.D;
    float w[NV][VE], dw[NV][VE], db[NV][VE];
    part.param(a.weight, 1.f, w);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VE; ++j)
            dw[v][j] = db[v][j] = 0.f;

    const IO* x = static_cast<const IO*>(a.x);
    const IO* dy = static_cast<const IO*>(a.dy);
    int row = blockIdx.x * per + row_of_thread<TPR>();
    for (int r0 = blockIdx.x * per; r0 < a.rows; r0 += step, row += step) {
        const int at = min(row, a.rows - 1);
        Vec<IO, VE> rx[NV], ry[NV];
        part.load(x + (size_t)at * a.xs, rx);
        part.load(dy + (size_t)at * a.D, ry);
        const float mean = a.mean[at], rstd = a.rstd[at];
        const bool mine = row < a.rows;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const float xh = (to_f32(rx[v].v[j]) - mean) * rstd, d = to_f32(ry[v].v[j]);
                if (j >= part.n[v])
                    continue;
                const float g = d * w[v][j];
                s1 += g;
                s2 = fmaf(g, xh, s2);
                if (mine) {
                    dw[v][j] = fmaf(d, xh, dw[v][j]);
                    db[v][j] += d;
                }
            }
        const float2 m = row_sum<TPR>(s1, s2, red);
        const float m1 = m.x * inv, m2 = m.y * inv;
        if (mine) {
            IO* dx = static_cast<IO*>(a.dx) + (size_t)row * a.D;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float o[VE];
#pragma unroll
                for (int j = 0; j < VE; ++j) {
                    const float xh = (to_f32(rx[v].v[j]) - mean) * rstd;
                    o[j] = rstd * (to_f32(ry[v].v[j]) * w[v][j] - m1 - xh * m2);
                }
                part.store(dx, v, o);
            }
        }
    }

    if (!a.ws)
        return;
    // the workgroup's rows: lanes of one column within a wave, then the sets of
    // threads that hold all columns
    constexpr int SETS = TPR < 64 ? WAVES : THREADS / TPR;
    __shared__ float sums[SETS > 1 ? SETS : 1][SETS > 1 ? TPR * VE : 1];
    const int l = threadIdx.x % TPR, set = TPR < 64 ? threadIdx.x >> 6 : threadIdx.x / TPR;
    const bool first = TPR >= 64 || (threadIdx.x & 63) < TPR;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float* out = a.ws + ((size_t)blockIdx.x * 2 + k) * a.D;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float s[VE];
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                s[j] = k ? db[v][j] : dw[v][j];
#pragma unroll
                for (int o = TPR; o < 64; o *= 2)
                    s[j] += __shfl_xor(s[j], o);
            }
            if constexpr (SETS > 1) {
                __syncthreads();
                if (first) {
#pragma unroll
                    for (int j = 0; j < VE; ++j)
                        sums[set][l * VE + j] = s[j];
                }
                __syncthreads();
                for (int i = threadIdx.x; i < TPR * VE; i += THREADS) {
                    const int c = v * TPR * VE + i;
                    if (c < a.D) {
                        float t = 0.f;
#pragma unroll
                        for (int q = 0; q < SETS; ++q)
                            t += sums[q][i];
                        out[c] = t;
                    }
                }
            } else {
                part.store(out, v, s);
            }
        }
    }
}

// Adds the partial sums [groups][2 D]: 64 columns a workgroup, 16 shares of the
// groups each, joined in order.
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormArgs a, int groups)
{
    __shared__ float share[16][64];
    const int l = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + l, n = 2 * a.D;
    float s = 0.f;
    if (c < n) {
#pragma unroll 8
        for (int g = q; g < groups; g += 16)
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
    float* out = c < a.D ? a.dweight : a.dbias;
    if (out)
        out[c < a.D ? c : c - a.D] = s;
}

// ---- rows too wide for registers: walked three times, from L2 --------------------
// A value a load: 512 x 32768 bf16 forward 32 us (2.1 TB/s of inputs and outputs), backward
// 32 us and 17 + 5 us for the sums; fp32 51 us (2.6 TB/s), 60 and 21 + 5 us.

__device__ __forceinline__ float wide_sum(float v, float2* red) { return row_sum<1024>(v, 0.f, red).x; }

template <typename IO>
__global__ __launch_bounds__(1024) void norm_fwd_wide_kernel(NormArgs a)
{
    __shared__ float2 red[16];
    const IO* x = static_cast<const IO*>(a.x) + (size_t)blockIdx.x * a.xs;
    IO* y = static_cast<IO*>(a.y) + (size_t)blockIdx.x * a.D;
    float s = 0.f;
    for (int i = threadIdx.x; i < a.D; i += 1024)
        s += to_f32(x[i]);
    const float mean = wide_sum(s, red) / a.D;
    s = 0.f;
    for (int i = threadIdx.x; i < a.D; i += 1024) {
        const float d = to_f32(x[i]) - mean;
        s = fmaf(d, d, s);
    }
    const float rstd = 1.f / sqrtf(wide_sum(s, red) / a.D + a.eps);
    for (int i = threadIdx.x; i < a.D; i += 1024) {
        const float xh = (to_f32(x[i]) - mean) * rstd;
        y[i] = from_f32<IO>(xh * (a.weight ? a.weight[i] : 1.f) + (a.bias ? a.bias[i] : 0.f));
    }
    if (threadIdx.x == 0) {
        if (a.mean)
            a.mean[blockIdx.x] = mean;
        if (a.rstd)
            a.rstd[blockIdx.x] = rstd;
    }
}

template <typename IO>
__global__ __launch_bounds__(1024) void norm_bwd_wide_kernel(NormArgs a)
{
    __shared__ float2 red[16];
    const IO* x = static_cast<const IO*>(a.x) + (size_t)blockIdx.x * a.xs;
    const IO* dy = static_cast<const IO*>(a.dy) + (size_t)blockIdx.x * a.D;
    IO* dx = static_cast<IO*>(a.dx) + (size_t)blockIdx.x * a.D;
    const float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
    float s1 = 0.f, s2 = 0.f;
    for (int i = threadIdx.x; i < a.D; i += 1024) {
        const float g = to_f32(dy[i]) * (a.weight ? a.weight[i] : 1.f);
        s1 += g;
        s2 = fmaf(g, (to_f32(x[i]) - mean) * rstd, s2);
    }
    const float2 m = row_sum<1024>(s1, s2, red);
    s1 = m.x / a.D;
    s2 = m.y / a.D;
    for (int i = threadIdx.x; i < a.D; i += 1024) {
        const float g = to_f32(dy[i]) * (a.weight ? a.weight[i] : 1.f);
        const float xh = (to_f32(x[i]) - mean) * rstd;
        dx[i] = from_f32<IO>(rstd * (g - s1 - xh * s2));
    }
}

// the wide rows' sums: one thread a column, over every gridDim.x-th row
template <typename IO>
__global__ __launch_bounds__(256) void norm_bwd_wide_sums_kernel(NormArgs a)
{
    const int c = blockIdx.y * 256 + threadIdx.x;
    if (c >= a.D)
        return;
    float dw = 0.f, db = 0.f;
    for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float dy = to_f32(static_cast<const IO*>(a.dy)[(size_t)r * a.D + c]);
        const float x = to_f32(static_cast<const IO*>(a.x)[(size_t)r * a.xs + c]);
        dw = fmaf(dy, (x - a.mean[r]) * a.rstd[r], dw);
        db += dy;
    }
    a.ws[((size_t)blockIdx.x * 2) * a.D + c] = dw;
    a.ws[((size_t)blockIdx.x * 2 + 1) * a.D + c] = db;
}

// ---- which kernel -------------------------------------------------------------------

// Threads and vectors for a row of `vecs` vectors of 16 bytes: the fewest threads
// whose registers hold it (a wave or less needs no barrier to add a row up).
struct Shape {
    int tpr, nv;  // tpr 0: too wide
};
Shape fwd_shape(int D, bool bf)
{
    const int vecs = (D + (bf ? 7 : 3)) / (bf ? 8 : 4);
    if (vecs <= 64)
        return {vecs <= 8 ? 8 : vecs <= 16 ? 16 : vecs <= 32 ? 32 : 64, 1};
    if (vecs <= 256)
        return {64, vecs <= 128 ? 2 : 4};
    if (vecs <= 1024)
        return {256, vecs <= 512 ? 2 : 4};
    if (vecs <= 2048)
        return {1024, 2};
    // room for 16 values a thread, not for 32
    if (vecs <= 4096 && !bf)
        return {1024, 4};
    return {0, 0};
}

// The backward holds x, dy, w and two sums: as many threads as the row has vectors,
// and two or four each only where 1024 threads do not suffice.
Shape bwd_shape(int D, bool bf)
{
    const int vecs = (D + (bf ? 7 : 3)) / (bf ? 8 : 4);
    if (vecs > 512)
        return vecs <= 1024 ? Shape{512, 2} : fwd_shape(D, bf);
    int t = 8;
    while (t < vecs)
        t *= 2;
    return {t, 1};
}

// calls f(threads, vectors) with the shape as constants, if it is that one
template <int T, int N, typename F>
bool with_shape(Shape s, F f)
{
    if (s.tpr != T || s.nv != N)
        return false;
    f(std::integral_constant<int, T>{}, std::integral_constant<int, N>{});
    return true;
}

template <typename IO>
hipError_t norm_fwd(const NormArgs& a, hipStream_t stream)
{
    const Shape s = fwd_shape(a.D, sizeof(IO) == 2);
    if (!s.tpr) {
        norm_fwd_wide_kernel<IO><<<a.rows, 1024, 0, stream>>>(a);
        return hipGetLastError();
    }
    // few rows: one wave a workgroup, so that they spread over the chip (256 x 2048
    // bf16 3.6 us, four waves 4.8)
    const bool few = s.tpr <= 64 && (long long)a.rows * s.tpr <= 64 * 1024;
    const int threads = s.tpr > 256 ? s.tpr : few ? 64 : 256;
    const int per = threads / s.tpr, groups = (a.rows + per - 1) / per;
    // more rows a workgroup than that loads w and b less often, but 1024 leaves loads
    // unasked for (524288 x 128 bf16 1024, 2048, 4096: 64, 51, 53 us; 32768 x 2048 49,
    // 48, 46 us)
    const int grid = groups < 2048 ? groups : 2048;
    auto run = [&](auto t, auto n) {
        norm_fwd_kernel<IO, decltype(t)::value, decltype(n)::value><<<grid, threads, 0, stream>>>(a);
    };
    with_shape<8, 1>(s, run) || with_shape<16, 1>(s, run) || with_shape<32, 1>(s, run) ||
        with_shape<64, 1>(s, run) || with_shape<64, 2>(s, run) || with_shape<64, 4>(s, run) ||
        with_shape<256, 2>(s, run) || with_shape<256, 4>(s, run) || with_shape<1024, 2>(s, run);
    if constexpr (sizeof(IO) == 4)
        with_shape<1024, 4>(s, run);
    return hipGetLastError();
}

// workgroups of the backward (and partial sums): two a compute unit, or the one
// that fits with several vectors a thread; for rows too wide for registers, so few
// that the partial sums stay small beside the rows
int bwd_groups(int rows, Shape s)
{
    const int per = s.tpr ? kBwdThreads / s.tpr : 16;
    const int groups = (rows - 1) / per + 1, most = s.nv == 1 ? 512 : 256;  // (0 for no rows)
    return rows < 1 ? 0 : groups < most ? groups : most;
}

template <typename IO>
hipError_t norm_bwd(const NormArgs& args, hipStream_t stream)
{
    NormArgs a = args;
    const Shape s = bwd_shape(a.D, sizeof(IO) == 2);
    const int groups = bwd_groups(a.rows, s);
    const bool sums = a.dweight || a.dbias;
    if (!sums)
        a.ws = nullptr;
    if (a.rows && !s.tpr) {
        norm_bwd_wide_kernel<IO><<<a.rows, 1024, 0, stream>>>(a);
        if (sums)
            norm_bwd_wide_sums_kernel<IO><<<dim3(groups, (a.D + 255) / 256), 256, 0, stream>>>(a);
    } else if (a.rows) {
        auto run = [&](auto t, auto n) {
            norm_bwd_kernel<IO, decltype(t)::value, decltype(n)::value><<<groups, kBwdThreads, 0, stream>>>(a);
        };
        with_shape<8, 1>(s, run) || with_shape<16, 1>(s, run) || with_shape<32, 1>(s, run) ||
            with_shape<64, 1>(s, run) || with_shape<128, 1>(s, run) || with_shape<256, 1>(s, run) ||
            with_shape<512, 1>(s, run) || with_shape<512, 2>(s, run) || with_shape<1024, 2>(s, run);
        if constexpr (sizeof(IO) == 4)
            with_shape<1024, 4>(s, run);
    }
    if (sums)
        norm_sum_kernel<<<(2 * a.D + 63) / 64, 1024, 0, stream>>>(a, groups);
    return hipGetLastError();
}

}  // namespace

int norm_bwd_groups(int rows, int D)
{
    // the larger of the two types' numbers, so that one workspace fits both
    const int f = bwd_groups(rows, bwd_shape(D, false)), h = bwd_groups(rows, bwd_shape(D, true));
    return f > h ? f : h;
}

hipError_t launch_norm_fwd(const NormArgs& a, bool bf, hipStream_t stream)
{
    if (a.rows == 0)
        return hipSuccess;
    return bf ? norm_fwd<bf16>(a, stream) : norm_fwd<float>(a, stream);
}

hipError_t launch_norm_bwd(const NormArgs& a, bool bf, hipStream_t stream)
{
    return bf ? norm_bwd<bf16>(a, stream) : norm_bwd<float>(a, stream);
}

}  // namespace kdn
