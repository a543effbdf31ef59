// kdn_conv.hip -- short causal convolution per channel, forward, backward and
// single-token step, gfx950.
#include "kdn_block_device.h"

namespace kdn {

namespace {

// x of the token j before token t of row b, whose sequence is s: from the
// sequence's state where that is before its first token
template <typename IO>
__device__ __forceinline__ float tap(const ConvArgs& a, Span s, int b, int t, int j, int c)
{
    if (t - j >= s.p)
        return to_f32(static_cast<const IO*>(a.x)[((size_t)b * a.T + t - j) * a.xs + c]);
    const int i = a.W - 1 + t - j - s.p;  // row of the state
    return a.state0 ? to_f32(static_cast<const IO*>(a.state0)[((size_t)s.n * (a.W - 1) + i) * a.D + c])
                    : 0.f;
}

template <typename IO>
__device__ __forceinline__ float conv_z(const ConvArgs& a, Span s, int b, int t, int c)
{
    float z = a.bias ? a.bias[c] : 0.f;
    for (int j = 0; j < a.W; ++j)
        z = fmaf(a.weight[(size_t)(a.W - 1 - j) * a.D + c], tap<IO>(a, s, b, t, j, c), z);
    return z;
}

template <typename IO>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a)
{
    const int c = blockIdx.y * 256 + threadIdx.x;
    const int b = blockIdx.x / a.T, t = blockIdx.x - b * a.T;
    if (c >= a.D)
        return;
    const Span s = span_of(a.cu, a.N, b, t, a.T);
    if (s.n < 0)
        return;
    const float z = conv_z<IO>(a, s, b, t, c);
    static_cast<IO*>(a.y)[((size_t)b * a.T + t) * a.D + c] =
        from_f32<IO>(a.silu ? z * gate_sigmoid(z) : z);
}

// Row i of a sequence's state after its last token is the token W-1-i before
// its end.
template <typename IO>
__global__ __launch_bounds__(256) void conv_state_kernel(ConvArgs a)
{
    const int c = blockIdx.y * 256 + threadIdx.x;
    const int n = blockIdx.x / (a.W - 1), i = blockIdx.x - n * (a.W - 1);
    if (c >= a.D)
        return;
    Span s{n, a.cu ? a.cu[n] : 0, a.cu ? a.cu[n + 1] : a.T};
    if (s.p < 0 || s.q > a.T || s.q < s.p)
        return;
    static_cast<IO*>(a.state_T)[(size_t)blockIdx.x * a.D + c] =
        from_f32<IO>(tap<IO>(a, s, a.cu ? 0 : n, s.q, a.W - 1 - i, c));
}

// g_t = dy_t act'(z_t)
template <typename IO>
__device__ __forceinline__ float conv_g(const ConvArgs& a, Span s, int b, int t, int c)
{
    const float dy = to_f32(static_cast<const IO*>(a.dy)[((size_t)b * a.T + t) * a.D + c]);
    if (!a.silu)
        return dy;
    const float z = conv_z<IO>(a, s, b, t, c), p = gate_sigmoid(z);
    return dy * (p * (1.f + z * (1.f - p)));
}

// gradient by the input at place t of the sequence (t < s.p: its state)
template <typename IO>
__device__ __forceinline__ float conv_dx(const ConvArgs& a, Span s, int b, int t, int c)
{
    float d = 0.f;
    for (int j = 0; j < a.W; ++j)
        if (t + j >= s.p && t + j < s.q)
            d = fmaf(a.weight[(size_t)(a.W - 1 - j) * a.D + c], conv_g<IO>(a, s, b, t + j, c), d);
    const int i = t - (s.q - (a.W - 1));
    if (i >= 0 && a.dstate_T)
        d += to_f32(static_cast<const IO*>(a.dstate_T)[((size_t)s.n * (a.W - 1) + i) * a.D + c]);
    return d;
}

template <typename IO>
__global__ __launch_bounds__(256) void conv_bwd_dx_kernel(ConvArgs a)
{
    const int c = blockIdx.y * 256 + threadIdx.x;
    const int b = blockIdx.x / a.T, t = blockIdx.x - b * a.T;
    if (c >= a.D)
        return;
    const Span s = span_of(a.cu, a.N, b, t, a.T);
    if (s.n >= 0)
        static_cast<IO*>(a.dx)[((size_t)b * a.T + t) * a.D + c] =
            from_f32<IO>(conv_dx<IO>(a, s, b, t, c));
}

template <typename IO>
__global__ __launch_bounds__(256) void conv_bwd_state_kernel(ConvArgs a)
{
    const int c = blockIdx.y * 256 + threadIdx.x;
    const int n = blockIdx.x / (a.W - 1), i = blockIdx.x - n * (a.W - 1);
    if (c >= a.D)
        return;
    Span s{n, a.cu ? a.cu[n] : 0, a.cu ? a.cu[n + 1] : a.T};
    if (s.p < 0 || s.q > a.T || s.q < s.p)
        return;
    static_cast<IO*>(a.dstate0)[(size_t)blockIdx.x * a.D + c] =
        from_f32<IO>(conv_dx<IO>(a, s, a.cu ? 0 : n, s.p - (a.W - 1) + i, c));
}

template <typename IO>
__global__ __launch_bounds__(256) void conv_bwd_param_kernel(ConvArgs a)
{
    const int c = blockIdx.y * 256 + threadIdx.x;
    if (c >= a.D)
        return;
    float dw[4] = {0.f, 0.f, 0.f, 0.f}, db = 0.f;
    for (int r = blockIdx.x; r < a.B * a.T; r += gridDim.x) {
        const int b = r / a.T, t = r - b * a.T;
        const Span s = span_of(a.cu, a.N, b, t, a.T);
        if (s.n < 0)
            continue;
        const float g = conv_g<IO>(a, s, b, t, c);
        db += g;
        for (int j = 0; j < a.W; ++j)
            dw[a.W - 1 - j] += g * tap<IO>(a, s, b, t, j, c);
    }
    for (int j = 0; j < a.W; ++j)
        a.ws[((size_t)blockIdx.x * (a.W + 1) + j) * a.D + c] = dw[j];
    a.ws[((size_t)blockIdx.x * (a.W + 1) + a.W) * a.D + c] = db;
}

__global__ __launch_bounds__(256) void conv_bwd_sum_kernel(ConvArgs a, int groups)
{
    const int c = blockIdx.y * 256 + threadIdx.x, j = blockIdx.x;
    if (c >= a.D)
        return;
    float s = 0.f;
    for (int g = 0; g < groups; ++g)
        s += a.ws[((size_t)g * (a.W + 1) + j) * a.D + c];
    if (j < a.W)
        a.dweight[(size_t)j * a.D + c] = s;
    else if (a.dbias)
        a.dbias[c] = s;
}

template <typename IO>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a)
{
    const int c = blockIdx.y * 256 + threadIdx.x, b = blockIdx.x, W = a.W;
    if (c >= a.D)
        return;
    IO* st = static_cast<IO*>(a.state_T) + (size_t)b * (W - 1) * a.D + c;
    float z = a.bias ? a.bias[c] : 0.f;
    IO next = static_cast<const IO*>(a.x)[(size_t)b * a.xs + c];
    z = fmaf(a.weight[(size_t)(W - 1) * a.D + c], to_f32(next), z);
    for (int i = W - 2; i >= 0; --i) {
        const IO old = st[(size_t)i * a.D];
        z = fmaf(a.weight[(size_t)i * a.D + c], to_f32(old), z);
        st[(size_t)i * a.D] = next;
        next = old;
    }
    static_cast<IO*>(a.y)[(size_t)b * a.D + c] = from_f32<IO>(a.silu ? z * gate_sigmoid(z) : z);
}

}  // namespace

int conv_bwd_groups(int B, int T, int D)
{
    const long long rows = (long long)B * T;
    return rows < 512 ? (int)rows : 512;
}

template <typename IO>
static hipError_t conv_fwd(const ConvArgs& a, hipStream_t stream)
{
    const unsigned cols = (a.D + 255) / 256;
    if (a.T)
        conv_fwd_kernel<IO><<<dim3((unsigned)(a.B * a.T), cols), 256, 0, stream>>>(a);
    if (a.state_T)
        conv_state_kernel<IO><<<dim3((unsigned)(a.N * (a.W - 1)), cols), 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename IO>
static hipError_t conv_bwd(const ConvArgs& a, hipStream_t stream)
{
    const unsigned cols = (a.D + 255) / 256;
    const int groups = conv_bwd_groups(a.B, a.T, a.D);
    if (a.T) {
        conv_bwd_dx_kernel<IO><<<dim3((unsigned)(a.B * a.T), cols), 256, 0, stream>>>(a);
        conv_bwd_param_kernel<IO><<<dim3(groups, cols), 256, 0, stream>>>(a);
    }
    if (a.dstate0)
        conv_bwd_state_kernel<IO><<<dim3((unsigned)(a.N * (a.W - 1)), cols), 256, 0, stream>>>(a);
    conv_bwd_sum_kernel<<<dim3(a.W + 1, cols), 256, 0, stream>>>(a, groups);
    return hipGetLastError();
}

hipError_t launch_conv_fwd(const ConvArgs& a, bool bf, hipStream_t stream)
{
    return bf ? conv_fwd<bf16>(a, stream) : conv_fwd<float>(a, stream);
}

hipError_t launch_conv_bwd(const ConvArgs& a, bool bf, hipStream_t stream)
{
    return bf ? conv_bwd<bf16>(a, stream) : conv_bwd<float>(a, stream);
}

hipError_t launch_conv_step(const ConvArgs& a, bool bf, hipStream_t stream)
{
    const dim3 grid(a.B, (a.D + 255) / 256);
    if (bf)
        conv_step_kernel<bf16><<<grid, 256, 0, stream>>>(a);
    else
        conv_step_kernel<float><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace kdn
