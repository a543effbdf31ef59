// kdn_norm.hip -- layer norm over rows, forward and backward, gfx950.
#include "kdn_block_device.h"

namespace kdn {

namespace {

// Sum of v over the 256 threads of a workgroup, in every thread.
__device__ __forceinline__ float block_sum(float v, float* red)
{
#pragma unroll
    for (int o = 32; o; o >>= 1)
        v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

template <typename IO>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs a)
{
    __shared__ float red[4];
    const IO* x = static_cast<const IO*>(a.x) + (size_t)blockIdx.x * a.xs;
    IO* y = static_cast<IO*>(a.y) + (size_t)blockIdx.x * a.D;
    float s = 0.f;
    for (int i = threadIdx.x; i < a.D; i += 256)
        s += to_f32(x[i]);
    const float mean = block_sum(s, red) / a.D;
    s = 0.f;
    for (int i = threadIdx.x; i < a.D; i += 256) {
        const float d = to_f32(x[i]) - mean;
        s += d * d;
    }
    const float rstd = 1.f / sqrtf(block_sum(s, red) / a.D + a.eps);
    for (int i = threadIdx.x; i < a.D; i += 256) {
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
__global__ __launch_bounds__(256) void norm_bwd_dx_kernel(NormArgs a)
{
    __shared__ float red[4];
    const IO* x = static_cast<const IO*>(a.x) + (size_t)blockIdx.x * a.xs;
    const IO* dy = static_cast<const IO*>(a.dy) + (size_t)blockIdx.x * a.D;
    IO* dx = static_cast<IO*>(a.dx) + (size_t)blockIdx.x * a.D;
    const float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
    float s1 = 0.f, s2 = 0.f;
    for (int i = threadIdx.x; i < a.D; i += 256) {
        const float g = to_f32(dy[i]) * (a.weight ? a.weight[i] : 1.f);
        s1 += g;
        s2 += g * ((to_f32(x[i]) - mean) * rstd);
    }
    s1 = block_sum(s1, red) / a.D;
    s2 = block_sum(s2, red) / a.D;
    for (int i = threadIdx.x; i < a.D; i += 256) {
        const float g = to_f32(dy[i]) * (a.weight ? a.weight[i] : 1.f);
        const float xh = (to_f32(x[i]) - mean) * rstd;
        dx[i] = from_f32<IO>(rstd * (g - s1 - xh * s2));
    }
}

// partial sums of the parameter gradients over one group of rows
template <typename IO>
__global__ __launch_bounds__(256) void norm_bwd_param_kernel(NormArgs a)
{
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.D)
        return;
    float dw = 0.f, db = 0.f;
    for (int r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float dy = to_f32(static_cast<const IO*>(a.dy)[(size_t)r * a.D + c]);
        const float x = to_f32(static_cast<const IO*>(a.x)[(size_t)r * a.xs + c]);
        dw += dy * ((x - a.mean[r]) * a.rstd[r]);
        db += dy;
    }
    a.ws[((size_t)blockIdx.y * 2) * a.D + c] = dw;
    a.ws[((size_t)blockIdx.y * 2 + 1) * a.D + c] = db;
}

__global__ __launch_bounds__(256) void norm_bwd_sum_kernel(NormArgs a, int groups)
{
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.D)
        return;
    float dw = 0.f, db = 0.f;
    for (int g = 0; g < groups; ++g) {
        dw += a.ws[((size_t)g * 2) * a.D + c];
        db += a.ws[((size_t)g * 2 + 1) * a.D + c];
    }
    if (a.dweight)
        a.dweight[c] = dw;
    if (a.dbias)
        a.dbias[c] = db;
}

}  // namespace

int norm_bwd_groups(int rows, int D) { return rows < 1 ? 0 : rows < 512 ? rows : 512; }

hipError_t launch_norm_fwd(const NormArgs& a, bool bf, hipStream_t stream)
{
    if (a.rows == 0)
        return hipSuccess;
    if (bf)
        norm_fwd_kernel<bf16><<<a.rows, 256, 0, stream>>>(a);
    else
        norm_fwd_kernel<float><<<a.rows, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs& a, bool bf, hipStream_t stream)
{
    const int groups = norm_bwd_groups(a.rows, a.D);
    const dim3 cols((a.D + 255) / 256, groups);
    if (a.rows) {
        if (bf)
            norm_bwd_dx_kernel<bf16><<<a.rows, 256, 0, stream>>>(a);
        else
            norm_bwd_dx_kernel<float><<<a.rows, 256, 0, stream>>>(a);
    }
    if (a.dweight || a.dbias) {
        if (a.rows) {
            if (bf)
                norm_bwd_param_kernel<bf16><<<cols, 256, 0, stream>>>(a);
            else
                norm_bwd_param_kernel<float><<<cols, 256, 0, stream>>>(a);
        }
        norm_bwd_sum_kernel<<<cols.x, 256, 0, stream>>>(a, groups);
    }
    return hipGetLastError();
}

}  // namespace kdn
