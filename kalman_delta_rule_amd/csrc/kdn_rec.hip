// kdn_rec.hip -- gated recurrence per channel, forward, backward and
// single-token step, gfx950.
#include "kdn.h"
#include "kdn_block_device.h"

namespace kdn {

namespace {

constexpr int kChk = KDN_REC_CHECKPOINT;

// alpha and 1 - alpha of a gate value; from a pre-activation both without
// cancellation: with e = exp(-a), 1 / (1 + e) and e / (1 + e)
__device__ __forceinline__ void gate_of(float a, bool preact, float& alpha, float& rest)
{
    if (!preact) {
        alpha = a;
        rest = 1.f - a;
        return;
    }
    alpha = gate_sigmoid(a);
    rest = gate_sigmoid(-a);
}

__device__ __forceinline__ float load_gate(const void* a, size_t i, bool preact, bool bf)
{
    return preact && bf ? to_f32(static_cast<const bf16*>(a)[i]) : static_cast<const float*>(a)[i];
}

// one lane walks one channel of one row
template <typename IO>
__global__ __launch_bounds__(64) void rec_fwd_kernel(RecArgs a)
{
    constexpr bool bf = sizeof(IO) == 2;
    const int c = blockIdx.y * 64 + threadIdx.x, b = blockIdx.x;
    if (c >= a.D)
        return;
    for (int n = a.cu ? 0 : b; n < (a.cu ? a.N : b + 1); ++n) {
        const int p = a.cu ? a.cu[n] : 0, q = a.cu ? a.cu[n + 1] : a.T;
        if (p < 0 || q > a.T)
            continue;
        float h = a.h0 ? a.h0[(size_t)n * a.D + c] : 0.f;
        for (int t = p; t < q; ++t) {
            const size_t r = (size_t)b * a.T + t;
            if (a.ckpt && t % kChk == 0)
                a.ckpt[((size_t)b * ((a.T + kChk - 1) / kChk) + t / kChk) * a.D + c] = h;
            float alpha, rest;
            gate_of(load_gate(a.a, r * a.as + c, a.preact, bf), a.preact, alpha, rest);
            const float x = to_f32(static_cast<const IO*>(a.x)[r * a.xs + c]);
            h = fmaf(alpha, h, a.blend ? rest * x : x);
            static_cast<IO*>(a.h)[r * a.D + c] = from_f32<IO>(h);
        }
        if (a.h_T)
            a.h_T[(size_t)n * a.D + c] = h;
    }
}

template <typename IO>
__global__ __launch_bounds__(64) void rec_bwd_kernel(RecArgs a)
{
    constexpr bool bf = sizeof(IO) == 2;
    __shared__ float prev[kChk][64];  // the state before each token of a block
    const int c = blockIdx.y * 64 + threadIdx.x, b = blockIdx.x;
    if (c >= a.D)
        return;
    const int blocks = (a.T + kChk - 1) / kChk;
    for (int n = a.cu ? a.N - 1 : b; n >= (a.cu ? 0 : b); --n) {
        const int p = a.cu ? a.cu[n] : 0, q = a.cu ? a.cu[n + 1] : a.T;
        if (p < 0 || q > a.T)
            continue;
        const float h0 = a.h0 ? a.h0[(size_t)n * a.D + c] : 0.f;
        float g = a.dh_T ? a.dh_T[(size_t)n * a.D + c] : 0.f;  // alpha lam of the next token
        int end = q;
        while (end > p) {
            const int blk = (end - 1) / kChk, begin = max(p, blk * kChk);
            float h = begin == p ? h0 : a.ckpt[((size_t)b * blocks + blk) * a.D + c];
            for (int t = begin; t < end; ++t) {
                const size_t r = (size_t)b * a.T + t;
                float alpha, rest;
                gate_of(load_gate(a.a, r * a.as + c, a.preact, bf), a.preact, alpha, rest);
                const float x = to_f32(static_cast<const IO*>(a.x)[r * a.xs + c]);
                prev[t - begin][threadIdx.x] = h;
                h = fmaf(alpha, h, a.blend ? rest * x : x);
            }
            for (int t = end - 1; t >= begin; --t) {
                const size_t r = (size_t)b * a.T + t;
                float alpha, rest;
                gate_of(load_gate(a.a, r * a.as + c, a.preact, bf), a.preact, alpha, rest);
                const float x = to_f32(static_cast<const IO*>(a.x)[r * a.xs + c]);
                const float lam = to_f32(static_cast<const IO*>(a.dh)[r * a.D + c]) + g;
                const float hp = prev[t - begin][threadIdx.x];
                const float da = lam * (a.blend ? hp - x : hp);
                static_cast<IO*>(a.dx)[r * a.D + c] = from_f32<IO>(a.blend ? lam * rest : lam);
                if (a.preact)
                    static_cast<IO*>(a.da)[r * a.D + c] = from_f32<IO>(da * alpha * rest);
                else
                    static_cast<float*>(a.da)[r * a.D + c] = da;
                g = alpha * lam;
            }
            end = begin;
        }
        if (a.dh0)
            a.dh0[(size_t)n * a.D + c] = g;
    }
}

template <typename IO>
__global__ __launch_bounds__(256) void rec_step_kernel(RecArgs a)
{
    constexpr bool bf = sizeof(IO) == 2;
    const int c = blockIdx.y * 256 + threadIdx.x, b = blockIdx.x;
    if (c >= a.D)
        return;
    float alpha, rest;
    gate_of(load_gate(a.a, (size_t)b * a.as + c, a.preact, bf), a.preact, alpha, rest);
    const float x = to_f32(static_cast<const IO*>(a.x)[(size_t)b * a.xs + c]);
    const float h = fmaf(alpha, a.h_T[(size_t)b * a.D + c], a.blend ? rest * x : x);
    a.h_T[(size_t)b * a.D + c] = h;
    static_cast<IO*>(a.h)[(size_t)b * a.D + c] = from_f32<IO>(h);
}

}  // namespace

size_t rec_workspace_bytes(int B, int T, int D) { return 0; }

hipError_t launch_rec_fwd(const RecArgs& a, bool bf, hipStream_t stream)
{
    const dim3 grid(a.B, (a.D + 63) / 64);
    if (bf)
        rec_fwd_kernel<bf16><<<grid, 64, 0, stream>>>(a);
    else
        rec_fwd_kernel<float><<<grid, 64, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_rec_bwd(const RecArgs& a, bool bf, hipStream_t stream)
{
    const dim3 grid(a.B, (a.D + 63) / 64);
    if (bf)
        rec_bwd_kernel<bf16><<<grid, 64, 0, stream>>>(a);
    else
        rec_bwd_kernel<float><<<grid, 64, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_rec_step(const RecArgs& a, bool bf, hipStream_t stream)
{
    const dim3 grid(a.B, (a.D + 255) / 256);
    if (bf)
        rec_step_kernel<bf16><<<grid, 256, 0, stream>>>(a);
    else
        rec_step_kernel<float><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace kdn
