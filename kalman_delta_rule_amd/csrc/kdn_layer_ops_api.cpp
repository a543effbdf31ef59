// kdn_layer_ops_api.cpp -- host side of the C ABI of group norm and dropout: synchronous
// argument validation and launch.  Nothing here allocates device memory or throws across
// the ABI.
#include <hip/hip_runtime.h>

#include <cmath>

#include "kdn.h"
#include "kdn_checks.h"
#include "kdn_layer_ops.h"

using namespace kdn;

static kdn_status check_group_norm(int N, int S, int C, int G, int io, int act)
{
    KDN_TRY(check_io(io));
    if (act != KDN_ACT_NONE && act != KDN_ACT_SILU)
        return fail(KDN_ERR_INVALID_ARG, "activation must be KDN_ACT_NONE (0) or KDN_ACT_SILU (1), got %d", act);
    if (N < 0 || S < 0)
        return fail(KDN_ERR_INVALID_ARG, "need N >= 0, S >= 0 (got N=%d S=%d)", N, S);
    KDN_TRY(check_width(C));
    if (G < 1 || C % G)
        return fail(KDN_ERR_INVALID_ARG, "C must be a multiple of G >= 1 (got C=%d G=%d)", C, G);
    if ((__int128)N * S * C >= kMaxElems || (__int128)N * G >= kMaxElems / 128)
        return fail(KDN_ERR_UNSUPPORTED, "N S C must stay below 2^31, N G below 2^24");
    if ((long long)N * S > kMaxTokens)
        return fail(KDN_ERR_UNSUPPORTED, "N S is at most 2^30 (got N=%d S=%d)", N, S);
    return KDN_OK;
}

static bool group_norm_sizes(int N, int S, int C, int G)
{
    return N >= 0 && S >= 0 && C >= 1 && C <= kMaxD && G >= 1 && C % G == 0 && (__int128)N * S * C < kMaxElems &&
           (__int128)N * G < kMaxElems / 128 && (long long)N * S <= kMaxTokens;
}

static kdn_status check_dropout(int rows, int D, int io, double p)
{
    KDN_TRY(check_io(io));
    if (rows < 0)
        return fail(KDN_ERR_INVALID_ARG, "need rows >= 0 (got %d)", rows);
    KDN_TRY(check_width(D));
    if ((long long)rows * D >= kMaxElems)
        return fail(KDN_ERR_UNSUPPORTED, "tensor sizes must stay below 2^31 elements");
    if (!(p >= 0.0 && p <= 1.0))
        return fail(KDN_ERR_INVALID_ARG, "p must be in [0, 1] (got %g)", p);
    return KDN_OK;
}

static void set_share(DropoutArgs& a, double p)
{
    a.least = (uint32_t)std::nearbyint(p * 65536.0);
    a.scale = a.least < 65536 ? (float)(65536.0 / (65536 - a.least)) : 0.f;
}

extern "C" {

size_t kdn_group_norm_fwd_workspace_size(int N, int S, int C, int G)
{
    return group_norm_sizes(N, S, C, G) ? group_norm_fwd_workspace_bytes(N, S, C, G) : 0;
}

kdn_status kdn_group_norm_fwd(int N, int S, int C, int G, int io_dtype, int activation, float eps, const void* x,
                              long long x_stride, const float* weight, const float* bias, void* y, float* mean,
                              float* rstd, void* workspace, size_t workspace_bytes, void* stream)
{
    KDN_TRY(check_group_norm(N, S, C, G, io_dtype, activation));
    if (!(eps >= 0.f) || !std::isfinite(eps))
        return fail(KDN_ERR_INVALID_ARG, "eps must be finite and >= 0 (got %g)", (double)eps);
    const long long rows = (long long)N * S, units = (long long)N * G;
    long long span;
    KDN_TRY(check_rows(rows, C, x_stride, "x", span));
    const size_t need = kdn_group_norm_fwd_workspace_size(N, S, C, G);
    KDN_TRY(check_workspace(workspace, workspace_bytes, need));
    const int e = io_size(io_dtype);
    const Buf bufs[] = {{x, span, e, "x", false, true},
                        {weight, C, 4, "weight", false, false},
                        {bias, C, 4, "bias", false, false},
                        {y, rows * C, e, "y", true, true},
                        {mean, units, 4, "mean", true, false},
                        {rstd, units, 4, "rstd", true, false},
                        {need ? workspace : nullptr, (long long)need, 1, "workspace", true, false}};
    KDN_TRY(check_buffers(bufs));
    GroupNormArgs a{};
    a.N = N, a.S = S, a.C = C, a.G = G, a.silu = activation == KDN_ACT_SILU, a.eps = eps;
    a.x = x, a.xs = x_stride, a.weight = weight, a.bias = bias, a.y = y, a.mean = mean, a.rstd = rstd;
    a.ws = workspace;
    return launched(launch_group_norm_fwd(a, io_dtype == KDN_BF16, (hipStream_t)stream), "kdn_group_norm_fwd");
}

size_t kdn_group_norm_bwd_workspace_size(int N, int S, int C, int G)
{
    return group_norm_sizes(N, S, C, G) ? group_norm_bwd_workspace_bytes(N, S, C, G) : 0;
}

kdn_status kdn_group_norm_bwd(int N, int S, int C, int G, int io_dtype, int activation, const void* dy, const void* x,
                              long long x_stride, const float* mean, const float* rstd, const float* weight,
                              const float* bias, void* dx, float* dweight, float* dbias, void* workspace,
                              size_t workspace_bytes, void* stream)
{
    KDN_TRY(check_group_norm(N, S, C, G, io_dtype, activation));
    const long long rows = (long long)N * S, units = (long long)N * G;
    long long span;
    KDN_TRY(check_rows(rows, C, x_stride, "x", span));
    const size_t need = kdn_group_norm_bwd_workspace_size(N, S, C, G);
    KDN_TRY(check_workspace(workspace, workspace_bytes, need));
    const int e = io_size(io_dtype);
    const Buf bufs[] = {{dy, rows * C, e, "dy", false, true},
                        {x, span, e, "x", false, true},
                        {mean, rows ? units : 0, 4, "mean", false, true},
                        {rstd, rows ? units : 0, 4, "rstd", false, true},
                        {weight, C, 4, "weight", false, false},
                        {bias, C, 4, "bias", false, false},
                        {dx, rows * C, e, "dx", true, true},
                        {dweight, C, 4, "dweight", true, false},
                        {dbias, C, 4, "dbias", true, false},
                        {need ? workspace : nullptr, (long long)need, 1, "workspace", true, false}};
    KDN_TRY(check_buffers(bufs));
    GroupNormArgs a{};
    a.N = N, a.S = S, a.C = C, a.G = G, a.silu = activation == KDN_ACT_SILU;
    a.x = x, a.xs = x_stride, a.weight = weight, a.bias = bias;
    a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
    a.dy = dy, a.dx = dx, a.dweight = dweight, a.dbias = dbias, a.ws = workspace;
    return launched(launch_group_norm_bwd(a, io_dtype == KDN_BF16, (hipStream_t)stream), "kdn_group_norm_bwd");
}

kdn_status kdn_dropout_fwd(int rows, int D, int io_dtype, double p, unsigned long long seed, unsigned long long offset,
                           const long long* seed_offset, const void* x, long long x_stride, const void* residual,
                           void* y, void* stream)
{
    KDN_TRY(check_dropout(rows, D, io_dtype, p));
    long long span;
    KDN_TRY(check_rows(rows, D, x_stride, "x", span));
    const int e = io_size(io_dtype);
    const long long n = (long long)rows * D;
    const Buf bufs[] = {{x, span, e, "x", false, true},
                        {residual, n, e, "residual", false, false},
                        {seed_offset, 2, 8, "seed_offset", false, false},
                        {y, n, e, "y", true, true}};
    KDN_TRY(check_buffers(bufs));
    DropoutArgs a{};
    a.rows = rows, a.D = D, a.seed = seed, a.offset = offset, a.state = seed_offset;
    a.x = x, a.xs = x_stride, a.residual = residual, a.y = y;
    set_share(a, p);
    return launched(launch_dropout(a, io_dtype == KDN_BF16, (hipStream_t)stream), "kdn_dropout_fwd");
}

kdn_status kdn_dropout_bwd(int rows, int D, int io_dtype, double p, unsigned long long seed, unsigned long long offset,
                           const long long* seed_offset, const void* dy, void* dx, void* stream)
{
    KDN_TRY(check_dropout(rows, D, io_dtype, p));
    const int e = io_size(io_dtype);
    const long long n = (long long)rows * D;
    const Buf bufs[] = {{dy, n, e, "dy", false, true},
                        {seed_offset, 2, 8, "seed_offset", false, false},
                        {dx, n, e, "dx", true, true}};
    KDN_TRY(check_buffers(bufs));
    DropoutArgs a{};
    a.rows = rows, a.D = D, a.seed = seed, a.offset = offset, a.state = seed_offset;
    a.x = dy, a.xs = D, a.y = dx;
    set_share(a, p);
    return launched(launch_dropout(a, io_dtype == KDN_BF16, (hipStream_t)stream), "kdn_dropout_bwd");
}

}  // extern "C"
