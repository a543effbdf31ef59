// kdn_linattn_api.cpp -- host side of the C ABI of linear attention: synchronous
// argument validation and launch.  Nothing here allocates device memory or
// throws across the ABI.
#include <hip/hip_runtime.h>

#include <cmath>

#include "kdn.h"
#include "kdn_checks.h"
#include "kdn_linattn.h"

using namespace kdn;

static kdn_status check_linattn(int B, int T, int H, int Hk, int dk, int dv, int io, float scale, const int* cu, int& N)
{
    KDN_TRY(check_io(io));
    if (H < 1 || Hk < 1 || H % Hk)
        return fail(KDN_ERR_INVALID_ARG, "need H >= 1 a multiple of Hk >= 1 (got H=%d Hk=%d)", H, Hk);
    if (dk < 1 || dv < 1)
        return fail(KDN_ERR_INVALID_ARG, "need dk >= 1, dv >= 1 (got dk=%d dv=%d)", dk, dv);
    if (dk > 256 || dv > 256)
        return fail(KDN_ERR_UNSUPPORTED, "dk and dv are at most 256 (got dk=%d dv=%d)", dk, dv);
    if (!std::isfinite(scale))
        return fail(KDN_ERR_INVALID_ARG, "scale must be finite (got %g)", (double)scale);
    if (H > kMaxD / 256)
        return fail(KDN_ERR_UNSUPPORTED, "H is at most 4096, got %d", H);
    KDN_TRY(check_sequence(B, T, H * (dk > dv ? dk : dv), cu, N));
    if ((__int128)N * H * dk * dv >= kMaxElems)
        return fail(KDN_ERR_UNSUPPORTED, "tensor sizes must stay below 2^31 elements");
    if ((long long)B * H * ((dk > dv ? dk : dv) + 63) / 64 * 3 >= 1 << 24)  // workgroups of a launch
        return fail(KDN_ERR_UNSUPPORTED, "too many heads for one launch (B=%d H=%d)", B, H);
    return KDN_OK;
}

// tokens of `heads` heads of `dim` elements: elements from the first to the last
static kdn_status check_heads(long long tokens, int heads, int dim, long long ts, long long hs, const char* name,
                              long long& span)
{
    if (heads > 1 && hs < dim)
        return fail(KDN_ERR_INVALID_ARG, "%s_head_stride must be at least %d, got %lld", name, dim, hs);
    if (heads > 1 && hs > kMaxRecStride)
        return fail(KDN_ERR_UNSUPPORTED, "%s_head_stride is at most %lld, got %lld", name, kMaxRecStride, hs);
    const long long row = heads > 1 ? (heads - 1) * hs + dim : dim;
    if (ts < row)
        return fail(KDN_ERR_INVALID_ARG, "%s_stride must be at least %lld, got %lld", name, row, ts);
    if (ts > kMaxRecStride)
        return fail(KDN_ERR_UNSUPPORTED, "%s_stride is at most %lld, got %lld", name, kMaxRecStride, ts);
    span = tokens ? (tokens - 1) * ts + row : 0;
    return KDN_OK;
}

static kdn::LinTensor lin_tensor(const void* p, long long ts, long long hs, int div)
{
    kdn::LinTensor t{};
    t.p = p, t.ts = ts, t.hs = (int)hs, t.div = div;
    return t;
}

static bool linattn_sizes(int B, int T, int H, int dk, int dv)
{
    return B >= 1 && T >= 0 && H >= 1 && H <= kMaxD / 256 && dk >= 1 && dk <= 256 && dv >= 1 && dv <= 256 &&
           (__int128)B * T * H * (dk > dv ? dk : dv) < kMaxElems && (long long)B * T <= kMaxTokens && B < 1 << 24;
}

extern "C" {

size_t kdn_linattn_fwd_workspace_size(int B, int T, int H, int dk, int dv)
{
    return linattn_sizes(B, T, H, dk, dv) ? kdn::linattn_fwd_workspace_bytes(B, T, H, dk, dv) : 0;
}

kdn_status kdn_linattn_fwd(int B, int T, int H, int Hk, int dk, int dv, int io_dtype, float scale, const void* q,
                           long long q_stride, long long q_head_stride, const void* k, long long k_stride,
                           long long k_head_stride, const void* v, long long v_stride, long long v_head_stride,
                           const float* decay, const float* S0, const int* cu_seqlens, int N, void* o, float* S_T,
                           void* workspace, size_t workspace_bytes, void* stream)
{
    bool clear;
    KDN_TRY(check_packed_io(io_dtype, clear));
    KDN_TRY(check_linattn(B, T, H, Hk, dk, dv, io_dtype, scale, cu_seqlens, N));
    const long long tokens = (long long)B * T, ns = (long long)N * H * dk * dv;
    long long qspan, kspan, vspan;
    KDN_TRY(check_heads(tokens, Hk, dk, q_stride, q_head_stride, "q", qspan));
    KDN_TRY(check_heads(tokens, Hk, dk, k_stride, k_head_stride, "k", kspan));
    KDN_TRY(check_heads(tokens, H, dv, v_stride, v_head_stride, "v", vspan));
    const size_t need = kdn_linattn_fwd_workspace_size(B, T, H, dk, dv);
    KDN_TRY(check_workspace(workspace, workspace_bytes, need));
    const int e = io_size(io_dtype);
    const Buf bufs[] = {{q, qspan, e, "q", false, true},
                        {k, kspan, e, "k", false, true},
                        {v, vspan, e, "v", false, true},
                        {decay, H, 4, "decay", false, true},
                        {S0, ns, 4, "S0", false, false},
                        {cu_seqlens, (long long)N + 1, 4, "cu_seqlens", false, false},
                        {o, tokens * H * dv, e, "o", true, true},
                        {S_T, ns, 4, "S_T", true, false},
                        {need ? workspace : nullptr, (long long)need, 1, "workspace", true, false}};
    KDN_TRY(check_buffers(bufs));
    kdn::LinCall c{};
    c.B = B, c.T = T, c.H = H, c.Hk = Hk, c.dk = dk, c.dv = dv, c.N = N, c.scale = scale, c.clear = clear;
    c.q = lin_tensor(q, q_stride, q_head_stride, H / Hk), c.k = lin_tensor(k, k_stride, k_head_stride, H / Hk);
    c.v = lin_tensor(v, v_stride, v_head_stride, 1);
    c.decay = decay, c.S0 = S0, c.cu = cu_seqlens, c.o = o, c.S_T = S_T, c.ws = workspace;
    return launched(kdn::launch_linattn_fwd(c, io_dtype == KDN_BF16, (hipStream_t)stream), "kdn_linattn_fwd");
}

size_t kdn_linattn_bwd_workspace_size(int B, int T, int H, int Hk, int dk, int dv)
{
    if (Hk < 1 || !linattn_sizes(B, T, H, dk, dv) || H % Hk)
        return 0;
    return kdn::linattn_bwd_workspace_bytes(B, T, H, Hk, dk, dv);
}

kdn_status kdn_linattn_bwd(int B, int T, int H, int Hk, int dk, int dv, int io_dtype, float scale, const void* d_o,
                           const void* q, long long q_stride, long long q_head_stride, const void* k,
                           long long k_stride, long long k_head_stride, const void* v, long long v_stride,
                           long long v_head_stride, const float* decay, const float* S0, const int* cu_seqlens, int N,
                           const float* dS_T, void* dq, void* dk_out, void* dv_out, float* dS0, void* workspace,
                           size_t workspace_bytes, void* stream)
{
    bool clear;
    KDN_TRY(check_packed_io(io_dtype, clear));
    KDN_TRY(check_linattn(B, T, H, Hk, dk, dv, io_dtype, scale, cu_seqlens, N));
    const long long tokens = (long long)B * T, ns = (long long)N * H * dk * dv;
    long long qspan, kspan, vspan;
    KDN_TRY(check_heads(tokens, Hk, dk, q_stride, q_head_stride, "q", qspan));
    KDN_TRY(check_heads(tokens, Hk, dk, k_stride, k_head_stride, "k", kspan));
    KDN_TRY(check_heads(tokens, H, dv, v_stride, v_head_stride, "v", vspan));
    const size_t need = kdn_linattn_bwd_workspace_size(B, T, H, Hk, dk, dv);
    KDN_TRY(check_workspace(workspace, workspace_bytes, need));
    const int e = io_size(io_dtype);
    const Buf bufs[] = {{d_o, tokens * H * dv, e, "d_o", false, true},
                        {q, qspan, e, "q", false, true},
                        {k, kspan, e, "k", false, true},
                        {v, vspan, e, "v", false, true},
                        {decay, H, 4, "decay", false, true},
                        {S0, ns, 4, "S0", false, false},
                        {cu_seqlens, (long long)N + 1, 4, "cu_seqlens", false, false},
                        {dS_T, ns, 4, "dS_T", false, false},
                        {dq, tokens * Hk * dk, e, "dq", true, true},
                        {dk_out, tokens * Hk * dk, e, "dk_out", true, true},
                        {dv_out, tokens * H * dv, e, "dv_out", true, true},
                        {dS0, ns, 4, "dS0", true, false},
                        {need ? workspace : nullptr, (long long)need, 1, "workspace", true, false}};
    KDN_TRY(check_buffers(bufs));
    kdn::LinCall c{};
    c.B = B, c.T = T, c.H = H, c.Hk = Hk, c.dk = dk, c.dv = dv, c.N = N, c.scale = scale, c.clear = clear;
    c.q = lin_tensor(q, q_stride, q_head_stride, H / Hk), c.k = lin_tensor(k, k_stride, k_head_stride, H / Hk);
    c.v = lin_tensor(v, v_stride, v_head_stride, 1), c.d_o = lin_tensor(d_o, (long long)H * dv, dv, 1);
    c.decay = decay, c.S0 = S0, c.cu = cu_seqlens, c.dS_T = dS_T;
    c.dq = dq, c.dk_out = dk_out, c.dv_out = dv_out, c.dS0 = dS0, c.ws = workspace;
    return launched(kdn::launch_linattn_bwd(c, io_dtype == KDN_BF16, (hipStream_t)stream), "kdn_linattn_bwd");
}

kdn_status kdn_linattn_step(int B, int H, int Hk, int dk, int dv, int io_dtype, float scale, const void* q,
                            long long q_stride, long long q_head_stride, const void* k, long long k_stride,
                            long long k_head_stride, const void* v, long long v_stride, long long v_head_stride,
                            const float* decay, float* state, void* o, void* stream)
{
    int N = 0;
    KDN_TRY(check_linattn(B, 1, H, Hk, dk, dv, io_dtype, scale, nullptr, N));
    long long qspan, kspan, vspan;
    KDN_TRY(check_heads(B, Hk, dk, q_stride, q_head_stride, "q", qspan));
    KDN_TRY(check_heads(B, Hk, dk, k_stride, k_head_stride, "k", kspan));
    KDN_TRY(check_heads(B, H, dv, v_stride, v_head_stride, "v", vspan));
    const int e = io_size(io_dtype);
    const Buf bufs[] = {{q, qspan, e, "q", false, true},
                        {k, kspan, e, "k", false, true},
                        {v, vspan, e, "v", false, true},
                        {decay, H, 4, "decay", false, true},
                        {state, (long long)B * H * dk * dv, 4, "state", true, true},
                        {o, (long long)B * H * dv, e, "o", true, true}};
    KDN_TRY(check_buffers(bufs));
    kdn::LinStepArgs a{};
    a.B = B, a.H = H, a.G = H / Hk, a.dk = dk, a.dv = dv, a.scale = scale;
    a.q = q, a.qs = q_stride, a.qh = q_head_stride, a.k = k, a.ks = k_stride, a.kh = k_head_stride;
    a.v = v, a.vs = v_stride, a.vh = v_head_stride, a.decay = decay, a.S = state, a.o = o;
    return launched(kdn::launch_linattn_step(a, io_dtype == KDN_BF16, (hipStream_t)stream), "kdn_linattn_step");
}

}  // extern "C"
