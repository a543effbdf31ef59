// kdn_block_api.cpp -- host side of the C ABI of the operators around the
// mixer: synchronous argument validation and launch.  Nothing here allocates
// device memory or throws across the ABI.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "kdn.h"
#include "kdn_block.h"
#include "kdn_errors.h"

namespace {

using kdn::fail;
using kdn::ok;

constexpr long long kMaxElems = 1ll << 31;  // of every dense tensor
constexpr long long kMaxStride = 1ll << 30;
// the recurrence steps over a tile of rows with 32-bit byte offsets
constexpr long long kMaxRecStride = 1ll << 22;
constexpr int kMaxD = 1 << 20, kMaxTokens = 1 << 30;

// One buffer of a call: its bytes (0: not given) and what the call does to it.
struct Buf {
    const void* p;
    long long elems;
    int size;  // bytes of an element, and its alignment
    const char* name;
    bool out;
    bool required;  // when elems > 0
};

long long bytes_of(const Buf& b) { return b.p ? b.elems * b.size : 0; }

// NULL where a buffer is needed, misaligned pointers, outputs that overlap
template <int N>
kdn_status check_buffers(const Buf (&bufs)[N])
{
    for (const Buf& b : bufs) {
        if (b.required && b.elems > 0 && !b.p)
            return fail(KDN_ERR_INVALID_ARG, "%s must not be NULL", b.name);
        if (reinterpret_cast<uintptr_t>(b.p) % (unsigned)b.size)
            return fail(KDN_ERR_INVALID_ARG, "%s must be %d-byte aligned", b.name, b.size);
    }
    for (const Buf& o : bufs) {
        if (!o.out || !bytes_of(o))
            continue;
        const uintptr_t o0 = reinterpret_cast<uintptr_t>(o.p), o1 = o0 + bytes_of(o);
        for (const Buf& b : bufs) {
            const uintptr_t b0 = reinterpret_cast<uintptr_t>(b.p), b1 = b0 + bytes_of(b);
            if (&b != &o && o0 < b1 && b0 < o1)
                return fail(KDN_ERR_INVALID_ARG, "%s must not overlap %s", o.name, b.name);
        }
    }
    return KDN_OK;
}

kdn_status check_io(int io)
{
    if (io != KDN_F32 && io != KDN_BF16)
        return fail(KDN_ERR_INVALID_ARG, "io_dtype must be KDN_F32 (0) or KDN_BF16 (1), got %d", io);
    return KDN_OK;
}

// an io_dtype that may hold KDN_CLEAR_TAIL, which is taken out of it
kdn_status check_packed_io(int& io, bool& clear)
{
    clear = io & KDN_CLEAR_TAIL;
    io &= ~KDN_CLEAR_TAIL;
    if (io != KDN_F32 && io != KDN_BF16)
        return fail(KDN_ERR_INVALID_ARG, "io_dtype must be KDN_F32 (0) or KDN_BF16 (1), with KDN_CLEAR_TAIL (0x400) "
                    "if wanted, got %d", clear ? io | KDN_CLEAR_TAIL : io);
    return KDN_OK;
}

kdn_status check_width(int D)
{
    if (D < 1)
        return fail(KDN_ERR_INVALID_ARG, "need D >= 1 (got %d)", D);
    if (D > kMaxD)
        return fail(KDN_ERR_UNSUPPORTED, "D is at most 2^20, got %d", D);
    return KDN_OK;
}

// rows of D elements, stride apart: the elements from the first to the last
kdn_status check_rows(long long rows, int D, long long stride, const char* name, long long& span,
                      long long most = kMaxStride)
{
    if (stride < D)
        return fail(KDN_ERR_INVALID_ARG, "%s_stride must be at least D = %d, got %lld", name, D, stride);
    if (stride > most)
        return fail(KDN_ERR_UNSUPPORTED, "%s_stride is at most %lld, got %lld", name, most, stride);
    span = rows ? (rows - 1) * stride + D : 0;
    return KDN_OK;
}

// [B,T,D] and the sequences in it; N becomes B where rows are not packed
kdn_status check_sequence(int B, int T, int D, const int* cu, int& N)
{
    if (B < 1 || T < 0)
        return fail(KDN_ERR_INVALID_ARG, "need B >= 1, T >= 0 (got B=%d T=%d)", B, T);
    const kdn_status st = check_width(D);
    if (st != KDN_OK)
        return st;
    if (cu && B != 1)
        return fail(KDN_ERR_INVALID_ARG, "packed sequences (cu_seqlens) need B = 1, got %d", B);
    if (cu && N < 1)
        return fail(KDN_ERR_INVALID_ARG, "packed sequences need N >= 1, got %d", N);
    if (!cu)
        N = B;
    // 128-bit products: three factors below 2^31
    if ((__int128)B * T * D >= kMaxElems || (__int128)N * D >= kMaxElems)
        return fail(KDN_ERR_UNSUPPORTED, "tensor sizes must stay below 2^31 elements");
    // token numbers, and those a tile further, are ints; a row is a workgroup or more
    if ((long long)B * T > kMaxTokens || B >= 1 << 24)
        return fail(KDN_ERR_UNSUPPORTED, "B T is at most 2^30 and B below 2^24 (got B=%d T=%d)", B, T);
    return KDN_OK;
}

kdn_status check_workspace(const void* ws, size_t bytes, size_t need)
{
    if (!need)
        return KDN_OK;
    if (!ws || bytes < need)
        return fail(KDN_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, ws ? bytes : (size_t)0);
    if (reinterpret_cast<uintptr_t>(ws) & 15u)
        return fail(KDN_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    return KDN_OK;
}

kdn_status launched(hipError_t e, const char* what)
{
    return e == hipSuccess ? ok() : fail(KDN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

#define KDN_TRY(call)               \
    do {                            \
        const kdn_status st_ = call; \
        if (st_ != KDN_OK)          \
            return st_;             \
    } while (0)

int io_size(int io) { return io == KDN_BF16 ? 2 : 4; }

kdn_status check_norm(int rows, int D, int io)
{
    KDN_TRY(check_io(io));
    if (rows < 0)
        return fail(KDN_ERR_INVALID_ARG, "need rows >= 0 (got %d)", rows);
    KDN_TRY(check_width(D));
    if ((long long)rows * D >= kMaxElems)
        return fail(KDN_ERR_UNSUPPORTED, "tensor sizes must stay below 2^31 elements");
    if (rows > kMaxTokens)  // row numbers, and those a stride further, are ints
        return fail(KDN_ERR_UNSUPPORTED, "rows is at most 2^30, got %d", rows);
    return KDN_OK;
}

kdn_status check_conv(int W, int io, int act)
{
    KDN_TRY(check_io(io));
    if (W < 2 || W > 4)
        return fail(KDN_ERR_UNSUPPORTED, "the convolution has 2 to 4 taps, got %d", W);
    if (act != KDN_ACT_NONE && act != KDN_ACT_SILU)
        return fail(KDN_ERR_INVALID_ARG, "activation must be KDN_ACT_NONE (0) or KDN_ACT_SILU (1), got %d", act);
    return KDN_OK;
}

kdn_status check_rec(int io, int gate, int blend)
{
    KDN_TRY(check_io(io));
    if (gate != KDN_GATE_ALPHA && gate != KDN_GATE_PREACT)
        return fail(KDN_ERR_INVALID_ARG, "gate must be KDN_GATE_ALPHA (0) or KDN_GATE_PREACT (1), got %d", gate);
    if (blend != 0 && blend != 1)
        return fail(KDN_ERR_INVALID_ARG, "blend must be 0 or 1, got %d", blend);
    return KDN_OK;
}

}  // namespace

extern "C" {

kdn_status kdn_layer_norm_fwd(int rows, int D, int io_dtype, float eps, const void* x,
                              long long x_stride, const float* weight, const float* bias,
                              void* y, float* mean, float* rstd, void* stream)
{
    KDN_TRY(check_norm(rows, D, io_dtype));
    if (!(eps >= 0.f) || !std::isfinite(eps))
        return fail(KDN_ERR_INVALID_ARG, "eps must be finite and >= 0 (got %g)", (double)eps);
    long long span;
    KDN_TRY(check_rows(rows, D, x_stride, "x", span));
    const int e = io_size(io_dtype);
    const Buf bufs[] = {{x, span, e, "x", false, true},
                        {weight, D, 4, "weight", false, false},
                        {bias, D, 4, "bias", false, false},
                        {y, (long long)rows * D, e, "y", true, true},
                        {mean, rows, 4, "mean", true, false},
                        {rstd, rows, 4, "rstd", true, false}};
    KDN_TRY(check_buffers(bufs));
    kdn::NormArgs a{};
    a.rows = rows, a.D = D, a.eps = eps;
    a.x = x, a.xs = x_stride, a.weight = weight, a.bias = bias;
    a.y = y, a.mean = mean, a.rstd = rstd;
    return launched(kdn::launch_norm_fwd(a, io_dtype == KDN_BF16, (hipStream_t)stream),
                    "kdn_layer_norm_fwd");
}

size_t kdn_layer_norm_bwd_workspace_size(int rows, int D)
{
    if (rows < 0 || rows > kMaxTokens || D < 1 || D > kMaxD || (long long)rows * D >= kMaxElems)
        return 0;
    return (size_t)kdn::norm_bwd_groups(rows, D) * 2 * D * sizeof(float);
}

kdn_status kdn_layer_norm_bwd(int rows, int D, int io_dtype, const void* dy, const void* x,
                              long long x_stride, const float* mean, const float* rstd,
                              const float* weight, void* dx, float* dweight, float* dbias,
                              void* workspace, size_t workspace_bytes, void* stream)
{
    KDN_TRY(check_norm(rows, D, io_dtype));
    long long span;
    KDN_TRY(check_rows(rows, D, x_stride, "x", span));
    const int e = io_size(io_dtype);
    const size_t need = dweight || dbias ? kdn_layer_norm_bwd_workspace_size(rows, D) : 0;
    KDN_TRY(check_workspace(workspace, workspace_bytes, need));
    const long long n = (long long)rows * D;
    const Buf bufs[] = {{dy, n, e, "dy", false, true},
                        {x, span, e, "x", false, true},
                        {mean, rows, 4, "mean", false, true},
                        {rstd, rows, 4, "rstd", false, true},
                        {weight, D, 4, "weight", false, false},
                        {dx, n, e, "dx", true, true},
                        {dweight, D, 4, "dweight", true, false},
                        {dbias, D, 4, "dbias", true, false},
                        {need ? workspace : nullptr, (long long)need, 1, "workspace", true, false}};
    KDN_TRY(check_buffers(bufs));
    kdn::NormArgs a{};
    a.rows = rows, a.D = D;
    a.x = x, a.xs = x_stride, a.weight = weight;
    a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
    a.dy = dy, a.dx = dx, a.dweight = dweight, a.dbias = dbias;
    a.ws = static_cast<float*>(workspace);
    return launched(kdn::launch_norm_bwd(a, io_dtype == KDN_BF16, (hipStream_t)stream),
                    "kdn_layer_norm_bwd");
}

kdn_status kdn_conv_fwd(int B, int T, int D, int W, int io_dtype, int activation, const void* x,
                        long long x_stride, const float* weight, const float* bias,
                        const void* state0, const int* cu_seqlens, int N, void* y, void* state_T,
                        void* stream)
{
    bool clear;
    KDN_TRY(check_packed_io(io_dtype, clear));
    KDN_TRY(check_conv(W, io_dtype, activation));
    KDN_TRY(check_sequence(B, T, D, cu_seqlens, N));
    if ((__int128)N * (W - 1) * D >= kMaxElems)
        return fail(KDN_ERR_UNSUPPORTED, "tensor sizes must stay below 2^31 elements");
    long long span;
    KDN_TRY(check_rows((long long)B * T, D, x_stride, "x", span));
    const int e = io_size(io_dtype);
    const long long n = (long long)B * T * D, ns = (long long)N * (W - 1) * D;
    const Buf bufs[] = {{x, span, e, "x", false, true},
                        {weight, (long long)W * D, 4, "weight", false, true},
                        {bias, D, 4, "bias", false, false},
                        {state0, ns, e, "state0", false, false},
                        {cu_seqlens, (long long)N + 1, 4, "cu_seqlens", false, false},
                        {y, n, e, "y", true, true},
                        {state_T, ns, e, "state_T", true, false}};
    KDN_TRY(check_buffers(bufs));
    kdn::ConvArgs a{};
    a.B = B, a.T = T, a.D = D, a.W = W, a.silu = activation == KDN_ACT_SILU, a.clear = clear;
    a.x = x, a.xs = x_stride, a.weight = weight, a.bias = bias;
    a.state0 = state0, a.cu = cu_seqlens, a.N = N, a.y = y, a.state_T = state_T;
    return launched(kdn::launch_conv_fwd(a, io_dtype == KDN_BF16, (hipStream_t)stream),
                    "kdn_conv_fwd");
}

size_t kdn_conv_bwd_workspace_size(int B, int T, int D, int W)
{
    if (B < 1 || T < 0 || D < 1 || D > kMaxD || W < 2 || W > 4 ||
        (__int128)B * T * D >= kMaxElems || (long long)B * T > kMaxTokens)
        return 0;
    return (size_t)kdn::conv_bwd_groups(B, T, D) * (W + 1) * D * sizeof(float);
}

kdn_status kdn_conv_bwd(int B, int T, int D, int W, int io_dtype, int activation, const void* dy,
                        const void* x, long long x_stride, const float* weight, const float* bias,
                        const void* state0, const int* cu_seqlens, int N, const void* dstate_T,
                        void* dx, float* dweight, float* dbias, void* dstate0, void* workspace,
                        size_t workspace_bytes, void* stream)
{
    bool clear;
    KDN_TRY(check_packed_io(io_dtype, clear));
    KDN_TRY(check_conv(W, io_dtype, activation));
    KDN_TRY(check_sequence(B, T, D, cu_seqlens, N));
    if ((__int128)N * (W - 1) * D >= kMaxElems)
        return fail(KDN_ERR_UNSUPPORTED, "tensor sizes must stay below 2^31 elements");
    long long span;
    KDN_TRY(check_rows((long long)B * T, D, x_stride, "x", span));
    const size_t need = kdn_conv_bwd_workspace_size(B, T, D, W);
    KDN_TRY(check_workspace(workspace, workspace_bytes, need));
    const int e = io_size(io_dtype);
    const long long n = (long long)B * T * D, ns = (long long)N * (W - 1) * D;
    const Buf bufs[] = {{dy, n, e, "dy", false, true},
                        {x, span, e, "x", false, true},
                        {weight, (long long)W * D, 4, "weight", false, true},
                        {bias, D, 4, "bias", false, false},
                        {state0, ns, e, "state0", false, false},
                        {cu_seqlens, (long long)N + 1, 4, "cu_seqlens", false, false},
                        {dstate_T, ns, e, "dstate_T", false, false},
                        {dx, n, e, "dx", true, true},
                        {dweight, (long long)W * D, 4, "dweight", true, true},
                        {dbias, D, 4, "dbias", true, false},
                        {dstate0, ns, e, "dstate0", true, false},
                        {need ? workspace : nullptr, (long long)need, 1, "workspace", true, false}};
    KDN_TRY(check_buffers(bufs));
    kdn::ConvArgs a{};
    a.B = B, a.T = T, a.D = D, a.W = W, a.silu = activation == KDN_ACT_SILU, a.clear = clear;
    a.x = x, a.xs = x_stride, a.weight = weight, a.bias = bias;
    a.state0 = state0, a.cu = cu_seqlens, a.N = N;
    a.dy = dy, a.dstate_T = dstate_T, a.dx = dx, a.dweight = dweight, a.dbias = dbias;
    a.dstate0 = dstate0, a.ws = static_cast<float*>(workspace);
    return launched(kdn::launch_conv_bwd(a, io_dtype == KDN_BF16, (hipStream_t)stream),
                    "kdn_conv_bwd");
}

kdn_status kdn_conv_step(int B, int D, int W, int io_dtype, int activation, const void* x,
                         long long x_stride, const float* weight, const float* bias, void* state,
                         void* y, void* stream)
{
    KDN_TRY(check_conv(W, io_dtype, activation));
    int N = 0;
    KDN_TRY(check_sequence(B, 1, D, nullptr, N));
    if ((__int128)B * (W - 1) * D >= kMaxElems)
        return fail(KDN_ERR_UNSUPPORTED, "tensor sizes must stay below 2^31 elements");
    long long span;
    KDN_TRY(check_rows(B, D, x_stride, "x", span));
    const int e = io_size(io_dtype);
    const Buf bufs[] = {{x, span, e, "x", false, true},
                        {weight, (long long)W * D, 4, "weight", false, true},
                        {bias, D, 4, "bias", false, false},
                        {state, (long long)B * (W - 1) * D, e, "state", true, true},
                        {y, (long long)B * D, e, "y", true, true}};
    KDN_TRY(check_buffers(bufs));
    kdn::ConvArgs a{};
    a.B = B, a.T = 1, a.D = D, a.W = W, a.silu = activation == KDN_ACT_SILU;
    a.x = x, a.xs = x_stride, a.weight = weight, a.bias = bias;
    a.N = B, a.y = y, a.state_T = state;
    return launched(kdn::launch_conv_step(a, io_dtype == KDN_BF16, (hipStream_t)stream),
                    "kdn_conv_step");
}

// a launch has fewer than 2^32 threads: only many rows of a few tokens come near
static kdn_status check_rec_grid(int B, int T, int D, bool backward)
{
    if (kdn::rec_threads(B, T, D, backward) >> 32)
        return fail(KDN_ERR_UNSUPPORTED, "too many short rows for one launch (B=%d T=%d D=%d)", B, T, D);
    return KDN_OK;
}

static size_t rec_workspace_size(int B, int T, int D, bool backward)
{
    if (B < 1 || T < 0 || D < 1 || D > kMaxD || (__int128)B * T * D >= kMaxElems ||
        (long long)B * T > kMaxTokens)
        return 0;
    return kdn::rec_workspace_bytes(B, T, D, backward);
}

size_t kdn_rec_fwd_workspace_size(int B, int T, int D) { return rec_workspace_size(B, T, D, false); }
size_t kdn_rec_bwd_workspace_size(int B, int T, int D) { return rec_workspace_size(B, T, D, true); }

kdn_status kdn_rec_fwd(int B, int T, int D, int io_dtype, int gate, int blend, const void* x,
                       long long x_stride, const void* a, long long a_stride, const float* h0,
                       const int* cu_seqlens, int N, void* h, float* h_T, float* checkpoints,
                       void* workspace, size_t workspace_bytes, void* stream)
{
    bool clear;
    KDN_TRY(check_packed_io(io_dtype, clear));
    KDN_TRY(check_rec(io_dtype, gate, blend));
    KDN_TRY(check_sequence(B, T, D, cu_seqlens, N));
    long long xspan, aspan;
    KDN_TRY(check_rows((long long)B * T, D, x_stride, "x", xspan, kMaxRecStride));
    KDN_TRY(check_rows((long long)B * T, D, a_stride, "a", aspan, kMaxRecStride));
    KDN_TRY(check_rec_grid(B, T, D, false));
    const size_t need = kdn_rec_fwd_workspace_size(B, T, D);
    KDN_TRY(check_workspace(workspace, workspace_bytes, need));
    const int e = io_size(io_dtype), ea = gate == KDN_GATE_PREACT ? e : 4;
    const long long ns = (long long)N * D;
    const long long nc = (long long)B * (((long long)T + KDN_REC_CHECKPOINT - 1) / KDN_REC_CHECKPOINT) * D;
    const Buf bufs[] = {{x, xspan, e, "x", false, true},
                        {a, aspan, ea, "a", false, true},
                        {h0, ns, 4, "h0", false, false},
                        {cu_seqlens, (long long)N + 1, 4, "cu_seqlens", false, false},
                        {h, (long long)B * T * D, e, "h", true, true},
                        {h_T, ns, 4, "h_T", true, false},
                        {checkpoints, nc, 4, "checkpoints", true, false},
                        {need ? workspace : nullptr, (long long)need, 1, "workspace", true, false}};
    KDN_TRY(check_buffers(bufs));
    kdn::RecArgs r{};
    r.B = B, r.T = T, r.D = D, r.preact = gate == KDN_GATE_PREACT, r.blend = blend == 1, r.clear = clear;
    r.x = x, r.xs = x_stride, r.a = a, r.as = a_stride, r.h0 = h0, r.cu = cu_seqlens, r.N = N;
    r.h = h, r.h_T = h_T, r.ckpt = checkpoints, r.ws = workspace;
    return launched(kdn::launch_rec_fwd(r, io_dtype == KDN_BF16, (hipStream_t)stream), "kdn_rec_fwd");
}

kdn_status kdn_rec_bwd(int B, int T, int D, int io_dtype, int gate, int blend, const void* dh,
                       const void* x, long long x_stride, const void* a, long long a_stride,
                       const float* checkpoints, const float* h0, const int* cu_seqlens, int N,
                       const float* dh_T, void* dx, void* da, float* dh0, void* workspace,
                       size_t workspace_bytes, void* stream)
{
    bool clear;
    KDN_TRY(check_packed_io(io_dtype, clear));
    KDN_TRY(check_rec(io_dtype, gate, blend));
    KDN_TRY(check_sequence(B, T, D, cu_seqlens, N));
    long long xspan, aspan;
    KDN_TRY(check_rows((long long)B * T, D, x_stride, "x", xspan, kMaxRecStride));
    KDN_TRY(check_rows((long long)B * T, D, a_stride, "a", aspan, kMaxRecStride));
    KDN_TRY(check_rec_grid(B, T, D, true));
    const size_t need = kdn_rec_bwd_workspace_size(B, T, D);
    KDN_TRY(check_workspace(workspace, workspace_bytes, need));
    const int e = io_size(io_dtype), ea = gate == KDN_GATE_PREACT ? e : 4;
    const long long n = (long long)B * T * D, ns = (long long)N * D;
    const long long nc = (long long)B * (((long long)T + KDN_REC_CHECKPOINT - 1) / KDN_REC_CHECKPOINT) * D;
    const Buf bufs[] = {{dh, n, e, "dh", false, true},
                        {x, xspan, e, "x", false, true},
                        {a, aspan, ea, "a", false, true},
                        {checkpoints, nc, 4, "checkpoints", false, true},
                        {h0, ns, 4, "h0", false, false},
                        {cu_seqlens, (long long)N + 1, 4, "cu_seqlens", false, false},
                        {dh_T, ns, 4, "dh_T", false, false},
                        {dx, n, e, "dx", true, true},
                        {da, n, ea, "da", true, true},
                        {dh0, ns, 4, "dh0", true, false},
                        {need ? workspace : nullptr, (long long)need, 1, "workspace", true, false}};
    KDN_TRY(check_buffers(bufs));
    kdn::RecArgs r{};
    r.B = B, r.T = T, r.D = D, r.preact = gate == KDN_GATE_PREACT, r.blend = blend == 1, r.clear = clear;
    r.x = x, r.xs = x_stride, r.a = a, r.as = a_stride, r.h0 = h0, r.cu = cu_seqlens, r.N = N;
    r.ckpt = const_cast<float*>(checkpoints), r.dh = dh, r.dh_T = dh_T;
    r.dx = dx, r.da = da, r.dh0 = dh0, r.ws = workspace;
    return launched(kdn::launch_rec_bwd(r, io_dtype == KDN_BF16, (hipStream_t)stream), "kdn_rec_bwd");
}

kdn_status kdn_rec_step(int B, int D, int io_dtype, int gate, int blend, const void* x,
                        long long x_stride, const void* a, long long a_stride, float* state,
                        void* h, void* stream)
{
    KDN_TRY(check_rec(io_dtype, gate, blend));
    int N = 0;
    KDN_TRY(check_sequence(B, 1, D, nullptr, N));
    long long xspan, aspan;
    KDN_TRY(check_rows(B, D, x_stride, "x", xspan));
    KDN_TRY(check_rows(B, D, a_stride, "a", aspan));
    const int e = io_size(io_dtype), ea = gate == KDN_GATE_PREACT ? e : 4;
    const Buf bufs[] = {{x, xspan, e, "x", false, true},
                        {a, aspan, ea, "a", false, true},
                        {state, (long long)B * D, 4, "state", true, true},
                        {h, (long long)B * D, e, "h", true, true}};
    KDN_TRY(check_buffers(bufs));
    kdn::RecArgs r{};
    r.B = B, r.T = 1, r.D = D, r.preact = gate == KDN_GATE_PREACT, r.blend = blend == 1;
    r.x = x, r.xs = x_stride, r.a = a, r.as = a_stride, r.h_T = state, r.h = h, r.N = B;
    return launched(kdn::launch_rec_step(r, io_dtype == KDN_BF16, (hipStream_t)stream),
                    "kdn_rec_step");
}

}  // extern "C"
