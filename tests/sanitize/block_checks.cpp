// The host code of the operators around the mixer (validation, overlap rules,
// sizes) driven through every entry point with stand-in device addresses,
// built with the address and undefined-behaviour sanitizers.  Exits nonzero
// after a failed expectation.
#include <cmath>
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "kdn.h"

extern int g_launches;

static int failures = 0;

static void* at(uint64_t a) { return reinterpret_cast<void*>(a); }
static float* fat(uint64_t a) { return reinterpret_cast<float*>(a); }
static const int* iat(uint64_t a) { return reinterpret_cast<const int*>(a); }

// A call must end with `code`, say `needle`, and launch only where it got past
// validation (KDN_ERR_HIP from the stand-ins).
static void expect(int line, kdn_status st, kdn_status code, const char* needle)
{
    static int seen = 0;
    const bool launched = g_launches != seen;
    seen = g_launches;
    if (st != code || !std::strstr(kdn_last_error_message(), needle) || launched != (code == KDN_ERR_HIP)) {
        std::printf("FAILED line %d: status %d, launched %d, last error: %s\n", line, (int)st,
                    (int)launched, kdn_last_error_message());
        ++failures;
    }
}
#define BAD(call, code, needle) expect(__LINE__, (call), (code), (needle))
#define RUNS(call) expect(__LINE__, (call), KDN_ERR_HIP, "launch stand-in")

static const uint64_t G = 1ull << 36;  // far enough apart for any size below

struct Norm {
    int rows = 10, D = 64, io = KDN_BF16;
    float eps = 1e-5f;
    long long xs = 64;
    uint64_t x = 1 * G, w = 2 * G, b = 3 * G, y = 4 * G, mean = 5 * G, rstd = 6 * G;
    uint64_t dy = 7 * G, dx = 8 * G, dw = 9 * G, db = 10 * G, ws = 11 * G;
    long long ws_bytes = -1;
    kdn_status fwd() const
    {
        return kdn_layer_norm_fwd(rows, D, io, eps, at(x), xs, fat(w), fat(b), at(y), fat(mean),
                                  fat(rstd), nullptr);
    }
    kdn_status bwd() const
    {
        const size_t n = ws_bytes < 0 ? kdn_layer_norm_bwd_workspace_size(rows, D) : (size_t)ws_bytes;
        return kdn_layer_norm_bwd(rows, D, io, at(dy), at(x), xs, fat(mean), fat(rstd), fat(w),
                                  at(dx), fat(dw), fat(db), at(ws), n, nullptr);
    }
};

#define WITH(T, expr) ([] { T c; expr; return c; }())

static void norm_checks()
{
    RUNS(Norm().fwd());
    RUNS(Norm().bwd());
    RUNS(WITH(Norm, (c.w = c.b = c.mean = c.rstd = 0)).fwd());
    RUNS(WITH(Norm, (c.dw = c.db = c.ws = 0)).bwd());
    RUNS(WITH(Norm, (c.rows = 0, c.x = c.y = 0)).fwd());
    RUNS(WITH(Norm, (c.xs = 1 << 20)).fwd());
    RUNS(WITH(Norm, (c.x += 2, c.y += 2)).fwd());
    BAD(WITH(Norm, c.io = 2).fwd(), KDN_ERR_INVALID_ARG, "io_dtype");
    BAD(WITH(Norm, c.io = 0x101).bwd(), KDN_ERR_INVALID_ARG, "io_dtype");
    BAD(WITH(Norm, c.rows = -1).fwd(), KDN_ERR_INVALID_ARG, "rows");
    BAD(WITH(Norm, c.D = 0).fwd(), KDN_ERR_INVALID_ARG, "D >= 1");
    BAD(WITH(Norm, (c.D = 1 << 21, c.xs = 1 << 21)).fwd(), KDN_ERR_UNSUPPORTED, "2^20");
    BAD(WITH(Norm, (c.rows = INT_MAX)).bwd(), KDN_ERR_UNSUPPORTED, "2^31");
    BAD(WITH(Norm, (c.rows = (1 << 30) + 1, c.D = 1, c.xs = 1)).fwd(), KDN_ERR_UNSUPPORTED, "2^30");
    BAD(WITH(Norm, c.eps = -1.f).fwd(), KDN_ERR_INVALID_ARG, "eps");
    BAD(WITH(Norm, c.eps = std::nanf("")).fwd(), KDN_ERR_INVALID_ARG, "eps");
    BAD(WITH(Norm, c.xs = 63).fwd(), KDN_ERR_INVALID_ARG, "x_stride");
    BAD(WITH(Norm, c.xs = -64).fwd(), KDN_ERR_INVALID_ARG, "x_stride");
    BAD(WITH(Norm, c.xs = LLONG_MAX).fwd(), KDN_ERR_UNSUPPORTED, "1073741824");
    BAD(WITH(Norm, c.x = 0).fwd(), KDN_ERR_INVALID_ARG, "x must not be NULL");
    BAD(WITH(Norm, c.y = 0).fwd(), KDN_ERR_INVALID_ARG, "y must not be NULL");
    BAD(WITH(Norm, c.mean = 0).bwd(), KDN_ERR_INVALID_ARG, "mean must not be NULL");
    BAD(WITH(Norm, c.x += 1).fwd(), KDN_ERR_INVALID_ARG, "x must be 2-byte aligned");
    BAD(WITH(Norm, (c.io = KDN_F32, c.x += 2)).fwd(), KDN_ERR_INVALID_ARG, "x must be 4-byte aligned");
    BAD(WITH(Norm, c.y = c.x + 128).fwd(), KDN_ERR_INVALID_ARG, "y must not overlap x");
    BAD(WITH(Norm, (c.xs = 640, c.y = c.x + 5 * 1280 + 128)).fwd(), KDN_ERR_INVALID_ARG, "overlap");
    BAD(WITH(Norm, c.dw = c.db + 4).bwd(), KDN_ERR_INVALID_ARG, "dweight must not overlap dbias");
    BAD(WITH(Norm, c.dx = c.dy).bwd(), KDN_ERR_INVALID_ARG, "dx must not overlap dy");
    BAD(WITH(Norm, c.ws = 0).bwd(), KDN_ERR_WORKSPACE, "workspace");
    BAD(WITH(Norm, c.ws_bytes = 64).bwd(), KDN_ERR_WORKSPACE, "workspace");
    BAD(WITH(Norm, c.ws += 4).bwd(), KDN_ERR_INVALID_ARG, "workspace must be 16-byte");
    BAD(WITH(Norm, c.ws = c.dy).bwd(), KDN_ERR_INVALID_ARG, "overlap");
    if (kdn_layer_norm_bwd_workspace_size(-1, 4) || kdn_layer_norm_bwd_workspace_size(INT_MAX, 1 << 20))
        ++failures, std::printf("FAILED norm workspace size of a bad shape\n");
}

struct Conv {
    int B = 2, T = 100, D = 64, W = 4, io = KDN_BF16, act = KDN_ACT_SILU, N = 0;
    long long xs = 64;
    uint64_t x = 1 * G, w = 2 * G, b = 3 * G, s0 = 4 * G, cu = 0, y = 5 * G, sT = 6 * G;
    uint64_t dy = 7 * G, dsT = 8 * G, dx = 9 * G, dw = 10 * G, db = 11 * G, ds0 = 12 * G, ws = 13 * G;
    long long ws_bytes = -1;
    kdn_status fwd() const
    {
        return kdn_conv_fwd(B, T, D, W, io, act, at(x), xs, fat(w), fat(b), at(s0), iat(cu), N,
                            at(y), at(sT), nullptr);
    }
    kdn_status bwd() const
    {
        const size_t n = ws_bytes < 0 ? kdn_conv_bwd_workspace_size(B, T, D, W) : (size_t)ws_bytes;
        return kdn_conv_bwd(B, T, D, W, io, act, at(dy), at(x), xs, fat(w), fat(b), at(s0), iat(cu),
                            N, at(dsT), at(dx), fat(dw), fat(db), at(ds0), at(ws), n, nullptr);
    }
    kdn_status step() const
    {
        return kdn_conv_step(B, D, W, io, act, at(x), xs, fat(w), fat(b), at(s0), at(y), nullptr);
    }
};

static void conv_checks()
{
    RUNS(Conv().fwd());
    RUNS(Conv().bwd());
    RUNS(Conv().step());
    RUNS(WITH(Conv, (c.b = c.s0 = c.sT = 0)).fwd());
    RUNS(WITH(Conv, (c.b = c.s0 = c.dsT = c.ds0 = c.db = 0)).bwd());
    RUNS(WITH(Conv, (c.T = 0, c.x = c.y = 0)).fwd());
    RUNS(WITH(Conv, (c.B = 1, c.cu = 14 * G, c.N = 5)).fwd());
    BAD(WITH(Conv, (c.cu = 14 * G, c.N = 5)).fwd(), KDN_ERR_INVALID_ARG, "B = 1");
    BAD(WITH(Conv, (c.B = 1, c.cu = 14 * G, c.N = 0)).bwd(), KDN_ERR_INVALID_ARG, "N >= 1");
    BAD(WITH(Conv, (c.B = 1, c.cu = 14 * G, c.N = INT_MAX)).fwd(), KDN_ERR_UNSUPPORTED, "2^31");
    BAD(WITH(Conv, (c.B = 1, c.cu = 14 * G, c.D = 1, c.xs = 1, c.N = 1 << 30)).fwd(), KDN_ERR_UNSUPPORTED, "2^31");
    BAD(WITH(Conv, (c.B = 1, c.cu = 14 * G + 2, c.N = 2)).fwd(), KDN_ERR_INVALID_ARG, "cu_seqlens must be 4-byte");
    BAD(WITH(Conv, c.W = 1).fwd(), KDN_ERR_UNSUPPORTED, "taps");
    BAD(WITH(Conv, c.W = 5).bwd(), KDN_ERR_UNSUPPORTED, "taps");
    BAD(WITH(Conv, c.W = -1).step(), KDN_ERR_UNSUPPORTED, "taps");
    BAD(WITH(Conv, c.act = 2).fwd(), KDN_ERR_INVALID_ARG, "activation");
    BAD(WITH(Conv, c.B = 0).fwd(), KDN_ERR_INVALID_ARG, "B >= 1");
    BAD(WITH(Conv, c.T = -1).fwd(), KDN_ERR_INVALID_ARG, "T >= 0");
    BAD(WITH(Conv, (c.B = INT_MAX, c.T = INT_MAX)).fwd(), KDN_ERR_UNSUPPORTED, "2^31");
    BAD(WITH(Conv, (c.B = INT_MAX)).step(), KDN_ERR_UNSUPPORTED, "2^31");
    BAD(WITH(Conv, c.w = 0).fwd(), KDN_ERR_INVALID_ARG, "weight must not be NULL");
    BAD(WITH(Conv, c.dw = 0).bwd(), KDN_ERR_INVALID_ARG, "dweight must not be NULL");
    BAD(WITH(Conv, c.s0 = 0).step(), KDN_ERR_INVALID_ARG, "state must not be NULL");
    BAD(WITH(Conv, c.sT = c.s0).fwd(), KDN_ERR_INVALID_ARG, "state_T must not overlap state0");
    BAD(WITH(Conv, c.y = c.x).step(), KDN_ERR_INVALID_ARG, "y must not overlap x");
    BAD(WITH(Conv, c.y = c.s0 + 64).step(), KDN_ERR_INVALID_ARG, "overlap");
    BAD(WITH(Conv, c.ds0 = c.dsT).bwd(), KDN_ERR_INVALID_ARG, "dstate0 must not overlap dstate_T");
    BAD(WITH(Conv, c.ws_bytes = 16).bwd(), KDN_ERR_WORKSPACE, "workspace");
    if (kdn_conv_bwd_workspace_size(1, 10, 8, 5) || kdn_conv_bwd_workspace_size(INT_MAX, INT_MAX, 1, 4))
        ++failures, std::printf("FAILED conv workspace size of a bad shape\n");
}

struct Rec {
    int B = 2, T = 300, D = 64, io = KDN_BF16, gate = KDN_GATE_PREACT, blend = 1, N = 0;
    long long xs = 64, as = 64;
    uint64_t x = 1 * G, a = 2 * G, h0 = 3 * G, cu = 0, h = 4 * G, hT = 5 * G, chk = 6 * G, ws = 7 * G;
    uint64_t dh = 8 * G, dhT = 9 * G, dx = 10 * G, da = 11 * G, dh0 = 12 * G;
    long long ws_bytes = -1;
    size_t bytes(size_t n) const { return ws_bytes < 0 ? n : (size_t)ws_bytes; }
    kdn_status fwd() const
    {
        return kdn_rec_fwd(B, T, D, io, gate, blend, at(x), xs, at(a), as, fat(h0), iat(cu), N,
                           at(h), fat(hT), fat(chk), at(ws), bytes(kdn_rec_fwd_workspace_size(B, T, D)),
                           nullptr);
    }
    kdn_status bwd() const
    {
        return kdn_rec_bwd(B, T, D, io, gate, blend, at(dh), at(x), xs, at(a), as, fat(chk),
                           fat(h0), iat(cu), N, fat(dhT), at(dx), at(da), fat(dh0), at(ws),
                           bytes(kdn_rec_bwd_workspace_size(B, T, D)), nullptr);
    }
    kdn_status step() const
    {
        return kdn_rec_step(B, D, io, gate, blend, at(x), xs, at(a), as, fat(hT), at(h), nullptr);
    }
};

static void rec_checks()
{
    RUNS(Rec().fwd());
    RUNS(Rec().bwd());
    RUNS(Rec().step());
    RUNS(WITH(Rec, (c.h0 = c.hT = c.chk = 0)).fwd());
    RUNS(WITH(Rec, (c.h0 = c.dhT = c.dh0 = 0)).bwd());
    RUNS(WITH(Rec, (c.T = 0, c.x = c.a = c.h = c.chk = c.ws = 0)).fwd());
    RUNS(WITH(Rec, (c.T = 0, c.x = c.a = c.dh = c.dx = c.da = c.chk = c.ws = 0)).bwd());
    RUNS(WITH(Rec, (c.T = 100, c.ws = 0)).fwd());
    RUNS(WITH(Rec, (c.B = 1, c.cu = 14 * G, c.N = 5)).bwd());
    RUNS(WITH(Rec, (c.x = c.a)).fwd());  // inputs may be the same
    BAD(WITH(Rec, c.gate = 2).fwd(), KDN_ERR_INVALID_ARG, "gate");
    BAD(WITH(Rec, c.blend = 2).bwd(), KDN_ERR_INVALID_ARG, "blend");
    BAD(WITH(Rec, c.io = -1).step(), KDN_ERR_INVALID_ARG, "io_dtype");
    BAD(WITH(Rec, (c.cu = 14 * G, c.N = 1)).bwd(), KDN_ERR_INVALID_ARG, "B = 1");
    BAD(WITH(Rec, (c.B = 1, c.cu = 14 * G, c.N = -4)).fwd(), KDN_ERR_INVALID_ARG, "N >= 1");
    BAD(WITH(Rec, c.as = 1).fwd(), KDN_ERR_INVALID_ARG, "a_stride");
    BAD(WITH(Rec, c.xs = 1).step(), KDN_ERR_INVALID_ARG, "x_stride");
    BAD(WITH(Rec, c.as = (1 << 22) + 1).bwd(), KDN_ERR_UNSUPPORTED, "a_stride is at most 4194304");
    RUNS(WITH(Rec, (c.as = c.xs = (1 << 22) + 1)).step());
    RUNS(WITH(Rec, (c.as = c.xs = 1 << 22)).fwd());
    BAD(WITH(Rec, (c.gate = KDN_GATE_ALPHA, c.a += 2)).fwd(), KDN_ERR_INVALID_ARG, "a must be 4-byte");
    RUNS(WITH(Rec, (c.a += 2)).fwd());
    BAD(WITH(Rec, c.chk = 0).bwd(), KDN_ERR_INVALID_ARG, "checkpoints must not be NULL");
    BAD(WITH(Rec, c.hT = 0).step(), KDN_ERR_INVALID_ARG, "state must not be NULL");
    BAD(WITH(Rec, c.hT = c.h0).fwd(), KDN_ERR_INVALID_ARG, "h_T must not overlap h0");
    BAD(WITH(Rec, c.h = c.x).fwd(), KDN_ERR_INVALID_ARG, "h must not overlap x");
    BAD(WITH(Rec, c.dx = c.dh).bwd(), KDN_ERR_INVALID_ARG, "dx must not overlap dh");
    BAD(WITH(Rec, c.dh0 = c.dhT).bwd(), KDN_ERR_INVALID_ARG, "dh0 must not overlap dh_T");
    BAD(WITH(Rec, c.h = c.hT).step(), KDN_ERR_INVALID_ARG, "overlap");
    BAD(WITH(Rec, c.ws = 0).fwd(), KDN_ERR_WORKSPACE, "workspace");
    BAD(WITH(Rec, c.ws_bytes = 1).bwd(), KDN_ERR_WORKSPACE, "workspace");
    BAD(WITH(Rec, c.ws = c.chk).bwd(), KDN_ERR_INVALID_ARG, "overlap");
    BAD(WITH(Rec, (c.B = 1 << 23, c.T = 2, c.D = 64)).bwd(), KDN_ERR_UNSUPPORTED, "too many short rows");
    BAD(WITH(Rec, (c.B = 1 << 24, c.T = 1, c.D = 1, c.xs = c.as = 1)).step(), KDN_ERR_UNSUPPORTED, "2^24");
    BAD(WITH(Rec, (c.B = 1, c.T = (1 << 30) + 1, c.D = 1, c.xs = c.as = 1)).fwd(), KDN_ERR_UNSUPPORTED, "2^30");
    BAD(WITH(Rec, (c.T = INT_MAX)).fwd(), KDN_ERR_UNSUPPORTED, "2^31");
    if (kdn_rec_fwd_workspace_size(1, 10, 0) || kdn_rec_bwd_workspace_size(INT_MAX, INT_MAX, 4))
        ++failures, std::printf("FAILED rec workspace size of a bad shape\n");
}

int main()
{
    norm_checks();
    conv_checks();
    rec_checks();
    if (failures)
        return 1;
    std::printf("all checks passed\n");
    return 0;
}
