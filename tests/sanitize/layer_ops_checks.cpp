// The host code of linear attention, group norm and dropout (validation, overlap rules,
// sizes) driven through every entry point with stand-in device addresses, built with the
// address and undefined-behaviour sanitizers.  Exits nonzero after a failed expectation.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "kdn.h"

extern int g_launches;

static int failures = 0;

static void* at(uint64_t a) { return reinterpret_cast<void*>(a); }
static float* fat(uint64_t a) { return reinterpret_cast<float*>(a); }
static const int* iat(uint64_t a) { return reinterpret_cast<const int*>(a); }
static const long long* lat(uint64_t a) { return reinterpret_cast<const long long*>(a); }

// A call must end with `code`, say `needle`, and launch only where it got past
// validation (KDN_ERR_HIP from the stand-ins).
static void expect(int line, kdn_status st, kdn_status code, const char* needle)
{
    static int seen = 0;
    const bool launched = g_launches != seen;
    seen = g_launches;
    if (st != code || !std::strstr(kdn_last_error_message(), needle) || launched != (code == KDN_ERR_HIP)) {
        std::printf("FAILED line %d: status %d, launched %d, last error: %s\n", line, (int)st, (int)launched,
                    kdn_last_error_message());
        ++failures;
    }
}
#define BAD(call, code, needle) expect(__LINE__, (call), (code), (needle))
#define RUNS(call) expect(__LINE__, (call), KDN_ERR_HIP, "launch stand-in")
#define WITH(T, expr) ([] { T c; expr; return c; }())

static const uint64_t G = 1ull << 36;  // far enough apart for any size below

struct Lin {
    int B = 2, T = 100, H = 4, Hk = 2, dk = 32, dv = 48, io = KDN_BF16, N = 0;
    float scale = 0.5f;
    long long qs = 64, qh = 32, ks = 64, kh = 32, vs = 192, vh = 48;
    uint64_t q = 1 * G, k = 2 * G, v = 3 * G, decay = 4 * G, S0 = 5 * G, cu = 0, o = 6 * G, S_T = 7 * G, ws = 8 * G;
    uint64_t d_o = 9 * G, dS = 10 * G, dq = 11 * G, dk_ = 12 * G, dv_ = 13 * G, dS0 = 14 * G;
    long long ws_bytes = -1;
    kdn_status fwd() const
    {
        const size_t n = ws_bytes < 0 ? kdn_linattn_fwd_workspace_size(B, T, H, dk, dv) : (size_t)ws_bytes;
        return kdn_linattn_fwd(B, T, H, Hk, dk, dv, io, scale, at(q), qs, qh, at(k), ks, kh, at(v), vs, vh, fat(decay),
                               fat(S0), iat(cu), N, at(o), fat(S_T), at(ws), n, nullptr);
    }
    kdn_status bwd() const
    {
        const size_t n = ws_bytes < 0 ? kdn_linattn_bwd_workspace_size(B, T, H, Hk, dk, dv) : (size_t)ws_bytes;
        return kdn_linattn_bwd(B, T, H, Hk, dk, dv, io, scale, at(d_o), at(q), qs, qh, at(k), ks, kh, at(v), vs, vh,
                               fat(decay), fat(S0), iat(cu), N, fat(dS), at(dq), at(dk_), at(dv_), fat(dS0), at(ws), n,
                               nullptr);
    }
    kdn_status step() const
    {
        return kdn_linattn_step(B, H, Hk, dk, dv, io, scale, at(q), qs, qh, at(k), ks, kh, at(v), vs, vh, fat(decay),
                                fat(S0), at(o), nullptr);
    }
};

static void linattn()
{
    RUNS(Lin().fwd());
    RUNS(Lin().bwd());
    RUNS(Lin().step());
    RUNS(WITH(Lin, c.T = 0).fwd());
    RUNS(WITH(Lin, (c.S0 = c.S_T = 0)).fwd());
    RUNS(WITH(Lin, (c.S0 = c.dS = c.dS0 = 0)).bwd());
    RUNS(WITH(Lin, (c.B = 1, c.cu = 15 * G, c.N = 3)).fwd());
    RUNS(WITH(Lin, (c.B = 1, c.cu = 15 * G, c.N = 3, c.io = KDN_F32 | KDN_CLEAR_TAIL)).bwd());
    RUNS(WITH(Lin, (c.qs = 1 << 22, c.qh = 40)).fwd());
    RUNS(WITH(Lin, (c.Hk = c.H = 1, c.qh = c.kh = c.vh = -7)).fwd());  // one head has no head stride
    for (int i = 0; i < 3; ++i) {
        auto call = [i](const Lin& c) { return i == 0 ? c.fwd() : i == 1 ? c.bwd() : c.step(); };
        BAD(call(WITH(Lin, c.io = 7)), KDN_ERR_INVALID_ARG, "io_dtype");
        BAD(call(WITH(Lin, c.Hk = 3)), KDN_ERR_INVALID_ARG, "multiple of Hk");
        BAD(call(WITH(Lin, c.Hk = 0)), KDN_ERR_INVALID_ARG, "multiple of Hk");
        BAD(call(WITH(Lin, c.H = INT_MIN)), KDN_ERR_INVALID_ARG, "multiple of Hk");
        BAD(call(WITH(Lin, c.dk = 0)), KDN_ERR_INVALID_ARG, "dk >= 1");
        BAD(call(WITH(Lin, c.dv = 257)), KDN_ERR_UNSUPPORTED, "at most 256");
        BAD(call(WITH(Lin, c.scale = NAN)), KDN_ERR_INVALID_ARG, "scale");
        BAD(call(WITH(Lin, c.B = 0)), KDN_ERR_INVALID_ARG, "B >= 1");
        BAD(call(WITH(Lin, c.H = 8192)), KDN_ERR_UNSUPPORTED, "H is at most");
        BAD(call(WITH(Lin, (c.B = 1 << 23, c.T = 1))), KDN_ERR_UNSUPPORTED, "");
        BAD(call(WITH(Lin, c.qs = 63)), KDN_ERR_INVALID_ARG, "q_stride");
        BAD(call(WITH(Lin, c.kh = 31)), KDN_ERR_INVALID_ARG, "k_head_stride");
        BAD(call(WITH(Lin, c.vs = (1ll << 22) + 1)), KDN_ERR_UNSUPPORTED, "v_stride");
        BAD(call(WITH(Lin, c.vh = LLONG_MAX)), KDN_ERR_UNSUPPORTED, "v_head_stride");
        BAD(call(WITH(Lin, c.q = 0)), KDN_ERR_INVALID_ARG, "q must not be NULL");
        BAD(call(WITH(Lin, c.decay = 0)), KDN_ERR_INVALID_ARG, "decay must not be NULL");
        BAD(call(WITH(Lin, c.k += 1)), KDN_ERR_INVALID_ARG, "aligned");
    }
    BAD(WITH(Lin, c.B = INT_MAX).step(), KDN_ERR_UNSUPPORTED, "");
    BAD(WITH(Lin, c.T = -1).fwd(), KDN_ERR_INVALID_ARG, "T >= 0");
    BAD(WITH(Lin, c.T = INT_MAX).bwd(), KDN_ERR_UNSUPPORTED, "2^31");
    BAD(WITH(Lin, (c.B = 1, c.cu = 15 * G, c.N = INT_MAX)).fwd(), KDN_ERR_UNSUPPORTED, "2^31");
    BAD(WITH(Lin, (c.cu = 15 * G, c.N = 3)).fwd(), KDN_ERR_INVALID_ARG, "B = 1");
    BAD(WITH(Lin, (c.B = 1, c.cu = 15 * G)).bwd(), KDN_ERR_INVALID_ARG, "N >= 1");
    BAD(WITH(Lin, c.io = KDN_BF16 | KDN_CLEAR_TAIL).step(), KDN_ERR_INVALID_ARG, "io_dtype");
    BAD(WITH(Lin, c.o = c.v + 64).fwd(), KDN_ERR_INVALID_ARG, "o must not overlap v");
    BAD(WITH(Lin, c.S_T = c.S0).fwd(), KDN_ERR_INVALID_ARG, "S_T must not overlap S0");
    BAD(WITH(Lin, c.dq = c.dk_).bwd(), KDN_ERR_INVALID_ARG, "overlap");
    BAD(WITH(Lin, c.dv_ = c.d_o).bwd(), KDN_ERR_INVALID_ARG, "dv_out must not overlap d_o");
    BAD(WITH(Lin, c.S0 = 0).step(), KDN_ERR_INVALID_ARG, "state must not be NULL");
    BAD(WITH(Lin, c.o = c.S0).step(), KDN_ERR_INVALID_ARG, "overlap");
    BAD(WITH(Lin, (c.T = 5000, c.ws_bytes = 4095)).fwd(), KDN_ERR_WORKSPACE, "4096");
    BAD(WITH(Lin, (c.T = 5000, c.ws = 0)).bwd(), KDN_ERR_WORKSPACE, "8192");
    BAD(WITH(Lin, (c.T = 5000, c.ws += 8)).fwd(), KDN_ERR_INVALID_ARG, "16-byte");
    BAD(WITH(Lin, (c.T = 5000, c.ws = c.q)).bwd(), KDN_ERR_INVALID_ARG, "workspace must not overlap");
    if (kdn_linattn_fwd_workspace_size(0, 4096, 4, 32, 32) || kdn_linattn_bwd_workspace_size(1, 4096, 4, 3, 32, 32) ||
        kdn_linattn_fwd_workspace_size(1, INT_MAX, INT_MAX, 256, 256)) {
        std::printf("FAILED: workspace of a shape that is refused\n");
        ++failures;
    }
}

struct Norm {
    int N = 6, S = 10, C = 64, groups = 4, io = KDN_BF16, act = KDN_ACT_SILU;
    float eps = 1e-5f;
    long long xs = 64;
    uint64_t x = 1 * G, w = 2 * G, b = 3 * G, y = 4 * G, mean = 5 * G, rstd = 6 * G;
    uint64_t dy = 7 * G, dx = 8 * G, dw = 9 * G, db = 10 * G, ws = 11 * G;
    long long ws_bytes = -1;
    kdn_status fwd() const
    {
        const size_t n = ws_bytes < 0 ? kdn_group_norm_fwd_workspace_size(N, S, C, groups) : (size_t)ws_bytes;
        return kdn_group_norm_fwd(N, S, C, groups, io, act, eps, at(x), xs, fat(w), fat(b), at(y), fat(mean), fat(rstd),
                                  at(ws), n, nullptr);
    }
    kdn_status bwd() const
    {
        const size_t n = ws_bytes < 0 ? kdn_group_norm_bwd_workspace_size(N, S, C, groups) : (size_t)ws_bytes;
        return kdn_group_norm_bwd(N, S, C, groups, io, act, at(dy), at(x), xs, fat(mean), fat(rstd), fat(w), fat(b),
                                  at(dx), fat(dw), fat(db), at(ws), n, nullptr);
    }
};

static void group_norm()
{
    RUNS(Norm().fwd());
    RUNS(Norm().bwd());
    RUNS(WITH(Norm, c.N = 0).fwd());
    RUNS(WITH(Norm, (c.w = c.b = c.mean = c.rstd = 0)).fwd());
    RUNS(WITH(Norm, (c.w = c.b = c.dw = c.db = 0)).bwd());
    RUNS(WITH(Norm, c.xs = 1ll << 30).fwd());
    for (int i = 0; i < 2; ++i) {
        auto call = [i](const Norm& c) { return i == 0 ? c.fwd() : c.bwd(); };
        BAD(call(WITH(Norm, c.io = KDN_BF16 | KDN_CLEAR_TAIL)), KDN_ERR_INVALID_ARG, "io_dtype");
        BAD(call(WITH(Norm, c.act = 2)), KDN_ERR_INVALID_ARG, "activation");
        BAD(call(WITH(Norm, c.N = -1)), KDN_ERR_INVALID_ARG, "N >= 0");
        BAD(call(WITH(Norm, c.S = -1)), KDN_ERR_INVALID_ARG, "S >= 0");
        BAD(call(WITH(Norm, c.C = 0)), KDN_ERR_INVALID_ARG, "D >= 1");
        BAD(call(WITH(Norm, c.C = INT_MAX)), KDN_ERR_UNSUPPORTED, "2^20");
        BAD(call(WITH(Norm, c.groups = 3)), KDN_ERR_INVALID_ARG, "multiple of G");
        BAD(call(WITH(Norm, c.groups = 0)), KDN_ERR_INVALID_ARG, "multiple of G");
        BAD(call(WITH(Norm, (c.N = c.S = INT_MAX))), KDN_ERR_UNSUPPORTED, "2^31");
        BAD(call(WITH(Norm, (c.N = 1 << 23, c.S = 1, c.C = c.groups = 4, c.xs = 4))), KDN_ERR_UNSUPPORTED, "2^24");
        BAD(call(WITH(Norm, c.xs = 63)), KDN_ERR_INVALID_ARG, "x_stride");
        BAD(call(WITH(Norm, c.x = 0)), KDN_ERR_INVALID_ARG, "x must not be NULL");
        BAD(call(WITH(Norm, c.w += 2)), KDN_ERR_INVALID_ARG, "aligned");
    }
    BAD(WITH(Norm, c.eps = -1.f).fwd(), KDN_ERR_INVALID_ARG, "eps");
    BAD(WITH(Norm, c.y = c.x).fwd(), KDN_ERR_INVALID_ARG, "y must not overlap x");
    BAD(WITH(Norm, c.rstd = c.mean).fwd(), KDN_ERR_INVALID_ARG, "overlap");
    BAD(WITH(Norm, c.mean = 0).bwd(), KDN_ERR_INVALID_ARG, "mean must not be NULL");
    BAD(WITH(Norm, c.dx = c.dy).bwd(), KDN_ERR_INVALID_ARG, "dx must not overlap dy");
    BAD(WITH(Norm, (c.S = 5000, c.ws_bytes = 100)).fwd(), KDN_ERR_WORKSPACE, "4096");
    BAD(WITH(Norm, c.ws = 0).bwd(), KDN_ERR_WORKSPACE, "4096");
}

struct Drop {
    int rows = 10, D = 33, io = KDN_BF16;
    double p = 0.1;
    long long xs = 40;
    uint64_t x = 1 * G, res = 2 * G, y = 3 * G, state = 0;
    kdn_status fwd() const
    {
        return kdn_dropout_fwd(rows, D, io, p, ULLONG_MAX, 1, lat(state), at(x), xs, at(res), at(y), nullptr);
    }
    kdn_status bwd() const { return kdn_dropout_bwd(rows, D, io, p, 0, 0, lat(state), at(x), at(y), nullptr); }
};

static void dropout()
{
    RUNS(Drop().fwd());
    RUNS(Drop().bwd());
    RUNS(WITH(Drop, (c.res = 0, c.p = 1.0, c.state = 4 * G)).fwd());
    RUNS(WITH(Drop, (c.rows = 0, c.x = c.y = 0)).bwd());
    for (int i = 0; i < 2; ++i) {
        auto call = [i](const Drop& c) { return i == 0 ? c.fwd() : c.bwd(); };
        BAD(call(WITH(Drop, c.io = 2)), KDN_ERR_INVALID_ARG, "io_dtype");
        BAD(call(WITH(Drop, c.rows = -1)), KDN_ERR_INVALID_ARG, "rows >= 0");
        BAD(call(WITH(Drop, c.D = 0)), KDN_ERR_INVALID_ARG, "D >= 1");
        BAD(call(WITH(Drop, (c.rows = INT_MAX, c.D = 2))), KDN_ERR_UNSUPPORTED, "2^31");
        BAD(call(WITH(Drop, c.p = -0.01)), KDN_ERR_INVALID_ARG, "p must be");
        BAD(call(WITH(Drop, c.p = 1.01)), KDN_ERR_INVALID_ARG, "p must be");
        BAD(call(WITH(Drop, c.p = NAN)), KDN_ERR_INVALID_ARG, "p must be");
        BAD(call(WITH(Drop, c.state = 4 * G + 4)), KDN_ERR_INVALID_ARG, "seed_offset must be 8-byte");
        BAD(call(WITH(Drop, c.y = c.x + 2)), KDN_ERR_INVALID_ARG, "overlap");
        BAD(call(WITH(Drop, c.y = 0)), KDN_ERR_INVALID_ARG, "NULL");
    }
    BAD(WITH(Drop, c.xs = 32).fwd(), KDN_ERR_INVALID_ARG, "x_stride");
    BAD(WITH(Drop, c.y = c.res).fwd(), KDN_ERR_INVALID_ARG, "y must not overlap residual");
}

int main()
{
    linattn();
    group_norm();
    dropout();
    if (!failures)
        std::printf("all checks passed\n");
    return failures != 0;
}
