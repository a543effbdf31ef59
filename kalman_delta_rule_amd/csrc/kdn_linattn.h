// kdn_linattn.h -- argument blocks and launchers of linear attention with a decay for
// each head.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace kdn {

// q, k, v or a gradient: token t of head h at p + t ts + (h / div) hs elements
struct LinTensor {
    const void* p;
    long long ts;
    int hs, div;
};

struct LinCall {
    int B, T, H, Hk, dk, dv, N;
    float scale;
    LinTensor q, k, v;
    const float* decay;  // [H]
    const float* S0;     // nullable [N,H,dk,dv]
    const int* cu;       // nullable [N+1]
    bool clear;          // zeros behind the last sequence
    void* o;             // [B,T,H,dv]
    float* S_T;          // nullable
    // backward
    LinTensor d_o;
    const float* dS_T;  // nullable
    void* dq;
    void* dk_out;
    void* dv_out;
    float* dS0;  // nullable
    void* ws;
};
size_t linattn_fwd_workspace_bytes(int B, int T, int H, int dk, int dv);
size_t linattn_bwd_workspace_bytes(int B, int T, int H, int Hk, int dk, int dv);
hipError_t launch_linattn_fwd(const LinCall& c, bool bf, hipStream_t stream);
hipError_t launch_linattn_bwd(const LinCall& c, bool bf, hipStream_t stream);

// One walk over the tokens (kdn_linattn.hip says which there are)
struct LinRole {
    LinTensor q, k, v;
    void* out;  // [B,T,H,vd]
    bool out_f32;
    const float* X0;  // nullable; element (i, j) of a state at i rs + j cs
    float* XT;        // nullable
    float* seg;       // [B,S,H] states handed from segment to segment
    int4* spans;      // [B,S] the tokens they are of, and the sequence if it begins there (or -1)
    int srs, scs;     // strides of an element in seg
    int kd, vd, rs, cs, rev;
    bool exact;  // its state is an fp32 output
    float of_p, of_x, of_u;
};
struct LinArgs {
    int B, T, H, N;
    const int* cu;
    const float* decay;
    bool clear;
    int S, L;  // segments of each row, and their tokens
    int parts, tokens;  // of a segment that go to a workgroup each, by where sequences begin; tokens of one
    int roles, slices;  // walks of a launch, and the most slices that one has
    bool odd;  // rows of some input begin in the middle of a word
    LinRole role[3];
};

// sums over the heads of a group
struct LinSums {
    const float* x[2];
    void* y[2];
};

struct LinStepArgs {
    int B, H, G, dk, dv;
    float scale;
    const void* q;
    long long qs, qh;  // elements between rows, between heads
    const void* k;
    long long ks, kh;
    const void* v;
    long long vs, vh;
    const float* decay;
    float* S;
    void* o;
};
hipError_t launch_linattn_step(const LinStepArgs& a, bool bf, hipStream_t stream);

}  // namespace kdn
