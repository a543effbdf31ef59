// kdn_block.h -- argument blocks and launchers of the operators around the
// mixer (layer norm, short convolution, gated recurrence).  Not part of the
// public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kdn {

struct NormArgs {
    int rows, D;
    float eps;
    const void* x;
    long long xs;         // elements from one row of x to the next
    const float* weight;  // nullable [D]
    const float* bias;    // nullable [D]
    void* y;
    float* mean;  // forward: nullable; backward: read
    float* rstd;
    // backward
    const void* dy;
    void* dx;
    float* dweight;  // nullable
    float* dbias;    // nullable
    float* ws;       // [norm_bwd_groups][2][D] partial sums
};
int norm_bwd_groups(int rows, int D);
hipError_t launch_norm_fwd(const NormArgs& a, bool bf, hipStream_t stream);
hipError_t launch_norm_bwd(const NormArgs& a, bool bf, hipStream_t stream);

struct ConvArgs {
    int B, T, D, W;
    bool silu;
    const void* x;
    long long xs;
    const float* weight;  // [W,D]
    const float* bias;    // nullable [D]
    const void* state0;   // nullable [N,W-1,D]
    const int* cu;        // nullable [N+1]
    int N;
    bool clear;  // zeros behind the last sequence, in y or dx
    void* y;
    void* state_T;  // nullable
    // backward
    const void* dy;
    const void* dstate_T;  // nullable
    void* dx;
    float* dweight;
    float* dbias;   // nullable
    void* dstate0;  // nullable
    float* ws;      // [conv_bwd_groups][W+1][D] partial sums
};
int conv_bwd_groups(int B, int T, int D);
hipError_t launch_conv_fwd(const ConvArgs& a, bool bf, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvArgs& a, bool bf, hipStream_t stream);
hipError_t launch_conv_step(const ConvArgs& a, bool bf, hipStream_t stream);

struct RecArgs {
    int B, T, D;
    bool preact, blend;
    const void* x;
    long long xs;
    const void* a;
    long long as;
    const float* h0;  // nullable [N,D]
    const int* cu;    // nullable [N+1]
    int N;
    bool clear;  // zeros behind the last sequence, in h and ckpt or dx and da
    void* h;
    float* h_T;   // nullable [N,D]; step: the state, in place
    float* ckpt;  // [B, ceil(T / 64), D]; forward: nullable, written; backward: read
    // backward
    const void* dh;
    const float* dh_T;  // nullable [N,D]
    void* dx;
    void* da;
    float* dh0;  // nullable [N,D]
    void* ws;
};
size_t rec_workspace_bytes(int B, int T, int D, bool backward);
unsigned long long rec_threads(int B, int T, int D, bool backward);  // of its largest launch
hipError_t launch_rec_fwd(const RecArgs& a, bool bf, hipStream_t stream);
hipError_t launch_rec_bwd(const RecArgs& a, bool bf, hipStream_t stream);
hipError_t launch_rec_step(const RecArgs& a, bool bf, hipStream_t stream);

}  // namespace kdn
