// kdn_layer_ops.h -- argument blocks and launchers of group norm and dropout.  Not part
// of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kdn {

struct GroupNormArgs {
    int N, S, C, G;
    bool silu;
    float eps;
    const void* x;
    long long xs;         // elements from one position of x to the next
    const float* weight;  // nullable [C]
    const float* bias;    // nullable [C]
    void* y;
    float* mean;  // forward: nullable; backward: read; [N,G]
    float* rstd;
    // backward
    const void* dy;
    void* dx;
    float* dweight;  // nullable
    float* dbias;    // nullable
    void* ws;
};
size_t group_norm_fwd_workspace_bytes(int N, int S, int C, int G);
size_t group_norm_bwd_workspace_bytes(int N, int S, int C, int G);
hipError_t launch_group_norm_fwd(const GroupNormArgs& a, bool bf, hipStream_t stream);
hipError_t launch_group_norm_bwd(const GroupNormArgs& a, bool bf, hipStream_t stream);

struct DropoutArgs {
    int rows, D;
    uint32_t least;  // of an element's 16 bits, where it is kept
    float scale;     // 65536 / (65536 - least)
    uint64_t seed, offset;
    const long long* state;  // nullable: {seed, offset} on the device
    const void* x;
    long long xs;
    const void* residual;  // nullable
    void* y;
};
hipError_t launch_dropout(const DropoutArgs& a, bool bf, hipStream_t stream);

}  // namespace kdn
