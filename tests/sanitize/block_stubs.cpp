// Stand-ins for the launchers of the operators around the mixer, for the
// host-only sanitizer build (see launch_stubs.cpp).
#include <hip/hip_runtime.h>

#include "kdn_block.h"

extern int g_launches;

static hipError_t reached()
{
    ++g_launches;
    return hipErrorNotSupported;
}

namespace kdn {
int norm_bwd_groups(int rows, int) { return rows < 512 ? rows : 512; }
hipError_t launch_norm_fwd(const NormArgs&, bool, hipStream_t) { return reached(); }
hipError_t launch_norm_bwd(const NormArgs&, bool, hipStream_t) { return reached(); }
int conv_bwd_groups(int B, int T, int) { return B * (T / 64 + 1); }
hipError_t launch_conv_fwd(const ConvArgs&, bool, hipStream_t) { return reached(); }
hipError_t launch_conv_bwd(const ConvArgs&, bool, hipStream_t) { return reached(); }
hipError_t launch_conv_step(const ConvArgs&, bool, hipStream_t) { return reached(); }
size_t rec_workspace_bytes(int, int T, int, bool) { return T > 256 ? 4096 : 0; }
unsigned long long rec_threads(int B, int T, int D, bool)
{
    return 256ull * B * (T / 128 + 1) * (D / 64 + 1);
}
hipError_t launch_rec_fwd(const RecArgs&, bool, hipStream_t) { return reached(); }
hipError_t launch_rec_bwd(const RecArgs&, bool, hipStream_t) { return reached(); }
hipError_t launch_rec_step(const RecArgs&, bool, hipStream_t) { return reached(); }
}  // namespace kdn
