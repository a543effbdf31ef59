// Stand-ins for the launchers of linear attention, group norm and dropout, for the
// host-only sanitizer build (see launch_stubs.cpp).
#include <hip/hip_runtime.h>

#include "kdn_layer_ops.h"
#include "kdn_linattn.h"

extern int g_launches;

static hipError_t reached()
{
    ++g_launches;
    return hipErrorNotSupported;
}

namespace kdn {
size_t linattn_fwd_workspace_bytes(int, int T, int, int, int) { return T > 1024 ? 4096 : 0; }
size_t linattn_bwd_workspace_bytes(int, int T, int H, int Hk, int, int) { return (T > 1024 ? 4096 : 0) + (H > Hk ? 4096 : 0); }
hipError_t launch_linattn_fwd(const LinCall&, bool, hipStream_t) { return reached(); }
hipError_t launch_linattn_bwd(const LinCall&, bool, hipStream_t) { return reached(); }
hipError_t launch_linattn_step(const LinStepArgs&, bool, hipStream_t) { return reached(); }
size_t group_norm_fwd_workspace_bytes(int, int S, int, int) { return S > 4096 ? 4096 : 0; }
size_t group_norm_bwd_workspace_bytes(int, int, int, int) { return 4096; }
hipError_t launch_group_norm_fwd(const GroupNormArgs&, bool, hipStream_t) { return reached(); }
hipError_t launch_group_norm_bwd(const GroupNormArgs&, bool, hipStream_t) { return reached(); }
hipError_t launch_dropout(const DropoutArgs&, bool, hipStream_t) { return reached(); }
}  // namespace kdn
