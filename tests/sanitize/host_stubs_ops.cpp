// Host-only stand-ins for the operators' kernel launchers, as host_stubs.cpp has for the GEMMs':
// every launch reports an error.
#include "ops_internal.h"

namespace tefp8 {
hipError_t launch_rmsnorm_fwd(const NormFwdArgs&, hipStream_t) { return hipErrorNoDevice; }
int64_t rmsnorm_bwd_blocks(int64_t rows, int64_t) { return rows < 1024 ? rows : 1024; }
hipError_t launch_rmsnorm_bwd(const NormBwdArgs&, hipStream_t) { return hipErrorNoDevice; }
int64_t router_fwd_blocks(int64_t tokens, int64_t, bool) { return tokens < 1024 ? 1 : 1024; }
int64_t router_fwd_workspace_bytes(int64_t tokens, int64_t experts) { return tokens < 1024 ? 0 : 8 * 1024 * (experts + 2); }
hipError_t launch_router_fwd(const RouterArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_router_bwd(const RouterBwdArgs&, hipStream_t) { return hipErrorNoDevice; }
int64_t clip_chunks(int64_t n) { return (n + 8191) / 8192; }
int64_t clip_blocks(const ClipBatch& b) { return b.chunks < 1 ? 1 : b.chunks < kClipBlocks ? b.chunks : kClipBlocks; }
int64_t clip_workspace_bytes() { return kClipBlocks * 8; }
hipError_t launch_grad_sumsq(const ClipBatch&, double*, int64_t, bool, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_grad_scale(const ClipBatch&, const double*, int64_t, float, float*, bool, hipStream_t) { return hipErrorNoDevice; }
}  // namespace tefp8
