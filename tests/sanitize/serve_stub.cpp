// Host-only stand-ins for the serving operators' launchers, so that their run entry points (serve_api.cpp),
// validation and planning link into a library without device code: calls that reach a launch report success.
#include "serve_kernels.h"

namespace wq {
hipError_t launch_lora(const LoraProblem&, const LoraPlan&, void*, hipStream_t) { return hipSuccess; }
hipError_t launch_rope(const RopeProblem&, hipStream_t) { return hipSuccess; }
hipError_t launch_tree(const TreeProblem&, const TreePlan&, float, void*, hipStream_t) { return hipSuccess; }
}  // namespace wq
