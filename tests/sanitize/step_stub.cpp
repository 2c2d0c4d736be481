// Host-only stand-ins for the launchers of the serving operators around a step's attention: calls that reach a
// launch report success.
#include "serve_step_kernels.h"

namespace wq {
hipError_t launch_norm_rope(const NormRopeProblem&, hipStream_t) { return hipSuccess; }
hipError_t launch_layout(const LayoutProblem&, hipStream_t) { return hipSuccess; }
hipError_t launch_prefix(const PrefixProblem&, const PrefixPlan&, float, void*, hipStream_t) { return hipSuccess; }
hipError_t launch_verify(const VerifyProblem&, const VerifyPlan&, void*, hipStream_t) { return hipSuccess; }
}  // namespace wq
