// The gated feed-forward's backward kernels on tiles (gated.cuh); a file of their own, because they compile as long as the
// forward's.
#include "gated.cuh"

namespace fp8lin {

int launch_gated_bwd(const GatedArgs& g, const Ctx& c) { return launch_gated_epi<kGateBwd>(g, c); }

}  // namespace fp8lin
