// The gated feed-forward's forward kernels on tiles (gated.cuh), and the choice among its kernels.
#include "gated.cuh"

namespace fp8lin {

int launch_gated_bwd(const GatedArgs& g, const Ctx& c);  // gated_bwd.cu

int launch_gated(const GatedArgs& g, const Ctx& c) {
  if (g.backward) return launch_gated_bwd(g, c);
  if (g.a_dtype != FP8_DT_BF16 && g.M <= kFewRows) return launch_few_gated(g, c);
  return launch_gated_epi<kGate>(g, c);
}

}  // namespace fp8lin
