// k_ffn_weight_grad.cu -- the ring's kernels of the gradient of a product's weight: both operands are stored summed axis
// (tokens) first.
#include "ffn_ring.cuh"

namespace gp {

cudaError_t launch_ffn_weight_grad(FfnProduct& p, const void** kernel) { return launch_tile<false, true, true>(p, kernel); }

}  // namespace gp
