// k_ffn_input_grad.cu -- the ring's kernels of the gradient of a product's input: rows of dz run along the summed axis,
// the weight is stored summed axis first.
#include "ffn_ring.cuh"

namespace gp {

cudaError_t launch_ffn_input_grad(FfnProduct& p, const void** kernel) { return launch_tile<false, false, true>(p, kernel); }

}  // namespace gp
