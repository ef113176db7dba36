// k_ffn_linear.cu -- the ring's kernels of the forward product with its epilogue, and of the gradient of its input.
#include "ffn_ring.cuh"

namespace gp {

cudaError_t launch_ffn_linear(FfnProduct& p, const void** kernel) {
  return p.plan.cta_pair ? launch_ring<256, true, false, false, false>(p, kernel)
                         : launch_ring<128, false, false, false, false>(p, kernel);
}

// dz rows run along the summed axis; the weight is stored summed axis first.
cudaError_t launch_ffn_input_grad(FfnProduct& p, const void** kernel) {
  return p.plan.cta_pair ? launch_ring<256, true, false, false, true>(p, kernel)
                         : launch_ring<128, false, false, false, true>(p, kernel);
}

}  // namespace gp
