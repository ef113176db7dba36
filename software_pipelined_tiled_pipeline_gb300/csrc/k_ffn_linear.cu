// k_ffn_linear.cu -- the ring's kernels of the forward product with its epilogue.
#include "ffn_ring.cuh"

namespace gp {

cudaError_t launch_ffn_linear(FfnProduct& p, const void** kernel) { return launch_tile<false, false, false>(p, kernel); }

}  // namespace gp
