// Forward of the layer norm (norm.cuh).
#include "norm_fwd.cuh"

namespace bl {

cudaError_t launch_layer_norm_fwd(int dtype, const LayerNormFwd& a, cudaStream_t st) {
  return launch_fwd_of<true>(dtype, a, st);
}

}  // namespace bl
