// Backward of the layer norm (norm.cuh).
#include "norm_bwd.cuh"

namespace bl {

int layer_norm_bwd_parts(int64_t rows, int64_t cols) { return bwd_parts_of<true>(rows, cols); }

cudaError_t launch_layer_norm_bwd(int dtype, const NormBwd& a, void* g_w, void* g_b,
                                  cudaStream_t st) {
  return launch_bwd_of<true>(dtype, a, g_w, g_b, st);
}

}  // namespace bl
