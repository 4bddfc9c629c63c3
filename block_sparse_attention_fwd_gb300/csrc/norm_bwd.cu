// Backward of the root-mean-square norm (norm.cuh).
#include "norm_bwd.cuh"

namespace bl {

int norm_bwd_parts(int64_t rows, int64_t cols) { return bwd_parts_of<false>(rows, cols); }

cudaError_t launch_norm_bwd(int dtype, const NormBwd& a, void* g_w, cudaStream_t st) {
  return launch_bwd_of<false>(dtype, a, g_w, nullptr, st);
}

}  // namespace bl
