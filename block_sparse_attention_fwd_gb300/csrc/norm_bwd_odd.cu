// The backward's ring kernel on rows that start anywhere.
#include "norm_bwd.cuh"

namespace bl {

namespace norm {

cudaError_t bwd_odd(int dtype, const NormBwd& a, int* blocks, cudaStream_t st) {
  if (dtype == 2) return a.codes ? cudaErrorNotSupported : bwd_ring<float, 0, true, false>(a, blocks, st);
  auto launch = [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    return !a.codes            ? bwd_ring<T, 0, true, false>(a, blocks, st)
           : a.fmt == kFmtInt8 ? bwd_ring<T, kFmtInt8, true, false>(a, blocks, st)
                               : bwd_ring<T, kFmtE4m3, true, false>(a, blocks, st);
  };
  return dtype == 0 ? launch((__nv_bfloat16*)nullptr) : launch((__half*)nullptr);
}

}  // namespace norm

}  // namespace bl
