// The layer norm's forward on rows of 16-bit types that start anywhere.
#include "norm_fwd.cuh"

namespace bl {

namespace norm {

cudaError_t layer_fwd_odd(int dtype, const LayerNormFwd& a, cudaStream_t st) {
  if (dtype > 1) return cudaErrorNotSupported;       // fp32
  const int fmt = a.codes ? a.fmt : 0;
  auto launch = [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    return fmt == 0          ? fwd_ring<T, 0, true, true, true>(a, st)
           : fmt == kFmtInt8 ? fwd_ring<T, kFmtInt8, true, true, true>(a, st)
                             : fwd_ring<T, kFmtE4m3, true, true, true>(a, st);
  };
  return dtype == 0 ? launch((__nv_bfloat16*)nullptr) : launch((__half*)nullptr);
}

}  // namespace norm

}  // namespace bl
