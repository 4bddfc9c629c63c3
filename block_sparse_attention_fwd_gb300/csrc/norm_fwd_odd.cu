// The forward's ring kernel on rows of 16-bit types that start anywhere.
#include "norm_fwd.cuh"

namespace bl {

namespace norm {

cudaError_t fwd_odd(int dtype, bool norm, const NormFwd& a, cudaStream_t st) {
  if (dtype > 1) return cudaErrorNotSupported;       // fp32
  const int fmt = a.codes ? a.fmt : 0;
  auto launch = [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    if (!norm)
      return fmt == kFmtInt8 ? fwd_ring<T, kFmtInt8, false, true, false>(a, st)
                             : fwd_ring<T, kFmtE4m3, false, true, false>(a, st);
    return fmt == 0          ? fwd_ring<T, 0, true, true, false>(a, st)
           : fmt == kFmtInt8 ? fwd_ring<T, kFmtInt8, true, true, false>(a, st)
                             : fwd_ring<T, kFmtE4m3, true, true, false>(a, st);
  };
  return dtype == 0 ? launch((__nv_bfloat16*)nullptr) : launch((__half*)nullptr);
}

}  // namespace norm

}  // namespace bl
