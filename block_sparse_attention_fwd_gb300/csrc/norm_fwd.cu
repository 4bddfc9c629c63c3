// Forward of the root-mean-square norm (norm.cuh) and row-wise saving in 8 bits.
#include "norm_fwd.cuh"

namespace bl {

cudaError_t launch_norm_fwd(int dtype, const NormFwd& a, cudaStream_t st) {
  return launch_fwd_of<false>(dtype, a, st);
}

cudaError_t launch_row_save(int dtype, const ActSave& s, cudaStream_t st) {
  if (s.cols > 16384) return cudaErrorNotSupported;
  NormFwd a{};
  a.rows = s.rows; a.cols = s.cols; a.x_stride = s.x_stride; a.groups = s.groups;
  a.x = s.x; a.codes = s.codes; a.scales = s.scales;
  a.group = s.group; a.fmt = s.fmt; a.shift = group_shift(s.group);
  const bool vec = a.cols % 8 == 0 && a.x_stride % 8 == 0 &&
                   aligned_to(a.x, chunk_align(dtype)) && aligned_to(a.codes, 8);
  if (!vec) return fwd_odd(dtype, false, a, st);
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    return s.fmt == kFmtInt8 ? fwd_ring<T, kFmtInt8, false, false, false>(a, st)
                             : fwd_ring<T, kFmtE4m3, false, false, false>(a, st);
  });
}

}  // namespace bl
