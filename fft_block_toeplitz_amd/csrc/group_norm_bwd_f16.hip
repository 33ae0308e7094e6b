// Group normalisation, backward, for f16 elements.
#include "group_norm.hpp"

namespace fftmv {
hipError_t launch_group_norm_backward_f16(const fftmv_group_norm_t &g, hipStream_t s) {
  return launch_group_norm_backward_as<f16>(g, s);
}
}  // namespace fftmv
