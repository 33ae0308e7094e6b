// Group normalisation, backward, for float elements.
#include "group_norm.hpp"

namespace fftmv {
hipError_t launch_group_norm_backward_f32(const fftmv_group_norm_t &g, hipStream_t s) {
  return launch_group_norm_backward_as<float>(g, s);
}
}  // namespace fftmv
