// Group normalisation, backward, for bf16 elements.
#include "group_norm.hpp"

namespace fftmv {
hipError_t launch_group_norm_backward_bf16(const fftmv_group_norm_t &g, hipStream_t s) {
  return launch_group_norm_backward_as<bf16>(g, s);
}
}  // namespace fftmv
