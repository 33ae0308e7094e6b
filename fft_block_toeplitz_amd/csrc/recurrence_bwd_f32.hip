// The backward scan of the gated linear recurrence for float elements.
#include "recurrence_bwd.hpp"

namespace fftmv {
hipError_t launch_recurrence_backward_f32(const fftmv_recurrence_t &r, hipStream_t s) {
  return launch_recurrence_backward_as<float>(r, s);
}
}  // namespace fftmv
