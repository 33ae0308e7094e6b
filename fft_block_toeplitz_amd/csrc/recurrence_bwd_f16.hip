// The backward scan of the gated linear recurrence for f16 elements.
#include "recurrence_bwd.hpp"

namespace fftmv {
hipError_t launch_recurrence_backward_f16(const fftmv_recurrence_t &r, hipStream_t s) {
  return launch_recurrence_backward_as<f16>(r, s);
}
}  // namespace fftmv
