// The forward scan of the gated linear recurrence for f16 elements.
#include "recurrence_fwd.hpp"

namespace fftmv {
hipError_t launch_recurrence_forward_f16(const fftmv_recurrence_t &r, hipStream_t s) {
  return launch_recurrence_forward_as<f16>(r, s);
}
}  // namespace fftmv
