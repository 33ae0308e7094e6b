// The forward scan of the gated linear recurrence for float elements.
#include "recurrence_fwd.hpp"

namespace fftmv {
hipError_t launch_recurrence_forward_f32(const fftmv_recurrence_t &r, hipStream_t s) {
  return launch_recurrence_forward_as<float>(r, s);
}
}  // namespace fftmv
