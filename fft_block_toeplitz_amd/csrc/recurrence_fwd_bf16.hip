// The forward scan of the gated linear recurrence for bf16 elements.
#include "recurrence_fwd.hpp"

namespace fftmv {
hipError_t launch_recurrence_forward_bf16(const fftmv_recurrence_t &r, hipStream_t s) {
  return launch_recurrence_forward_as<bf16>(r, s);
}
}  // namespace fftmv
