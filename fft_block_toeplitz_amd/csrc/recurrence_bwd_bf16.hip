// The backward scan of the gated linear recurrence for bf16 elements.
#include "recurrence_bwd.hpp"

namespace fftmv {
hipError_t launch_recurrence_backward_bf16(const fftmv_recurrence_t &r, hipStream_t s) {
  return launch_recurrence_backward_as<bf16>(r, s);
}
}  // namespace fftmv
