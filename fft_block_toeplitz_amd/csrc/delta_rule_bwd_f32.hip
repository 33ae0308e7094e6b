// The delta rule's backward pass for f32 elements.
#include "delta_rule_bwd.hpp"

namespace fftmv {
hipError_t launch_delta_backward_f32(const fftmv_delta_rule_t &r, hipStream_t s) { return launch_delta_backward<float>(r, s); }
}  // namespace fftmv
