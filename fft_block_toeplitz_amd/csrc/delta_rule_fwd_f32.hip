// The delta rule's forward pass for f32 elements.
#include "delta_rule_fwd.hpp"

namespace fftmv {
hipError_t launch_delta_forward_f32(const fftmv_delta_rule_t &r, hipStream_t s) { return launch_delta_forward<float>(r, s); }
}  // namespace fftmv
