// The delta rule's forward pass for f16 elements.
#include "delta_rule_fwd.hpp"

namespace fftmv {
hipError_t launch_delta_forward_f16(const fftmv_delta_rule_t &r, hipStream_t s) { return launch_delta_forward<f16>(r, s); }
}  // namespace fftmv
