// The delta rule's backward pass for f16 elements.
#include "delta_rule_bwd.hpp"

namespace fftmv {
hipError_t launch_delta_backward_f16(const fftmv_delta_rule_t &r, hipStream_t s) { return launch_delta_backward<f16>(r, s); }
}  // namespace fftmv
