// One step of the gated linear recurrence for many streams against a cache
// of states, in place.
#include "recurrence.hpp"

namespace fftmv {
namespace {

template <typename T, int DECAY, int DRIVE>
__global__ __launch_bounds__(kBlock) void step_kernel(fftmv_recurrence_step_t r) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x, b = blockIdx.y;
  if (c >= r.channels) return;
  const int64_t slot = r.slots ? r.slots[b] : b;
  T *h = static_cast<T *>(r.h) + b * r.h_step + c;
  if (slot < 0 || slot >= r.places) {
    *h = static_cast<T>(0.0f);
    return;
  }
  const Terms e = decay_terms<T, DECAY>(static_cast<float>(static_cast<const T *>(r.gate)[b * r.gate_step + c]));
  float *state = r.state + slot * r.state_step + c;
  const float v =
      fmaf(e.a, *state, drive_of<DRIVE>(e, static_cast<float>(static_cast<const T *>(r.x)[b * r.x_step + c])));
  *state = v;
  *h = static_cast<T>(v);
}

}  // namespace

hipError_t launch_recurrence_step(const fftmv_recurrence_step_t &r, hipStream_t s) {
  const int64_t nx = (r.channels + kBlock - 1) / kBlock;
  if (r.batch > 65535 || !grid_fits(nx * r.batch, kBlock)) return hipErrorInvalidConfiguration;
  return by_dtype(r.dtype, [&](auto t) {
    return by_recurrence_kind(r.decay, r.drive, [&](auto d, auto u) {
      step_kernel<decltype(t), decltype(d)::value, decltype(u)::value>
          <<<dim3(static_cast<unsigned>(nx), static_cast<unsigned>(r.batch)), kBlock, 0, s>>>(r);
      return hipGetLastError();
    });
  });
}

}  // namespace fftmv
