// One step of the gated linear recurrence for many streams against a cache
// of states, in place.
//
// Memory traffic bounds it: x, gate and state read, state and h written, once
// each. A thread takes four neighbouring channels of one stream; the threads
// run through all streams' rows as one axis, so narrow rows fill workgroups
// too. The channels behind the last whole four go one by one: a vector moved
// back over its neighbour's channels would meet states already stepped.
//
// 512 streams of 5000 channels in bf16 take 7.6 us, 4.7 TB/s (one channel a
// thread: 9.1 us); 4 streams of 500, 2.2 us, a launch's latency.
#include "recurrence.hpp"

namespace fftmv {
namespace {

constexpr int kStepVec = 4;

template <typename T, int DECAY, int DRIVE, int VEC>
__device__ __forceinline__ void step_channels(const T *x, const T *gate, float *state, T *h) {
  const Vec<T, VEC> xv = load_vec<T, VEC>(x), gv = load_vec<T, VEC>(gate);
  float v[VEC];
  Vec<float, VEC> s = load_vec<float, VEC>(state);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const Terms t = decay_terms<T, DECAY>(gv[e]);
    s.v[e] = v[e] = fmaf(t.a, s.v[e], drive_of<DRIVE>(t, xv[e]));
  }
  // not streamed past the caches as h is: the next step reads the state
  if constexpr (VEC == 1) {
    *state = s.v[0];
  } else {
    *reinterpret_cast<u32x4_any *>(state) = __builtin_bit_cast(u32x4_any, s);
  }
  store_vec(h, v);
}

template <typename T, int DECAY, int DRIVE>
__global__ __launch_bounds__(kBlock) void step_kernel(fftmv_recurrence_step_t r, uint32_t columns) {
  const uint32_t i = blockIdx.x * kBlock + threadIdx.x, b = i / columns;
  if (b >= r.batch) return;
  const int64_t c = static_cast<int64_t>(i - b * columns) * kStepVec;
  const int most = static_cast<int>(min(static_cast<int64_t>(kStepVec), r.channels - c));
  const int64_t slot = r.slots ? r.slots[b] : static_cast<int64_t>(b);
  T *h = static_cast<T *>(r.h) + b * r.h_step + c;
  if (slot < 0 || slot >= r.places) {
    for (int e = 0; e < most; ++e) h[e] = static_cast<T>(0.0f);
    return;
  }
  const T *x = static_cast<const T *>(r.x) + b * r.x_step + c;
  const T *gate = static_cast<const T *>(r.gate) + b * r.gate_step + c;
  float *state = r.state + slot * r.state_step + c;
  if (most == kStepVec) {
    step_channels<T, DECAY, DRIVE, kStepVec>(x, gate, state, h);
  } else {
    for (int e = 0; e < most; ++e) step_channels<T, DECAY, DRIVE, 1>(x + e, gate + e, state + e, h + e);
  }
}

}  // namespace

hipError_t launch_recurrence_step(const fftmv_recurrence_step_t &r, hipStream_t s) {
  const int64_t columns = (r.channels + kStepVec - 1) / kStepVec;
  const int64_t blocks = (columns * r.batch + kBlock - 1) / kBlock;
  if (!grid_fits(blocks, kBlock)) return hipErrorInvalidConfiguration;
  return by_dtype(r.dtype, [&](auto t) {
    return by_recurrence_kind(r.decay, r.drive, [&](auto d, auto u) {
      step_kernel<decltype(t), decltype(d)::value, decltype(u)::value>
          <<<static_cast<unsigned>(blocks), kBlock, 0, s>>>(r, static_cast<uint32_t>(columns));
      return hipGetLastError();
    });
  });
}

}  // namespace fftmv
