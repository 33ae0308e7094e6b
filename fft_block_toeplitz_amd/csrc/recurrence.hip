// The gated linear recurrence h_t = a_t h_{t-1} + u_t: one thread per
// sequence and channel, step after step.
#include "common.hpp"
#include "internal.hpp"
#include "sequence.hpp"

namespace fftmv {
namespace {

// First row and number of steps of sequence b, and where its rows start.
struct Span {
  int64_t row, n;  // row: on the flattened time axis
  int64_t t0;      // step index of the first row within its batch stride
};

__device__ __forceinline__ Span span_of(const fftmv_recurrence_t &r, int64_t b) {
  Span s;
  if (r.offsets) {
    int64_t lo = r.offsets[b], hi = r.offsets[b + 1];
    lo = lo < 0 ? 0 : lo > r.steps ? r.steps : lo;
    hi = hi < lo ? lo : hi > r.steps ? r.steps : hi;
    s.row = s.t0 = lo;
    s.n = hi - lo;
  } else {
    s.row = b * r.steps;
    s.t0 = 0;
    s.n = r.steps;
    if (r.lengths) {
      const int64_t l = r.lengths[b];
      s.n = l < 0 ? 0 : l > r.steps ? r.steps : l;
    }
  }
  return s;
}

template <typename T>
__device__ __forceinline__ int64_t at(const fftmv_recurrence_t &r, int64_t b, int64_t t, int64_t sb, int64_t st) {
  return (r.offsets ? 0 : b * sb) + t * st;
}

// Zeros in channel c of the rows that no sequence holds.
template <typename T>
__device__ void clear_rest(const fftmv_recurrence_t &r, int64_t b, int64_t c, T *p, int64_t sb, int64_t st,
                           const Span &s) {
  if (r.offsets) {
    if (b == 0)
      for (int64_t t = 0; t < r.offsets[0] && t < r.steps; ++t) p[t * st + c] = static_cast<T>(0.0f);
    if (b == r.batch - 1)
      for (int64_t t = s.t0 + s.n; t < r.steps; ++t) p[t * st + c] = static_cast<T>(0.0f);
  } else {
    for (int64_t t = s.n; t < r.steps; ++t) p[b * sb + t * st + c] = static_cast<T>(0.0f);
  }
}

template <typename T, int DECAY, int DRIVE>
__global__ __launch_bounds__(kWave) void forward_kernel(fftmv_recurrence_t r) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kWave + threadIdx.x, b = blockIdx.y;
  if (c >= r.channels) return;
  const Span s = span_of(r, b);
  float h = r.h0 ? r.h0[b * r.channels + c] : 0.0f;
  for (int64_t t = 0; t < s.n; ++t) {
    const int64_t row = s.row + t;
    if (r.carries && row % FFTMV_RECURRENCE_CHUNK == 0)
      r.carries[row / FFTMV_RECURRENCE_CHUNK * r.channels + c] = h;
    const float x = static_cast<float>(static_cast<const T *>(r.x)[at<T>(r, b, s.t0 + t, r.x_batch, r.x_step) + c]);
    const float g =
        static_cast<float>(static_cast<const T *>(r.gate)[at<T>(r, b, s.t0 + t, r.gate_batch, r.gate_step) + c]);
    const Terms e = decay_terms<T, DECAY>(g);
    h = fmaf(e.a, h, drive_of<DRIVE>(e, x));
    static_cast<T *>(r.h)[at<T>(r, b, s.t0 + t, r.h_batch, r.h_step) + c] = static_cast<T>(h);
  }
  clear_rest(r, b, c, static_cast<T *>(r.h), r.h_batch, r.h_step, s);
  if (r.h_last) r.h_last[b * r.channels + c] = h;
}

template <typename T, int DECAY, int DRIVE>
__global__ __launch_bounds__(kWave) void backward_kernel(fftmv_recurrence_t r) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kWave + threadIdx.x, b = blockIdx.y;
  if (c >= r.channels) return;
  const Span s = span_of(r, b);
  const T *x = static_cast<const T *>(r.x), *g = static_cast<const T *>(r.gate), *dh = static_cast<const T *>(r.dh);
  T *dx = static_cast<T *>(r.dx), *dg = static_cast<T *>(r.dgate);
  float back = r.dh_last ? r.dh_last[b * r.channels + c] : 0.0f;  // a_{t+1} r_{t+1}
  const float h0 = r.h0 ? r.h0[b * r.channels + c] : 0.0f;
  float before[FFTMV_RECURRENCE_CHUNK];
  for (int64_t end = s.n; end > 0;) {
    // the steps of one chunk: [from, end)
    const int64_t chunk = (s.row + end - 1) / FFTMV_RECURRENCE_CHUNK;
    int64_t from = chunk * FFTMV_RECURRENCE_CHUNK - s.row;
    float h = h0;
    if (from > 0)
      h = r.carries[chunk * r.channels + c];
    else
      from = 0;
    for (int64_t t = from; t < end; ++t) {
      before[t - from] = h;
      const Terms e = decay_terms<T, DECAY>(static_cast<float>(g[at<T>(r, b, s.t0 + t, r.gate_batch, r.gate_step) + c]));
      h = fmaf(e.a, h, drive_of<DRIVE>(e, static_cast<float>(x[at<T>(r, b, s.t0 + t, r.x_batch, r.x_step) + c])));
    }
    for (int64_t t = end - 1; t >= from; --t) {
      const float xt = static_cast<float>(x[at<T>(r, b, s.t0 + t, r.x_batch, r.x_step) + c]);
      const Terms e = decay_terms<T, DECAY>(static_cast<float>(g[at<T>(r, b, s.t0 + t, r.gate_batch, r.gate_step) + c]));
      const float rt = static_cast<float>(dh[at<T>(r, b, s.t0 + t, r.dh_batch, r.dh_step) + c]) + back;
      back = e.a * rt;
      float da = rt * before[t - from], du = rt;
      if (DRIVE == FFTMV_DRIVE_COMPLEMENT) da -= rt * xt, du *= e.rest;
      dx[at<T>(r, b, s.t0 + t, r.dx_batch, r.dx_step) + c] = static_cast<T>(du);
      dg[at<T>(r, b, s.t0 + t, r.dgate_batch, r.dgate_step) + c] = static_cast<T>(da * e.slope);
    }
    end = from;
  }
  clear_rest(r, b, c, dx, r.dx_batch, r.dx_step, s);
  clear_rest(r, b, c, dg, r.dgate_batch, r.dgate_step, s);
  if (r.dh0) r.dh0[b * r.channels + c] = back;
}

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

template <typename F>
hipError_t by_kind(int dtype, int decay, int drive, F f) {
  return by_dtype(dtype, [&](auto t) {
    return by_three(decay, [&](auto d) { return by_two(drive, [&](auto u) { return f(t, d, u); }); });
  });
}

}  // namespace

hipError_t launch_recurrence_forward(const fftmv_recurrence_t &r, hipStream_t s) {
  const int64_t nx = (r.channels + kWave - 1) / kWave;
  if (r.batch > 65535 || !grid_fits(nx * r.batch, kWave)) return hipErrorInvalidConfiguration;
  return by_kind(r.dtype, r.decay, r.drive, [&](auto t, auto d, auto u) {
    forward_kernel<decltype(t), decltype(d)::value, decltype(u)::value>
        <<<dim3(static_cast<unsigned>(nx), static_cast<unsigned>(r.batch)), kWave, 0, s>>>(r);
    return hipGetLastError();
  });
}

hipError_t launch_recurrence_backward(const fftmv_recurrence_t &r, hipStream_t s) {
  const int64_t nx = (r.channels + kWave - 1) / kWave;
  if (r.batch > 65535 || !grid_fits(nx * r.batch, kWave)) return hipErrorInvalidConfiguration;
  return by_kind(r.dtype, r.decay, r.drive, [&](auto t, auto d, auto u) {
    backward_kernel<decltype(t), decltype(d)::value, decltype(u)::value>
        <<<dim3(static_cast<unsigned>(nx), static_cast<unsigned>(r.batch)), kWave, 0, s>>>(r);
    return hipGetLastError();
  });
}

hipError_t launch_recurrence_step(const fftmv_recurrence_step_t &r, hipStream_t s) {
  const int64_t nx = (r.channels + kBlock - 1) / kBlock;
  if (r.batch > 65535 || !grid_fits(nx * r.batch, kBlock)) return hipErrorInvalidConfiguration;
  return by_kind(r.dtype, r.decay, r.drive, [&](auto t, auto d, auto u) {
    step_kernel<decltype(t), decltype(d)::value, decltype(u)::value>
        <<<dim3(static_cast<unsigned>(nx), static_cast<unsigned>(r.batch)), kBlock, 0, s>>>(r);
    return hipGetLastError();
  });
}

}  // namespace fftmv
