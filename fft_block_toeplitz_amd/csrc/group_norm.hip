// Group normalisation with an activation: one workgroup per sample and
// group, three passes over its rows.
#include "common.hpp"
#include "internal.hpp"
#include "sequence.hpp"

namespace fftmv {
namespace {

// Sum over the workgroup, the same bits in every thread.
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kBlock / kWave];
  v = wave_sum(v);
  __syncthreads();  // the last use of part is over
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  float s = part[0];
  for (int i = 1; i < kBlock / kWave; ++i) s += part[i];
  return s;
}

__device__ __forceinline__ int64_t held_rows(const fftmv_group_norm_t &g, int64_t n) {
  if (!g.lengths) return g.rows;
  const int64_t l = g.lengths[n];
  return l < 0 ? 0 : l > g.rows ? g.rows : l;
}

template <typename T, int ACT>
__global__ __launch_bounds__(kBlock) void forward_kernel(fftmv_group_norm_t g) {
  const int64_t n = blockIdx.x / g.groups, q = blockIdx.x % g.groups, D = g.channels / g.groups;
  const int64_t held = held_rows(g, n), count = held * D;
  const T *x = static_cast<const T *>(g.x) + n * g.x_sample + q * D;
  T *y = static_cast<T *>(g.y) + n * g.y_sample + q * D;
  float s = 0.0f;
  for (int64_t i = threadIdx.x; i < count; i += kBlock) s += static_cast<float>(x[i / D * g.x_row + i % D]);
  const float mean = count ? block_sum(s) / static_cast<float>(count) : 0.0f;
  s = 0.0f;
  for (int64_t i = threadIdx.x; i < count; i += kBlock) {
    const float v = static_cast<float>(x[i / D * g.x_row + i % D]) - mean;
    s += v * v;
  }
  const float rstd = count ? 1.0f / sqrtf(block_sum(s) / static_cast<float>(count) + g.eps) : 0.0f;
  if (g.stats && threadIdx.x == 0) {
    g.stats[2 * static_cast<int64_t>(blockIdx.x)] = mean;
    g.stats[2 * static_cast<int64_t>(blockIdx.x) + 1] = rstd;
  }
  for (int64_t i = threadIdx.x; i < g.rows * D; i += kBlock) {
    float v = 0.0f;
    if (i < count) {
      const float w = g.weight ? g.weight[q * D + i % D] : 1.0f, b = g.bias ? g.bias[q * D + i % D] : 0.0f;
      v = activate<ACT>((static_cast<float>(x[i / D * g.x_row + i % D]) - mean) * rstd * w + b);
    }
    y[i / D * g.y_row + i % D] = static_cast<T>(v);
  }
}

template <typename T, int ACT>
__global__ __launch_bounds__(kBlock) void backward_kernel(fftmv_group_norm_t g) {
  const int64_t n = blockIdx.x / g.groups, q = blockIdx.x % g.groups, D = g.channels / g.groups;
  const int64_t held = held_rows(g, n), count = held * D;
  const T *x = static_cast<const T *>(g.x) + n * g.x_sample + q * D;
  const T *dy = static_cast<const T *>(g.dy) + n * g.dy_sample + q * D;
  T *dx = static_cast<T *>(g.dx) + n * g.dx_sample + q * D;
  float *sums = static_cast<float *>(g.workspace) + 2 * (n * g.channels + q * D);
  const float mean = g.stats[2 * static_cast<int64_t>(blockIdx.x)];
  const float rstd = g.stats[2 * static_cast<int64_t>(blockIdx.x) + 1];
  float m1 = 0.0f, m2 = 0.0f;
  for (int64_t c = 0; c < D; ++c) {
    const float w = g.weight ? g.weight[q * D + c] : 1.0f, b = g.bias ? g.bias[q * D + c] : 0.0f;
    float sb = 0.0f, sw = 0.0f;
    for (int64_t t = threadIdx.x; t < held; t += kBlock) {
      const float xh = (static_cast<float>(x[t * g.x_row + c]) - mean) * rstd;
      const float dz = static_cast<float>(dy[t * g.dy_row + c]) * activate_slope<ACT>(xh * w + b);
      sb += dz;
      sw += dz * xh;
    }
    sb = block_sum(sb);
    sw = block_sum(sw);
    if (threadIdx.x == 0) sums[2 * c] = sb, sums[2 * c + 1] = sw;
    m1 += sb * w;
    m2 += sw * w;
  }
  m1 = count ? m1 / static_cast<float>(count) : 0.0f;
  m2 = count ? m2 / static_cast<float>(count) : 0.0f;
  for (int64_t i = threadIdx.x; i < g.rows * D; i += kBlock) {
    float v = 0.0f;
    const int64_t t = i / D, c = i % D;
    if (t < held) {
      const float w = g.weight ? g.weight[q * D + c] : 1.0f, b = g.bias ? g.bias[q * D + c] : 0.0f;
      const float xh = (static_cast<float>(x[t * g.x_row + c]) - mean) * rstd;
      const float dz = static_cast<float>(dy[t * g.dy_row + c]) * activate_slope<ACT>(xh * w + b);
      v = rstd * (dz * w - m1 - xh * m2);
    }
    dx[t * g.dx_row + c] = static_cast<T>(v);
  }
}

__global__ __launch_bounds__(kBlock) void parameter_sums_kernel(fftmv_group_norm_t g) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  if (c >= g.channels) return;
  const float *sums = static_cast<const float *>(g.workspace);
  float sb = 0.0f, sw = 0.0f;
  for (int64_t n = 0; n < g.samples; ++n) {
    sb += sums[2 * (n * g.channels + c)];
    sw += sums[2 * (n * g.channels + c) + 1];
  }
  if (g.dbias) g.dbias[c] = sb;
  if (g.dweight) g.dweight[c] = sw;
}

template <typename F>
hipError_t by_kind(const fftmv_group_norm_t &g, F f) {
  return by_dtype(g.dtype, [&](auto t) { return by_three(g.activation, [&](auto a) { return f(t, a); }); });
}

}  // namespace

hipError_t launch_group_norm_forward(const fftmv_group_norm_t &g, hipStream_t s) {
  if (!grid_fits(g.samples * g.groups, kBlock)) return hipErrorInvalidConfiguration;
  return by_kind(g, [&](auto t, auto a) {
    forward_kernel<decltype(t), decltype(a)::value>
        <<<static_cast<unsigned>(g.samples * g.groups), kBlock, 0, s>>>(g);
    return hipGetLastError();
  });
}

hipError_t launch_group_norm_backward(const fftmv_group_norm_t &g, hipStream_t s) {
  if (!grid_fits(g.samples * g.groups, kBlock)) return hipErrorInvalidConfiguration;
  hipError_t e = by_kind(g, [&](auto t, auto a) {
    backward_kernel<decltype(t), decltype(a)::value>
        <<<static_cast<unsigned>(g.samples * g.groups), kBlock, 0, s>>>(g);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  parameter_sums_kernel<<<static_cast<unsigned>((g.channels + kBlock - 1) / kBlock), kBlock, 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace fftmv
