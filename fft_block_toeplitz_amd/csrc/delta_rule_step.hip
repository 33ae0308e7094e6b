// One step of the gated delta rule for many streams against a cache of states,
// in place.
//
// The states' bytes bound it: each goes through the registers of one workgroup,
// read once and written once. With p = S^T k and r = S^T q, both taken while S
// is on its way in,
//   e = v - a p,   S' = a S + b k e^T,   y = scale (a r + b (q.k) e)
// so one sum over the keys is all that the workgroup's threads wait for. A thread
// has 4 value columns of every GROUPS-th key; narrow heads take fewer threads along the
// values, so that none is idle (512 streams of 32 heads of 64 x 64 bf16: 16 threads 108
// us, 32 121; 1024 of 32 x 32: 8 threads 99, 32 115). 128 streams of 32 heads of 128 x
// 128: 88 us, 6.1 TB/s with a part of the states in the last cache, 116 with none there.
#include "delta_rule.hpp"

namespace fftmv {
namespace {

// LANES: threads across the values, 4 columns each
template <typename T, int KEYS, int LANES>
__global__ __launch_bounds__(kBlock) void delta_step_kernel(fftmv_delta_rule_step_t r) {
  constexpr int GROUPS = kBlock / LANES, ROWS = KEYS / GROUPS, WAVES = kBlock / kWave;
  static_assert(KEYS % GROUPS == 0, "whole rounds of the groups");
  __shared__ float keys_of[KEYS], queries[KEYS];
  __shared__ __align__(16) f32x4 sums[2][WAVES][LANES];
  const int thread = threadIdx.x, lane = thread % kWave, wave = thread / kWave;
  const uint32_t heads = static_cast<uint32_t>(r.heads), share = heads / static_cast<uint32_t>(r.key_heads);
  const int64_t b = blockIdx.x / heads, head = blockIdx.x % heads, key_head = blockIdx.x % heads / share;
  const int keys = static_cast<int>(r.keys), values = static_cast<int>(r.values);
  const int col = (blockIdx.y * LANES + thread % LANES) * 4, group = thread / LANES;
  const int most = min(4, values - col);
  const int64_t slot = r.slots ? r.slots[b] : b;
  T *y = head_row<T>(r.y, 0, b, head);
  if (slot < 0 || slot >= r.places) {
    if (group == 0)
      for (int e = 0; e < most; ++e) y[col + e] = static_cast<T>(0.0f);
    return;
  }
  float *state = r.state + slot * r.state_place + head * (r.keys * r.values);
  f32x4 s[ROWS];
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    const int key = j * GROUPS + group;
    s[j] = f32x4{0, 0, 0, 0};
    if (key < keys) {
      const float *p = state + static_cast<int64_t>(key) * values + col;
      if (most == 4) {
        s[j] = __builtin_bit_cast(f32x4, *reinterpret_cast<const u32x4_any *>(p));
      } else {
        for (int e = 0; e < most; ++e) s[j][e] = p[e];
      }
    }
  }
  for (int key = thread; key < KEYS; key += kBlock) {
    keys_of[key] = key < keys ? static_cast<float>(head_row<T>(r.k, 0, b, key_head)[key]) : 0.0f;
    queries[key] = key < keys ? static_cast<float>(head_row<T>(r.q, 0, b, key_head)[key]) : 0.0f;
  }
  const float a = expf(log_decay(r.decay, static_cast<float>(*head_row<T>(r.gate, 0, b, head))));
  const float rate = rate_of(r.rate, static_cast<float>(*head_row<T>(r.beta, 0, b, head)));
  f32x4 v = {0, 0, 0, 0};
  for (int e = 0; e < most; ++e) v[e] = static_cast<float>(head_row<T>(r.v, 0, b, head)[col + e]);
  __syncthreads();
  float qk = 0.0f;
#pragma unroll
  for (int key = lane; key < KEYS; key += kWave) qk = fmaf(keys_of[key], queries[key], qk);
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) qk += __shfl_xor(qk, d);
  f32x4 p = {0, 0, 0, 0}, q = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    const int key = j * GROUPS + group;
    p += s[j] * keys_of[key];
    q += s[j] * queries[key];
  }
#pragma unroll
  for (int d = LANES; d < kWave; d *= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[e] += __shfl_xor(p[e], d);
      q[e] += __shfl_xor(q[e], d);
    }
  if (lane < LANES) {
    sums[0][wave][lane] = p;
    sums[1][wave][lane] = q;
  }
  __syncthreads();
  p = q = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    p += sums[0][w][thread % LANES];
    q += sums[1][w][thread % LANES];
  }
  const f32x4 e = v - a * p;
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    const int key = j * GROUPS + group;
    if (key < keys) {
      const f32x4 next = a * s[j] + (rate * keys_of[key]) * e;
      float *to = state + static_cast<int64_t>(key) * values + col;
      if (most == 4) {
        *reinterpret_cast<u32x4_any *>(to) = __builtin_bit_cast(u32x4_any, next);
      } else {
        for (int i = 0; i < most; ++i) to[i] = next[i];
      }
    }
  }
  if (group == 0) {
    const f32x4 out = r.scale * (a * q + (rate * qk) * e);
    for (int i = 0; i < most; ++i) y[col + i] = static_cast<T>(out[i]);
  }
}

}  // namespace

hipError_t launch_delta_step(const fftmv_delta_rule_step_t &r, hipStream_t s) {
  auto launch = [&](auto t, auto keys, auto lanes) {
    constexpr int LANES = decltype(lanes)::value;
    const int64_t blocks = (r.values + 4 * LANES - 1) / (4 * LANES);
    if (!grid_fits(r.batch * r.heads * blocks, kBlock)) return hipErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(r.batch * r.heads), static_cast<unsigned>(blocks));
    delta_step_kernel<decltype(t), decltype(keys)::value, LANES><<<grid, kBlock, 0, s>>>(r);
    return hipGetLastError();
  };
  return by_dtype(r.dtype, [&](auto t) {
    return by_keys(r.keys, [&](auto k) {
      if (r.values <= 32) return launch(t, k, Const<8>{});
      if (r.values <= 64) return launch(t, k, Const<16>{});
      return launch(t, k, Const<32>{});
    });
  });
}

}  // namespace fftmv
