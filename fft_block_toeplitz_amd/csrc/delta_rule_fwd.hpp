// Forward pass of the gated delta rule: the runs of one sequence one after the
// other, its state in registers. A wave has 16 value columns of all keys, which
// no other wave needs anything from; the waves of a workgroup share the run's
// rows of keys and queries in LDS.
#pragma once

#include "delta_rule.hpp"

namespace fftmv {

constexpr int kChainWaves = 4;
constexpr int kChainThreads = kChainWaves * kWave;

template <typename T, int KEYS, bool SAVE>
__global__ __launch_bounds__(kChainThreads) void delta_chain_kernel(fftmv_delta_rule_t r, DeltaWorkspace w) {
  using Tri = Triangles<T, false>;
  constexpr int NP = kParts<T>, NO = kOut<T>, S = KEYS / 32;
  __shared__ __align__(16) uint16_t ktile[NP * kRun * kTileRow<KEYS>], qtile[NP * kRun * kTileRow<KEYS>];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, x = lane % 16, g = lane / 16;
  const int64_t head = blockIdx.x % r.heads, b = blockIdx.x / r.heads;
  const int64_t key_head = head / (r.heads / r.key_heads);
  const int keys = static_cast<int>(r.keys), values = static_cast<int>(r.values);
  const int col = (blockIdx.y * kChainWaves + wave) * 16 + x;
  const bool inside = col < values;
  const Span span = span_of(r, b);
  const int64_t states = r.keys * r.values;

  f32x4 state[KEYS / 16];
#pragma unroll
  for (int t = 0; t < KEYS / 16; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = key_of(t, g, i);
      state[t][i] = r.h0 && inside && key < keys
                        ? r.h0[(b * r.heads + head) * states + static_cast<int64_t>(key) * values + col]
                        : 0.0f;
    }

  auto keep = [&](float *to) {
#pragma unroll
    for (int t = 0; t < KEYS / 16; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key_of(t, g, i);
        if (inside && key < keys) to[static_cast<int64_t>(key) * values + col] = state[t][i];
      }
  };

  for (int first = 0; first < span.len; first += kRun) {
    const int n = min(kRun, span.len - first);
    const int64_t row = span.row + first, at = (span.run + first / kRun) * r.heads + head;
    const Factors &f = w.factors[at];
    const u32x4 *tri = w.triangles + at * Tri::kAll * kWave;
    if constexpr (SAVE) keep(r.carries + at * states);
    __syncthreads();
    fill_tile<T, KEYS, kChainThreads>(ktile, r.k, span.batch, row, n, key_head, keys);
    fill_tile<T, KEYS, kChainThreads>(qtile, r.q, span.batch, row, n, key_head, keys);
    f32x4 v[kTiles];
#pragma unroll
    for (int m = 0; m < kTiles; ++m) v[m] = load_column<T>(r.v, span.batch, row, n, head, m, g, col, inside);
    __syncthreads();

    f32x4 u[kTiles], y[kTiles];
#pragma unroll
    for (int m = 0; m < kTiles; ++m) u[m] = y[m] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const Cut<kFull> part = cut_tiles<kFull>(state[2 * s], state[2 * s + 1]);
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        multiply<kFull>(u[m], tile_rows<KEYS, NP>(ktile, m, s, lane), part);
        multiply<NO>(y[m], tile_rows<KEYS, NP>(qtile, m, s, lane), part);
      }
    }
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      const f32x4 into = *reinterpret_cast<const f32x4 *>(f.into + 16 * m + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[m][i] = fmaf(-into[i], u[m][i], v[m][i]);
        y[m][i] *= r.scale * into[i];
      }
    }
    {
      const Cut<kFull> a = cut_tiles<kFull>(u[0], u[1]), c = cut_tiles<kFull>(u[2], u[3]);
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        u[m] = f32x4{0, 0, 0, 0};
        multiply<kFull>(u[m], load_frag<kFull>(tri, lower_frag(m, 0), Tri::kTParts, lane), a);
        if (m >= 2) multiply<kFull>(u[m], load_frag<kFull>(tri, lower_frag(m, 1), Tri::kTParts, lane), c);
      }
    }
    {
      const Cut<NO> a = cut_tiles<NO>(u[0], u[1]), c = cut_tiles<NO>(u[2], u[3]);
      const u32x4 *p = tri + Tri::kP * kWave;
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        multiply<NO>(y[m], load_frag<NO>(p, lower_frag(m, 0), Tri::kPParts, lane), a);
        if (m >= 2) multiply<NO>(y[m], load_frag<NO>(p, lower_frag(m, 1), Tri::kPParts, lane), c);
      }
    }
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      const f32x4 out = *reinterpret_cast<const f32x4 *>(f.out + 16 * m + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * m + 4 * g + i;
        if (inside && t < n) head_row<T>(r.y, span.batch, row + t, head)[col] = static_cast<T>(y[m][i]);
      }
      u[m] *= out;
    }
    const float whole = f.into[kRun - 1];
    const Cut<kFull> a = cut_tiles<kFull>(u[0], u[1]), c = cut_tiles<kFull>(u[2], u[3]);
#pragma unroll
    for (int t = 0; t < KEYS / 16; ++t) {
      state[t] *= whole;
      multiply<kFull>(state[t], tile_columns<KEYS, NP>(ktile, t, 0, lane), a);
      multiply<kFull>(state[t], tile_columns<KEYS, NP>(ktile, t, 1, lane), c);
    }
  }
  if (r.h_last) keep(r.h_last + (b * r.heads + head) * states);
}

template <typename T>
hipError_t launch_delta_forward(const fftmv_delta_rule_t &r, hipStream_t s) {
  const int64_t runs = delta_runs(r.batch, r.steps, r.offsets != nullptr);
  DeltaWorkspace w;
  delta_workspace(runs, r.heads, r.keys, r.values, r.dtype, false, r.workspace, &w);
  const int64_t waves = (r.values + 15) / 16, blocks = (waves + kChainWaves - 1) / kChainWaves;
  if (!grid_fits(runs * r.heads, kWave) || !grid_fits(r.batch * r.heads * blocks, kChainThreads))
    return hipErrorInvalidConfiguration;
  return by_keys(r.keys, [&](auto k) {
    constexpr int KEYS = decltype(k)::value;
    if (runs > 0) {
      delta_factors_kernel<T, KEYS, false><<<static_cast<unsigned>(runs * r.heads), kWave, 0, s>>>(r, w);
      if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    const dim3 grid(static_cast<unsigned>(r.batch * r.heads), static_cast<unsigned>(blocks));
    if (r.carries)
      delta_chain_kernel<T, KEYS, true><<<grid, kChainThreads, 0, s>>>(r, w);
    else
      delta_chain_kernel<T, KEYS, false><<<grid, kChainThreads, 0, s>>>(r, w);
    return hipGetLastError();
  });
}

}  // namespace fftmv
