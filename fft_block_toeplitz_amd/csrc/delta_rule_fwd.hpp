// Forward pass of the gated delta rule: the runs of one sequence one after the
// other, its state in registers. A wave has 16 value columns of all keys, which
// no other wave needs anything from; the waves of a workgroup share the run's
// rows of keys and queries in LDS.
#pragma once

#include "delta_rule.hpp"

namespace fftmv {

// The state at a run's start goes to the back waves in parts, as the front waves need
// it, or (!PARTS) in FP32, two thirds of the bytes, to be cut there again.
template <typename T, int KEYS, int FRAGS, int BUFFERS, bool TILE, bool PARTS>
struct ForwardLds : ChainLds<T, KEYS, FRAGS, BUFFERS> {
  alignas(16) uint16_t q[TILE ? kParts<T> * kRun * kTileRow<KEYS, kParts<T>> : 8];
  static constexpr int S = KEYS / 32;
  alignas(16) u32x4 s[kFrontWaves][S][PARTS ? kFull : 2][kWave];
  alignas(16) f32x4 u[kFrontWaves][kTiles][kWave];  // X
};

// What a chain has in LDS, in this order as far as it fits: P's parts as T's (of 16-bit
// elements; two of three where only that leaves room for the queries), queries, two
// buffers of keys, the state in parts. (65536 steps of 8 heads of 128 x 128 bf16, two buffers
// and the state in FP32: 767 us, one and the state in parts 790.)
template <typename T, int KEYS, bool MAPS>
struct ForwardPlan {
  template <int P, int BUFFERS, bool TILE, bool PARTS>
  static constexpr bool fits() {
    return sizeof(ForwardLds<T, KEYS, kFrags * (kFull + P), BUFFERS, TILE, PARTS>) <= kLdsBytes;
  }
  static constexpr bool HALF = sizeof(T) == 2;
  static constexpr int P = MAPS || !HALF ? 0 : fits<kFull, 1, true, false>() ? kFull : kFull - 1;
  static constexpr bool TILE = fits<P, 1, true, false>();
  static constexpr int BUFFERS = fits<P, 2, TILE, false>() ? 2 : 1;
  static constexpr bool PARTS = fits<P, BUFFERS, TILE, true>();
  using Lds = ForwardLds<T, KEYS, kFrags * (kFull + P), BUFFERS, TILE, PARTS>;
};

// What a chain is for: the outputs, also with the states kept for the backward pass, or the maps of parts.
enum ChainUse { kOutputs, kCarries, kMaps };

template <typename T, int KEYS, bool WHOLE, int USE>
__global__ __launch_bounds__(kChainThreads) void delta_chain_kernel(fftmv_delta_rule_t r, DeltaWorkspace w) {
  using Tri = Triangles<false>;
  using Plan = ForwardPlan<T, KEYS, USE == kMaps>;
  constexpr int NP = kParts<T>, S = KEYS / 32, P = Plan::P, FRAGS = kFrags * (kFull + P), BUFFERS = Plan::BUFFERS;
  constexpr bool TILE = Plan::TILE;
  __shared__ typename Plan::Lds lds;
  const int side = __builtin_amdgcn_readfirstlane(threadIdx.x / kFrontThreads);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) % kFrontWaves;
  int thread = threadIdx.x % kFrontThreads, lane = threadIdx.x % kWave, x = lane % 16, g = lane / 16;
  auto again = [&]() __attribute__((always_inline)) {
    thread = afresh(thread), lane = thread % kWave, x = lane % 16, g = lane / 16;
  };
  const int keys = static_cast<int>(r.keys), values = static_cast<int>(r.values);
  // maps: blocks of value columns, then blocks of unit states without values
  const int value_blocks = (values + kValues - 1) / kValues, unit_blocks = USE == kMaps ? (keys + kValues - 1) / kValues : 0;
  const Place place(r.batch * r.heads * w.cuts.parts, value_blocks + unit_blocks);
  const uint32_t heads = static_cast<uint32_t>(r.heads), of_all = place.unit / w.cuts.parts;
  const int64_t head = of_all % heads, b = longest_first(r, w.cuts, of_all / heads, reinterpret_cast<int *>(&lds));
  const int64_t sequence = b * r.heads + head, key_head = head / (heads / static_cast<uint32_t>(r.key_heads));
  const bool units = USE == kMaps && static_cast<int>(place.which) >= value_blocks;
  const int first_col = (static_cast<int>(place.which) - (units ? value_blocks : 0)) * kValues, col = first_col + wave * 16 + x;
  const bool inside = col < (units ? keys : values);
  const Span span = span_of(r, b);
  const Part part(w.cuts, place.unit, span.len);
  if (USE == kMaps ? part.end >= span.len : part.part > 0 && part.begin >= span.len) return;
  const int64_t states = r.keys * r.values;

  if (side == 0) {
    f32x4 state[KEYS / 16];
#pragma unroll
    for (int t = 0; t < KEYS / 16; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key_of(t, g, i);
        state[t][i] = 0.0f;
        if constexpr (USE == kMaps) {
          state[t][i] = units && key == col ? 1.0f : 0.0f;
        } else {
          const float *from = part.part ? w.starts + place.unit * states : r.h0 ? r.h0 + sequence * states : nullptr;
          if (from && inside && key < keys) state[t][i] = from[static_cast<int64_t>(key) * values + col];
        }
      }
    auto keep = [&](float *to, int width) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < KEYS / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = key_of(t, g, i);
          if (inside && key < keys) to[static_cast<int64_t>(key) * width + col] = state[t][i];
        }
    };
    Cut<kFull> cuts[S];
    auto leave_state = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        cuts[s] = cut_tiles<kFull>(state[2 * s], state[2 * s + 1]);
        if constexpr (USE == kMaps) continue;
        if constexpr (Plan::PARTS) {
#pragma unroll
          for (int p = 0; p < kFull; ++p) lds.s[wave][s][p][lane] = cuts[s].p[p];
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) lds.s[wave][s][h][lane] = __builtin_bit_cast(u32x4, state[2 * s + h]);
        }
      }
    };
    leave_state();
    __syncthreads();
    for (int first = part.begin, buffer = 0; first < part.end; first += kRun, buffer = (buffer + 1) % BUFFERS) {
      const uint16_t *k = lds.k[buffer];
      again();
      f32x4 u[kTiles];
#pragma unroll
      for (int m = 0; m < kTiles; ++m) u[m] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < S; ++s) {
        Cut<NP> rows[kTiles];
        tile_rows<KEYS>(rows, k, s, lane);
        multiply_rows<kFull>(u, rows, cuts[s]);
      }
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
        u[m] = value_column(lds.v, m, 16 * wave, lane) - *reinterpret_cast<const f32x4 *>(lds.into + 16 * m + 4 * g) * u[m];
      {
        const Cut<kFull> a = cut_tiles<kFull>(u[0], u[1]), c = cut_tiles<kFull>(u[2], u[3]);
#pragma unroll
        for (int m = 0; m < kTiles; ++m) u[m] = f32x4{0, 0, 0, 0};
        multiply_triangle<kFull, kFull, kFull, false>(u, lds.frags, a, c, lane);
      }
      if constexpr (USE != kMaps) {
#pragma unroll
        for (int m = 0; m < kTiles; ++m) lds.u[wave][m][lane] = u[m];
      }
#pragma unroll
      for (int m = 0; m < kTiles; ++m) u[m] *= *reinterpret_cast<const f32x4 *>(lds.out + 16 * m + 4 * g);
      const float whole = lds.into[kRun - 1];
      if constexpr (USE == kCarries) keep(r.carries + ((span.run + first / kRun) * r.heads + head) * (states + kRun * r.values), values);
      __syncthreads();
      const Cut<kFull> a = cut_tiles<kFull>(u[0], u[1]), c = cut_tiles<kFull>(u[2], u[3]);
#pragma unroll
      for (int t = 0; t < KEYS / 16; ++t) state[t] *= whole;
      multiply_columns<KEYS, NP>(state, k, a, c, lane);
      if constexpr (BUFFERS == 1) __syncthreads();
      leave_state();
      __syncthreads();
    }
    if constexpr (USE == kMaps)
      keep(w.maps + static_cast<int64_t>(place.unit) * keys * (keys + values) + (units ? values : 0), keys + values);
    else if (r.h_last && part.end >= span.len)
      keep(r.h_last + sequence * states, values);
  } else {
    Fetched<T, KEYS, FRAGS, WHOLE> next;
    Raw8<T> own[KEYS / 32];       // queries, with a tile
    // without a tile (outputs of 65536 steps of 8 heads of 128 x 128 bf16 that way 329 us instead of 262, packed FP16 ones
    // 461 and 385, before third parts)
    QueryRows<T, KEYS, WHOLE> q;
    Cut<kFull> p[kFrags];
    constexpr int HOLD = QueryRows<T, KEYS, WHOLE>::HOLD;
    auto at = [&](int first) __attribute__((always_inline)) { return (span.run + first / kRun) * r.heads + head; };
    auto steps = [&](int first) __attribute__((always_inline)) { return min(kRun, span.len - first); };
    // behind the last run that one again: loads stand in no branch
    const int last = (part.end - 1) / kRun * kRun;
    auto fetch = [&](int first) __attribute__((always_inline)) {
      next.fetch_keys(thread, r.k, keys, span.batch, span.row + first, steps(first), key_head);
      next.fetch_values(thread, r.v, values, span.batch, span.row + first, steps(first), head, first_col);
      next.fetch_factors(thread, w.triangles + at(first) * Tri::kAll * kWave, w.factors[at(first)]);
      if constexpr (TILE && USE != kMaps)
        fetch_rows<T, KEYS, WHOLE>(own, thread, r.q, keys, span.batch, span.row + first, steps(first), key_head);
    };
    auto put = [&](int first) __attribute__((always_inline)) {
      if (units) {
#pragma unroll
        for (auto &v : next.v)
#pragma unroll
          for (auto &word : v.w) word = u32x4{0, 0, 0, 0};
      }
      next.put_values(thread, lds, values, steps(first), first_col);
      next.put_factors(thread, lds);
      if constexpr (TILE && USE != kMaps) put_rows<T, KEYS, WHOLE>(own, thread, lds.q, keys, steps(first));
    };
    auto fetch_triangle = [&](int first) __attribute__((always_inline)) {
      // from LDS as far as P is there. Each wave for itself from memory, four times the loads, made the outputs of 65536
      // steps (8 heads of 128 x 128 bf16) 276 us instead of 262, before third parts; FP32 elements leave no room
      const u32x4 *far = w.triangles + at(first) * Tri::kAll * kWave;
#pragma unroll
      for (int a = 0; a < kFull; ++a)
#pragma unroll
        for (int i = 0; i < kFrags; ++i) p[i].p[a] = at_lane((a < P ? lds.frags : far) + (Tri::kP + a * kFrags + i) * kWave, lane);
    };
    auto fetch_queries = [&](int first, auto s) __attribute__((always_inline)) {
      q.template fetch<decltype(s)::value>(r.q, keys, span.batch, span.row + first, steps(first), key_head, lane);
    };
    auto fetch_first_queries = [&](int first) __attribute__((always_inline)) { unrolled<0, HOLD>([&](auto s) __attribute__((always_inline)) { fetch_queries(first, s); }); };
    if (part.end > part.begin) {
      fetch(part.begin);
      if constexpr (!TILE && USE != kMaps) fetch_first_queries(part.begin);
      next.put_keys(thread, lds.k[0], keys, steps(part.begin));
      put(part.begin);
    }
    __syncthreads();
    for (int first = part.begin, buffer = 0; first < part.end; first += kRun, buffer = (buffer + 1) % BUFFERS) {
      again();
      const int n = steps(first), then = min(first + kRun, last);
      fetch(then);
      f32x4 y[kTiles];
#pragma unroll
      for (int m = 0; m < kTiles; ++m) y[m] = f32x4{0, 0, 0, 0};
      if constexpr (USE != kMaps) {
        unrolled<0, S>([&](auto i) __attribute__((always_inline)) {
          constexpr int s = decltype(i)::value;
          Cut<kFull> part;
          if constexpr (Plan::PARTS) {
#pragma unroll
            for (int p = 0; p < kFull; ++p) part.p[p] = lds.s[wave][s][p][lane];
          } else {
            part = cut_tiles<kFull>(__builtin_bit_cast(f32x4, lds.s[wave][s][0][lane]), __builtin_bit_cast(f32x4, lds.s[wave][s][1][lane]));
          }
          Cut<NP> rows[kTiles];
          if constexpr (TILE) {
            tile_rows<KEYS>(rows, lds.q, s, lane);
          } else {
#pragma unroll
            for (int m = 0; m < kTiles; ++m) rows[m] = q.template operand<s>(m, keys, n, lane);
            if constexpr (s + HOLD < S) fetch_queries(first, Const<s + HOLD>{});
          }
          multiply_rows_t<kFull>(y, rows, part);  // steps along the lanes
          if constexpr (!TILE) part_done();
        });
        fetch_triangle(first);  // only now: registers
#pragma unroll
        for (int m = 0; m < kTiles; ++m) y[m] *= r.scale * lds.into[16 * m + x];
      }
      __syncthreads();
      if constexpr (USE != kMaps) {
        f32x4 u[kTiles];
#pragma unroll
        for (int m = 0; m < kTiles; ++m) u[m] = lds.u[wave][m][lane];
        if constexpr (USE == kCarries) {
          float *to = r.carries + at(first) * (states + kRun * r.values) + states;
#pragma unroll
          for (int m = 0; m < kTiles; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (inside) to[static_cast<int64_t>(16 * m + 4 * g + i) * values + col] = u[m][i];
        }
        multiply_triangle<kFull, false, true>(y, p, cut_tiles<kFull>(u[0], u[1]), cut_tiles<kFull>(u[2], u[3]));
        if constexpr (!TILE) fetch_first_queries(then);
        const int c = first_col + 16 * wave + 4 * g;
        T *to = head_row<T>(r.y, span.batch, span.row + first, head);
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          const int t = 16 * m + x;
          if constexpr (WHOLE) {
            if (t < n && c < values) {
              const float e[4] = {y[m][0], y[m][1], y[m][2], y[m][3]};
              store_vec(&at_lane_of(to, t * static_cast<uint32_t>(r.y.step) + c), e, false);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (t < n && c + i < values) to[t * r.y.step + c + i] = static_cast<T>(y[m][i]);
          }
        }
      }
      again();
      put(then);
      if constexpr (BUFFERS == 2) {
        next.put_keys(thread, lds.k[1 - buffer], keys, steps(then));
      } else {
        __syncthreads();
        next.put_keys(thread, lds.k[0], keys, steps(then));
      }
      __syncthreads();
    }
  }
}

template <typename T>
hipError_t launch_delta_forward(const fftmv_delta_rule_t &r, hipStream_t s) {
  const int64_t runs = delta_runs(r.batch, r.steps, r.offsets != nullptr), sequences = r.batch * r.heads;
  DeltaWorkspace w;
  delta_workspace(r.batch, r.steps, r.heads, r.keys, r.values, r.offsets != nullptr, false, r.workspace, &w);
  const int64_t blocks = (r.values + kValues - 1) / kValues, units = (r.keys + kValues - 1) / kValues;
  if (!grid_fits(runs * r.heads, kFrontThreads) || !grid_fits(sequences * ((r.values + 15) / 16), 512) || !grid_fits(sequences * w.cuts.parts * (blocks + units), kChainThreads))
    return hipErrorInvalidConfiguration;
  return by_keys(r.keys, [&](auto k) {
    constexpr int KEYS = decltype(k)::value;
    if (runs > 0) {
      const hipError_t e = by_two(delta_whole_rows(r), [&](auto whole) {
        delta_factors_kernel<T, KEYS, decltype(whole)::value != 0, false>
            <<<static_cast<unsigned>(runs * r.heads), kFrontThreads, 0, s>>>(r, w);
        return hipGetLastError();
      });
      if (e != hipSuccess) return e;
    }
    return by_two(delta_whole(r, r.v, r.y), [&](auto whole) {
      constexpr bool WHOLE = decltype(whole)::value != 0;
      const unsigned chains = static_cast<unsigned>(sequences * w.cuts.parts), columns = static_cast<unsigned>(blocks);
      if (w.cuts.parts > 1) {
        const unsigned all = chains * static_cast<unsigned>(blocks + units);
        delta_chain_kernel<T, KEYS, WHOLE, kMaps><<<all, kChainThreads, 0, s>>>(r, w);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        delta_join_kernel<T, KEYS, false>
            <<<dim3(static_cast<unsigned>(sequences), static_cast<unsigned>((r.values + 15) / 16)), KEYS / 16 * kWave, 0, s>>>(r, w);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
      }
      if (r.carries)
        delta_chain_kernel<T, KEYS, WHOLE, kCarries><<<chains * columns, kChainThreads, 0, s>>>(r, w);
      else
        delta_chain_kernel<T, KEYS, WHOLE, kOutputs><<<chains * columns, kChainThreads, 0, s>>>(r, w);
      return hipGetLastError();
    });
  });
}

}  // namespace fftmv
