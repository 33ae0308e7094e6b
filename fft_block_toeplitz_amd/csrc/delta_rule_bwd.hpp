// Backward pass of the gated delta rule. With D the gradient of the state behind
// a run and dY that of its outputs,
//   Z   = (1 + diag(b) B)^-T (P^T dY + diag(e^{G_last - G}) K D)   the gradient of U = diag(b) X
//   D'  = e^{G_last} D + (scale diag(e^G) Q)^T dY - (diag(b e^G) K)^T Z
// goes from run to run, from the last to the first, as the state does forward;
// everything else belongs to one run:
//   dV  = diag(b) Z
//   dP  = dY U^T,  N = Z U^T, both lower triangles;  F = scale E o dP,  H = -diag(b) E o N
//   dQ  = scale diag(e^G) dY S^T + F K
//   dK  = F^T Q + (H + H^T) K + diag(e^{G_last - G}) U D^T - diag(b e^G) Z S^T
//   db_j = z_j . x_j
//   dG_i collects, with its sign, every product that e^{G_i} is a factor of; the
//   gradient of log a_t is the sum of dG_i over i >= t.
// So three kernels: the factors, the chain of D, and the gradients of all runs
// at once, from the states and X that the forward pass kept and the gradients and
// Z that the chain left. (Computing X and Z again from the states saves half of the
// bytes, 64 KB of a run of 128 values, and takes three triangles and K S, K D: 8 x 2048
// steps of 16 heads of 128 x 128 bf16 in 576 us instead of 437, with the chains 43
// faster, all in two parts an operand. Without them a run needs half of a CU's LDS, and
// two go side by side: 377 us in three parts.)
#pragma once

#include "delta_rule.hpp"

namespace fftmv {

// The chain of the states' gradients. P^T dY and (scale diag(e^G) Q)^T dY wait
// for no other run: the back waves compute them a run ahead of the front, which
// does K D, T^T (..) and K^T Z. (8 x 2048 steps of 16 heads of 128 x 128 bf16: 258 us, for
// 0.8 GB, half of them the gradients and Z that it leaves.)
template <typename T, int KEYS, int BUFFERS, bool TILE>
struct BackwardLds : ChainLds<T, KEYS, kFrags * kFull, BUFFERS> {
  alignas(16) uint16_t q[TILE ? kParts<T> * kRun * kTileRow<KEYS, kParts<T>> : 8];  // queries of the back waves' run
  alignas(16) f32x4 z[kFrontWaves][kTiles][kWave];                       // P^T dY of the front's
  alignas(16) f32x4 d[kFrontWaves][KEYS / 16][kWave];                    // Q^T (..) dY
};

template <typename T, int KEYS, bool WHOLE, bool MAPS>
__global__ __launch_bounds__(kChainThreads) void delta_back_chain_kernel(fftmv_delta_rule_t r, DeltaWorkspace w) {
  using Tri = Triangles<true>;
  constexpr int FRAGS = kFrags * kFull, NP = kParts<T>, S = KEYS / 32;
  constexpr bool TILE = sizeof(BackwardLds<T, KEYS, 1, true>) <= kLdsBytes;
  constexpr int BUFFERS = sizeof(BackwardLds<T, KEYS, 2, TILE>) <= kLdsBytes ? 2 : 1;
  using Lds = BackwardLds<T, KEYS, BUFFERS, TILE>;
  __shared__ Lds lds;
  const int side = __builtin_amdgcn_readfirstlane(threadIdx.x / kFrontThreads);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) % kFrontWaves;
  int thread = threadIdx.x % kFrontThreads, lane = threadIdx.x % kWave, x = lane % 16, g = lane / 16;
  auto again = [&]() __attribute__((always_inline)) {
    thread = afresh(thread), lane = thread % kWave, x = lane % 16, g = lane / 16;
  };
  const int keys = static_cast<int>(r.keys), values = static_cast<int>(r.values);
  // maps: blocks of value columns, then blocks of unit gradients without dY
  const int value_blocks = (values + kValues - 1) / kValues, unit_blocks = MAPS ? (keys + kValues - 1) / kValues : 0;
  const Place place(r.batch * r.heads * w.cuts.parts, value_blocks + unit_blocks);
  const uint32_t heads = static_cast<uint32_t>(r.heads), of_all = place.unit / w.cuts.parts;
  const int64_t head = of_all % heads, b = longest_first(r, w.cuts, of_all / heads, reinterpret_cast<int *>(&lds));
  const int64_t sequence = b * r.heads + head, key_head = head / (heads / static_cast<uint32_t>(r.key_heads));
  const bool units = MAPS && static_cast<int>(place.which) >= value_blocks;
  const int first_col = (static_cast<int>(place.which) - (units ? value_blocks : 0)) * kValues, col = first_col + wave * 16 + x;
  const bool inside = col < (units ? keys : values);
  const Span span = span_of(r, b);
  const Part part(w.cuts, place.unit, span.len);
  if (MAPS ? part.part == 0 || part.begin >= span.len : part.part > 0 && part.begin >= span.len) return;
  const int64_t states = r.keys * r.values;
  const int last = part.end > part.begin ? (part.end - 1) / kRun * kRun : part.begin - kRun;
  auto at = [&](int first) __attribute__((always_inline)) { return (span.run + first / kRun) * r.heads + head; };

  if (side == 0) {
    f32x4 grad[KEYS / 16];
#pragma unroll
    for (int t = 0; t < KEYS / 16; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key_of(t, g, i);
        grad[t][i] = 0.0f;
        if constexpr (MAPS) {
          grad[t][i] = units && key == col ? 1.0f : 0.0f;
        } else {
          const float *from = part.end < span.len ? w.starts + place.unit * states : r.dh_last ? r.dh_last + sequence * states : nullptr;
          if (from && inside && key < keys) grad[t][i] = from[static_cast<int64_t>(key) * values + col];
        }
      }
    auto keep = [&](float *to, int width) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < KEYS / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = key_of(t, g, i);
          if (inside && key < keys) to[static_cast<int64_t>(key) * width + col] = grad[t][i];
        }
    };
    __syncthreads();
    __syncthreads();
    __syncthreads();
    for (int first = last, buffer = 0; first >= part.begin; first -= kRun, buffer = (buffer + 1) % BUFFERS) {
      again();
      const uint16_t *k = lds.k[buffer];
      if constexpr (!MAPS) keep(w.grads + at(first) * (states + kRun * r.values), values);
      const float whole = lds.into[kRun - 1];
      f32x4 z[kTiles];
#pragma unroll
      for (int m = 0; m < kTiles; ++m) z[m] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const Cut<kFull> part = cut_tiles<kFull>(grad[2 * s], grad[2 * s + 1]);
        Cut<NP> rows[kTiles];
        tile_rows<KEYS>(rows, k, s, lane);
        multiply_rows<kFull>(z, rows, part);
#pragma unroll
        for (int t = 2 * s; t < 2 * s + 2; ++t) grad[t] = grad[t] * whole + lds.d[wave][t][lane];
      }
#pragma unroll
      for (int m = 0; m < kTiles; ++m) z[m] = z[m] * *reinterpret_cast<const f32x4 *>(lds.out + 16 * m + 4 * g) + lds.z[wave][m][lane];
      {
        const Cut<kFull> a = cut_tiles<kFull>(z[0], z[1]), c = cut_tiles<kFull>(z[2], z[3]);
#pragma unroll
        for (int m = 0; m < kTiles; ++m) z[m] = f32x4{0, 0, 0, 0};
        multiply_triangle<kFull, kFull, kFull, true>(z, lds.frags, a, c, lane);
      }
      if constexpr (!MAPS) {
        float *to = w.grads + at(first) * (states + kRun * r.values) + states;
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (inside) to[static_cast<int64_t>(16 * m + 4 * g + i) * values + col] = z[m][i];
      }
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
        z[m] *= -(*reinterpret_cast<const f32x4 *>(lds.rate + 16 * m + 4 * g) * *reinterpret_cast<const f32x4 *>(lds.into + 16 * m + 4 * g));
      __syncthreads();
      const Cut<kFull> a = cut_tiles<kFull>(z[0], z[1]), c = cut_tiles<kFull>(z[2], z[3]);
      multiply_columns<KEYS, NP>(grad, k, a, c, lane);
      if constexpr (BUFFERS == 1) __syncthreads();
      __syncthreads();
    }
    if constexpr (MAPS)
      keep(w.maps + static_cast<int64_t>(place.unit) * keys * (keys + values) + (units ? values : 0), keys + values);
    else if (r.dh0 && part.part == 0)
      keep(r.dh0 + sequence * states, values);
  } else {
    Fetched<T, KEYS, FRAGS, WHOLE> next;  // keys and T^T of the front's next run, dY of the run behind it
    Raw8<T> q[TILE ? KEYS / 32 : 1];
    auto steps = [&](int first) __attribute__((always_inline)) { return min(kRun, span.len - first); };
    auto fetch_front = [&](int first) __attribute__((always_inline)) {
      next.fetch_keys(thread, r.k, keys, span.batch, span.row + first, steps(first), key_head);
      next.fetch_factors(thread, w.triangles + (at(first) * Tri::kAll + Tri::kTt) * kWave, w.factors[at(first)]);
    };
    auto put_front = [&](int first, int buffer) __attribute__((always_inline)) {
      next.put_factors(thread, lds);
      next.put_keys(thread, lds.k[buffer], keys, steps(first));
    };
    auto fetch_back = [&](int first) __attribute__((always_inline)) {
      next.fetch_values(thread, r.dy, values, span.batch, span.row + first, steps(first), head, first_col);
      if constexpr (TILE)
        fetch_rows<T, KEYS, WHOLE>(q, thread, r.q, keys, span.batch, span.row + first, steps(first), key_head);
    };
    auto put_back = [&](int first) __attribute__((always_inline)) {
      if (units) {
#pragma unroll
        for (auto &v : next.v)
#pragma unroll
          for (auto &word : v.w) word = u32x4{0, 0, 0, 0};
      }
      next.put_values(thread, lds, values, steps(first), first_col);
      if constexpr (TILE) put_rows<T, KEYS, WHOLE>(q, thread, lds.q, keys, steps(first));
    };
    f32x4 z[kTiles], d[KEYS / 16], into[kTiles];
    Cut<kFull> p[kFrags];  // P^T
    auto fetch_own = [&](int first) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kFrags; ++i)
        p[i] = load_frag<kFull>(w.triangles + (at(first) * Tri::kAll + Tri::kP) * kWave, i, kFull, lane);
#pragma unroll
      for (int m = 0; m < kTiles; ++m) into[m] = *reinterpret_cast<const f32x4 *>(w.factors[at(first)].into + 16 * m + 4 * g);
    };
    auto compute = [&](int first) __attribute__((always_inline)) {
      f32x4 dy[kTiles];
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        dy[m] = value_column(lds.v, m, 16 * wave, lane);
        z[m] = f32x4{0, 0, 0, 0};
      }
      {
        const Cut<NP> a = cut_tiles<NP>(dy[0], dy[1]), c = cut_tiles<NP>(dy[2], dy[3]);
        multiply_triangle<kFull, true, false>(z, p, a, c);
      }
      part_done();
#pragma unroll
      for (int m = 0; m < kTiles; ++m) dy[m] *= r.scale * into[m];
      const Cut<kFull> a = cut_tiles<kFull>(dy[0], dy[1]), c = cut_tiles<kFull>(dy[2], dy[3]);
#pragma unroll
      for (int t = 0; t < KEYS / 16; ++t) d[t] = f32x4{0, 0, 0, 0};
      if constexpr (TILE) {
        multiply_columns<KEYS, NP>(d, lds.q, a, c, lane);
      } else {
#pragma unroll
        for (int t = 0; t < KEYS / 16; ++t) {  // straight from memory, as results hold the steps
          const int key = key_of(t, x / 4, x % 4), n = steps(first);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const f32x4 lo = load_column<T>(r.q, span.batch, span.row + first, n, key_head, 2 * s, g, key, key < keys);
            const f32x4 hi = load_column<T>(r.q, span.batch, span.row + first, n, key_head, 2 * s + 1, g, key, key < keys);
            multiply<kFull>(d[t], cut_tiles<NP>(lo, hi), s ? c : a);
          }
          part_done();
        }
      }
    };
    auto leave = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int m = 0; m < kTiles; ++m) lds.z[wave][m][lane] = z[m];
#pragma unroll
      for (int t = 0; t < KEYS / 16; ++t) lds.d[wave][t][lane] = d[t];
    };
    if (last >= part.begin) {
      fetch_own(last);
      fetch_front(last);
      fetch_back(last);
      put_front(last, 0);
      put_back(last);
    }
    __syncthreads();
    // the first run's products by themselves; then always one run ahead
    if (last >= part.begin) {
      compute(last);
      const int then = max(last - kRun, part.begin);
      fetch_back(then);
      fetch_own(then);
      leave();
    }
    __syncthreads();
    if (last >= part.begin) put_back(max(last - kRun, part.begin));
    __syncthreads();
    for (int first = last, buffer = 0; first >= part.begin; first -= kRun, buffer = (buffer + 1) % BUFFERS) {
      again();
      // in front of the first run that one again: loads stand in no branch
      const int then = max(first - kRun, part.begin), later = max(then - kRun, part.begin);
      fetch_front(then);
      fetch_back(later);
      compute(then);
      __syncthreads();
      again();
      leave();
      if constexpr (BUFFERS == 2) put_front(then, 1 - buffer);
      put_back(later);
      fetch_own(later);
      if constexpr (BUFFERS == 1) {
        __syncthreads();
        put_front(then, 0);
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------ one run's gradients
// A workgroup has one run of one head of queries and keys, and goes through the
// heads that share it, so that their gradients add up in registers. Values are
// taken 64 or 32 columns at a time: threads bring eight or four of a step of U, Z and dY
// each to LDS, then the waves take products over the values, each for keys (and steps)
// of its own, transposed, so that a lane has four neighbouring keys. What K S
// and K D would be needed for, the sums over a step's values, comes from Z S^T and U D^T
// by the step's key: z . S^T k = k . S z. States, X, Z and fields of a run of 128 x 128 are
// 290 KB, 1.3 GB for 8 x 2048 steps of 16 heads in 377 us: 3.5 TB/s, with the matrix units
// busy 24 % of the time and LDS conflicts 18 % (two parts an operand: 321 us).
constexpr int kGradWaves = 8;
constexpr int kGradThreads = kGradWaves * kWave;
constexpr int kGrams = 10;  // 16x16 tiles of a lower triangle of kRun
constexpr int kGradJobs = (2 * kGrams + kGradWaves - 1) / kGradWaves;

__host__ __device__ constexpr int gram_row(int t) { return t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3; }
__host__ __device__ constexpr int gram_col(int t) { return t - gram_row(t) * (gram_row(t) + 1) / 2; }

// The sum over 16 neighbouring lanes, in each of them.
__device__ __forceinline__ float across16(float v) {
  auto turned = [](float f, auto by) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(f), 0x120 + decltype(by)::value, 0xf, 0xf, true));
  };
  v += turned(v, Const<8>{});
  v += turned(v, Const<4>{});
  v += turned(v, Const<2>{});
  return v + turned(v, Const<1>{});
}
__device__ __forceinline__ float across_groups(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// QUERIES: a tile of their own for the queries, where it fits.
template <typename T, int KEYS, int COLS, bool QUERIES>
struct GradsLds {
  static constexpr int NP = kParts<T>, KR = KEYS + 8, VR = COLS + 8, FR = kRun + 8;  // elements between rows
  alignas(16) uint16_t k[NP * kRun * KR];  // keys, and without a tile of their own at the end queries
  alignas(16) uint16_t q[QUERIES ? NP * kRun * KR : 8];
  union {
    struct {
      alignas(16) uint16_t u[kFull * kRun * VR], z[kFull * kRun * VR], dy[NP * kRun * VR];
    } one;
    struct {
      alignas(16) uint16_t f[kFull * kRun * FR], h[kFull * kRun * FR];
    } two;
  };
  alignas(16) Factors f;
  float sums[KEYS / 16][kRun];  // what of dG goes through the states, of each 16 keys
  float rates[kRun];            // z . x
  float turns[KEYS / 16][kRun]; // q . dq of this head, of each 16 keys
  float lasts[kGradWaves];      // what the last step's G has beside
  float gram_rows[2 * kGrams][16], gram_cols[2 * kGrams][16];
};

// Two workgroups on a CU where LDS and registers hold them: one loads while the
// other computes. (8 x 2048 steps, 16 heads of 128 x 128 bf16: one, 64 columns at a time,
// 488 us, two by 32 columns 407 on the same card; 32 heads of 64 x 64 with 8 of queries
// and keys: bf16, 64 columns either way, 547 and 358, fp16, two by 32, 546 and 444. Shared
// heads' gradients take the registers of 128 keys.)
template <typename T, int KEYS, bool SHARED>
constexpr bool grads_twice() {
  return (!SHARED || KEYS <= 64) && 2 * sizeof(GradsLds<T, KEYS, 32, false>) <= kLdsBytes;
}
// Value columns at a time: half as many where only that leaves room for a second workgroup.
template <typename T, int KEYS, bool SHARED>
constexpr int grads_cols() {
  return grads_twice<T, KEYS, SHARED>() && 2 * sizeof(GradsLds<T, KEYS, 64, false>) > kLdsBytes ? 32 : 64;
}
template <typename T, int KEYS, bool SHARED>
constexpr bool grads_queries() {
  return (grads_twice<T, KEYS, SHARED>() ? 2 : 1) * sizeof(GradsLds<T, KEYS, grads_cols<T, KEYS, SHARED>(), true>) <= kLdsBytes;
}

// SHARED: several heads have the same queries and keys.
template <typename T, int KEYS, bool WHOLE, bool SHARED>
__global__ __launch_bounds__(kGradThreads, (grads_twice<T, KEYS, SHARED>() ? 4 : 2)) void delta_grads_kernel(
    fftmv_delta_rule_t r, DeltaWorkspace w) {
  constexpr bool QUERIES = grads_queries<T, KEYS, SHARED>();
  constexpr int COLS = grads_cols<T, KEYS, SHARED>(), PER = COLS / 8;  // of them a thread's
  using Lds = GradsLds<T, KEYS, COLS, QUERIES>;
  constexpr int NP = kParts<T>, NO = kFull, S = KEYS / 32, VR = Lds::VR, KR = Lds::KR, FR = Lds::FR;
  constexpr bool LATE = grads_twice<T, KEYS, SHARED>() && (KEYS == 128 || SHARED || (KEYS == 64 && COLS == 64 && !WHOLE));  // what the other workgroup hides need not be held
  constexpr int KT = KEYS / 16, MT = kTiles * KT / kGradWaves;  // tiles of keys, and of steps for one of them a wave
  __shared__ Lds lds;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int tile_k = wave % KT, tile_m = wave / KT * MT;  // this wave's keys and steps
  int thread = threadIdx.x, lane = thread % kWave, x = lane % 16, g = lane / 16;
  auto again = [&]() __attribute__((always_inline)) {
    thread = afresh(thread), lane = thread % kWave, x = lane % 16, g = lane / 16;
  };
  const uint32_t key_heads = static_cast<uint32_t>(r.key_heads);
  const int64_t slot = blockIdx.x / key_heads, key_head = blockIdx.x % key_heads;
  const Slot where = slot_of(r, slot);
  if (where.first < 0) return;
  const Span span = span_of(r, where.b);
  const int n = min(kRun, span.len - where.first);
  if (n <= 0) return;
  const int64_t row = span.row + where.first, states = r.keys * r.values;
  const int keys = static_cast<int>(r.keys), values = static_cast<int>(r.values);
  const int share = static_cast<int>(static_cast<uint32_t>(r.heads) / key_heads);

  // rows of 8 * CHUNKS elements into a tile
  auto fill = [&](uint16_t *tile, auto chunks, const Rows<T, WHOLE> &rows, int from) __attribute__((always_inline)) {
    constexpr int C = decltype(chunks)::value;
#pragma unroll
    for (int i = 0; i < (kRun * C + kGradThreads - 1) / kGradThreads; ++i) {
      const int u = thread + i * kGradThreads, t = u / C, c = u % C * 8;
      if (kRun * C % kGradThreads && u >= kRun * C) break;
      Raw8<T> v = rows.load(t, from + c);
      if (!WHOLE || from + 8 * C > rows.width) settle<WHOLE>(v, from + c, rows.width, t < n);
      const auto parts = cut_raw<T>(v);
#pragma unroll
      for (int p = 0; p < NP; ++p) *reinterpret_cast<u32x4 *>(tile + (p * kRun + t) * KR + c) = parts.p[p];
    }
  };

  // FP32 gradients of shared queries and keys add up in the outputs, others, which would round there, in registers. A
  // head's part of dq is whole before it joins them: its q . dq goes into this head's gates alone
  constexpr bool KEEP = SHARED && sizeof(T) == 2;
  f32x4 dq[MT], dk[MT];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < MT; ++m) dq[m] = dk[m] = f32x4{0, 0, 0, 0};
  };
  clear();
  auto store_gradients = [&](bool add) __attribute__((always_inline)) {
    again();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int t = 16 * (tile_m + m) + x, key = 16 * tile_k + 4 * g;
      if (t >= n) continue;
      T *q = head_row<T>(r.dq, span.batch, row + t, key_head) + key, *k = head_row<T>(r.dk, span.batch, row + t, key_head) + key;
      if (key + 4 <= keys) {
        float a[4] = {dq[m][0], dq[m][1], dq[m][2], dq[m][3]}, b[4] = {dk[m][0], dk[m][1], dk[m][2], dk[m][3]};
        if (SHARED && !KEEP && add) {
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] += static_cast<float>(q[i]), b[i] += static_cast<float>(k[i]);
        }
        store_vec(q, a, false);
        store_vec(k, b, false);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (key + i < keys) {
            const bool more = SHARED && !KEEP && add;
            q[i] = static_cast<T>(more ? dq[m][i] + static_cast<float>(q[i]) : dq[m][i]);
            k[i] = static_cast<T>(more ? dk[m][i] + static_cast<float>(k[i]) : dk[m][i]);
          }
      }
    }
  };

  int64_t head = key_head * share;
  do {
    again();
    const int64_t at = slot * r.heads + head;
    // states with X behind them, their gradients with Z: what is behind the last reads as zeros
    const int64_t each = states + kRun * r.values;
    const auto state = __builtin_amdgcn_make_buffer_rsrc(r.carries + at * each, 0, static_cast<int>(each * 4), kBufferFlags);
    const auto grad = __builtin_amdgcn_make_buffer_rsrc(w.grads + at * each, 0, static_cast<int>(each * 4), kBufferFlags);
    f32x4 gram[kGradJobs], yq[MT], zs[MT], ud[MT];  // the triangles' tiles; dY S^T (then dQ), Z S^T and U D^T, transposed
#pragma unroll
    for (int m = 0; m < MT; ++m) yq[m] = zs[m] = ud[m] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < kGradJobs; ++q) gram[q] = f32x4{0, 0, 0, 0};
    float last = 0.0f;  // of this wave's values: e^{G_last} <state, its gradient> and the sum of k . o
    __syncthreads();
    if (!QUERIES || head % share == 0) fill(lds.k, Const<KEYS / 8>{}, Rows<T, WHOLE>(r.k, span.batch, row, key_head, n, keys), 0);
    if (thread < static_cast<int>(sizeof(Factors) / 16))
      reinterpret_cast<u32x4 *>(&lds.f)[thread] = at_lane(reinterpret_cast<const u32x4 *>(w.factors + at), thread);
    if (QUERIES && head % share == 0) fill(lds.q, Const<KEYS / 8>{}, Rows<T, WHOLE>(r.q, span.batch, row, key_head, n, keys), 0);
    again();
    const float own_rate = w.factors[at].rate[thread / 8];
    float rate_sum = 0.0f;  // z . x of this thread's step and columns
    for (int from = 0; from < values; from += COLS) {
      if (from) __syncthreads();
      again();
      // rows of the state and its gradient, for the products with the values; behind the last key zeros
      u32x4 rows[COLS / 32][2][2];
      auto fetch_rows_of_states = [&](auto part) __attribute__((always_inline)) {
        constexpr int s = decltype(part)::value;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = 16 * tile_k + x;
          const int byte = (key < keys ? key * values + from + 32 * s + 8 * g + 4 * h : static_cast<int>(each)) * 4;
          rows[s][0][h] = __builtin_amdgcn_raw_buffer_load_b128(state, byte, 0, 0);
          rows[s][1][h] = __builtin_amdgcn_raw_buffer_load_b128(grad, byte, 0, 0);
        }
      };
      {  // a thread has PER columns of one step: U, Z and dY into LDS, dV out; dY by eights
        const int t = thread / 8, at_c = thread % 8 * PER, c = from + at_c, at_dy = at_c / 8 * 8;
        const int byte = static_cast<int>(states + t * values + c) * 4;
        u32x4 errors[PER / 4], zs_of[PER / 4];
#pragma unroll
        for (int h = 0; h < PER / 4; ++h) {
          errors[h] = __builtin_amdgcn_raw_buffer_load_b128(state, byte + 16 * h, 0, 0);
          zs_of[h] = __builtin_amdgcn_raw_buffer_load_b128(grad, byte + 16 * h, 0, 0);
        }
        Raw8<T> dy = Rows<T, WHOLE>(r.dy, span.batch, row, head, n, values).load(t, from + at_dy);
        if constexpr (!LATE) unrolled<0, COLS / 32>(fetch_rows_of_states);
        float u[8] = {}, z[8] = {};
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          const bool in = c + e < values;
          u[e] = in ? __uint_as_float(errors[e / 4][e % 4]) : 0.0f;
          z[e] = in ? __uint_as_float(zs_of[e / 4][e % 4]) : 0.0f;
          rate_sum = fmaf(z[e], u[e], rate_sum);
          u[e] *= own_rate;
        }
        const auto u_parts = cut<NO>(u), z_parts = cut<NO>(z);
        if (!WHOLE || from + COLS > values) settle<WHOLE>(dy, from + at_dy, values, t < n);
        const auto dy_parts = cut_raw<T>(dy);
        auto put = [&](uint16_t *tile, const u32x4 &part, int p) __attribute__((always_inline)) {
          uint16_t *to = tile + (p * kRun + t) * VR + at_c;
          if constexpr (PER == 8) {
            *reinterpret_cast<u32x4 *>(to) = part;
          } else {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            *reinterpret_cast<u32x2 *>(to) = u32x2{part[0], part[1]};
          }
        };
#pragma unroll
        for (int p = 0; p < NO; ++p) {
          put(lds.one.u, u_parts.p[p], p);
          put(lds.one.z, z_parts.p[p], p);
        }
        if (PER == 8 || thread % 2 == 0) {
#pragma unroll
          for (int p = 0; p < NP; ++p) *reinterpret_cast<u32x4 *>(lds.one.dy + (p * kRun + t) * VR + at_dy) = dy_parts.p[p];
        }
#pragma unroll
        for (int e = 0; e < PER; ++e) z[e] *= own_rate;
        if (t < n) {
          T *to = head_row<T>(r.dv, span.batch, row + t, head) + c;
          if (c + PER <= values) {
            if constexpr (sizeof(T) == 2 && PER == 8) {
              store_vec(to, z, false);
            } else {
              const float lo[4] = {z[0], z[1], z[2], z[3]}, hi[4] = {z[4], z[5], z[6], z[7]};
              store_vec(to, lo, false);
              if constexpr (PER == 8) store_vec(to + 4, hi, false);
            }
          } else {
#pragma unroll
            for (int e = 0; e < PER; ++e)
              if (c + e < values) to[e] = static_cast<T>(z[e]);
          }
        }
      }
      __syncthreads();
      again();
#pragma unroll
      for (int q = 0; q < kGradJobs; ++q) {
        const int job = wave + kGradWaves * q, tile = job < kGrams ? job : job - kGrams;
        if (job >= 2 * kGrams) break;
#pragma unroll
        for (int s = 0; s < COLS / 32; ++s) {
          const Cut<NO> u = plain_rows<VR, NO>(lds.one.u, gram_col(tile), s, lane);
          if (job < kGrams)
            multiply<NO>(gram[q], plain_rows<VR, NP>(lds.one.dy, gram_row(tile), s, lane), u);
          else
            multiply<NO>(gram[q], plain_rows<VR, NO>(lds.one.z, gram_row(tile), s, lane), u);
          if constexpr (KEYS == 128 && SHARED) part_done();
        }
      }
      part_done();
      again();
      unrolled<0, COLS / 32>([&](auto part) __attribute__((always_inline)) {
        constexpr int s = decltype(part)::value;
        if constexpr (LATE) fetch_rows_of_states(part);
        const int c = from + 32 * s + 8 * g;
        float b[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            b[0][4 * h + e] = __uint_as_float(rows[s][0][h][e]);
            b[1][4 * h + e] = __uint_as_float(rows[s][1][h][e]);
          }
        if (from + COLS > values) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            b[0][e] = c + e < values ? b[0][e] : 0.0f;
            b[1][e] = c + e < values ? b[1][e] : 0.0f;
          }
        }
        if (wave / KT == 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) last = fmaf(b[0][e] * lds.f.into[kRun - 1], b[1][e], last);
        }
        constexpr bool TIGHT = KEYS == 128 && (SHARED || sizeof(T) == 4);  // registers
        if constexpr (TIGHT) part_done();
        const Cut<NO> sp = cut<NO>(b[0]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          multiply<NO>(yq[m], sp, plain_rows<VR, NP>(lds.one.dy, tile_m + m, s, lane));
          multiply<NO>(zs[m], sp, plain_rows<VR, NO>(lds.one.z, tile_m + m, s, lane));
          if constexpr (TIGHT) part_done();
        }
        const Cut<NO> dp = cut<NO>(b[1]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          multiply<NO>(ud[m], dp, plain_rows<VR, NO>(lds.one.u, tile_m + m, s, lane));
          if constexpr (TIGHT) part_done();
        }
      });
    }
    again();
#pragma unroll
    for (int m = 0; m < MT; ++m) {  // a step's factors are a lane's here
      const int t = 16 * (tile_m + m) + x;
      const f32x4 o = ud[m] * lds.f.out[t], i = zs[m] * (lds.f.rate[t] * lds.f.into[t]);
      yq[m] *= r.scale * lds.f.into[t];
      dk[m] += o - i;
      float ends = 0.0f, sum = 0.0f;  // k . o, k . i
#pragma unroll
      for (int part = 0; part < NP; ++part) {
        const uint16_t *k = lds.k + (part * kRun + t) * KR + 16 * tile_k + 4 * g;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float key = __uint_as_float(static_cast<uint32_t>(k[e]) << 16);
          ends = fmaf(key, o[e], ends);
          sum = fmaf(key, i[e], sum);
        }
      }
      last += ends;
      sum = across_groups(sum + ends);
      if (g == 0) lds.sums[tile_k][t] = sum;
    }
    rate_sum += dpp<kDppQuadXor1>(rate_sum);
    rate_sum += dpp<kDppQuadXor2>(rate_sum);
    rate_sum += dpp<kDppRowHalfMirror>(rate_sum);
    if (thread % 8 == 0) lds.rates[thread / 8] = rate_sum;
    last = across_groups(across16(last));
    if (lane == 0) lds.lasts[wave] = last;
    __syncthreads();  // u, z and dy are done with

    // what goes through the triangles
#pragma unroll
    for (int q = 0; q < kGradJobs; ++q) {
      again();
      const int job = wave + kGradWaves * q, tile = job < kGrams ? job : job - kGrams;
      if (job >= 2 * kGrams) break;
      const int m = gram_row(tile), c = gram_col(tile), j = 16 * c + x;
      f32x4 raw = {0, 0, 0, 0};
      if (job < kGrams) {
        if constexpr (QUERIES) {
#pragma unroll
          for (int s = 0; s < S; ++s) multiply<NO>(raw, plain_rows<KR, NP>(lds.q, m, s, lane), plain_rows<KR, NP>(lds.k, c, s, lane));
        } else {
          const Rows<T, WHOLE> rows(r.q, span.batch, row, key_head, n, keys);
          Raw8<T> own[S];
#pragma unroll
          for (int s = 0; s < S; ++s) own[s] = rows.load(16 * m + x, 32 * s + 8 * g);
#pragma unroll
          for (int s = 0; s < S; ++s) {
            if (!WHOLE || keys < KEYS) settle<WHOLE>(own[s], 32 * s + 8 * g, keys, 16 * m + x < n);
            multiply<NO>(raw, cut_raw<T>(own[s]), plain_rows<KR, NP>(lds.k, c, s, lane));
          }
        }
      } else {
#pragma unroll
        for (int s = 0; s < S; ++s) multiply<NO>(raw, plain_rows<KR, NP>(lds.k, m, s, lane), plain_rows<KR, NP>(lds.k, c, s, lane));
      }
      uint16_t *to = job < kGrams ? lds.two.f : lds.two.h;
      const double sum_j = lds.f.sum[j];
      float down = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * m + 4 * g + i;
        const bool in = job < kGrams ? j <= t : j < t;
        const float e = in ? expf(static_cast<float>(lds.f.sum[t] - sum_j)) : 0.0f;
        // dG_t: q . dq holds this row of P but for its diagonal, which e^{G_t - G_t} is no factor of
        float v = (job < kGrams ? r.scale : -lds.f.rate[t]) * e * gram[q][i], line;
        if (!in) v = 0.0f;
        const float p = in ? v * raw[i] : 0.0f;
        if (job < kGrams) {
          line = across16(j == t ? -p : 0.0f);
          down += j < t ? p : 0.0f;
        } else {
          line = across16(p);
          down += p;
        }
        if (x == 0) lds.gram_rows[job][4 * g + i] = line;
#pragma unroll
        for (int a = 0; a < NO; ++a) {
          const __bf16 vb = static_cast<__bf16>(v);
          to[(a * kRun + t) * FR + j] = __builtin_bit_cast(uint16_t, vb);
          if (m % 2 == 0 && m == c) to[(a * kRun + t) * FR + j + 16] = 0;  // the tile right of it shares its slots
          v -= static_cast<float>(vb);
        }
      }
      down = across_groups(down);
      if (g == 0) lds.gram_cols[job][x] = down;
      part_done();
    }
    __syncthreads();

    again();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const Cut<NP> k = plain_columns<KR, NP>(lds.k, 32 * s, 16 * tile_k, lane);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (in_lower(tile_m + m, s)) {
          multiply<NO>(yq[m], k, plain_rows<FR, NO>(lds.two.f, tile_m + m, s, lane));
          multiply<NO>(dk[m], k, plain_rows<FR, NO>(lds.two.h, tile_m + m, s, lane));
        }
        if (in_upper(tile_m + m, s)) multiply<NO>(dk[m], k, plain_columns<FR, NO>(lds.two.h, 32 * s, 16 * (tile_m + m), lane));
      }
    }
    if constexpr (!QUERIES) {
      __syncthreads();
      fill(lds.k, Const<KEYS / 8>{}, Rows<T, WHOLE>(r.q, span.batch, row, key_head, n, keys), 0);
      __syncthreads();
    }
    const uint16_t *queries = QUERIES ? lds.q : lds.k;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const Cut<NP> q = plain_columns<KR, NP>(queries, 32 * s, 16 * tile_k, lane);
#pragma unroll
      for (int m = 0; m < MT; ++m)
        if (in_upper(tile_m + m, s)) multiply<NO>(dk[m], q, plain_columns<FR, NO>(lds.two.f, 32 * s, 16 * (tile_m + m), lane));
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {  // q . dq: step 16 m + x, four keys
      float sum = 0.0f;
      const int t = 16 * (tile_m + m) + x;
#pragma unroll
      for (int part = 0; part < NP; ++part) {
        const uint16_t *q = queries + (part * kRun + t) * KR + 16 * tile_k + 4 * g;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = fmaf(yq[m][i], __uint_as_float(static_cast<uint32_t>(q[i]) << 16), sum);
      }
      dq[m] += yq[m];
      sum = across_groups(sum);
      if (g == 0) lds.turns[tile_k][t] = sum;
    }
    __syncthreads();
    again();
    if (wave == 0) {  // the gates: lane i has step i
      double own = 0.0, end = 0.0;
#pragma unroll
      for (int v = 0; v < KT; ++v) own += static_cast<double>(lds.turns[v][lane]) - lds.sums[v][lane];
#pragma unroll
      for (int v = 0; v < kGradWaves; ++v) end += lds.lasts[v];
#pragma unroll
      for (int job = 0; job < 2 * kGrams; ++job) {
        const int tile = job % kGrams;
        if (gram_row(tile) == g) own += lds.gram_rows[job][x];
        if (gram_col(tile) == g) own -= lds.gram_cols[job][x];
      }
      // sum over this step and those behind it
      const double all = lane_sums(own, lane);
      const double grad_log = __shfl(all, kWave - 1) - all + own + end;
      if (lane < n) {
        const float gate = static_cast<float>(*head_row<T>(r.gate, span.batch, row + lane, head));
        const float beta = static_cast<float>(*head_row<T>(r.beta, span.batch, row + lane, head));
        const float slope = r.decay == FFTMV_DECAY_SIGMOID ? 1.0f / (1.0f + expf(gate)) : 1.0f;
        const float b = rate_of(r.rate, beta);
        const float turn = r.rate == FFTMV_RATE_SIGMOID ? b / (1.0f + expf(beta)) : 1.0f;
        *head_row<T>(r.dgate, span.batch, row + lane, head) = static_cast<T>(static_cast<float>(grad_log) * slope);
        *head_row<T>(r.dbeta, span.batch, row + lane, head) = static_cast<T>(lds.rates[lane] * turn);
      }
    }
    if constexpr (SHARED && !KEEP) {
      store_gradients(head > key_head * share);
      clear();
    }
  } while (SHARED && ++head < (key_head + 1) * share);
  if constexpr (!SHARED || KEEP) store_gradients(false);
}

template <typename T>
hipError_t launch_delta_backward(const fftmv_delta_rule_t &r, hipStream_t s) {
  const int64_t runs = delta_runs(r.batch, r.steps, r.offsets != nullptr), sequences = r.batch * r.heads;
  DeltaWorkspace w;
  delta_workspace(r.batch, r.steps, r.heads, r.keys, r.values, r.offsets != nullptr, true, r.workspace, &w);
  const int64_t blocks = (r.values + kValues - 1) / kValues, units = (r.keys + kValues - 1) / kValues;
  if (!grid_fits(runs * r.heads, kFrontThreads) || !grid_fits(sequences * ((r.values + 15) / 16), 512) || !grid_fits(runs * r.key_heads, kGradThreads) ||
      !grid_fits(sequences * w.cuts.parts * (blocks + units), kChainThreads))
    return hipErrorInvalidConfiguration;
  return by_keys(r.keys, [&](auto k) {
    constexpr int KEYS = decltype(k)::value;
    if (runs > 0) {
      const hipError_t e = by_two(delta_whole_rows(r), [&](auto whole) {
        delta_factors_kernel<T, KEYS, decltype(whole)::value != 0, true>
            <<<static_cast<unsigned>(runs * r.heads), kFrontThreads, 0, s>>>(r, w);
        return hipGetLastError();
      });
      if (e != hipSuccess) return e;
    }
    const hipError_t e = by_two(delta_whole(r, r.dy, r.dy), [&](auto whole) {
      constexpr bool WHOLE = decltype(whole)::value != 0;
      const unsigned chains = static_cast<unsigned>(sequences * w.cuts.parts), columns = static_cast<unsigned>(blocks);
      if (w.cuts.parts > 1) {
        const unsigned all = chains * static_cast<unsigned>(blocks + units);
        delta_back_chain_kernel<T, KEYS, WHOLE, true><<<all, kChainThreads, 0, s>>>(r, w);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        delta_join_kernel<T, KEYS, true>
            <<<dim3(static_cast<unsigned>(sequences), static_cast<unsigned>((r.values + 15) / 16)), KEYS / 16 * kWave, 0, s>>>(r, w);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
      }
      delta_back_chain_kernel<T, KEYS, WHOLE, false><<<chains * columns, kChainThreads, 0, s>>>(r, w);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    if (runs == 0) return hipSuccess;
    return by_two(delta_whole(r, r.dy, r.v), [&](auto whole) {
      return by_two(r.heads > r.key_heads, [&](auto shared) {
        delta_grads_kernel<T, KEYS, decltype(whole)::value != 0, decltype(shared)::value != 0>
            <<<static_cast<unsigned>(runs * r.key_heads), kGradThreads, 0, s>>>(r, w);
        return hipGetLastError();
      });
    });
  });
}

}  // namespace fftmv
