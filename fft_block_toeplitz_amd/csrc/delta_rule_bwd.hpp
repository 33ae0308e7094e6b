// Backward pass of the gated delta rule. With D the gradient of the state behind
// a run and dY that of its outputs,
//   Z   = T^T (P^T dY + diag(e^{G_last - G}) K D)      the gradient of U
//   D'  = e^{G_last} D + (scale diag(e^G) Q)^T dY - (diag(b e^G) K)^T Z
// goes from run to run, from the last to the first, as the state does forward;
// everything else belongs to one run:
//   dV  = diag(b) Z
//   dP  = dY U^T,  N = Z U^T, both lower triangles;  F = scale E o dP,  H = -diag(b) E o N
//   dQ  = scale diag(e^G) dY S^T + F K
//   dK  = F^T Q + (H + H^T) K + diag(e^{G_last - G}) U D^T - diag(b e^G) Z S^T
//   db_j = z_j . x_j - sum_i E_ji k_j.k_i N_ji   with X = V - diag(e^G) K S
//   dG_i collects, with its sign, every product that e^{G_i} is a factor of; the
//   gradient of log a_t is the sum of dG_i over i >= t.
// So three kernels: the factors, the chain of D, and the gradients of all runs
// at once, which compute U and Z again from the states that the passes kept:
// that costs a tenth of a run's products, and reading them back half of its bytes.
#pragma once

#include "delta_rule.hpp"

namespace fftmv {

constexpr int kBackWaves = 4;
constexpr int kBackThreads = kBackWaves * kWave;

template <typename T, int KEYS>
__global__ __launch_bounds__(kBackThreads) void delta_back_chain_kernel(fftmv_delta_rule_t r, DeltaWorkspace w) {
  using Tri = Triangles<T, true>;
  constexpr int NP = kParts<T>, S = KEYS / 32;
  __shared__ __align__(16) uint16_t ktile[NP * kRun * kTileRow<KEYS>], qtile[NP * kRun * kTileRow<KEYS>];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, x = lane % 16, g = lane / 16;
  const int64_t head = blockIdx.x % r.heads, b = blockIdx.x / r.heads;
  const int64_t key_head = head / (r.heads / r.key_heads);
  const int keys = static_cast<int>(r.keys), values = static_cast<int>(r.values);
  const int col = (blockIdx.y * kBackWaves + wave) * 16 + x;
  const bool inside = col < values;
  const Span span = span_of(r, b);
  const int64_t states = r.keys * r.values;

  f32x4 grad[KEYS / 16];
#pragma unroll
  for (int t = 0; t < KEYS / 16; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = key_of(t, g, i);
      grad[t][i] = r.dh_last && inside && key < keys
                       ? r.dh_last[(b * r.heads + head) * states + static_cast<int64_t>(key) * values + col]
                       : 0.0f;
    }
  auto keep = [&](float *to) {
#pragma unroll
    for (int t = 0; t < KEYS / 16; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key_of(t, g, i);
        if (inside && key < keys) to[static_cast<int64_t>(key) * values + col] = grad[t][i];
      }
  };

  for (int first = (span.len - 1) / kRun * kRun; first >= 0 && span.len > 0; first -= kRun) {
    const int n = min(kRun, span.len - first);
    const int64_t row = span.row + first, at = (span.run + first / kRun) * r.heads + head;
    const Factors &f = w.factors[at];
    const u32x4 *tri = w.triangles + at * Tri::kAll * kWave;
    keep(w.grads + at * states);
    __syncthreads();
    fill_tile<T, KEYS, kBackThreads>(ktile, r.k, span.batch, row, n, key_head, keys);
    fill_tile<T, KEYS, kBackThreads>(qtile, r.q, span.batch, row, n, key_head, keys);
    f32x4 dy[kTiles];
#pragma unroll
    for (int m = 0; m < kTiles; ++m) dy[m] = load_column<T>(r.dy, span.batch, row, n, head, m, g, col, inside);
    __syncthreads();

    f32x4 z[kTiles];
#pragma unroll
    for (int m = 0; m < kTiles; ++m) z[m] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const Cut<kFull> part = cut_tiles<kFull>(grad[2 * s], grad[2 * s + 1]);
#pragma unroll
      for (int m = 0; m < kTiles; ++m) multiply<kFull>(z[m], tile_rows<KEYS, NP>(ktile, m, s, lane), part);
    }
    {
      const Cut<NP> a = cut_tiles<NP>(dy[0], dy[1]), c = cut_tiles<NP>(dy[2], dy[3]);
      const u32x4 *p = tri + Tri::kP * kWave;
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        z[m] *= *reinterpret_cast<const f32x4 *>(f.out + 16 * m + 4 * g);
        if (m < 2) multiply<kFull>(z[m], load_frag<kFull>(p, upper_frag(m, 0), Tri::kPParts, lane), a);
        multiply<kFull>(z[m], load_frag<kFull>(p, upper_frag(m, 1), Tri::kPParts, lane), c);
      }
    }
    {
      const Cut<kFull> a = cut_tiles<kFull>(z[0], z[1]), c = cut_tiles<kFull>(z[2], z[3]);
      const u32x4 *p = tri + Tri::kTt * kWave;
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        z[m] = f32x4{0, 0, 0, 0};
        if (m < 2) multiply<kFull>(z[m], load_frag<kFull>(p, upper_frag(m, 0), Tri::kTtParts, lane), a);
        multiply<kFull>(z[m], load_frag<kFull>(p, upper_frag(m, 1), Tri::kTtParts, lane), c);
      }
    }
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      const f32x4 into = *reinterpret_cast<const f32x4 *>(f.into + 16 * m + 4 * g);
      const f32x4 rate = *reinterpret_cast<const f32x4 *>(f.rate + 16 * m + 4 * g);
      z[m] *= -(rate * into);
      dy[m] *= into * r.scale;
    }
    const float whole = f.into[kRun - 1];
    const Cut<kFull> za = cut_tiles<kFull>(z[0], z[1]), zc = cut_tiles<kFull>(z[2], z[3]);
    const Cut<kFull> ya = cut_tiles<kFull>(dy[0], dy[1]), yc = cut_tiles<kFull>(dy[2], dy[3]);
#pragma unroll
    for (int t = 0; t < KEYS / 16; ++t) {
      grad[t] *= whole;
      multiply<kFull>(grad[t], tile_columns<KEYS, NP>(ktile, t, 0, lane), za);
      multiply<kFull>(grad[t], tile_columns<KEYS, NP>(ktile, t, 1, lane), zc);
      multiply<kFull>(grad[t], tile_columns<KEYS, NP>(qtile, t, 0, lane), ya);
      multiply<kFull>(grad[t], tile_columns<KEYS, NP>(qtile, t, 1, lane), yc);
    }
  }
  if (r.dh0) keep(r.dh0 + (b * r.heads + head) * states);
}

// ------------------------------------------------------------ one run's gradients
// A workgroup has one run of one head of queries and keys, and goes through the
// heads that share it, so that their gradients add up in registers. Values are
// taken 64 columns at a time: 16 for a wave while U and Z are computed, then all
// of them for a wave's own keys.
constexpr int kValues = 64;
constexpr int kGrams = 10;  // 16x16 tiles of a lower triangle of kRun

__host__ __device__ constexpr int gram_row(int t) { return t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3; }
__host__ __device__ constexpr int gram_col(int t) { return t - gram_row(t) * (gram_row(t) + 1) / 2; }

__device__ __forceinline__ float across16(float v) {
#pragma unroll
  for (int d = 1; d < 16; d *= 2) v += __shfl_xor(v, d);
  return v;
}

template <typename T, int KEYS>
struct GradsLds {
  static constexpr int NP = kParts<T>, NO = kOut<T>, VR = kTileRow<kValues>;
  alignas(16) uint16_t k[NP * kRun * kTileRow<KEYS>];  // keys, and at the end queries
  union {
    struct {
      alignas(16) uint16_t u[NO * kRun * VR], z[NO * kRun * VR], dy[NP * kRun * VR];
    } one;
    struct {
      alignas(16) uint16_t f[NO * kRun * VR], h[NO * kRun * VR];
    } two;
  };
  float rows[kBackWaves][kRun];   // dG by row, of each wave's keys
  float lasts[kBackWaves];        // what the last step's G has beside
  float rates[kBackWaves][kRun];  // z . x by row, of each wave's values
  float gram_rows[2 * kGrams][16], gram_cols[2 * kGrams][16], gram_rates[kGrams][16];
};

template <typename T, int KEYS>
__global__ __launch_bounds__(kBackThreads) void delta_grads_kernel(fftmv_delta_rule_t r, DeltaWorkspace w) {
  using Tri = Triangles<T, true>;
  using Lds = GradsLds<T, KEYS>;
  constexpr int NP = kParts<T>, NO = kOut<T>, S = KEYS / 32, VR = Lds::VR;
  constexpr int KT = KEYS / 16 > kBackWaves ? KEYS / 16 / kBackWaves : 1;  // tiles of keys a wave
  constexpr int JOBS = 2 * kGrams / kBackWaves;
  __shared__ Lds lds;
  const int wave = threadIdx.x / kWave, lane0 = threadIdx.x % kWave;
  const int64_t slot = blockIdx.x / r.key_heads, key_head = blockIdx.x % r.key_heads;
  const Slot where = slot_of(r, slot);
  if (where.first < 0) return;
  const Span span = span_of(r, where.b);
  const int n = min(kRun, span.len - where.first);
  if (n <= 0) return;
  const int64_t row = span.row + where.first, states = r.keys * r.values;
  const int keys = static_cast<int>(r.keys), values = static_cast<int>(r.values);
  const int share = static_cast<int>(r.heads / r.key_heads);
  const bool mine = wave * KT < KEYS / 16;  // this wave has keys

  f32x4 dq[kTiles][KT], dk[kTiles][KT];
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int c = 0; c < KT; ++c) dq[m][c] = dk[m][c] = f32x4{0, 0, 0, 0};

  for (int64_t head = key_head * share; head < (key_head + 1) * share; ++head) {
    const int64_t at = slot * r.heads + head;
    const Factors &f = w.factors[at];
    const u32x4 *tri = w.triangles + at * Tri::kAll * kWave;
    const float *state = r.carries + at * states, *grad = w.grads + at * states;
    f32x4 aq[kTiles][KT], az[kTiles][KT], au[kTiles][KT], gram[JOBS], zx[kTiles];
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      zx[m] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < KT; ++c) aq[m][c] = az[m][c] = au[m][c] = f32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int q = 0; q < JOBS; ++q) gram[q] = f32x4{0, 0, 0, 0};
    int lane = afresh(lane0), x = lane % 16, g = lane / 16;
    auto again = [&] { lane = afresh(lane0), x = lane % 16, g = lane / 16; };
    float dot = 0.0f;  // <state, its gradient>, of this wave's values
    __syncthreads();
    fill_tile<T, KEYS, kBackThreads>(lds.k, r.k, span.batch, row, n, key_head, keys);

    for (int from = 0; from < values; from += kValues) {
      __syncthreads();
      fill_tile<T, kValues, kBackThreads>(lds.one.dy, r.dy, span.batch, row, n, head, values, from);
      again();
      const int col = from + 16 * wave + x;
      const bool inside = col < values;
      // U and Z of 16 columns
      f32x4 u[kTiles], z[kTiles];
#pragma unroll
      for (int m = 0; m < kTiles; ++m) u[m] = z[m] = f32x4{0, 0, 0, 0};
      __syncthreads();
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float a[8], d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int key = 32 * s + 8 * g + e;
          const bool there = inside && key < keys;
          a[e] = there ? state[static_cast<int64_t>(key) * values + col] : 0.0f;
          d[e] = there ? grad[static_cast<int64_t>(key) * values + col] : 0.0f;
          dot = fmaf(a[e], d[e], dot);
        }
        const Cut<NO> sp = cut<NO>(a), dp = cut<NO>(d);
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          const Cut<NP> k = tile_rows<KEYS, NP>(lds.k, m, s, lane);
          multiply<NO>(u[m], k, sp);
          multiply<NO>(z[m], k, dp);
        }
        part_done();
      }
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        again();
        const f32x4 v = load_column<T>(r.v, span.batch, row, n, head, m, g, col, inside);
        const f32x4 into = *reinterpret_cast<const f32x4 *>(f.into + 16 * m + 4 * g);
        u[m] = v - into * u[m];
        z[m] *= *reinterpret_cast<const f32x4 *>(f.out + 16 * m + 4 * g);
      }
      f32x4 xs[kTiles];
#pragma unroll
      for (int m = 0; m < kTiles; ++m) xs[m] = u[m];
      {
        const Cut<NO> a = cut_tiles<NO>(u[0], u[1]), c = cut_tiles<NO>(u[2], u[3]);
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          u[m] = f32x4{0, 0, 0, 0};
          multiply<NO>(u[m], load_frag<NO>(tri, lower_frag(m, 0), Tri::kTParts, lane), a);
          if (m >= 2) multiply<NO>(u[m], load_frag<NO>(tri, lower_frag(m, 1), Tri::kTParts, lane), c);
        }
      }
      part_done();
      {
        const u32x4 *p = tri + Tri::kP * kWave;
        const Cut<NP> a = plain_columns<VR, NP, 16>(lds.one.dy, 0, 16 * wave, lane);
        const Cut<NP> c = plain_columns<VR, NP, 16>(lds.one.dy, 32, 16 * wave, lane);
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          if (m < 2) multiply<NO>(z[m], load_frag<NO>(p, upper_frag(m, 0), Tri::kPParts, lane), a);
          multiply<NO>(z[m], load_frag<NO>(p, upper_frag(m, 1), Tri::kPParts, lane), c);
        }
      }
      part_done();
      {
        const Cut<NO> a = cut_tiles<NO>(z[0], z[1]), c = cut_tiles<NO>(z[2], z[3]);
        const u32x4 *p = tri + Tri::kTt * kWave;
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          z[m] = f32x4{0, 0, 0, 0};
          if (m < 2) multiply<NO>(z[m], load_frag<NO>(p, upper_frag(m, 0), Tri::kTtParts, lane), a);
          multiply<NO>(z[m], load_frag<NO>(p, upper_frag(m, 1), Tri::kTtParts, lane), c);
        }
      }
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        again();
        const f32x4 rate = *reinterpret_cast<const f32x4 *>(f.rate + 16 * m + 4 * g);
        zx[m] += z[m] * xs[m];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 16 * m + 4 * g + i;
          if (inside && t < n) head_row<T>(r.dv, span.batch, row + t, head)[col] = static_cast<T>(rate[i] * z[m][i]);
          float ur = u[m][i], zr = z[m][i];
#pragma unroll
          for (int p = 0; p < NO; ++p) {
            const __bf16 ub = static_cast<__bf16>(ur), zb = static_cast<__bf16>(zr);
            lds.one.u[(p * kRun + t) * VR + 16 * wave + x] = __builtin_bit_cast(uint16_t, ub);
            lds.one.z[(p * kRun + t) * VR + 16 * wave + x] = __builtin_bit_cast(uint16_t, zb);
            ur -= static_cast<float>(ub);
            zr -= static_cast<float>(zb);
          }
        }
      }
      __syncthreads();
      // products over the values: this wave's keys, and its tiles of the triangles
#pragma unroll
      for (int s = 0; s < kValues / 32; ++s) {
        again();
        const int c0 = from + 32 * s + 8 * g;
        if (mine) {
          Cut<NO> sp[KT], dp[KT];
#pragma unroll
          for (int c = 0; c < KT; ++c) {
            const int key = 16 * (wave * KT + c) + x;
            sp[c] = load_wide<NO>(state + static_cast<int64_t>(min(key, keys - 1)) * values, c0, values, key < keys);
            dp[c] = load_wide<NO>(grad + static_cast<int64_t>(min(key, keys - 1)) * values, c0, values, key < keys);
          }
#pragma unroll
          for (int m = 0; m < kTiles; ++m) {
            const Cut<NP> y = tile_rows<kValues, NP>(lds.one.dy, m, s, lane);
            const Cut<NO> zz = tile_rows<kValues, NO>(lds.one.z, m, s, lane), uu = tile_rows<kValues, NO>(lds.one.u, m, s, lane);
#pragma unroll
            for (int c = 0; c < KT; ++c) {
              multiply<NO>(aq[m][c], y, sp[c]);
              multiply<NO>(az[m][c], zz, sp[c]);
              multiply<NO>(au[m][c], uu, dp[c]);
            }
            part_done();
          }
        }
#pragma unroll
        for (int q = 0; q < JOBS; ++q) {
          const int job = wave + kBackWaves * q, tile = job < kGrams ? job : job - kGrams;
          const Cut<NO> uu = tile_rows<kValues, NO>(lds.one.u, gram_col(tile), s, lane);
          if (job < kGrams)
            multiply<NO>(gram[q], tile_rows<kValues, NP>(lds.one.dy, gram_row(tile), s, lane), uu);
          else
            multiply<NO>(gram[q], tile_rows<kValues, NO>(lds.one.z, gram_row(tile), s, lane), uu);
          part_done();
        }
      }
    }
    again();
    __syncthreads();  // u, z and dy are done with
    // what goes through the states
    f32x4 sums[kTiles];
    {
      float last = 0.0f;
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        const f32x4 into = *reinterpret_cast<const f32x4 *>(f.into + 16 * m + 4 * g);
        const f32x4 out = *reinterpret_cast<const f32x4 *>(f.out + 16 * m + 4 * g);
        const f32x4 rate = *reinterpret_cast<const f32x4 *>(f.rate + 16 * m + 4 * g);
        sums[m] = f32x4{0, 0, 0, 0};
        f32x4 behind = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < KT; ++c) {
          const f32x4 d = az[m][c] * (into * rate), o = au[m][c] * out;
          aq[m][c] *= into * r.scale;
          dq[m][c] += aq[m][c];
          dk[m][c] += o - d;
          if (mine) {
            const f32x4 k = tile_values<kTileRow<KEYS>, NP>(lds.k, m, 16 * (wave * KT + c), lane);
            sums[m] -= k * d;
            behind += k * o;
          }
        }
        sums[m] -= behind;
        last += behind[0] + behind[1] + behind[2] + behind[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float zr = across16(zx[m][i]);
          if (x == 0) lds.rates[wave][16 * m + 4 * g + i] = zr;
        }
      }
      last = fmaf(f.into[kRun - 1], dot, last);
      last = across16(last);
      last += __shfl_xor(last, 16);
      last += __shfl_xor(last, 32);
      if (lane == 0) lds.lasts[wave] = last;
    }
    part_done();
    // what goes through the triangles
#pragma unroll
    for (int q = 0; q < JOBS; ++q) {
      again();
      const int job = wave + kBackWaves * q, tile = job < kGrams ? job : job - kGrams;
      const int m = gram_row(tile), c = gram_col(tile), j = 16 * c + x;
      f32x4 raw = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const Cut<NP> kc = tile_rows<KEYS, NP>(lds.k, c, s, lane);
        if (job < kGrams)
          multiply<NO>(raw,
                       load_cut(head_row<T>(r.q, span.batch, row + min(16 * m + x, n - 1), key_head), 32 * s + 8 * g,
                                keys, 16 * m + x < n),
                       kc);
        else
          multiply<NO>(raw, tile_rows<KEYS, NP>(lds.k, m, s, lane), kc);
      }
      uint16_t *to = job < kGrams ? lds.two.f : lds.two.h;
      float down = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * m + 4 * g + i;
        const bool in = job < kGrams ? j <= t : j < t;
        const float e = in ? expf(static_cast<float>(f.sum[t] - f.sum[j])) : 0.0f;
        float v, rate = 0.0f;
        if (job < kGrams) {
          v = in ? r.scale * e * gram[q][i] : 0.0f;
        } else {
          v = in ? -f.rate[t] * e * gram[q][i] : 0.0f;
          rate = across16(in ? -e * raw[i] * gram[q][i] : 0.0f);
        }
        const float p = j < t ? v * raw[i] : 0.0f, line = across16(p);
        down += p;
        if (x == 0) {
          lds.gram_rows[job][4 * g + i] = line;
          if (job >= kGrams) lds.gram_rates[tile][4 * g + i] = rate;
        }
#pragma unroll
        for (int a = 0; a < NO; ++a) {
          const __bf16 vb = static_cast<__bf16>(v);
          to[(a * kRun + t) * VR + j] = __builtin_bit_cast(uint16_t, vb);
          if (m % 2 == 0 && m == c) to[(a * kRun + t) * VR + j + 16] = 0;  // the tile right of it shares its slots
          v -= static_cast<float>(vb);
        }
      }
      down += __shfl_xor(down, 16);
      down += __shfl_xor(down, 32);
      if (g == 0) lds.gram_cols[job][x] = down;
      part_done();
    }
    __syncthreads();

    if (mine) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Cut<NP> kc[KT];
        again();
#pragma unroll
        for (int c = 0; c < KT; ++c) kc[c] = plain_columns<kTileRow<KEYS>, NP, 4>(lds.k, 32 * s, 16 * (wave * KT + c), lane);
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          if (in_lower(m, s)) {
            const Cut<NO> f = tile_rows<kValues, NO>(lds.two.f, m, s, lane), h = tile_rows<kValues, NO>(lds.two.h, m, s, lane);
#pragma unroll
            for (int c = 0; c < KT; ++c) {
              multiply<NO>(dq[m][c], f, kc[c]);
              multiply<NO>(dk[m][c], h, kc[c]);
            }
          }
          if (in_upper(m, s)) {
            const Cut<NO> h = plain_columns<VR, NO, 4>(lds.two.h, 32 * s, 16 * m, lane);
#pragma unroll
            for (int c = 0; c < KT; ++c) multiply<NO>(dk[m][c], h, kc[c]);
          }
          part_done();
        }
      }
    }
    __syncthreads();
    fill_tile<T, KEYS, kBackThreads>(lds.k, r.q, span.batch, row, n, key_head, keys);
    __syncthreads();
    if (mine) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Cut<NP> qc[KT];
        again();
#pragma unroll
        for (int c = 0; c < KT; ++c) qc[c] = plain_columns<kTileRow<KEYS>, NP, 4>(lds.k, 32 * s, 16 * (wave * KT + c), lane);
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
          if (in_upper(m, s)) {
            const Cut<NO> f = plain_columns<VR, NO, 4>(lds.two.f, 32 * s, 16 * m, lane);
#pragma unroll
            for (int c = 0; c < KT; ++c) multiply<NO>(dk[m][c], f, qc[c]);
            part_done();
          }
      }
    }
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
#pragma unroll
      for (int c = 0; c < KT; ++c)
        if (mine) sums[m] += aq[m][c] * tile_values<kTileRow<KEYS>, NP>(lds.k, m, 16 * (wave * KT + c), lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = across16(sums[m][i]);
        if (x == 0) lds.rows[wave][16 * m + 4 * g + i] = s;
      }
    }
    __syncthreads();
    if (wave == 0) {  // the gates: lane i has step i
      double own = 0.0, rate = 0.0, last = 0.0;
#pragma unroll
      for (int v = 0; v < kBackWaves; ++v) {
        own += lds.rows[v][lane];
        rate += lds.rates[v][lane];
        last += lds.lasts[v];
      }
#pragma unroll
      for (int job = 0; job < 2 * kGrams; ++job) {
        const int tile = job % kGrams;
        if (gram_row(tile) == g) {
          own += lds.gram_rows[job][x];
          if (job >= kGrams) rate += lds.gram_rates[tile][x];
        }
        if (gram_col(tile) == g) own -= lds.gram_cols[job][x];
      }
      // sum over this step and those behind it
      const double all = lane_sums(own, lane);
      const double grad_log = __shfl(all, kWave - 1) - all + own + last;
      if (lane < n) {
        const float gate = static_cast<float>(*head_row<T>(r.gate, span.batch, row + lane, head));
        const float beta = static_cast<float>(*head_row<T>(r.beta, span.batch, row + lane, head));
        const float slope = r.decay == FFTMV_DECAY_SIGMOID ? 1.0f / (1.0f + expf(gate)) : 1.0f;
        const float b = rate_of(r.rate, beta);
        const float turn = r.rate == FFTMV_RATE_SIGMOID ? b / (1.0f + expf(beta)) : 1.0f;
        *head_row<T>(r.dgate, span.batch, row + lane, head) = static_cast<T>(static_cast<float>(grad_log) * slope);
        *head_row<T>(r.dbeta, span.batch, row + lane, head) = static_cast<T>(static_cast<float>(rate) * turn);
      }
    }
  }
  if (mine) {
    const int lane = afresh(lane0), x = lane % 16, g = lane / 16;
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int c = 0; c < KT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 16 * m + 4 * g + i, key = 16 * (wave * KT + c) + x;
          if (t < n && key < keys) {
            head_row<T>(r.dq, span.batch, row + t, key_head)[key] = static_cast<T>(dq[m][c][i]);
            head_row<T>(r.dk, span.batch, row + t, key_head)[key] = static_cast<T>(dk[m][c][i]);
          }
        }
  }
}

template <typename T>
hipError_t launch_delta_backward(const fftmv_delta_rule_t &r, hipStream_t s) {
  const int64_t runs = delta_runs(r.batch, r.steps, r.offsets != nullptr);
  DeltaWorkspace w;
  delta_workspace(runs, r.heads, r.keys, r.values, r.dtype, true, r.workspace, &w);
  const int64_t waves = (r.values + 15) / 16, blocks = (waves + kBackWaves - 1) / kBackWaves;
  if (!grid_fits(runs * r.heads, kWave) || !grid_fits(runs * r.key_heads, kBackThreads) ||
      !grid_fits(r.batch * r.heads * blocks, kBackThreads))
    return hipErrorInvalidConfiguration;
  return by_keys(r.keys, [&](auto k) {
    constexpr int KEYS = decltype(k)::value;
    if (runs > 0) {
      delta_factors_kernel<T, KEYS, true><<<static_cast<unsigned>(runs * r.heads), kWave, 0, s>>>(r, w);
      if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    const dim3 grid(static_cast<unsigned>(r.batch * r.heads), static_cast<unsigned>(blocks));
    delta_back_chain_kernel<T, KEYS><<<grid, kBackThreads, 0, s>>>(r, w);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (runs > 0) delta_grads_kernel<T, KEYS><<<static_cast<unsigned>(runs * r.key_heads), kBackThreads, 0, s>>>(r, w);
    return hipGetLastError();
  });
}

}  // namespace fftmv
