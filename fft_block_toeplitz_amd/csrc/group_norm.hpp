// Group normalisation with an activation over channels-last fields.
//
// A workgroup takes a slab of whole groups, neighbouring channels that its
// lanes read in 16-byte vectors, and spreads its rows over the rest of its
// threads. What fits a workgroup's registers is read once ("resident": short
// samples, single tokens); longer samples are read twice, once for the sums
// and once to be written ("split": rows shared out over many workgroups).
// The bound is memory traffic in all of them: 16000 tokens of 5000 channels in
// bf16 take 85 us forward (3.8 TB/s) and 182 us backward (2.6 TB/s; FP32 136 and
// 206, 4.7 TB/s), 8 x 4096 x 1024 fields 50 and 78 us (the split form's second
// reading, of 2 and 4 fields, comes from the last cache: 2.7 and 2.6 TB/s of the
// bytes that must move; FP32 86 and 133, 3.1 and 3.0 TB/s).
//
// A vector may cover channels of two groups (their width need not divide by
// eight): then sums go through LDS per channel, otherwise per thread (WHOLE).
// Variances are sums of squared deviations from the mean: deviations of
// registers from the sample's mean (resident), or per tile from the tile's own
// mean, joined by the pairwise formula (split); no difference of large sums.
// Every sum runs in a fixed order, and at most kInTurn terms or so one after the
// other: longer ones in blocks whose sums are added up in turn.
#pragma once

#include <algorithm>

#include "common.hpp"
#include "internal.hpp"
#include "sequence.hpp"

namespace fftmv {

constexpr int kNormThreads = 1024;  // at most
// of a resident workgroup that holds several rows a thread (256 registers each)
constexpr int kHeldThreads = 512;
constexpr int kInTurn = 32;
template <int Q, int P>
constexpr int kResidentThreads = Q * P > 1 ? kHeldThreads : kNormThreads;

// How a field is cut into slabs and workgroups.
struct NormShape {
  int64_t N;
  int S, D, G;
  int threads;      // of a workgroup
  int gs, slabs;    // groups of a slab, slabs of a row
  int lx, ty;       // lanes across a slab, rows of a sample side by side
  int sub;          // samples side by side (1 but for short samples)
  int team;         // threads that sum one group (a power of two, at most a wave)
  int across;       // workgroups over the samples of one slab (resident), or row ranges of a sample (split)
  int range;        // split: rows of a range
  int cut, width;   // split: slabs that one group is cut into where it is wider than the lanes (else 1), their channels
};

__device__ __forceinline__ int held_rows(const fftmv_group_norm_t &g, int64_t n) {
  const int S = static_cast<int>(g.rows);
  if (!g.lengths) return S;
  const int l = g.lengths[n];
  return l < 0 ? 0 : l > S ? S : l;
}

// Row `row` of a sample, zeros where row >= held. The load is unconditional (of
// row 0 in that case, which is there): loads behind branches wait one for
// another, and took three times as long.
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> load_held(const T *sample, int row, int held, int64_t stride) {
  const bool on = row < held;
  const Vec<T, VEC> v = load_vec<T, VEC>(sample + static_cast<int64_t>(on ? row : 0) * stride);
  if constexpr (VEC * sizeof(T) == 16) {
    const u32x4_any w = __builtin_bit_cast(u32x4_any, v), none = {0, 0, 0, 0};
    return __builtin_bit_cast(Vec<T, VEC>, on ? w : none);
  } else {
    return on ? v : Vec<T, VEC>{};
  }
}

// This thread's place in a slab. CUT: slabs are pieces of one group.
template <int VEC, bool CUT = false>
struct SlabLane {
  int ng, wd;           // groups and channels of this slab
  int g0;               // the slab's first group
  int lane, flat;       // flat: its row of lanes
  int sub, row;         // which of the samples side by side, and the first of its rows there (ty apart)
  int c;                // first of its VEC channels, within the slab. The last lane steps back to end with the slab:
                        // the channels that it repeats go to the same places with the same values
  int64_t ch0;          // the slab's first channel
  bool in;
  __device__ SlabLane(const NormShape &s, int slab) {
    if constexpr (CUT) {
      g0 = slab / s.cut;
      const int from = (slab - g0 * s.cut) * s.width;
      ng = 1;
      wd = s.D - from < s.width ? s.D - from : s.width;
      ch0 = static_cast<int64_t>(g0) * s.D + from;
    } else {
      g0 = slab * s.gs;
      ng = s.gs < s.G - g0 ? s.gs : s.G - g0;
      wd = ng * s.D;
      ch0 = static_cast<int64_t>(g0) * s.D;
    }
    lane = threadIdx.x % s.lx;
    flat = threadIdx.x / s.lx;
    sub = s.sub > 1 ? flat / s.ty : 0;
    row = flat - sub * s.ty;
    c = lane * VEC;
    in = flat < s.ty * s.sub && c < wd;
    if (c + VEC > wd) c = wd - VEC;
  }
  // sample q of this thread, kept inside the batch
  __device__ __forceinline__ int64_t sample(const NormShape &s, int64_t n0, int q) const {
    const int64_t n = n0 + q * s.sub + sub;
    return n < s.N ? n : s.N - 1;
  }
};

// Rows that each of a thread's samples holds (0 behind the last sample).
template <int VEC, int Q>
__device__ __forceinline__ void held_of(const fftmv_group_norm_t &g, const NormShape &s, const SlabLane<VEC> &l,
                                        int64_t n0, int (&held)[Q]) {
#pragma unroll
  for (int q = 0; q < Q; ++q) held[q] = s.S;
  if (g.lengths) {
#pragma unroll
    for (int q = 0; q < Q; ++q) held[q] = g.lengths[l.sample(s, n0, q)];
#pragma unroll
    for (int q = 0; q < Q; ++q) held[q] = held[q] < 0 ? 0 : held[q] > s.S ? s.S : held[q];
  }
#pragma unroll
  for (int q = 0; q < Q; ++q)
    if (!l.in || n0 + q * s.sub + l.sub >= s.N) held[q] = 0;
}

template <int VEC>
__device__ __forceinline__ void load_params(const float *p, int64_t ch, float none, float (&v)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = p ? p[ch + e] : none;
}

// Group of each of a thread's channels.
template <int VEC, bool WHOLE>
struct GroupOf {
  int g[WHOLE ? 1 : VEC];
  __device__ GroupOf(int c, int D) {
    if constexpr (WHOLE) {
      g[0] = c / D;
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[e] = (c + e) / D;
    }
  }
  __device__ __forceinline__ int operator[](int e) const { return g[WHOLE ? 0 : e]; }
};

// A thread's contribution to the sums of its groups, in `part` (a row of slots
// for each row of lanes): one slot a thread, or one a channel.
template <int VEC, bool WHOLE, typename Lane>
__device__ __forceinline__ void put_part(float *part, const NormShape &s, const Lane &l, const float (&v)[VEC]) {
  if (!l.in) return;
  if constexpr (WHOLE) {
    float sum = v[0];
#pragma unroll
    for (int e = 1; e < VEC; ++e) sum += v[e];
    part[l.flat * s.lx + l.lane] = sum;
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) part[l.flat * (s.lx * VEC) + l.c + e] = v[e];
  }
}
template <int VEC, bool WHOLE>
__device__ __forceinline__ int part_slots(const NormShape &s) {
  return s.sub * s.ty * s.lx * (WHOLE ? 1 : VEC);
}

// Sums of `sets` x ng groups, a set being the ty rows of slots of one sample:
// f(set * ng + group, sum) by one thread each. All threads call it.
template <int VEC, bool WHOLE, typename F>
__device__ __forceinline__ void team_sums(const float *part, const NormShape &s, int ng, int sets, F f) {
  const int gw = WHOLE ? s.D / VEC : s.D, lw = WHOLE ? s.lx : s.lx * VEC, slots = s.ty * lw;
  // the team as `across` threads along a row of slots, its rest over the rows
  int across = 1;
  while (across < gw && across < s.team) across *= 2;
  const int me = threadIdx.x & (s.team - 1), first = me & (across - 1), row = me / across, rows = s.team / across;
  for (int pair = threadIdx.x / s.team; pair < sets * ng; pair += blockDim.x / s.team) {
    const int set = pair / ng, g = pair - set * ng;
    const float *base = part + set * slots + g * gw;
    float sum = 0.0f;
    for (int t = row; t < s.ty; t += rows) {
      const float *p = base + t * lw;
      float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
      int j = first;
      for (; j + 3 * across < gw; j += 4 * across) {
        s0 += p[j];
        s1 += p[j + across];
        s2 += p[j + 2 * across];
        s3 += p[j + 3 * across];
      }
      for (; j < gw; j += across) s0 += p[j];
      sum += (s0 + s1) + (s2 + s3);
    }
    for (int m = s.team / 2; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
    if (me == 0) f(pair, sum);
  }
}

// ------------------------------------------------------------ resident
// Q samples at a time, up to P rows of each in a thread's registers.
template <typename T, int VEC, bool WHOLE, int ACT, int Q, int P>
__global__ __launch_bounds__((kResidentThreads<Q, P>)) void norm_forward_kernel(fftmv_group_norm_t g, NormShape s) {
  extern __shared__ float lds[];
  const int slots = part_slots<VEC, WHOLE>(s);
  float *part = lds, *mean = lds + Q * slots, *rstd = mean + Q * s.sub * s.gs;
  const int slab = blockIdx.x % s.slabs;
  const SlabLane<VEC> l(s, slab);
  const GroupOf<VEC, WHOLE> group(l.c, s.D);
  float w[VEC], b[VEC];
  load_params(g.weight, l.ch0 + l.c, 1.0f, w);
  load_params(g.bias, l.ch0 + l.c, 0.0f, b);
  const int64_t step = static_cast<int64_t>(gridDim.x / s.slabs) * (Q * s.sub);
  for (int64_t n0 = static_cast<int64_t>(blockIdx.x / s.slabs) * (Q * s.sub); n0 < s.N; n0 += step) {
    Vec<T, VEC> v[Q][P];
    int held[Q];
    held_of<VEC, Q>(g, s, l, n0, held);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const T *x = static_cast<const T *>(g.x) + l.sample(s, n0, q) * g.x_sample + l.ch0 + l.c;
#pragma unroll
      for (int p = 0; p < P; ++p) v[q][p] = load_held<T, VEC>(x, l.row + p * s.ty, held[q], g.x_row);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float sum[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        sum[e] = v[q][0][e];
#pragma unroll
        for (int p = 1; p < P; ++p) sum[e] += v[q][p][e];
      }
      put_part<VEC, WHOLE>(part + q * slots, s, l, sum);
    }
    __syncthreads();
    team_sums<VEC, WHOLE>(part, s, l.ng, Q * s.sub, [&](int pair, float sum) {
      const int64_t n = n0 + pair / l.ng;
      const int h = n < s.N ? held_rows(g, n) : 0;
      mean[pair] = h ? sum / (static_cast<float>(h) * s.D) : 0.0f;
    });
    __syncthreads();
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float sq[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float m = l.in ? mean[(q * s.sub + l.sub) * l.ng + group[e]] : 0.0f;
        sq[e] = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const float d = l.row + p * s.ty < held[q] ? v[q][p][e] - m : 0.0f;
          sq[e] = fmaf(d, d, sq[e]);
        }
      }
      put_part<VEC, WHOLE>(part + q * slots, s, l, sq);
    }
    __syncthreads();
    team_sums<VEC, WHOLE>(part, s, l.ng, Q * s.sub, [&](int pair, float sum) {
      const int64_t n = n0 + pair / l.ng;
      const int h = n < s.N ? held_rows(g, n) : 0;
      const float r = h ? 1.0f / sqrtf(sum / (static_cast<float>(h) * s.D) + g.eps) : 0.0f;
      rstd[pair] = r;
      if (g.stats && n < s.N) {
        float *to = g.stats + 2 * (n * s.G + static_cast<int64_t>(slab) * s.gs + pair % l.ng);
        to[0] = mean[pair];
        to[1] = r;
      }
    });
    __syncthreads();
    if (l.in) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int64_t n = n0 + q * s.sub + l.sub;
        if (n >= s.N) break;
        T *y = static_cast<T *>(g.y) + n * g.y_sample + l.ch0 + l.c;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int row = l.row + p * s.ty;
          if (row >= s.S) break;
          float o[VEC] = {};
          if (row < held[q]) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const int k = (q * s.sub + l.sub) * l.ng + group[e];
              o[e] = activate<T, ACT>(fmaf((v[q][p][e] - mean[k]) * rstd[k], w[e], b[e]));
            }
          }
          store_vec<T, VEC>(y + static_cast<int64_t>(row) * g.y_row, o);
        }
      }
    }
  }
}

// Sums of dz and dz xhat over the rows of all samples of this workgroup: row
// `first` of the workspace, or the results themselves where there is one; `more`:
// added to what an earlier call left there.
template <int VEC, typename Lane>
__device__ __forceinline__ void put_param_sums(const fftmv_group_norm_t &g, const NormShape &s,
                                               const Lane &l, float *lds, int first, bool alone,
                                               const float (&db)[VEC], const float (&dw)[VEC], bool more = false) {
  const int lw = s.lx * VEC;
  const int64_t C = static_cast<int64_t>(s.G) * s.D;
  float2 *to = static_cast<float2 *>(g.workspace) + first * C + l.ch0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
    put_part<VEC, false>(lds, s, l, k ? dw : db);
    __syncthreads();
    for (int c = threadIdx.x; c < l.wd; c += blockDim.x) {
      float sum = 0.0f;
      const int rows = s.sub * s.ty;
      for (int t0 = 0; t0 < rows; t0 += 16) {
        float some = 0.0f;
        for (int t = t0; t < rows && t < t0 + 16; ++t) some += lds[t * lw + c];
        sum += some;
      }
      float *out = k ? g.dweight : g.dbias;
      if (!alone) out = k ? &to[c].y : &to[c].x;
      else if (out) out += l.ch0 + c;
      if (out) *out = more ? *out + sum : sum;
    }
  }
}

template <typename T, int VEC, bool WHOLE, int ACT, int Q, int P>
__global__ __launch_bounds__((kResidentThreads<Q, P>)) void norm_backward_kernel(fftmv_group_norm_t g, NormShape s) {
  extern __shared__ float lds[];
  const int slots = part_slots<VEC, WHOLE>(s);
  float *part = lds, *stat = lds + 2 * Q * slots, *m = stat + 2 * Q * s.sub * s.gs;
  const int slab = blockIdx.x % s.slabs, first = blockIdx.x / s.slabs;
  const SlabLane<VEC> l(s, slab);
  const GroupOf<VEC, WHOLE> group(l.c, s.D);
  float w[VEC], b[VEC], db[VEC], dw[VEC];
  load_params(g.weight, l.ch0 + l.c, 1.0f, w);
  load_params(g.bias, l.ch0 + l.c, 0.0f, b);
  constexpr int kTurns = 3 * kInTurn;  // under the hundred roundings that the sums are held to
  const int64_t step = static_cast<int64_t>(gridDim.x / s.slabs) * (Q * s.sub);
  const bool alone = gridDim.x == static_cast<unsigned>(s.slabs);
  int64_t n0 = static_cast<int64_t>(first) * (Q * s.sub);
  bool more = false;
  do {  // kTurns samples of each thread, whose sums go out in front of the next
#pragma unroll
    for (int e = 0; e < VEC; ++e) db[e] = dw[e] = 0.0f;
    const int64_t end = s.N - n0 > kTurns / Q * step ? n0 + kTurns / Q * step : s.N;
    for (; n0 < end; n0 += step) {
      Vec<T, VEC> v[Q][P], d[Q][P];
      int held[Q];
      held_of<VEC, Q>(g, s, l, n0, held);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int64_t n = l.sample(s, n0, q);
        const T *x = static_cast<const T *>(g.x) + n * g.x_sample + l.ch0 + l.c;
        const T *dy = static_cast<const T *>(g.dy) + n * g.dy_sample + l.ch0 + l.c;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          v[q][p] = load_held<T, VEC>(x, l.row + p * s.ty, held[q], g.x_row);
          d[q][p] = load_held<T, VEC>(dy, l.row + p * s.ty, held[q], g.dy_row);
        }
      }
      for (int i = threadIdx.x; i < Q * s.sub * l.ng; i += blockDim.x) {
        const int64_t n = n0 + i / l.ng;
        if (n < s.N) {
          const float *from = g.stats + 2 * (n * s.G + static_cast<int64_t>(slab) * s.gs + i % l.ng);
          stat[2 * i] = from[0];
          stat[2 * i + 1] = from[1];
        } else {
          stat[2 * i] = stat[2 * i + 1] = 0.0f;
        }
      }
      __syncthreads();
      // dz and xhat of one element; where no row is held, dy and dz are 0. In FP32
      // dz takes dy's place, so that no slope is evaluated again behind the sums
      // (16000 x 5000 tokens with SiLU 199 us, evaluated twice 220); the place of a
      // 16-bit element cannot hold it
      constexpr bool kKeep = sizeof(T) == 4;
      auto terms = [&](int q, int p, int e, bool kept, float &xh, float &dz) {
        const int k = 2 * ((q * s.sub + l.sub) * l.ng + group[e]);
        xh = (v[q][p][e] - stat[k]) * stat[k + 1];
        dz = d[q][p][e];
        if (!kept) dz *= activate_slope<T, ACT>(fmaf(xh, w[e], b[e]));
      };
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        float t1[VEC], t2[VEC];
        if (l.in) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            float sb = 0.0f, sw = 0.0f;
#pragma unroll
            for (int p = 0; p < P; ++p) {
              float xh, dz;
              terms(q, p, e, false, xh, dz);
              if constexpr (kKeep) d[q][p].v[e] = dz;
              sb += dz;
              sw = fmaf(dz, xh, sw);
            }
            db[e] += sb;
            dw[e] += sw;
            t1[e] = sb * w[e];
            t2[e] = sw * w[e];
          }
        }
        put_part<VEC, WHOLE>(part + q * slots, s, l, t1);
        put_part<VEC, WHOLE>(part + (Q + q) * slots, s, l, t2);
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        forget(v[q]);
        forget(d[q]);
      }
      team_sums<VEC, WHOLE>(part, s, l.ng, 2 * Q * s.sub, [&](int pair, float sum) {
        const int64_t n = n0 + pair / l.ng % (Q * s.sub);
        const int h = n < s.N ? held_rows(g, n) : 0;
        m[pair] = h ? sum / (static_cast<float>(h) * s.D) : 0.0f;
      });
      __syncthreads();
      if (l.in) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int64_t n = n0 + q * s.sub + l.sub;
          if (n >= s.N) break;
          T *dx = static_cast<T *>(g.dx) + n * g.dx_sample + l.ch0 + l.c;
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const int row = l.row + p * s.ty;
            if (row >= s.S) break;
            float o[VEC] = {};
            if (row < held[q]) {
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                float xh, dz;
                terms(q, p, e, kKeep, xh, dz);
                const int k = (q * s.sub + l.sub) * l.ng + group[e];
                o[e] = stat[2 * k + 1] * (fmaf(dz, w[e], -m[k]) - xh * m[Q * s.sub * l.ng + k]);
              }
            }
            store_vec<T, VEC>(dx + static_cast<int64_t>(row) * g.dx_row, o);
            row_done();
          }
        }
      }
      __syncthreads();  // stat is written again
    }
    put_param_sums<VEC>(g, s, l, lds, first, alone, db, dw, more);
    __syncthreads();
    more = true;
  } while (n0 < s.N);
}

// --------------------------------------------------------------- split
// One range of rows of one sample and slab.
struct Range {
  int64_t n;
  int slab, part, from, to;  // to: behind the last held row
  __device__ Range(const fftmv_group_norm_t &g, const NormShape &s) {
    slab = blockIdx.x % s.slabs;
    const int64_t rest = blockIdx.x / s.slabs;
    part = static_cast<int>(rest % s.across);
    n = rest / s.across;
    from = part * s.range;
    const int held = held_rows(g, n);
    to = held - from < s.range ? held : from + s.range;
  }
};

// What the ranges leave for each of their slab's groups (CUT: for the slab, a
// piece of one group): one pair of numbers; a row of pairs for each range.
template <bool CUT>
__device__ __forceinline__ int64_t pairs_of_range(const NormShape &s) {
  return CUT ? s.slabs : s.G;
}
// Where part i of a group stands behind its first: range i, or piece i % cut of range i / cut.
template <bool CUT>
__device__ __forceinline__ int64_t range_pair(const NormShape &s, int64_t pairs, int i) {
  if constexpr (!CUT) return i * pairs;
  const int part = i / s.cut;
  return part * pairs + (i - part * s.cut);
}
// The shape as team_sums takes it: a slab of one group as wide as the slab.
template <bool CUT, typename Lane>
__device__ __forceinline__ NormShape summed(const NormShape &s, const Lane &l) {
  NormShape t = s;
  if constexpr (CUT) t.D = l.wd;
  return t;
}

constexpr int kTile = 4;  // rows of a thread in one tile (eight measured the same, and spilled)

// (mean, sum of squared deviations) of each group over one range, from
// tiles of kTile rows a thread, each about its own mean and joined pairwise.
template <typename T, int VEC, bool CUT>
__global__ __launch_bounds__(kNormThreads) void norm_ranges_kernel(fftmv_group_norm_t g, NormShape s) {
  extern __shared__ float lds[];
  float *part = lds, *mean = lds + s.ty * s.lx * VEC;
  const Range r(g, s);
  const SlabLane<VEC, CUT> l(s, r.slab);
  const NormShape sum_of = summed<CUT>(s, l);
  const GroupOf<VEC, false> group(l.c, s.D);
  const T *x = static_cast<const T *>(g.x) + r.n * g.x_sample + l.ch0 + l.c;
  float mu[VEC], m2[VEC], count = 0.0f;        // of a block of tiles
  float fmu[VEC], fm2[VEC], fcount = 0.0f;     // of the blocks in front of it
#pragma unroll
  for (int e = 0; e < VEC; ++e) mu[e] = m2[e] = fmu[e] = fm2[e] = 0.0f;
  // the block joined to those in front
  auto join_front = [&] {
    const float all = fcount + count, share = all > 0.0f ? count / all : 0.0f, weight = fcount * share;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float d = mu[e] - fmu[e];
      mu[e] = fmaf(d, share, fmu[e]);
      m2[e] = fm2[e] + fmaf(d * d, weight, m2[e]);
    }
    count = all;
  };
  if (l.in) {
    int turn = 0;
    for (int t = r.from + l.row; t < r.to; t += kTile * s.ty) {
      Vec<T, VEC> v[kTile];
      int rows = (r.to - t + s.ty - 1) / s.ty;
      rows = rows < kTile ? rows : kTile;
#pragma unroll
      for (int p = 0; p < kTile; ++p) v[p] = load_held<T, VEC>(x, t + p * s.ty, r.to, g.x_row);
      const float k = static_cast<float>(rows), all = count + k, share = k / all, weight = count * share;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float sum = 0.0f, sq = 0.0f;
#pragma unroll
        for (int p = 0; p < kTile; ++p) sum += v[p][e];
        const float m = sum / k;
#pragma unroll
        for (int p = 0; p < kTile; ++p) {
          const float d = p < rows ? v[p][e] - m : 0.0f;
          sq = fmaf(d, d, sq);
        }
        const float d = m - mu[e];
        mu[e] = fmaf(d, share, mu[e]);
        m2[e] += fmaf(d * d, weight, sq);
      }
      count = all;
      if (++turn == kInTurn) {
        join_front();
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          fmu[e] = mu[e];
          fm2[e] = m2[e];
          mu[e] = m2[e] = 0.0f;
        }
        fcount = count;
        count = 0.0f;
        turn = 0;
      }
    }
    if (fcount > 0.0f) join_front();
  }
  const int rows = r.to - r.from;
  float v[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = count * mu[e];
  put_part<VEC, false>(part, s, l, v);
  __syncthreads();
  team_sums<VEC, false>(part, sum_of, l.ng, 1, [&](int k, float sum) {
    mean[k] = rows > 0 ? sum / (static_cast<float>(rows) * sum_of.D) : 0.0f;
  });
  __syncthreads();
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const float d = l.in ? mu[e] - mean[group[e]] : 0.0f;
    v[e] = fmaf(d * d, count, m2[e]);
  }
  put_part<VEC, false>(part, s, l, v);
  __syncthreads();
  float2 *to = static_cast<float2 *>(g.workspace) + (r.n * s.across + r.part) * pairs_of_range<CUT>(s) +
               (CUT ? r.slab : l.g0);
  team_sums<VEC, false>(part, sum_of, l.ng, 1, [&](int k, float sum) { to[k] = make_float2(mean[k], sum); });
}

// Joins the ranges' sums, then normalises one range.
template <typename T, int VEC, int ACT, bool CUT>
__global__ __launch_bounds__(kNormThreads) void norm_apply_kernel(fftmv_group_norm_t g, NormShape s) {
  extern __shared__ float lds[];
  float *mean = lds, *rstd = lds + s.gs;
  const Range r(g, s);
  const SlabLane<VEC, CUT> l(s, r.slab);
  const GroupOf<VEC, false> group(l.c, s.D);
  const int held = held_rows(g, r.n);
  const int64_t pairs = pairs_of_range<CUT>(s);
  const float2 *from = static_cast<const float2 *>(g.workspace) + r.n * s.across * pairs + l.g0 * s.cut;
  const int parts = s.across * s.cut;  // of a group: the pieces of one range, then of the next
  // one team of threads a group, four ranges of a thread at a time, joined
  // pairwise: (count, mean, sum of squared deviations)
  const int me = threadIdx.x % s.team, teams = blockDim.x / s.team;
  for (int k = threadIdx.x / s.team; k < l.ng; k += teams) {
    float count = 0.0f, mu = 0.0f, sq = 0.0f;  // of the blocks of ranges so far
    auto join = [](float &count, float &mu, float &sq, float n, float m, float q) {
      const float all = count + n, share = all > 0.0f ? n / all : 0.0f, d = m - mu;
      sq += q + d * d * count * share;
      mu = fmaf(d, share, mu);
      count = all;
    };
    for (int b0 = me; b0 < parts; b0 += kInTurn * s.team) {
      float bcount = 0.0f, bmu = 0.0f, bsq = 0.0f;  // of a block of ranges
      for (int i0 = b0; i0 < parts && i0 < b0 + kInTurn * s.team; i0 += 4 * s.team) {
        float2 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = i0 + j * s.team;
          v[j] = from[range_pair<CUT>(s, pairs, i < parts ? i : 0) + k];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = i0 + j * s.team, part = CUT ? i / s.cut : i, piece = CUT ? i - part * s.cut : 0;
          const int rows = held - part * s.range, rest = s.D - piece * s.width;
          if (i < parts && rows > 0)
            join(bcount, bmu, bsq, static_cast<float>(rows < s.range ? rows : s.range) * (CUT && rest > s.width ? s.width : rest),
                 v[j].x, v[j].y);
        }
      }
      if (b0 == me) count = bcount, mu = bmu, sq = bsq;
      else join(count, mu, sq, bcount, bmu, bsq);
    }
    for (int m = 1; m < s.team; m <<= 1) {
      const float n = __shfl_xor(count, m), mm = __shfl_xor(mu, m), qq = __shfl_xor(sq, m);
      join(count, mu, sq, n, mm, qq);  // lane 0's order is the one that counts
    }
    if (me == 0) {
      mean[k] = mu;
      rstd[k] = held ? 1.0f / sqrtf(sq / (static_cast<float>(held) * s.D) + g.eps) : 0.0f;
      if (g.stats && r.part == 0) {  // (CUT: every piece the same)
        float *to = g.stats + 2 * (r.n * s.G + l.g0 + k);
        to[0] = mu;
        to[1] = rstd[k];
      }
    }
  }
  __syncthreads();
  if (!l.in) return;
  // y = act(x scale + (bias - mean scale)) would cancel for large means
  float w[VEC], b[VEC], mu[VEC], rs[VEC];
  load_params(g.weight, l.ch0 + l.c, 1.0f, w);
  load_params(g.bias, l.ch0 + l.c, 0.0f, b);
#pragma unroll
  for (int e = 0; e < VEC; ++e) mu[e] = mean[group[e]], rs[e] = rstd[group[e]];
  const T *x = static_cast<const T *>(g.x) + r.n * g.x_sample + l.ch0 + l.c;
  T *y = static_cast<T *>(g.y) + r.n * g.y_sample + l.ch0 + l.c;
  const int end = s.S - r.from < s.range ? s.S : r.from + s.range;
  for (int t = r.from + l.row; t < end; t += 4 * s.ty) {
    Vec<T, VEC> v[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = load_held<T, VEC>(x, t + p * s.ty, r.to, g.x_row);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int row = t + p * s.ty;
      if (row >= end) break;
      float o[VEC] = {};
      if (row < r.to) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = activate<T, ACT>(fmaf((v[p][e] - mu[e]) * rs[e], w[e], b[e]));
      }
      store_vec<T, VEC>(y + static_cast<int64_t>(row) * g.y_row, o);
    }
  }
}

// Sums of dz and dz xhat over one range: of each channel, in row (n, range) of
// the workspace, and, times the weight, of each group, behind those rows.
template <typename T, int VEC, int ACT, bool CUT>
__global__ __launch_bounds__(kNormThreads) void norm_sums_kernel(fftmv_group_norm_t g, NormShape s) {
  extern __shared__ float lds[];
  const Range r(g, s);
  const SlabLane<VEC, CUT> l(s, r.slab);
  const NormShape sum_of = summed<CUT>(s, l);
  float w[VEC], db[VEC], dw[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) w[e] = db[e] = dw[e] = 0.0f;
  if (l.in && r.to > r.from) {  // (without rows there may be no statistics)
    const GroupOf<VEC, false> group(l.c, s.D);
    float b[VEC], mu[VEC], rs[VEC];
    load_params(g.weight, l.ch0 + l.c, 1.0f, w);
    load_params(g.bias, l.ch0 + l.c, 0.0f, b);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float *from = g.stats + 2 * (r.n * s.G + l.g0 + group[e]);
      mu[e] = from[0];
      rs[e] = from[1];
    }
    const T *x = static_cast<const T *>(g.x) + r.n * g.x_sample + l.ch0 + l.c;
    const T *dy = static_cast<const T *>(g.dy) + r.n * g.dy_sample + l.ch0 + l.c;
    float pb[VEC], pw[VEC];  // of a block of tiles
#pragma unroll
    for (int e = 0; e < VEC; ++e) pb[e] = pw[e] = 0.0f;
    int turn = 0;
    for (int t = r.from + l.row; t < r.to; t += 4 * s.ty) {
      Vec<T, VEC> v[4], d[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        v[p] = load_held<T, VEC>(x, t + p * s.ty, r.to, g.x_row);
        d[p] = load_held<T, VEC>(dy, t + p * s.ty, r.to, g.dy_row);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float sb = 0.0f, sw = 0.0f;
#pragma unroll
        for (int p = 0; p < 4; ++p) {  // rows that are not there have dy = 0
          const float xh = (v[p][e] - mu[e]) * rs[e], dz = d[p][e] * activate_slope<T, ACT>(fmaf(xh, w[e], b[e]));
          sb += dz;
          sw = fmaf(dz, xh, sw);
        }
        pb[e] += sb;
        pw[e] += sw;
      }
      if (++turn == kInTurn) {
        turn = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          db[e] += pb[e];
          dw[e] += pw[e];
          pb[e] = pw[e] = 0.0f;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      db[e] += pb[e];
      dw[e] += pw[e];
    }
  }
  const int64_t row = r.n * s.across + r.part, C = static_cast<int64_t>(s.G) * s.D;
  put_param_sums<VEC>(g, s, l, lds, static_cast<int>(row), false, db, dw);
  float2 *to = static_cast<float2 *>(g.workspace) + s.N * s.across * C + row * pairs_of_range<CUT>(s) +
               (CUT ? r.slab : l.g0);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float t[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) t[e] = (k ? dw[e] : db[e]) * w[e];
    __syncthreads();
    put_part<VEC, false>(lds, s, l, t);
    __syncthreads();
    team_sums<VEC, false>(lds, sum_of, l.ng, 1, [&](int i, float sum) { (k ? to[i].y : to[i].x) = sum; });
  }
}

// dweight and dbias of kSumChannels channels (a line of the workspace) from its
// `rows` rows, shared out over the rest of the threads.
constexpr int kSumChannels = 16;
__device__ __forceinline__ void param_sums(const fftmv_group_norm_t &g, int64_t rows, int64_t block, float *lds) {
  const int c = threadIdx.x % kSumChannels, part = threadIdx.x / kSumChannels, parts = blockDim.x / kSumChannels;
  const int64_t ch = block * kSumChannels + c;
  const float2 *from = static_cast<const float2 *>(g.workspace);
  float sb = 0.0f, sw = 0.0f;
  if (ch < g.channels)
    for (int64_t b0 = part; b0 < rows; b0 += kInTurn * 16 * parts) {
      float tb = 0.0f, tw = 0.0f;
      for (int64_t i0 = b0; i0 < rows && i0 < b0 + kInTurn * 16 * parts; i0 += 16 * parts) {
        float b = 0.0f, w = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int64_t i = i0 + k * parts;
          const float2 v = from[(i < rows ? i : i0) * g.channels + ch];
          b += i < rows ? v.x : 0.0f;
          w += i < rows ? v.y : 0.0f;
        }
        tb += b;
        tw += w;
      }
      sb += tb;
      sw += tw;
    }
  lds[threadIdx.x] = sb;
  lds[blockDim.x + threadIdx.x] = sw;
  __syncthreads();
  if (part == 0 && ch < g.channels) {
    for (int k = 1; k < parts; ++k) {
      sb += lds[k * kSumChannels + c];
      sw += lds[blockDim.x + k * kSumChannels + c];
    }
    if (g.dbias) g.dbias[ch] = sb;
    if (g.dweight) g.dweight[ch] = sw;
  }
}

// dx of one range, the means of dz w and dz w xhat joined from all ranges; and,
// in the workgroups behind the first `main`, the parameters' sums.
template <typename T, int VEC, int ACT, bool CUT>
__global__ __launch_bounds__(kNormThreads) void norm_grad_kernel(fftmv_group_norm_t g, NormShape s, int64_t main) {
  extern __shared__ float lds[];
  if (blockIdx.x >= main) {
    param_sums(g, s.N * s.across, blockIdx.x - main, lds);
    return;
  }
  float *m1 = lds, *m2 = lds + s.gs;
  const Range r(g, s);
  const SlabLane<VEC, CUT> l(s, r.slab);
  const GroupOf<VEC, false> group(l.c, s.D);
  const int held = held_rows(g, r.n);
  const int64_t C = static_cast<int64_t>(s.G) * s.D;
  const int64_t pairs = pairs_of_range<CUT>(s);
  const float2 *from = static_cast<const float2 *>(g.workspace) + s.N * s.across * C + r.n * s.across * pairs + l.g0 * s.cut;
  const int parts = s.across * s.cut;
  const int me = threadIdx.x % s.team, teams = blockDim.x / s.team;
  for (int k = threadIdx.x / s.team; k < l.ng; k += teams) {
    float a = 0.0f, b = 0.0f;
    for (int b0 = me; b0 < parts; b0 += kInTurn * s.team) {
      float pa = 0.0f, pb = 0.0f;
      for (int i0 = b0; i0 < parts && i0 < b0 + kInTurn * s.team; i0 += 4 * s.team) {
        float2 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = i0 + j * s.team;
          v[j] = from[range_pair<CUT>(s, pairs, i < parts ? i : 0) + k];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i0 + j * s.team < parts) pa += v[j].x, pb += v[j].y;
      }
      a += pa;
      b += pb;
    }
    for (int m = s.team / 2; m > 0; m >>= 1) {
      a += __shfl_xor(a, m);
      b += __shfl_xor(b, m);
    }
    if (me == 0) {
      const float n = static_cast<float>(held) * s.D;
      m1[k] = held ? a / n : 0.0f;
      m2[k] = held ? b / n : 0.0f;
    }
  }
  __syncthreads();
  const int end = s.S - r.from < s.range ? s.S : r.from + s.range;
  if (!l.in || r.from >= end) return;
  float w[VEC], b[VEC], mu[VEC], rs[VEC], k1[VEC], k2[VEC];
  load_params(g.weight, l.ch0 + l.c, 1.0f, w);
  load_params(g.bias, l.ch0 + l.c, 0.0f, b);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const float *st = g.stats + 2 * (r.n * s.G + l.g0 + group[e]);
    mu[e] = st[0];
    rs[e] = st[1];
    k1[e] = m1[group[e]];
    k2[e] = m2[group[e]];
  }
  const T *x = static_cast<const T *>(g.x) + r.n * g.x_sample + l.ch0 + l.c;
  const T *dy = static_cast<const T *>(g.dy) + r.n * g.dy_sample + l.ch0 + l.c;
  T *dx = static_cast<T *>(g.dx) + r.n * g.dx_sample + l.ch0 + l.c;
  for (int t = r.from + l.row; t < end; t += 2 * s.ty) {
    Vec<T, VEC> v[2], d[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      v[p] = load_held<T, VEC>(x, t + p * s.ty, r.to, g.x_row);
      d[p] = load_held<T, VEC>(dy, t + p * s.ty, r.to, g.dy_row);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int row = t + p * s.ty;
      if (row >= end) break;
      float o[VEC] = {};
      if (row < r.to) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (v[p][e] - mu[e]) * rs[e], dz = d[p][e] * activate_slope<T, ACT>(fmaf(xh, w[e], b[e]));
          o[e] = rs[e] * (fmaf(dz, w[e], -k1[e]) - xh * k2[e]);
        }
      }
      store_vec<T, VEC>(dx + static_cast<int64_t>(row) * g.dx_row, o);
    }
  }
}

// ---------------------------------------------------------------- wide
// A row or two of groups wider than a workgroup's lanes (8192 channels at 16
// bits, 4096 in FP32): one workgroup per sample and group, its threads along the
// channels, the rows in turn, read again from the caches for each pass.
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kBlock / kWave];
  v = wave_sum(v);
  __syncthreads();  // the last use of part is over
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  float s = part[0];
#pragma unroll
  for (int i = 1; i < kBlock / kWave; ++i) s += part[i];
  return s;
}

// The sum of f(t, c) over a sample's held rows and this thread's channels, in
// blocks of kInTurn channels.
template <typename F>
__device__ __forceinline__ float wide_sum(int held, int64_t D, F f) {
  float sum = 0.0f;
  for (int t = 0; t < held; ++t)
    for (int64_t c0 = threadIdx.x; c0 < D; c0 += kInTurn * kBlock) {
      float part = 0.0f;
      for (int64_t c = c0; c < D && c < c0 + kInTurn * kBlock; c += kBlock) part += f(t, c);
      sum += part;
    }
  return sum;
}

template <typename T, int ACT>
__global__ __launch_bounds__(kBlock) void norm_wide_forward_kernel(fftmv_group_norm_t g) {
  const int64_t n = blockIdx.x / g.groups, q = blockIdx.x % g.groups, D = g.channels / g.groups;
  const int held = held_rows(g, n);
  const float count = static_cast<float>(held) * D;
  const T *x = static_cast<const T *>(g.x) + n * g.x_sample + q * D;
  T *y = static_cast<T *>(g.y) + n * g.y_sample + q * D;
  const float mean =
      block_sum(wide_sum(held, D, [&](int t, int64_t c) { return static_cast<float>(x[t * g.x_row + c]); })) /
      fmaxf(count, 1.0f);
  const float sum = block_sum(wide_sum(held, D, [&](int t, int64_t c) {
    const float d = static_cast<float>(x[t * g.x_row + c]) - mean;
    return d * d;
  }));
  const float rstd = held ? 1.0f / sqrtf(sum / count + g.eps) : 0.0f;
  if (g.stats && threadIdx.x == 0) {
    g.stats[2 * static_cast<int64_t>(blockIdx.x)] = mean;
    g.stats[2 * static_cast<int64_t>(blockIdx.x) + 1] = rstd;
  }
  for (int t = 0; t < static_cast<int>(g.rows); ++t)
    for (int64_t c = threadIdx.x; c < D; c += kBlock) {
      float v = 0.0f;
      if (t < held) {
        const float w = g.weight ? g.weight[q * D + c] : 1.0f, b = g.bias ? g.bias[q * D + c] : 0.0f;
        v = activate<T, ACT>(fmaf((static_cast<float>(x[t * g.x_row + c]) - mean) * rstd, w, b));
      }
      y[t * g.y_row + c] = static_cast<T>(v);
    }
}

// Writes its sums of each channel in row n of the workspace.
template <typename T, int ACT>
__global__ __launch_bounds__(kBlock) void norm_wide_backward_kernel(fftmv_group_norm_t g) {
  const int64_t n = blockIdx.x / g.groups, q = blockIdx.x % g.groups, D = g.channels / g.groups;
  const int held = held_rows(g, n);
  const float count = fmaxf(static_cast<float>(held) * D, 1.0f);
  const T *x = static_cast<const T *>(g.x) + n * g.x_sample + q * D;
  const T *dy = static_cast<const T *>(g.dy) + n * g.dy_sample + q * D;
  T *dx = static_cast<T *>(g.dx) + n * g.dx_sample + q * D;
  float2 *sums = static_cast<float2 *>(g.workspace) + n * g.channels + q * D;
  const float mean = g.stats[2 * static_cast<int64_t>(blockIdx.x)];
  const float rstd = g.stats[2 * static_cast<int64_t>(blockIdx.x) + 1];
  float m1 = 0.0f, m2 = 0.0f, n1 = 0.0f, n2 = 0.0f;
  int turn = 0;
  for (int64_t c = threadIdx.x; c < D; c += kBlock) {
    const float w = g.weight ? g.weight[q * D + c] : 1.0f, b = g.bias ? g.bias[q * D + c] : 0.0f;
    float sb = 0.0f, sw = 0.0f;
    for (int t = 0; t < held; ++t) {
      const float xh = (static_cast<float>(x[t * g.x_row + c]) - mean) * rstd;
      const float dz = static_cast<float>(dy[t * g.dy_row + c]) * activate_slope<T, ACT>(fmaf(xh, w, b));
      sb += dz;
      sw = fmaf(dz, xh, sw);
    }
    sums[c] = make_float2(sb, sw);
    n1 = fmaf(sb, w, n1);
    n2 = fmaf(sw, w, n2);
    if (++turn == kInTurn) {
      m1 += n1;
      m2 += n2;
      n1 = n2 = 0.0f;
      turn = 0;
    }
  }
  m1 += n1;
  m2 += n2;
  m1 = block_sum(m1) / count;
  m2 = block_sum(m2) / count;
  for (int t = 0; t < static_cast<int>(g.rows); ++t)
    for (int64_t c = threadIdx.x; c < D; c += kBlock) {
      float v = 0.0f;
      if (t < held) {
        const float w = g.weight ? g.weight[q * D + c] : 1.0f, b = g.bias ? g.bias[q * D + c] : 0.0f;
        const float xh = (static_cast<float>(x[t * g.x_row + c]) - mean) * rstd;
        const float dz = static_cast<float>(dy[t * g.dy_row + c]) * activate_slope<T, ACT>(fmaf(xh, w, b));
        v = rstd * (fmaf(dz, w, -m1) - xh * m2);
      }
      dx[t * g.dx_row + c] = static_cast<T>(v);
    }
}

// ---------------------------------------------------------------- plans
// What a call launches; decided by sizes alone.
struct NormPlan {
  enum Kind { kSplit, kTokens, kRow, kResident, kWide } kind = kSplit;
  bool whole = false;
  int vec = 1;
  NormShape s{};
  int64_t rows = 0;      // rows of sums that backward leaves in the workspace
  size_t lds = 0, workspace = 0;
};

NormPlan norm_plan(int64_t samples, int64_t rows, int64_t channels, int64_t groups, int dtype, bool backward);

hipError_t launch_param_sums(const fftmv_group_norm_t &g, int64_t rows, hipStream_t s);

// Groups are cut only where they are wider than the lanes, so into whole vectors.
template <int VEC, typename F>
hipError_t by_cut(const NormShape &h, F f) {
  if constexpr (VEC > 1)
    if (h.cut > 1) return f(Const<true>{});
  return f(Const<false>{});
}

template <typename T, int ACT, int VEC>
hipError_t launch_norm_forward_vec(const fftmv_group_norm_t &g, const NormPlan &p, hipStream_t s) {
  const NormShape &h = p.s;
  const unsigned threads = static_cast<unsigned>(h.threads);
  if (p.kind == NormPlan::kSplit) {
    const int64_t blocks = h.N * h.slabs * h.across;
    if (!grid_fits(blocks, h.threads)) return hipErrorInvalidConfiguration;
    return by_cut<VEC>(h, [&](auto cut) {
      constexpr bool CUT = decltype(cut)::value;
      norm_ranges_kernel<T, VEC, CUT><<<static_cast<unsigned>(blocks), threads, p.lds, s>>>(g, h);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      norm_apply_kernel<T, VEC, ACT, CUT><<<static_cast<unsigned>(blocks), threads, 2 * h.gs * sizeof(float), s>>>(g, h);
      return hipGetLastError();
    });
  }
  const unsigned blocks = static_cast<unsigned>(h.slabs * h.across);
  if (p.kind == NormPlan::kTokens) {
    if (p.whole) norm_forward_kernel<T, VEC, true, ACT, 4, 1><<<blocks, threads, p.lds, s>>>(g, h);
    else norm_forward_kernel<T, VEC, false, ACT, 4, 1><<<blocks, threads, p.lds, s>>>(g, h);
  } else if (p.kind == NormPlan::kRow) {
    if (p.whole) norm_forward_kernel<T, VEC, true, ACT, 1, 1><<<blocks, threads, p.lds, s>>>(g, h);
    else norm_forward_kernel<T, VEC, false, ACT, 1, 1><<<blocks, threads, p.lds, s>>>(g, h);
  } else {
    if (p.whole) norm_forward_kernel<T, VEC, true, ACT, 1, 8><<<blocks, threads, p.lds, s>>>(g, h);
    else norm_forward_kernel<T, VEC, false, ACT, 1, 8><<<blocks, threads, p.lds, s>>>(g, h);
  }
  return hipGetLastError();
}

template <typename T, int ACT, int VEC>
hipError_t launch_norm_backward_vec(const fftmv_group_norm_t &g, const NormPlan &p, hipStream_t s) {
  const NormShape &h = p.s;
  const unsigned threads = static_cast<unsigned>(h.threads);
  if (p.kind == NormPlan::kSplit) {
    const int64_t blocks = h.N * h.slabs * h.across, more = (g.channels + kSumChannels - 1) / kSumChannels;
    if (!grid_fits(blocks + more, h.threads)) return hipErrorInvalidConfiguration;
    return by_cut<VEC>(h, [&](auto cut) {
      constexpr bool CUT = decltype(cut)::value;
      norm_sums_kernel<T, VEC, ACT, CUT><<<static_cast<unsigned>(blocks), threads, p.lds, s>>>(g, h);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      const size_t lds = std::max<size_t>(2 * h.gs, 2 * h.threads) * sizeof(float);
      norm_grad_kernel<T, VEC, ACT, CUT><<<static_cast<unsigned>(blocks + more), threads, lds, s>>>(g, h, blocks);
      return hipGetLastError();
    });
  }
  const unsigned blocks = static_cast<unsigned>(h.slabs * h.across);
  if (p.kind == NormPlan::kTokens) {
    if (p.whole) norm_backward_kernel<T, VEC, true, ACT, 2, 1><<<blocks, threads, p.lds, s>>>(g, h);
    else norm_backward_kernel<T, VEC, false, ACT, 2, 1><<<blocks, threads, p.lds, s>>>(g, h);
  } else if (p.kind == NormPlan::kRow) {
    if (p.whole) norm_backward_kernel<T, VEC, true, ACT, 1, 1><<<blocks, threads, p.lds, s>>>(g, h);
    else norm_backward_kernel<T, VEC, false, ACT, 1, 1><<<blocks, threads, p.lds, s>>>(g, h);
  } else {
    if (p.whole) norm_backward_kernel<T, VEC, true, ACT, 1, 4><<<blocks, threads, p.lds, s>>>(g, h);
    else norm_backward_kernel<T, VEC, false, ACT, 1, 4><<<blocks, threads, p.lds, s>>>(g, h);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || h.across == 1) return e;
  return launch_param_sums(g, h.across, s);
}

template <typename T>
hipError_t launch_group_norm_forward_as(const fftmv_group_norm_t &g, hipStream_t s) {
  const NormPlan p = norm_plan(g.samples, g.rows, g.channels, g.groups, g.dtype, false);
  return by_three(g.activation, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    if (p.kind == NormPlan::kWide) {
      if (!grid_fits(g.samples * g.groups, kBlock)) return hipErrorInvalidConfiguration;
      norm_wide_forward_kernel<T, ACT><<<static_cast<unsigned>(g.samples * g.groups), kBlock, 0, s>>>(g);
      return hipGetLastError();
    }
    return p.vec > 1 ? launch_norm_forward_vec<T, ACT, kVec<T>>(g, p, s) : launch_norm_forward_vec<T, ACT, 1>(g, p, s);
  });
}

template <typename T>
hipError_t launch_group_norm_backward_as(const fftmv_group_norm_t &g, hipStream_t s) {
  const NormPlan p = norm_plan(g.samples, g.rows, g.channels, g.groups, g.dtype, true);
  return by_three(g.activation, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    if (p.kind == NormPlan::kWide) {
      if (!grid_fits(g.samples * g.groups, kBlock)) return hipErrorInvalidConfiguration;
      norm_wide_backward_kernel<T, ACT><<<static_cast<unsigned>(g.samples * g.groups), kBlock, 0, s>>>(g);
      const hipError_t e = hipGetLastError();
      return e != hipSuccess ? e : launch_param_sums(g, g.samples, s);
    }
    return p.vec > 1 ? launch_norm_backward_vec<T, ACT, kVec<T>>(g, p, s)
                     : launch_norm_backward_vec<T, ACT, 1>(g, p, s);
  });
}

}  // namespace fftmv
