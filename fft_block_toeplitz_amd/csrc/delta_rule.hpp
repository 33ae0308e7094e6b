// The gated delta rule in runs of kRun = 64 steps: what its kernels share.
//
// Within a run that the state S enters, with G_i the sum of log a up to step i,
// E_ij = exp(G_i - G_j) and
//   B_ij = E_ij k_i.k_j  (j < i),      P_ij = scale E_ij q_i.k_j  (j <= i),
//   T    = (1 + B diag(b))^-1          (unit lower triangular),
// the errors X (row i is what step i finds wrong under its key: it writes U =
// diag(b) X there) are
//   X  = T (V - diag(e^G) K S)
//   Y  = scale diag(e^G) Q S + P diag(b) X
//   S' = e^{G_last} S + K^T diag(b e^{G_last - G}) X
// so that a run is products of matrices, and only K S, T (..) and K^T (..) X wait
// for the run before. T, P diag(b) and the factors need no state: a kernel of
// their own computes them for all runs at once.
//
// Products go to the bf16 matrix instructions with FP32 sums. An FP32 operand
// is cut into bf16 parts, the leading 8 bits, the next 8, the last 8: three parts
// hold all 24 bits. bf16 inputs are one part, fp16 inputs two, both exact. All
// products of parts down to 2^-24 are taken, whatever the outputs' type: a result
// of 16 bits is then the 32-bit one rounded once, and the gates' gradients, which
// are differences of sums, have 32-bit sums' digits. (An FP32 matrix instruction has
// a sixteenth of the rate: three parts against one exact operand are 5.3 times as
// fast, six products 2.7. Two parts for what becomes 16 bits, three products instead
// of six, put one value in 135 of bf16 results and one in 20 of fp16 ones on the other
// side of a rounding, for 744 us instead of 764 at 65536 steps of 8 heads of 128 x 128
// bf16 and 882 instead of 958 at 8 x 2048 steps of 16 such heads with gradients.)
//
// Layouts of a 16x16x32 product in a wave: operands have index lane % 16 and 8
// slots of the contracted axis, the result column lane % 16 and rows 4 (lane /
// 16) + 0..3. Which rows of the contracted axis the slots stand for is free as
// long as both operands agree, so a result is the next product's operand as it
// lies in the registers: slots 0..3 from one 16-row tile, 4..7 from the next.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "internal.hpp"
#include "sequence.hpp"

namespace fftmv {

hipError_t launch_delta_forward_f32(const fftmv_delta_rule_t &r, hipStream_t s);
hipError_t launch_delta_forward_bf16(const fftmv_delta_rule_t &r, hipStream_t s);
hipError_t launch_delta_forward_f16(const fftmv_delta_rule_t &r, hipStream_t s);
hipError_t launch_delta_backward_f32(const fftmv_delta_rule_t &r, hipStream_t s);
hipError_t launch_delta_backward_bf16(const fftmv_delta_rule_t &r, hipStream_t s);
hipError_t launch_delta_backward_f16(const fftmv_delta_rule_t &r, hipStream_t s);
hipError_t launch_delta_step(const fftmv_delta_rule_step_t &r, hipStream_t s);

constexpr int kRun = FFTMV_DELTA_RUN;
constexpr int kTiles = kRun / 16;
static_assert(kRun == 64, "one lane for each step of a run");
constexpr int kFrags = 6;  // operands of 16 rows x 32 slots that a triangle of kRun holds something in

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// bf16 parts of an element, exact; and of an FP32 value next to it
template <typename T>
constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
template <>
inline constexpr int kParts<f16> = 2;
constexpr int kFull = 3;

// f(Const<0>), ..., f(Const<N - 1>): loops whose numbers choose registers.
template <int I, int N, typename F>
__device__ __forceinline__ void unrolled(F &&f) {
  if constexpr (I < N) {
    f(Const<I>{});
    unrolled<I + 1, N>(f);
  }
}

// ------------------------------------------------------------------ operands
template <int N>
struct Cut {
  u32x4 p[N];  // 8 slots of each part
};

__device__ __forceinline__ uint32_t high_halves(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x07060302);
}

// Eight values as N parts. All but the last are cut off, which leaves the rest
// exact; the last is rounded (exact where the bits end there).
template <int N>
__device__ __forceinline__ Cut<N> cut(const float (&x)[8]) {
  Cut<N> c;
  float r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (n == N - 1) {
      bf16x8 b;
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = static_cast<__bf16>(r[e]);
      c.p[n] = __builtin_bit_cast(u32x4, b);
    } else {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t lo = __float_as_uint(r[2 * w]), hi = __float_as_uint(r[2 * w + 1]);
        c.p[n][w] = high_halves(lo, hi);
        r[2 * w] -= __uint_as_float(lo & 0xffff0000u);
        r[2 * w + 1] -= __uint_as_float(hi & 0xffff0000u);
      }
    }
  }
  return c;
}

// Two result tiles of 16 rows as the next product's operand.
template <int N>
__device__ __forceinline__ Cut<N> cut_tiles(f32x4 first, f32x4 second) {
  const float x[8] = {first[0], first[1], first[2], first[3], second[0], second[1], second[2], second[3]};
  return cut<N>(x);
}

// c += a b over the parts' products down to 2^(-8 LIMIT), the small ones first.
template <int LIMIT, int NA, int NB>
__device__ __forceinline__ void multiply(f32x4 &c, const Cut<NA> &a, const Cut<NB> &b) {
#pragma unroll
  for (int s = LIMIT - 1; s >= 0; --s) {
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = s - i;
      if (j >= 0 && j < NB)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.p[i]),
                                                    __builtin_bit_cast(bf16x8, b.p[j]), c, 0, 0, 0);
    }
  }
}

// The same for several results: neighbouring instructions add to different ones, which need not wait for each other.
template <int LIMIT, int M, int NA, int NB>
__device__ __forceinline__ void multiply_rows(f32x4 *c, const Cut<NA> (&a)[M], const Cut<NB> &b) {
#pragma unroll
  for (int s = LIMIT - 1; s >= 0; --s) {
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = s - i;
      if (j < 0 || j >= NB) continue;
#pragma unroll
      for (int m = 0; m < M; ++m)
        c[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[m].p[i]),
                                                       __builtin_bit_cast(bf16x8, b.p[j]), c[m], 0, 0, 0);
    }
  }
}

// The transposed results: b's index in rows 4 (lane / 16) + 0..3, a's in column lane % 16.
template <int LIMIT, int M, int NA, int NB>
__device__ __forceinline__ void multiply_rows_t(f32x4 *c, const Cut<NA> (&a)[M], const Cut<NB> &b) {
#pragma unroll
  for (int s = LIMIT - 1; s >= 0; --s) {
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = s - i;
      if (j < 0 || j >= NB) continue;
#pragma unroll
      for (int m = 0; m < M; ++m)
        c[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b.p[j]),
                                                       __builtin_bit_cast(bf16x8, a[m].p[i]), c[m], 0, 0, 0);
    }
  }
}

// ------------------------------------------------------------------- fields
template <typename I>
__device__ __forceinline__ I clamp_to(I v, I most) {
  return v < 0 ? 0 : v > most ? most : v;
}
template <typename T>
__device__ __forceinline__ T *head_row(const fftmv_heads_t &f, int64_t b, int64_t t, int64_t n) {
  return static_cast<T *>(f.data) + b * f.batch + t * f.step + n * f.head;
}

// Elements c..c+7 of a row of n, those behind it as zeros. Exact.
template <typename T>
__device__ __forceinline__ void load8(const T *p, int c, int n, float (&x)[8]) {
  if (c + 8 <= n) {
    constexpr int V = kVec<T>;
#pragma unroll
    for (int h = 0; h < 8 / V; ++h) {
      const Vec<T, V> v = load_vec<T, V>(p + c + h * V);
#pragma unroll
      for (int e = 0; e < V; ++e) x[h * V + e] = v[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = c + e < n ? static_cast<float>(p[c + e]) : 0.0f;
  }
}
// Eight elements c.. of row t of n elements as they lie in memory: loaded now,
// settled (what is behind the row's end, or in rows that are not there, cleared)
// when they are needed. A run's rows are loaded a run ahead, so nothing here may
// wait for them.
//   WHOLE  rows are multiples of eight elements, words, and not far apart
//          (delta_whole): a chunk is in a row or behind it, and the hardware's
//          bounds check on the run's bytes gives zeros for rows behind the last.
//          Addresses take one instruction, and no branch stands between loads
//   else   where the row ends inside, the load is moved back to end with the row,
//          and shifted afterwards
// (45 packed sequences of 30011 steps, 16 heads of 64 x 128 fp16: 490 us whole, 650 by
// the other way; 8 x 2048 steps of 16 heads of 128 x 128 bf16 with gradients 1120 and 1194.)
template <typename T>
struct Raw8 {
  u32x4 w[sizeof(T) / 2];
};
constexpr int kBufferFlags = 0x00027000;  // plain words
template <typename T, bool WHOLE>
struct Rows {
  const T *first;
  int64_t step;
  int n, width;
  __amdgpu_buffer_rsrc_t buffer;
  __device__ __forceinline__ Rows(const fftmv_heads_t &f, int64_t b, int64_t row, int64_t head, int n, int width)
      : first(head_row<const T>(f, b, row, head)), step(f.step), n(n), width(width) {
    if constexpr (WHOLE)
      buffer = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<T *>(first), 0, static_cast<int>(((n - 1) * step + width) * static_cast<int64_t>(sizeof(T))), kBufferFlags);
  }
  __device__ __forceinline__ Raw8<T> load(int t, int c) const {
    Raw8<T> r;
    if constexpr (WHOLE) {
      const int at = (t * static_cast<int>(step) + c) * static_cast<int>(sizeof(T));
#pragma unroll
      for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h)
        r.w[h] = __builtin_amdgcn_raw_buffer_load_b128(buffer, at + 16 * h, 0, 0);
    } else {
      const T *p = first + min(t, n - 1) * step;
      if (width >= 8) {
        p += min(c, width - 8);
#pragma unroll
        for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h) {
          const u32x4_any v = reinterpret_cast<const u32x4_any *>(p)[h];
          r.w[h] = u32x4{v[0], v[1], v[2], v[3]};
        }
      } else {
        T e[8] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c == 0 && i < width) e[i] = p[i];
        __builtin_memcpy(&r, e, sizeof(e));
      }
    }
    return r;
  }
};
template <bool WHOLE, typename T>
__device__ __forceinline__ void settle(Raw8<T> &r, int c, int n, bool held) {
  if constexpr (WHOLE) {
    const bool in = c < n;
#pragma unroll
    for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[h][i] = in ? r.w[h][i] : 0u;
    return;
  }
  const int drop = !held ? 8 : n >= 8 ? clamp_to(c + 8 - n, 8) : 0;  // elements at the front that are not the chunk's
  if constexpr (sizeof(T) == 2) {
    uint64_t lo = r.w[0][0] | static_cast<uint64_t>(r.w[0][1]) << 32, hi = r.w[0][2] | static_cast<uint64_t>(r.w[0][3]) << 32;
    if (drop >= 4) lo = hi, hi = 0;
    const int bits = drop % 4 * 16;
    if (drop == 8) lo = 0;
    lo = bits ? lo >> bits | hi << (64 - bits) : lo;
    hi >>= bits;
    r.w[0] = u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
  } else {
#pragma unroll
    for (int step = 4; step >= 1; step /= 2) {
      const bool by = drop & step;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t moved = i + step < 8 ? r.w[(i + step) / 4 % 2][(i + step) % 4] : 0u;
        r.w[i / 4][i % 4] = by ? moved : r.w[i / 4][i % 4];
      }
    }
    if (drop == 8) r.w[0] = r.w[1] = u32x4{0, 0, 0, 0};
  }
}
template <typename T>
__device__ __forceinline__ Cut<kParts<T>> cut_raw(const Raw8<T> &r) {
  if constexpr (kParts<T> == 1) {
    return Cut<1>{{r.w[0]}};
  } else {
    T e[8];
    __builtin_memcpy(e, &r, sizeof(e));
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(e[i]);
    return cut<kParts<T>>(x);
  }
}

// The steps of sequence b: flat rows (packed) or rows of its own, and the
// number of its first run.
struct Span {
  int64_t batch, row, run;
  int len;
};
inline __host__ __device__ int64_t runs_of(int64_t steps) { return (steps + kRun - 1) / kRun; }
inline __host__ __device__ int64_t delta_runs(int64_t batch, int64_t steps, bool packed) {
  return steps == 0 ? 0 : packed ? steps / kRun + batch : batch * runs_of(steps);
}
__device__ __forceinline__ Span span_of(const fftmv_delta_rule_t &r, int64_t b) {
  const int steps = static_cast<int>(r.steps);
  if (r.offsets) {
    const int lo = clamp_to(r.offsets[b], steps), hi = clamp_to(r.offsets[b + 1], steps);
    return {0, lo, lo / kRun + b, hi > lo ? hi - lo : 0};
  }
  return {b, 0, b * runs_of(steps), r.lengths ? clamp_to(r.lengths[b], steps) : steps};
}
// The sequence of run slot i and the run's first step in it, -1 where the slot
// holds no run. Packed: sequences begin at slots offsets[b] / kRun + b, which
// ascend; slots between one's last run and the next one's first stay empty.
struct Slot {
  int64_t b;
  int first;
};
__device__ __forceinline__ Slot slot_of(const fftmv_delta_rule_t &r, int64_t i) {
  const int steps = static_cast<int>(r.steps);
  if (!r.offsets) {
    const uint32_t n = static_cast<uint32_t>(runs_of(steps)), b = static_cast<uint32_t>(i) / n;  // a grid's workgroups
    return {b, static_cast<int>(i - static_cast<int64_t>(b) * n) * kRun};
  }
  int64_t lo = 0, hi = r.batch - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) / 2;
    if (clamp_to(r.offsets[mid], steps) / kRun + mid <= i)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int64_t place = i - (clamp_to(r.offsets[lo], steps) / kRun + lo);
  return {lo, place < 0 || place * kRun > INT32_MAX ? -1 : static_cast<int>(place) * kRun};
}

// ---------------------------------------------------------------- workspace
// What the first kernel leaves for each run slot and head.
struct Factors {
  double sum[kRun];  // G_i
  // e^{G_i}, e^{G_last - G_i} (forward times b_i), b_i; into[kRun - 1] is the whole run's decay
  float into[kRun], out[kRun], rate[kRun];
};
// Fragments (one part of an operand, 64 lanes x 16 bytes) of T and P diag(b)
// forward, of P^T and (1 + diag(b) B)^-T backward.
template <bool BACK>
struct Triangles {
  static constexpr int kT = 0, kTParts = BACK ? 0 : kFull;
  static constexpr int kP = kT + kFrags * kTParts;  // backward a fragment's parts side by side, forward those of one rank
  static constexpr int kTt = kP + kFrags * kFull, kTtParts = BACK ? kFull : 0;
  static constexpr int kAll = kTt + kFrags * kTtParts;
};
// Fragment of rows tile m and slots 32 s.. of a lower or upper triangle.
__host__ __device__ constexpr int lower_frag(int m, int s) { return m < 2 ? m : 2 * m - 2 + s; }
__host__ __device__ constexpr int upper_frag(int m, int s) { return m < 2 ? 2 * m + s : m + 2; }
__host__ __device__ constexpr bool in_lower(int m, int s) { return s == 0 || m >= 2; }
__host__ __device__ constexpr bool in_upper(int m, int s) { return s == 1 || m < 2; }

// p[i] with an offset of 32 bits beside an address that all lanes share.
template <typename T>
__device__ __forceinline__ const T &at_lane(const T *p, uint32_t i) {
  return *reinterpret_cast<const T *>(reinterpret_cast<const char *>(p) + i * static_cast<uint32_t>(sizeof(T)));
}
template <typename T>
__device__ __forceinline__ T &at_lane_of(T *p, uint32_t i) {
  return *reinterpret_cast<T *>(reinterpret_cast<char *>(p) + i * static_cast<uint32_t>(sizeof(T)));
}
template <int N>
__device__ __forceinline__ Cut<N> load_frag(const u32x4 *f, int frag, int parts, int lane) {
  Cut<N> c;
#pragma unroll
  for (int n = 0; n < N; ++n) c.p[n] = at_lane(f + (frag * parts + n) * kWave, lane);
  return c;
}

template <int LIMIT, bool UPPER, bool TRANSPOSED, int N, int NB>
__device__ __forceinline__ void multiply_triangle(f32x4 (&c)[kTiles], const Cut<N> (&a)[kFrags], const Cut<NB> &lo,
                                                  const Cut<NB> &hi) {
#pragma unroll
  for (int s = LIMIT - 1; s >= 0; --s) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = s - i;
      if (j < 0 || j >= NB) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          if (!(UPPER ? in_upper(m, h) : in_lower(m, h))) continue;
          const bf16x8 f = __builtin_bit_cast(bf16x8, a[UPPER ? upper_frag(m, h) : lower_frag(m, h)].p[i]);
          const bf16x8 x = __builtin_bit_cast(bf16x8, (h ? hi : lo).p[j]);
          c[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(TRANSPOSED ? x : f, TRANSPOSED ? f : x, c[m], 0, 0, 0);
        }
    }
  }
}
// c += the lower (upper) triangle in f, PARTS parts of a fragment, times the operands of steps 0..31 and 32..63.
template <int LIMIT, int N, int PARTS, bool UPPER, int NB>
__device__ __forceinline__ void multiply_triangle(f32x4 (&c)[kTiles], const u32x4 *f, const Cut<NB> &lo, const Cut<NB> &hi,
                                                  int lane) {
  Cut<N> a[kFrags];
#pragma unroll
  for (int i = 0; i < kFrags; ++i) a[i] = load_frag<N>(f, i, PARTS, lane);
  multiply_triangle<LIMIT, UPPER, false>(c, a, lo, hi);
}

// Long sequences with few heads leave most of the card without work: they are
// cut into parts. The state behind a part is M S + N of the state S in front of
// it; M and N of all parts but the last are computed at once (the same chain, from
// no state and from each unit state without values), joined one after another, and
// then every part goes through its runs from its own state: two and a half times
// the work, by as many times the workgroups. The gradients' chain is cut likewise.
struct DeltaCuts {
  int parts;  // of a sequence, at most
  int runs;   // of a part
};
// Times in tenths of a run of the chain, on 256 CUs: a map's run takes 0.8 of one, a joint 1.2, the
// two more launches 4. (bf16, whole and in parts: one sequence of 65536 steps, 8 heads of
// 128 x 128 3637 and 747 us; 5 of 1999 steps, 7 heads of 75 x 41 168 and 121; FP32 with gradients,
// 6 of up to 1000 steps, 4 heads of 64 x 64 255 and 202.) Packed sequences stay whole: places
// of parts by what the host knows, as runs have them (slot_of), have not been built, and one
// packed sequence of 65536 steps takes the 3.6 ms.
inline DeltaCuts delta_cuts(int64_t batch, int64_t steps, int64_t heads, int64_t keys, int64_t values, bool packed) {
  const int64_t runs = (steps + kRun - 1) / kRun, chains = batch * heads;
  DeltaCuts best = {1, static_cast<int>(runs > 0 ? runs : 1)};
  if (packed || runs < 8 || chains >= 256) return best;
  const int64_t vb = (values + 63) / 64, kb = (keys + 63) / 64;
  int64_t least = (chains * vb + 255) / 256 * runs * 10;
  for (int64_t n = 2; n <= 64 && n <= runs / 4; ++n) {
    const int64_t per = (runs + n - 1) / n, parts = (runs + per - 1) / per;
    const int64_t time = (chains * vb * parts + 255) / 256 * per * 10 +
                         (chains * (parts - 1) * (vb + kb) + 255) / 256 * per * 8 + (parts - 1) * 12 + 40;
    if (time < least) {
      least = time;
      best = {static_cast<int>(parts), static_cast<int>(per)};
    }
  }
  return best;
}

// The workspace of a call in its parts.
struct DeltaWorkspace {
  Factors *factors;
  u32x4 *triangles;
  float *grads;  // backward: the gradients of the states behind each run and Z, [runs][heads][keys + kRun][values]
  // of each part of a sequence: (N, M) [keys][values + keys], and the state in front of it (backward: behind it)
  float *maps, *starts;
  DeltaCuts cuts;
};
inline size_t delta_workspace(int64_t batch, int64_t steps, int64_t heads, int64_t keys, int64_t values, bool packed,
                              bool back, void *at = nullptr, DeltaWorkspace *w = nullptr) {
  const size_t n = static_cast<size_t>(delta_runs(batch, steps, packed)) * heads;
  const DeltaCuts cuts = delta_cuts(batch, steps, heads, keys, values, packed);
  const size_t parts = cuts.parts > 1 ? static_cast<size_t>(batch) * heads * cuts.parts : 0;
  const size_t factors = n * sizeof(Factors), triangles = n * 2 * kFull * kFrags * kWave * sizeof(u32x4);
  const size_t grads = (back ? n * (keys + kRun) * values * sizeof(float) + 15 : 0) & ~size_t{15};
  const size_t maps = (parts * keys * (keys + values) * sizeof(float) + 15) & ~size_t{15};
  const size_t starts = parts * keys * values * sizeof(float);
  static_assert(sizeof(Factors) % 16 == 0, "fragments are 16-byte aligned");
  if (w) {
    char *p = static_cast<char *>(at);
    w->factors = reinterpret_cast<Factors *>(p);
    w->triangles = reinterpret_cast<u32x4 *>(p + factors);
    w->grads = reinterpret_cast<float *>(p + factors + triangles);
    w->maps = reinterpret_cast<float *>(p + factors + triangles + grads);
    w->starts = reinterpret_cast<float *>(p + factors + triangles + grads + maps);
    w->cuts = cuts;
  }
  return factors + triangles + grads + maps + starts;
}

// ------------------------------------------------------ gates of 64 steps
// log a, bounded below: e^-1e5 is zero, and a sum with it still tells the others
// apart in 64 bits.
__device__ __forceinline__ float log_decay(int decay, float g) {
  float l = g;
  if (decay == FFTMV_DECAY_SIGMOID) l = fminf(g, 0.0f) - log1pf(expf(-fabsf(g)));
  if (g != g) l = g;
  return l < -1e5f ? -1e5f : l;
}
__device__ __forceinline__ float rate_of(int rate, float v) {
  return rate == FFTMV_RATE_SIGMOID ? 1.0f / (1.0f + expf(-v)) : v;
}
__device__ __forceinline__ double lane_sums(double v, int lane) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const double o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// ------------------------------------------------------------ the inverse
// By one wave, in blocks: a lane solves one column of a diagonal block of 16 by
// substitution (products of powers would lose what cancels where keys are
// alike), and the blocks below are joined in FP32 products,
// T_21 = -T_22 A_21 T_11.
constexpr int kTri = kRun + 4;  // floats between rows of the triangle in LDS

template <bool TRANSPOSED>
__device__ __forceinline__ f32x4 load4(const float *a, int row, int col) {
  if constexpr (TRANSPOSED) return f32x4{a[col * kTri + row], a[(col + 1) * kTri + row], a[(col + 2) * kTri + row], a[(col + 3) * kTri + row]};
  const float4 v = *reinterpret_cast<const float4 *>(a + row * kTri + col);
  return f32x4{v.x, v.y, v.z, v.w};
}

// c += L X for a 16x16 block of LDS (rows at r, contracted columns at k) and X in a result's layout.
__device__ __forceinline__ void block_multiply(f32x4 &c, const float *a, int r, int k, f32x4 x, int lane) {
  const f32x4 l = load4<false>(a, r + lane % 16, k + 4 * (lane / 16));
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(l[i], x[i], c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 block_load(const float *a, int r, int c, int lane) {
  return load4<true>(a, c + lane % 16, r + 4 * (lane / 16));
}
__device__ __forceinline__ void block_store(float *a, int r, int c, f32x4 v, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a[(r + 4 * (lane / 16) + i) * kTri + c + lane % 16] = v[i];
}

// What the wave's lanes have written to LDS is there for all of them: its accesses stay in order.
__device__ __forceinline__ void wave_done() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Turns the strictly lower A in LDS into (1 + A)^-1 (its upper blocks are not written).
__device__ __forceinline__ void invert(float *a, int lane) {
  {  // the diagonal blocks: block lane / 16, column lane % 16
    const int b = lane / 16 * 16, col = lane % 16;
    float x[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float s = r == col ? 1.0f : 0.0f;
#pragma unroll
      for (int k = 0; k < (r + 3) / 4; ++k) {
        const f32x4 v = load4<false>(a, b + r, b + 4 * k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * k + i < r) s = fmaf(-v[i], x[4 * k + i], s);
      }
      x[r] = s;
    }
    wave_done();
#pragma unroll
    for (int r = 0; r < 16; ++r) a[(b + r) * kTri + b + col] = x[r];
    wave_done();
  }
#pragma unroll
  for (int b = 0; b < kRun; b += 32) {
    f32x4 y = {0, 0, 0, 0}, t = {0, 0, 0, 0};
    block_multiply(y, a, b + 16, b, block_load(a, b, b, lane), lane);
    block_multiply(t, a, b + 16, b + 16, -y, lane);
    wave_done();
    block_store(a, b + 16, b, t, lane);
    wave_done();
  }
  f32x4 y[2][2], t[2][2];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      y[r][c] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = c; k < 2; ++k) block_multiply(y[r][c], a, 32 + 16 * r, 16 * k, block_load(a, 16 * k, 16 * c, lane), lane);
    }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      t[r][c] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k <= r; ++k) block_multiply(t[r][c], a, 32 + 16 * r, 32 + 16 * k, -y[k][c], lane);
    }
  wave_done();
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int c = 0; c < 2; ++c) block_store(a, 32 + 16 * r, 16 * c, t[r][c], lane);
  wave_done();
}

// ------------------------------------------------------ tiles of keys in LDS
// Rows of kRun steps, KEYS elements each, parts one behind the other. The bytes
// between rows keep off each other's banks both eight rows read by 16 bytes
// (tile_rows) and four by 8 (tile_columns): 16 of them do the former alone at 128 keys,
// 48 all but in pairs; more parts leave no room for that. (The maps of 65536 steps of 8
// heads of 128 x 128 bf16 381 and 366 us, outputs 262 either way.)
template <int KEYS, int NP>
constexpr int kTileRow = KEYS + (KEYS == 128 && NP == 1 ? 24 : 8);

// Operand with index row 16 m + lane % 16 and slots of elements 32 s + 8 g ...
template <int ROW, int NP>
__device__ __forceinline__ Cut<NP> plain_rows(const uint16_t *tile, int m, int s, int lane) {
  Cut<NP> c;
#pragma unroll
  for (int p = 0; p < NP; ++p)
    c.p[p] = *reinterpret_cast<const u32x4 *>(tile + (p * kRun + 16 * m + lane % 16) * ROW + 32 * s + 8 * (lane / 16));
  return c;
}
template <int KEYS, int NP>
__device__ __forceinline__ Cut<NP> tile_rows(const uint16_t *tile, int m, int s, int lane) {
  return plain_rows<kTileRow<KEYS, NP>, NP>(tile, m, s, lane);
}
template <int KEYS, int NP>
__device__ __forceinline__ void tile_rows(Cut<NP> (&c)[kTiles], const uint16_t *tile, int s, int lane) {
#pragma unroll
  for (int m = 0; m < kTiles; ++m) c[m] = tile_rows<KEYS, NP>(tile, m, s, lane);
}
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
// Four rows of one column for each lane: within 16 lanes, lane l reads 4
// elements of row l / 4 and receives column l of the 4 x 16 that they read.
__device__ __forceinline__ s16x4 transposed4(const uint16_t *p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
}
__device__ __forceinline__ u32x4 join8(s16x4 a, s16x4 b) {
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 v = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return __builtin_bit_cast(u32x4, v);
}
// Key that row (lane group g, i) of the state's tile t stands for: eight
// neighbouring keys of a lane then lie in the tiles 2 s and 2 s + 1, the slots
// of tile_rows.
__host__ __device__ constexpr int key_of(int t, int g, int i) { return 32 * (t / 2) + 8 * g + 4 * (t % 2) + i; }
// Operand with index the keys of state tile t and slots of the steps as results hold them.
template <int KEYS, int NP>
__device__ __forceinline__ Cut<NP> tile_columns(const uint16_t *tile, int t, int s, int lane) {
  Cut<NP> c;
  const int l = lane % 16, row = 32 * s + 4 * (lane / 16) + l / 4, col = key_of(t, l % 4, 0);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const uint16_t *q = tile + (p * kRun + row) * kTileRow<KEYS, NP> + col;
    c.p[p] = join8(transposed4(q), transposed4(q + 16 * kTileRow<KEYS, NP>));
  }
  return c;
}

// state += (columns of the tile)^T times the operands of steps 0..31 and 32..63, four tiles of keys at a time.
template <int KEYS, int NP>
__device__ __forceinline__ void multiply_columns(f32x4 (&state)[KEYS / 16], const uint16_t *tile, const Cut<kFull> &lo,
                                                 const Cut<kFull> &hi, int lane) {
  constexpr int M = KEYS / 16 < 4 ? KEYS / 16 : 4;
#pragma unroll
  for (int t = 0; t < KEYS / 16; t += M) {
    Cut<NP> k[2][M];
#pragma unroll
    for (int i = 0; i < M; ++i) {
      k[0][i] = tile_columns<KEYS, NP>(tile, t + i, 0, lane);
      k[1][i] = tile_columns<KEYS, NP>(tile, t + i, 1, lane);
    }
    multiply_rows<kFull>(state + t, k[0], lo);
    multiply_rows<kFull>(state + t, k[1], hi);
  }
}
// Operand with index columns col.. (lane % 16) and slots of rows row + 8 g + 0..7.
template <int ROW, int NP>
__device__ __forceinline__ Cut<NP> plain_columns(const uint16_t *tile, int row, int col, int lane) {
  Cut<NP> c;
  const int l = lane % 16;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const uint16_t *q = tile + (p * kRun + row + 8 * (lane / 16) + l / 4) * ROW + col + 4 * (l % 4);
    c.p[p] = join8(transposed4(q), transposed4(q + 4 * ROW));
  }
  return c;
}

// Keeps the scheduler from moving work across: it would start on later loads and products and spill.
__device__ __forceinline__ void part_done() { __builtin_amdgcn_sched_barrier(0); }

// The same number, of unknown origin: addresses and conditions made from it are
// computed where they are used. The compiler would else compute those of a whole
// loop's body in front of the loop, hundreds of them, and spill.
__device__ __forceinline__ int afresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Steps 16 m + 4 g + 0..3 of one value column, zeros where nothing is held.
template <typename T>
__device__ __forceinline__ f32x4 load_column(const fftmv_heads_t &f, int64_t b, int64_t row, int n, int64_t head,
                                             int m, int g, int col, bool inside) {
  f32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 16 * m + 4 * g + i;
    if (inside && t < n) v[i] = static_cast<float>(head_row<T>(f, b, row + t, head)[col]);
  }
  return v;
}

// ------------------------------------------------------- runs one after another
// The chains (of states, and of their gradients) go through a sequence's runs.
// Only K S, T (..) and K^T (..) X of a run wait for the run before: four waves, the
// front, do those, 16 value columns each with the state in registers; four more,
// one on each SIMD beside a front wave, do all else: they bring the next run's
// rows and triangles from memory to LDS and make the outputs from what the front
// leaves there, operands of the state at a run's start and of X in its middle. A
// run has two halves between barriers:
//   front  R = V - e^G K S, X = T R     | S' = e^{G_last} S + K^T (..) X
//   back   Q S; the next run's loads    | Y = .. + P diag(b) X; the next run into LDS
// The back waves set the pace of outputs: at 128 bf16 keys, nothing kept, a run takes 4.6
// us, 8.9 k clocks, of which the front works 5.1 (2.8 and 2.3 in its halves) and waits
// for the back's 4.7 (the next loads 1.7, Q S 3.0) and 4.3 (P diag(b) X and stores 2.5, the
// next run into LDS 1.8). The matrix units are busy 38 % of the time and 516 KB go through
// LDS, 58 bytes a clock of the 107 to 114 that a kernel of reads alone reaches. Maps, which
// have no outputs, take 2.7 us a run by the front's products in line; where states are kept,
// memory counts too. (8 x 2048 steps of 16 heads of 128 x 128 in bf16, 210 us with the
// states and errors kept, took 235 without the errors and all of it in one wave a SIMD,
// both before third parts: 225 with them. Loads two runs ahead were slower.)
constexpr int kFrontWaves = 4;
constexpr int kFrontThreads = kFrontWaves * kWave;
constexpr int kChainThreads = 2 * kFrontThreads;
constexpr int kValues = 16 * kFrontWaves;  // value columns of a workgroup
constexpr int kLdsBytes = 160 << 10;
constexpr int kCus = 256;

template <typename T>
constexpr int kValueRow = kValues + 16 / sizeof(T);

template <typename T, int KEYS, int FRAGS, int BUFFERS>
struct ChainLds {
  static constexpr int NP = kParts<T>, S = KEYS / 32;
  alignas(16) uint16_t k[BUFFERS][NP * kRun * kTileRow<KEYS, NP>];
  alignas(16) T v[kRun * kValueRow<T>];
  alignas(16) u32x4 frags[FRAGS * kWave];
  alignas(16) float into[kRun], out[kRun], rate[kRun];
};

// A thread's part of a run's rows of keys on their way to LDS.
template <typename T, int KEYS, bool WHOLE>
__device__ __forceinline__ void fetch_rows(Raw8<T> (&k)[KEYS / 32], int thread, const fftmv_heads_t &f, int keys,
                                           int64_t b, int64_t row, int n, int64_t head) {
  const Rows<T, WHOLE> rows(f, b, row, head, n, keys);
#pragma unroll
  for (int i = 0; i < KEYS / 32; ++i) k[i] = rows.load(thread / (KEYS / 8) + i * (kFrontThreads * 8 / KEYS), thread % (KEYS / 8) * 8);
}
template <typename T, int KEYS, bool WHOLE>
__device__ __forceinline__ void put_rows(Raw8<T> (&k)[KEYS / 32], int thread, uint16_t *tile, int keys, int n) {
#pragma unroll
  for (int i = 0; i < KEYS / 32; ++i) {
    const int u = thread + i * kFrontThreads, t = u / (KEYS / 8), c = u % (KEYS / 8) * 8;
    if (!WHOLE || keys < KEYS) settle<WHOLE>(k[i], c, keys, t < n);
    const auto parts = cut_raw<T>(k[i]);
#pragma unroll
    for (int p = 0; p < kParts<T>; ++p)
      *reinterpret_cast<u32x4 *>(tile + (p * kRun + t) * kTileRow<KEYS, kParts<T>> + c) = parts.p[p];
  }
}

// ------------------------------------------------------ T, P and the factors
// Zeros in the rows of `n` elements that belong to no sequence: those of a
// padded run behind its length; of the packed axis, rows 64 i.. outside all.
template <typename T>
__device__ __forceinline__ void clear_rows(const fftmv_delta_rule_t &r, const fftmv_heads_t &f, int64_t slot,
                                           int64_t b, int first, int64_t head, int n) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  constexpr int WAVES = kFrontWaves;
  if (!f.data) return;
  const int steps = static_cast<int>(r.steps);
  if (r.offsets) {
    const int lo = clamp_to(r.offsets[0], steps), hi = clamp_to(r.offsets[r.batch], steps);
    const int64_t at = slot * kRun;
    for (int64_t t = at + wave; t < at + kRun && t < steps; t += WAVES) {
      if (t >= lo && t < hi) continue;
      T *row = head_row<T>(f, 0, t, head);
      for (int c = lane; c < n; c += kWave) row[c] = static_cast<T>(0.0f);
    }
  } else if (r.lengths) {
    const int len = clamp_to(r.lengths[b], steps);
    for (int t = max(first, len) + wave; t < min(first + kRun, steps); t += WAVES) {
      T *row = head_row<T>(f, b, t, head);
      for (int c = lane; c < n; c += kWave) row[c] = static_cast<T>(0.0f);
    }
  }
}

// The kernel of a run's factors, for each run slot and head. Only the inverse is
// in line; products, decays and outputs go by fragments, the pieces that the
// chains load, two of P's tiles and the same two of the triangle each, so that a
// decay is computed once for both: four waves have three or two tiles each. Rows
// lie in LDS as they are in memory: products of 16-bit elements are exact in
// FP32, FP32 ones are cut where they are read. Memory bounds it: a run of 128 keys
// in 16 bits reads 32 KB and leaves 37 (8 x 2048 steps of 16 heads: 71 us forward, 74
// backward, 4.3 TB/s). One wave a run, with the rows in registers, took 8 % longer,
// and 20 us instead of 12 for 4 runs of 20 heads in FP32, where the latency of one
// counts. Heads that share keys follow each other: 30011 packed fp16 steps of 16 heads, 8
// of keys, 91 us instead of 96 (107 with P's third parts).
template <typename T, int KEYS>
struct FactorLds {
  static constexpr int ROW = KEYS + 16 / sizeof(T);
  alignas(16) T k[kRun * ROW];
  union {
    alignas(16) T q[kRun * ROW];
    alignas(16) float tri[kRun * kTri];  // once the products are there
  };
  double total[kRun];
  float rates[kRun];
};

// Workgroups that read the same rows follow each other on one XCD (workgroup i runs on
// XCD i % 8), which has them in its cache: `sharing` of them for each of `count` units,
// from a grid of all of them in one row.
struct Place {
  uint32_t unit, which;
  __device__ __forceinline__ Place(int64_t units, int sharing) {  // a grid's workgroups are counted in 32 bits
    const uint32_t count = static_cast<uint32_t>(units), each = static_cast<uint32_t>(sharing), i = blockIdx.x;
    const uint32_t whole = count / kXcds * kXcds, width = i < whole * each ? kXcds : count % kXcds;  // the last few units
    const uint32_t j = i < whole * each ? i : i - whole * each, row = j / width;
    unit = (i < whole * each ? row / each * kXcds : whole) + (j - row * width);
    which = row % each;
  }
};

// Fragment i of a wave: three of six tiles' worth to the first two waves, two to the others.
template <bool UPPER>
__device__ __forceinline__ int fragment_of(int wave, int i) {
  return UPPER ? (wave == 0 ? 1 + i : wave == 1 ? 4 + i : wave == 2 ? 0 : 3) : (wave < 2 ? 2 * wave + i : wave + 2);
}
__device__ __forceinline__ int fragments_of(int wave) { return wave < 2 ? 2 : 1; }
// The rows' tile and the slots' half of a fragment.
template <bool UPPER>
__device__ __forceinline__ int fragment_tile(int f) {
  return UPPER ? (f < 4 ? f / 2 : f - 2) : (f < 2 ? f : f / 2 + 1);
}
template <bool UPPER>
__device__ __forceinline__ int fragment_half(int f) {
  return UPPER ? (f < 4 ? f % 2 : 1) : (f < 2 ? 0 : f % 2);
}

// c += (rows of tile a of one) (rows of tile b of the other)^T, 32 elements.
template <typename T, int ROW>
struct RowOperand {
  using Raw = std::conditional_t<sizeof(T) == 4, Cut<kFull>, Cut<1>>;
  static __device__ __forceinline__ Raw load(const T *rows, int tile, int s, int lane) {
    const u32x4 *p = reinterpret_cast<const u32x4 *>(rows + (16 * tile + lane % 16) * ROW + 32 * s + 8 * (lane / 16));
    if constexpr (sizeof(T) == 4)
      return cut_raw<T>(Raw8<T>{{p[0], p[1]}});
    else
      return Raw{{p[0]}};
  }
  static __device__ __forceinline__ void multiply_into(f32x4 &c, const Raw &a, const Raw &b) {
    if constexpr (std::is_same_v<T, f16>)
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a.p[0]), __builtin_bit_cast(f16x8, b.p[0]), c, 0, 0, 0);
    else
      multiply<kFull>(c, a, b);
  }
};

template <typename T, int KEYS, bool WHOLE, bool BACK>
__global__ __launch_bounds__(kFrontThreads) void delta_factors_kernel(fftmv_delta_rule_t r, DeltaWorkspace w) {
  using Lds = FactorLds<T, KEYS>;
  using Tri = Triangles<BACK>;
  __shared__ Lds lds;
  const int thread = threadIdx.x, lane = thread % kWave, wave = thread / kWave, x = lane % 16, g = lane / 16;
  const uint32_t key_heads = static_cast<uint32_t>(r.key_heads), share = static_cast<uint32_t>(r.heads) / key_heads;
  const Place place(gridDim.x / share, share);
  const int64_t slot = place.unit / key_heads, key_head = place.unit % key_heads, head = key_head * share + place.which;
  const int64_t at = slot * r.heads + head;
  const Slot where = slot_of(r, slot);
  if constexpr (BACK) {
    clear_rows<T>(r, r.dv, slot, where.b, where.first, head, static_cast<int>(r.values));
    clear_rows<T>(r, r.dgate, slot, where.b, where.first, head, 1);
    clear_rows<T>(r, r.dbeta, slot, where.b, where.first, head, 1);
    if (place.which == 0) {
      clear_rows<T>(r, r.dq, slot, where.b, where.first, key_head, static_cast<int>(r.keys));
      clear_rows<T>(r, r.dk, slot, where.b, where.first, key_head, static_cast<int>(r.keys));
    }
  } else {
    clear_rows<T>(r, r.y, slot, where.b, where.first, head, static_cast<int>(r.values));
  }
  if (where.first < 0) return;
  const Span span = span_of(r, where.b);
  const int n = min(kRun, span.len - where.first);  // steps of this run
  if (n <= 0) return;
  const int64_t row = span.row + where.first;
  const int keys = static_cast<int>(r.keys);

  float gate = 0.0f, beta = 0.0f;
  if (wave == 0 && lane < n) {
    gate = static_cast<float>(*head_row<T>(r.gate, span.batch, row + lane, head));
    beta = static_cast<float>(*head_row<T>(r.beta, span.batch, row + lane, head));
  }
  Raw8<T> rows[2][KEYS / 32];
  fetch_rows<T, KEYS, WHOLE>(rows[0], thread, r.k, keys, span.batch, row, n, key_head);
  fetch_rows<T, KEYS, WHOLE>(rows[1], thread, r.q, keys, span.batch, row, n, key_head);
  if (wave == 0) {  // gates: lane i has step i; steps behind the last leave the state as it is
    const bool held = lane < n;
    const double sum = lane_sums(held ? static_cast<double>(log_decay(r.decay, gate)) : 0.0, lane);
    const double last = __shfl(sum, kRun - 1);
    const float rate = held ? rate_of(r.rate, beta) : 0.0f;
    Factors &f = w.factors[at];
    f.into[lane] = expf(static_cast<float>(sum));
    f.out[lane] = expf(static_cast<float>(last - sum)) * (BACK ? 1.0f : rate);
    f.sum[lane] = sum;
    f.rate[lane] = lds.rates[lane] = rate;
    lds.total[lane] = sum;
  }
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int i = 0; i < KEYS / 32; ++i) {
      const int u = thread + i * kFrontThreads, t = u / (KEYS / 8), c = u % (KEYS / 8) * 8;
      if (!WHOLE || keys < KEYS) settle<WHOLE>(rows[which][i], c, keys, t < n);
      u32x4 *to = reinterpret_cast<u32x4 *>((which ? lds.q : lds.k) + t * Lds::ROW + c);
#pragma unroll
      for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h) to[h] = rows[which][i].w[h];
    }
  __syncthreads();

  // products and decays: rows of tile `own` at lane % 16, two tiles of slots. Forward
  // rows are those of T and P, backward those of their transposes
  using Op = RowOperand<T, Lds::ROW>;
  u32x4 *out = w.triangles + at * Tri::kAll * kWave;
  const int count = fragments_of(wave);
  f32x4 below[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i >= count) break;
    const int f = fragment_of<BACK>(wave, i), own = fragment_tile<BACK>(f), half = fragment_half<BACK>(f);
    f32x4 p[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int other = 2 * half + h;
      p[h] = below[i][h] = f32x4{0, 0, 0, 0};
      if (BACK ? other < own : other > own) continue;
#pragma unroll
      for (int s = 0; s < KEYS / 32; ++s) {
        const auto a = Op::load(lds.k, other, s, lane), b = Op::load(lds.k, own, s, lane);
        Op::multiply_into(below[i][h], a, b);
        if constexpr (BACK)
          Op::multiply_into(p[h], Op::load(lds.q, other, s, lane), b);
        else
          Op::multiply_into(p[h], a, Op::load(lds.q, own, s, lane));
      }
      const int one = 16 * own + x, first = 16 * other + 4 * g;
      const double mine = lds.total[one];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int step = BACK ? first + e : one, past = BACK ? one : first + e;
        const double between = BACK ? lds.total[step] - mine : mine - lds.total[past];
        const float decay = past <= step ? expf(static_cast<float>(between)) : 0.0f;
        // A = B diag(b) forward, diag(b) B backward
        p[h][e] = past <= step ? r.scale * (BACK ? 1.0f : lds.rates[past]) * decay * p[h][e] : 0.0f;
        below[i][h][e] = past < step ? lds.rates[BACK ? step : past] * decay * below[i][h][e] : 0.0f;
      }
    }
    const auto c = cut_tiles<kFull>(p[0], p[1]);
#pragma unroll
    for (int a = 0; a < kFull; ++a) out[(Tri::kP + (BACK ? f * kFull + a : a * kFrags + f)) * kWave + lane] = c.p[a];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i >= count) break;
    const int f = fragment_of<BACK>(wave, i), own = fragment_tile<BACK>(f), half = fragment_half<BACK>(f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int other = 2 * half + h;
      if (BACK ? other < own : other > own) continue;
      if constexpr (BACK)
        block_store(lds.tri, 16 * other, 16 * own, below[i][h], lane);
      else
        *reinterpret_cast<f32x4 *>(lds.tri + (16 * own + x) * kTri + 16 * other + 4 * g) = below[i][h];
    }
  }
  __syncthreads();
  if (wave == 0) invert(lds.tri, lane);
  __syncthreads();

#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i >= count) break;
    const int f = fragment_of<BACK>(wave, i), own = 16 * fragment_tile<BACK>(f) + x, first = 32 * fragment_half<BACK>(f) + 4 * g;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int other = first + 16 * (e / 4) + e % 4, t = BACK ? other : own, j = BACK ? own : other;
      v[e] = j <= t ? lds.tri[t * kTri + j] : 0.0f;
    }
    const auto c = cut<kFull>(v);
#pragma unroll
    for (int q = 0; q < kFull; ++q) out[((BACK ? Tri::kTt : Tri::kT) + f * kFull + q) * kWave + lane] = c.p[q];
  }
}

// The same for all that a run needs: keys, values, a triangle's fragments, factors.
template <typename T, int KEYS, int FRAGS, bool WHOLE>
struct Fetched {
  static constexpr int NV = kValues / 32, NF = (FRAGS * kWave + kFrontThreads - 1) / kFrontThreads;
  Raw8<T> k[KEYS / 32], v[NV];
  u32x4 frags[NF], factors;

  __device__ __forceinline__ void fetch_keys(int thread, const fftmv_heads_t &f, int keys, int64_t b, int64_t row, int n,
                                             int64_t head) {
    fetch_rows<T, KEYS, WHOLE>(k, thread, f, keys, b, row, n, head);
  }
  __device__ __forceinline__ void put_keys(int thread, uint16_t *tile, int keys, int n) {
    put_rows<T, KEYS, WHOLE>(k, thread, tile, keys, n);
  }
  __device__ __forceinline__ void fetch_values(int thread, const fftmv_heads_t &f, int values, int64_t b, int64_t row,
                                               int n, int64_t head, int first_col) {
    const Rows<T, WHOLE> rows(f, b, row, head, n, values);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      v[i] = rows.load(thread / (kValues / 8) + i * (kFrontThreads * 8 / kValues), first_col + thread % (kValues / 8) * 8);
  }
  template <typename L>
  __device__ __forceinline__ void put_values(int thread, L &lds, int values, int n, int first_col) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = thread + i * kFrontThreads, t = u / (kValues / 8), c = u % (kValues / 8) * 8;
      if (!WHOLE || first_col + kValues > values) settle<WHOLE>(v[i], first_col + c, values, t < n);
#pragma unroll
      for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h)
        reinterpret_cast<u32x4 *>(lds.v + t * kValueRow<T> + c)[h] = v[i].w[h];
    }
  }
  __device__ __forceinline__ void fetch_factors(int thread, const u32x4 *from, const Factors &f) {
#pragma unroll
    for (int i = 0; i < NF; ++i) frags[i] = at_lane(from, min(thread + i * kFrontThreads, FRAGS * kWave - 1));
    factors = at_lane(reinterpret_cast<const u32x4 *>(f.into), min(thread, 3 * kRun / 4 - 1));
  }
  template <typename L>
  __device__ __forceinline__ void put_factors(int thread, L &lds) {
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const int u = thread + i * kFrontThreads;
      if (FRAGS * kWave % kFrontThreads == 0 || u < FRAGS * kWave) lds.frags[u] = frags[i];
    }
    if (thread < 3 * kRun / 4) reinterpret_cast<u32x4 *>(lds.into)[thread] = factors;
  }
};

// Rows of queries as operands straight from memory, HOLD of their S parts of 32 keys at a time.
template <typename T, int KEYS, bool WHOLE>
struct QueryRows {
  static constexpr int S = KEYS / 32, HOLD = sizeof(T) == 2 ? S : 1;
  Raw8<T> q[HOLD][kTiles];
  template <int s>
  __device__ __forceinline__ void fetch(const fftmv_heads_t &f, int keys, int64_t b, int64_t row, int n,
                                        int64_t head, int lane) {
    const Rows<T, WHOLE> rows(f, b, row, head, n, keys);
#pragma unroll
    for (int m = 0; m < kTiles; ++m) q[s % HOLD][m] = rows.load(16 * m + lane % 16, 32 * s + 8 * (lane / 16));
  }
  template <int s>
  __device__ __forceinline__ Cut<kParts<T>> operand(int m, int keys, int n, int lane) {
    if (!WHOLE || keys < KEYS)
      settle<WHOLE>(q[s % HOLD][m], 32 * s + 8 * (lane / 16), keys, 16 * m + lane % 16 < n);
    return cut_raw<T>(q[s % HOLD][m]);
  }
};

// Steps 16 m + 4 g + 0..3 of column col + lane % 16 of the values in LDS.
template <typename T>
__device__ __forceinline__ f32x4 value_column(const T *v, int m, int col, int lane) {
  const int l = lane % 16, row = 16 * m + 4 * (lane / 16);
  f32x4 r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = v[(row + i) * kValueRow<T> + col + l];
  } else {
    typedef T T4 __attribute__((ext_vector_type(4)));
    const uint16_t *p = reinterpret_cast<const uint16_t *>(v) + (row + l / 4) * kValueRow<T> + col + 4 * (l % 4);
    const T4 q = __builtin_bit_cast(T4, transposed4(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = static_cast<float>(q[i]);
  }
  return r;
}

// Rows that are multiples of eight elements, begin at words, do not overlap, and
// whose run of 64 is addressed in 31 bits.
inline bool delta_whole(const fftmv_heads_t &f, int64_t width, int dtype) {
  const int64_t es = dtype == FFTMV_F32 ? 4 : 2;
  return width % 8 == 0 && f.step >= width && f.step <= (1 << 22) && f.batch * es % 4 == 0 && f.step * es % 4 == 0 &&
         f.head * es % 4 == 0 && reinterpret_cast<uintptr_t>(f.data) % 4 == 0;
}
inline bool delta_whole_rows(const fftmv_delta_rule_t &r) {
  return delta_whole(r.q, r.keys, r.dtype) && delta_whole(r.k, r.keys, r.dtype);
}
inline bool delta_whole(const fftmv_delta_rule_t &r, const fftmv_heads_t &valued, const fftmv_heads_t &other) {
  return delta_whole_rows(r) && delta_whole(valued, r.values, r.dtype) && delta_whole(other, r.values, r.dtype);
}
// A part of a sequence, in its steps.
struct Part {
  int part, begin, end;
  __device__ __forceinline__ Part(const DeltaCuts &cuts, int64_t index, int len)
      : part(static_cast<int>(index % cuts.parts)) {
    const int64_t each = static_cast<int64_t>(cuts.runs) * kRun;
    begin = static_cast<int>(min(part * each, static_cast<int64_t>(len)));
    end = static_cast<int>(part == cuts.parts - 1 ? len : min((part + 1) * each, static_cast<int64_t>(len)));
  }
};

// The sequence of a place, longest first, so that none of the long ones begins when
// the others end. `lens`: kChainThreads + 1 words of LDS. More sequences than threads,
// sequences in parts and those that all run at once keep their order. (45 packed
// sequences of 30011 steps, 16 heads of 64 x 128 fp16: 288 us, in their order 350, with a
// chain's blocks far apart too 385; 310 with third parts.)
__device__ __forceinline__ int64_t longest_first(const fftmv_delta_rule_t &r, const DeltaCuts &cuts, int64_t place, int *lens) {
  if (!(r.offsets || r.lengths) || r.batch > kChainThreads || cuts.parts > 1 || gridDim.x <= kCus) return place;
  const int me = threadIdx.x, n = static_cast<int>(r.batch);
  if (me < n) lens[me] = span_of(r, me).len;
  __syncthreads();
  if (me < n) {
    const int mine = lens[me];
    int rank = 0;
    for (int i = 0; i < n; ++i) rank += lens[i] > mine || (lens[i] == mine && i < me);
    if (rank == place) lens[kChainThreads] = me;
  }
  __syncthreads();
  const int b = __builtin_amdgcn_readfirstlane(lens[kChainThreads]);
  __syncthreads();
  return b;
}

// The states in front of the parts (backward: the gradients of those behind
// them) one after another. A workgroup has 16 value columns and a wave 16 keys of
// them; the waves pass each other the state through LDS, and load the next map
// while they wait: 3.1 us a joint at 128 x 128 (one wave for all keys: 18).
// (T keeps the instances of one element type's source apart from the others'.)
template <typename T, int KEYS, bool BACK>
__global__ __launch_bounds__(KEYS / 16 * kWave) void delta_join_kernel(fftmv_delta_rule_t r, DeltaWorkspace w) {
  constexpr int S = KEYS / 32, TILES = KEYS / 16;
  __shared__ f32x4 shared[2][TILES][kWave];
  const int t = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave, x = lane % 16, g = lane / 16;
  const int keys = static_cast<int>(r.keys), values = static_cast<int>(r.values), width = keys + values;
  const int col = blockIdx.y * 16 + x, row = key_of(t, x / 4, x % 4);
  const bool inside = col < values;
  const int64_t sequence = blockIdx.x, states = r.keys * r.values;
  const Span span = span_of(r, sequence / r.heads);
  const int64_t each = static_cast<int64_t>(w.cuts.runs) * kRun;
  const int joints = static_cast<int>((span.len + each - 1) / each) - 1;
  auto part_of = [&](int i) { return BACK ? joints - i : i; };
  struct Map {
    float m[S][8];
    f32x4 n;
  };
  auto fetch = [&](Map &to, int i) __attribute__((always_inline)) {
    const float *map = w.maps + (sequence * w.cuts.parts + part_of(i)) * keys * width;
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int e = 0; e < 8; ++e) to.m[s][e] = 0.0f;
      if (row < keys) load8(map + static_cast<int64_t>(row) * width + values, 32 * s + 8 * g, keys, to.m[s]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = key_of(t, g, e);
      to.n[e] = inside && key < keys ? map[static_cast<int64_t>(key) * width + col] : 0.0f;
    }
  };
  const float *from = BACK ? r.dh_last : r.h0;
  f32x4 state;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = key_of(t, g, i);
    state[i] = from && inside && key < keys ? from[sequence * states + static_cast<int64_t>(key) * values + col] : 0.0f;
  }
  auto join = [&](const Map &map, int i) __attribute__((always_inline)) {
    shared[i % 2][t][lane] = state;
    __syncthreads();
    state = map.n;
#pragma unroll
    for (int s = 0; s < S; ++s)
      multiply<kFull>(state, cut<kFull>(map.m[s]), cut_tiles<kFull>(shared[i % 2][2 * s][lane], shared[i % 2][2 * s + 1][lane]));
    float *to = w.starts + (sequence * w.cuts.parts + part_of(i) + (BACK ? -1 : 1)) * states;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = key_of(t, g, e);
      if (inside && key < keys) to[static_cast<int64_t>(key) * values + col] = state[e];
    }
  };
  Map even, odd;
  if (joints > 0) fetch(even, 0);
  for (int i = 0; i < joints; i += 2) {
    if (i + 1 < joints) fetch(odd, i + 1);
    join(even, i);
    if (i + 1 >= joints) break;
    if (i + 2 < joints) fetch(even, i + 2);
    join(odd, i + 1);
  }
}

template <typename F>
hipError_t by_keys(int64_t keys, F f) {
  if (keys <= 32) return f(Const<32>{});
  if (keys <= 64) return f(Const<64>{});
  return f(Const<128>{});
}

}  // namespace fftmv
