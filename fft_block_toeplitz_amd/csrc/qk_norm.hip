#include "qk_norm.hpp"

namespace fftmv {
namespace {

// Where a lane's elements are: slots 0..3 and 4..7 from `first` and `second`
// on, or each by itself. Rotated halves: pair e in slots e and e + 4;
// neighbours: in slots 2 e and 2 e + 1.
struct Lane {
  int first, second;
  bool whole;      // by fours
  bool joined;     // all eight in a row
  uint32_t owned;  // slots that are this lane's alone, bit by bit
  int turns;       // its cosines
};
// The element of a slot of a lane that takes them one by one, or -1.
__device__ __forceinline__ int element_of(const NormPlan &s, bool halves, int l, int slot) {
  const int p = kNormPairs * l + (halves ? slot % kNormPairs : slot / 2);
  const bool odd = halves ? slot >= kNormPairs : slot % 2;
  const int i = halves && p < s.turned ? p + (odd ? s.turned : 0) : 2 * p + odd;
  return i < s.dim ? i : -1;
}
// The rotated pair of a lane's e-th.
template <bool WHOLE>
__device__ __forceinline__ int pair_of(const NormPlan &s, int l, int e) {
  const int p = kNormPairs * l;
  return (WHOLE ? min(p, s.turned - kNormPairs) : p) + e;
}
template <bool WHOLE>
__device__ __forceinline__ Lane lane_of(const NormPlan &s, bool halves, int l) {
  Lane r = {0, 4, true, false, 0, min(l, s.turned_lanes) * kNormPairs};
  const int p = kNormPairs * l;
  if constexpr (WHOLE) {
    if (l < s.turned_lanes) {
      const int from = pair_of<WHOLE>(s, l, 0), shared = p - from;
      r.first = halves ? from : 2 * from;
      r.second = halves ? from + s.turned : 2 * from + 4;
      r.owned = halves ? (0xfu & (0xfu << shared)) * 0x11u : 0xffu & (0xffu << 2 * shared);
    } else {
      const int at = 2 * s.turned + kNormElements * (l - s.turned_lanes), from = min(at, s.dim - kNormElements);
      r.first = from;
      r.second = from + 4;
      r.owned = at < s.dim ? 0xffu & (0xffu << (at - from)) : 0;
    }
  } else {
    r.whole = halves && p < s.turned ? p + kNormPairs <= s.turned : 2 * p + kNormElements <= s.dim;
    r.first = halves && p < s.turned ? p : 2 * p;
    r.second = halves && p < s.turned ? p + s.turned : 2 * p + 4;
#pragma unroll
    for (int e = 0; e < kNormElements; ++e)
      if (element_of(s, halves, l, e) >= 0) r.owned |= 1u << e;
  }
  r.joined = r.whole && r.second == r.first + 4;
  return r;
}

// A lane's elements as they lie in memory, in words: as elements of 16 bits the
// compiler takes them apart where they are loaded, and waits there (8 x 2048 rows
// of 32 heads of 128 bf16, gradients: 83 us, so 72).
template <typename T>
struct Raw {
  uint32_t w[2 * sizeof(T)];
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(w[e]);
    else
      return static_cast<float>(__builtin_bit_cast(T, static_cast<uint16_t>(w[e / 2] >> e % 2 * 16)));
  }
};
// Lanes without elements read some of their neighbours' where all are taken by fours.
template <bool WHOLE, typename T>
__device__ __forceinline__ void fetch(Raw<T> &r, const T *x, const Lane &at, const NormPlan &s, bool halves, int l) {
  using W = typename Words<4 * sizeof(T)>::type;
  constexpr int N = sizeof(T);  // words of four elements
  if (at.joined && sizeof(T) == 2) {
    const u32x4_any v = *reinterpret_cast<const u32x4_any *>(x + at.first);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = v[i];
  } else if (WHOLE || at.whole) {
    const W u = *reinterpret_cast<const W *>(x + at.first), v = *reinterpret_cast<const W *>(x + at.second);
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = u[i], r.w[N + i] = v[i];
  } else if (at.owned) {
    T each[kNormElements];
#pragma unroll
    for (int e = 0; e < kNormElements; ++e) {
      const int i = element_of(s, halves, l, e);
      each[e] = i >= 0 ? x[i] : static_cast<T>(0.0f);
    }
    __builtin_memcpy(&r, each, sizeof(r));
  }
}
template <bool WHOLE, typename T>
__device__ __forceinline__ void put(T *y, const float (&v)[kNormElements], const Lane &at, const NormPlan &s, bool halves,
                                    int l) {
  if (!at.owned) return;
  if (at.joined && sizeof(T) == 2) {
    // in one: lines streamed by halves partly leave twice (neighbours, 128 MB of results: 150 MB written, 52 us instead
    // of 47; gradients 80 instead of 72)
    if constexpr (sizeof(T) == 2) store_vec(y + at.first, v);
  } else if (WHOLE || at.whole) {
    const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
    store_vec(y + at.first, lo);
    store_vec(y + at.second, hi);
  } else {
#pragma unroll
    for (int e = 0; e < kNormElements; ++e) {
      const int i = element_of(s, halves, l, e);
      if (i >= 0) y[i] = static_cast<T>(v[e]);
    }
  }
}

// The pairs of a lane turned by their angles.
__device__ __forceinline__ void turn(float (&v)[kNormElements], const float4 &cosines, const float4 &sines, bool halves) {
  const float c[4] = {cosines.x, cosines.y, cosines.z, cosines.w}, s[4] = {sines.x, sines.y, sines.z, sines.w};
  const auto pair = [&](int e, float &a, float &b) {
    const float x = a, y = b;
    a = fmaf(x, c[e], -(y * s[e]));
    b = fmaf(y, c[e], x * s[e]);
  };
  if (halves) {
#pragma unroll
    for (int e = 0; e < kNormPairs; ++e) pair(e, v[e], v[e + 4]);
  } else {
#pragma unroll
    for (int e = 0; e < kNormPairs; ++e) pair(e, v[2 * e], v[2 * e + 1]);
  }
}

// The sum over the LANES lanes of a head, the same in each of them.
template <int LANES>
__device__ __forceinline__ float across(float v) {
  v += dpp<kDppQuadXor1>(v);
  v += dpp<kDppQuadXor2>(v);
  v += dpp<kDppRowHalfMirror>(v);
  if constexpr (LANES >= 16) v += dpp<kDppRowMirror>(v);
  if constexpr (LANES >= 32) v += __shfl_xor(v, 16);
  if constexpr (LANES >= 64) v += __shfl_xor(v, 32);
  return v;
}

// A row of a workgroup: where it begins in x, dy and y (dx), in elements, and
// its position. Rows behind their sequence have nothing to read.
struct NormRow {
  int64_t x, dy, to;
  double position;
  int held;
};

template <typename T, int LANES, bool WHOLE, bool BACK>
__global__ __launch_bounds__(kBlock) void qk_norm_kernel(fftmv_qk_norm_t n, NormPlan s, float *partials) {
  constexpr int GROUPS = kBlock / LANES, SLOTS = LANES * kNormElements;
  __shared__ float4 turns[2][kNormTurns / 4];
  __shared__ NormRow table[kNormRows];
  const bool halves = n.pairs == FFTMV_PAIRS_HALVES, query = static_cast<int>(blockIdx.x) < s.blocks[0];
  const int block = query ? blockIdx.x : blockIdx.x - s.blocks[0], blocks = s.blocks[query ? 0 : 1];
  const int most = s.rows[query ? 0 : 1], heads = static_cast<int>(query ? n.query_heads : n.key_heads);
  const fftmv_heads_t from = query ? n.q : n.k, grad = query ? n.dqy : n.dky;
  const fftmv_heads_t to = BACK ? (query ? n.dq : n.dk) : (query ? n.qy : n.ky);
  const float *weight = query ? n.q_weight : n.k_weight;
  const int l = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const Lane at = lane_of<WHOLE>(s, halves, l);
  const uint32_t rows = static_cast<uint32_t>(n.batch * n.steps), steps = static_cast<uint32_t>(n.steps);
  const float over = n.norm == FFTMV_NORM_RMS ? 1.0f / s.dim : 1.0f;
  float w[kNormElements], dw[kNormElements] = {};
  Raw<float> weights;
#pragma unroll
  for (int e = 0; e < kNormElements; ++e) weights.w[e] = __float_as_uint(1.0f);
  if (weight) fetch<WHOLE>(weights, weight, at, s, halves, l);
#pragma unroll
  for (int e = 0; e < kNormElements; ++e) w[e] = weights[e];
  // the next of a group's heads, `GROUPS` further along the rows
  const int down = GROUPS / heads, along = GROUPS - down * heads;
  for (uint32_t first = static_cast<uint32_t>(block) * most; first < rows; first += static_cast<uint32_t>(blocks) * most) {
    const int count = static_cast<int>(min(static_cast<uint32_t>(most), rows - first));
    int r = group / heads, h = group - r * heads;
    Raw<T> x = {}, dy = {};
    const auto take = [&](int64_t x0, int64_t dy0) {
      fetch<WHOLE>(x, static_cast<const T *>(from.data) + x0 + h * from.head, at, s, halves, l);
      if constexpr (BACK) fetch<WHOLE>(dy, static_cast<const T *>(grad.data) + dy0 + h * grad.head, at, s, halves, l);
    };
    if (r < count) {  // the first head needs no table, and is fetched held or not
      const uint32_t b = (first + r) / steps, t = first + r - b * steps;
      take(b * from.batch + t * from.step, b * grad.batch + t * grad.step);
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < count) {
      const uint32_t row = first + threadIdx.x, b = row / steps, t = row - b * steps;
      table[threadIdx.x] = {b * from.batch + t * from.step, b * grad.batch + t * grad.step, b * to.batch + t * to.step,
                            n.positions ? static_cast<double>(n.positions[b * n.position_batch + t]) : static_cast<double>(t),
                            !n.lengths || static_cast<int>(t) < n.lengths[b]};
    }
    __syncthreads();
    if (s.turned) {
      float *cosines = reinterpret_cast<float *>(turns[0]), *sines = reinterpret_cast<float *>(turns[1]);
      for (int i = threadIdx.x; i < count * s.turns; i += kBlock) {
        const int row = i / s.turns, slot = i - row * s.turns;
        const int p = pair_of<WHOLE>(s, slot / kNormPairs, slot % kNormPairs);
        float sn = 0.0f, cs = 1.0f;
        if (slot < s.turns - kNormPairs && p < s.turned) {
          double angle = table[row].position * n.frequency[p] * 0.15915494309189533577;  // 1 / (2 pi)
          angle -= rint(angle);
          sincospif(2.0f * static_cast<float>(angle), &sn, &cs);
        }
        cosines[i] = cs;
        sines[i] = sn;
      }
      __syncthreads();
    }
    while (r < count) {
      float v[kNormElements], g[kNormElements];
#pragma unroll
      for (int e = 0; e < kNormElements; ++e) v[e] = x[e], g[e] = dy[e];
      const int row = r;
      const bool held = table[row].held;
      T *y = static_cast<T *>(to.data) + table[row].to + h * to.head;
      r += down, h += along;
      if (h >= heads) h -= heads, ++r;
      if (r < count && table[r].held) take(table[r].x, table[r].dy);
      if (!held) {
#pragma unroll
        for (int e = 0; e < kNormElements; ++e) v[e] = 0.0f;
        put<WHOLE>(y, v, at, s, halves, l);
        continue;
      }
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < kNormElements; ++e) {
        const float u = at.owned >> e & 1 ? v[e] : 0.0f;
        sum = fmaf(u, u, sum);
      }
      const float inverse = 1.0f / sqrtf(fmaf(across<LANES>(sum), over, n.eps));
      float4 cs = {}, sn = {};
      if (s.turned) {
        const int i = (row * s.turns + at.turns) / 4;
        cs = turns[0][i], sn = turns[1][i];
      }
      if constexpr (!BACK) {
#pragma unroll
        for (int e = 0; e < kNormElements; ++e) v[e] *= inverse * w[e];
        if (s.turned) turn(v, cs, sn, halves);
      } else {
        if (s.turned) turn(g, cs, make_float4(-sn.x, -sn.y, -sn.z, -sn.w), halves);
        float inner = 0.0f;
#pragma unroll
        for (int e = 0; e < kNormElements; ++e) {
          v[e] *= inverse;  // x / n
          dw[e] = fmaf(g[e], v[e], dw[e]);
          g[e] *= w[e];
          inner = fmaf(at.owned >> e & 1 ? g[e] : 0.0f, v[e], inner);
        }
        inner = across<LANES>(inner) * over;
#pragma unroll
        for (int e = 0; e < kNormElements; ++e) v[e] = inverse * fmaf(-v[e], inner, g[e]);
      }
      put<WHOLE>(y, v, at, s, halves, l);
    }
  }
  if constexpr (BACK) {
    if (!partials) return;
    // the groups' sums, joined in a fixed order
    float *sums = reinterpret_cast<float *>(turns);
    static_assert(sizeof(turns) >= kBlock * kNormElements * sizeof(float), "eight sums of each thread");
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kNormElements; ++e) sums[group * SLOTS + e * LANES + l] = dw[e];
    __syncthreads();
    for (int i = threadIdx.x; i < SLOTS; i += kBlock) {
      const int e = i / LANES;  // of this thread's own lane: LANES divides kBlock
      if (!(at.owned >> e & 1)) continue;
      const int j = !WHOLE && !at.whole ? element_of(s, halves, l, e) : e < 4 ? at.first + e : at.second + e - 4;
      float sum = 0.0f;
#pragma unroll 4
      for (int q = 0; q < GROUPS; ++q) sum += sums[q * SLOTS + i];
      partials[static_cast<int64_t>(blockIdx.x) * s.dim + j] = sum;
    }
  }
}

// The workgroups' sums for one element of one weight each: a wave's lanes take
// every 64th, and add up across.
__global__ __launch_bounds__(kWave) void qk_norm_sums_kernel(const float *partials, int queries, int keys, int dim, float *dq,
                                                             float *dk) {
  const bool query = static_cast<int>(blockIdx.x) < dim;
  const int i = query ? blockIdx.x : blockIdx.x - dim, blocks = query ? queries : keys;
  float *to = query ? dq : dk;
  if (!to) return;
  if (!query) partials += static_cast<int64_t>(queries) * dim;
  float sum = 0.0f;
#pragma unroll 8
  for (int b = threadIdx.x; b < blocks; b += kWave) sum += partials[static_cast<int64_t>(b) * dim + i];
  sum = across<kWave>(sum);
  if (threadIdx.x == 0) to[i] = sum;
}

template <typename F>
hipError_t by_lanes(int lanes, F f) {
  if (lanes <= 8) return f(Const<8>{});
  if (lanes <= 16) return f(Const<16>{});
  if (lanes <= 32) return f(Const<32>{});
  return f(Const<64>{});
}

template <bool BACK>
hipError_t launch(const fftmv_qk_norm_t &n, const NormPlan &p, float *partials, hipStream_t s) {
  return by_dtype(n.dtype, [&](auto t) {
    return by_lanes(p.lanes, [&](auto lanes) {
      constexpr int L = decltype(lanes)::value;
      const int blocks = p.blocks[0] + p.blocks[1];
      if (p.apart)
        qk_norm_kernel<decltype(t), L, true, BACK><<<blocks, kBlock, 0, s>>>(n, p, partials);
      else
        qk_norm_kernel<decltype(t), L, false, BACK><<<blocks, kBlock, 0, s>>>(n, p, partials);
      return hipGetLastError();
    });
  });
}

}  // namespace

hipError_t launch_qk_norm_forward(const fftmv_qk_norm_t &n, hipStream_t s) {
  const int64_t rows = n.batch * n.steps;
  if (rows == 0) return hipSuccess;
  return launch<false>(n, qk_norm_plan(rows, n.query_heads, n.key_heads, n.dim, n.frequencies, false), nullptr, s);
}

hipError_t launch_qk_norm_backward(const fftmv_qk_norm_t &n, hipStream_t s) {
  const int64_t rows = n.batch * n.steps;
  NormPlan p = {};
  float *partials = n.dq_weight || n.dk_weight ? static_cast<float *>(n.workspace) : nullptr;
  if (rows > 0) {
    p = qk_norm_plan(rows, n.query_heads, n.key_heads, n.dim, n.frequencies, true);
    const hipError_t e = launch<true>(n, p, partials, s);
    if (e != hipSuccess) return e;
  }
  if (!n.dq_weight && !n.dk_weight) return hipSuccess;
  const int dim = static_cast<int>(n.dim);
  qk_norm_sums_kernel<<<2 * dim, kWave, 0, s>>>(partials, p.blocks[0], p.blocks[1], dim, n.dq_weight, n.dk_weight);
  return hipGetLastError();
}

}  // namespace fftmv
