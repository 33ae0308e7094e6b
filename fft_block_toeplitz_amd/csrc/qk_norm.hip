#include "qk_norm.hpp"

namespace fftmv {
namespace {

// The elements of a lane's pairs 4 l..4 l + 3 of one head: two runs of four
// (rotated halves), one run of eight (neighbours, and what is not rotated), or
// whatever is left at borders, one by one.
struct Lane {
  int first, second;  // element of pair 0's halves
  int mode;           // 0: four and four, 1: eight, 2: one by one, 3: nothing
};
__device__ __forceinline__ int pair_first(int p, int turned, bool halves) { return halves && p < turned ? p : 2 * p; }
__device__ __forceinline__ int pair_second(int p, int turned, bool halves) {
  return halves && p < turned ? p + turned : 2 * p + 1;
}
__device__ __forceinline__ Lane lane_of(int l, int turned, bool halves, int dim) {
  const int p = kNormPairs * l, end = p + kNormPairs;
  Lane r = {pair_first(p, turned, halves), pair_second(p, turned, halves), 2};
  if (2 * p >= dim && (!halves || p >= turned))
    r.mode = 3;
  else if (halves && end <= turned)
    r.mode = 0;
  else if ((!halves || p >= turned) && 2 * end <= dim)
    r.mode = 1;
  return r;
}

template <typename T>
__device__ __forceinline__ void load_pairs(const T *x, const Lane &at, int l, int turned, bool halves, int dim,
                                           float (&a)[kNormPairs], float (&b)[kNormPairs]) {
  if (at.mode == 0) {
    const Vec<T, 4> u = load_vec<T, 4>(x + at.first), v = load_vec<T, 4>(x + at.second);
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = u[e], b[e] = v[e];
  } else if (at.mode == 1) {
    const Vec<T, 4> u = load_vec<T, 4>(x + at.first), v = load_vec<T, 4>(x + at.first + 4);
    a[0] = u[0], b[0] = u[1], a[1] = u[2], b[1] = u[3];
    a[2] = v[0], b[2] = v[1], a[3] = v[2], b[3] = v[3];
  } else {
#pragma unroll
    for (int e = 0; e < kNormPairs; ++e) {
      const int p = kNormPairs * l + e, i = pair_first(p, turned, halves), j = pair_second(p, turned, halves);
      a[e] = at.mode == 2 && i < dim ? static_cast<float>(x[i]) : 0.0f;
      b[e] = at.mode == 2 && j < dim ? static_cast<float>(x[j]) : 0.0f;
    }
  }
}
template <typename T>
__device__ __forceinline__ void store_pairs(T *y, const Lane &at, int l, int turned, bool halves, int dim,
                                            const float (&a)[kNormPairs], const float (&b)[kNormPairs]) {
  if (at.mode == 0) {
    store_vec(y + at.first, a);
    store_vec(y + at.second, b);
  } else if (at.mode == 1) {
    const float u[8] = {a[0], b[0], a[1], b[1], a[2], b[2], a[3], b[3]};
    if constexpr (sizeof(T) == 2) {
      store_vec(y + at.first, u);
    } else {
      const float lo[4] = {u[0], u[1], u[2], u[3]}, hi[4] = {u[4], u[5], u[6], u[7]};
      store_vec(y + at.first, lo);
      store_vec(y + at.first + 4, hi);
    }
  } else if (at.mode == 2) {
#pragma unroll
    for (int e = 0; e < kNormPairs; ++e) {
      const int p = kNormPairs * l + e, i = pair_first(p, turned, halves), j = pair_second(p, turned, halves);
      if (i < dim) y[i] = static_cast<T>(a[e]);
      if (j < dim) y[j] = static_cast<T>(b[e]);
    }
  }
}

template <int LANES>
__device__ __forceinline__ float across(float v) {
#pragma unroll
  for (int d = 1; d < LANES; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// 1 / sqrt(v): 16-bit elements take the hardware's (1 ulp), FP32 ones two roundings.
template <typename T>
__device__ __forceinline__ float inverse_root(float v) {
  if constexpr (sizeof(T) == 4) return 1.0f / sqrtf(v);
  return __builtin_amdgcn_rsqf(v);
}

template <typename T>
__device__ __forceinline__ T *row_of(const fftmv_heads_t &f, int64_t b, int64_t t, int64_t head) {
  return static_cast<T *>(f.data) + b * f.batch + t * f.step + head * f.head;
}

template <typename T, int LANES, bool BACK>
__global__ __launch_bounds__(kBlock) void qk_norm_kernel(fftmv_qk_norm_t n, NormPlan plan, float *partials) {
  constexpr int GROUPS = kBlock / LANES;
  __shared__ float2 turns[kNormTurns];
  const int turned = static_cast<int>(n.frequencies), dim = static_cast<int>(n.dim);
  const bool halves = n.pairs == FFTMV_PAIRS_HALVES;
  const int l = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const Lane at = lane_of(l, turned, halves, dim);
  const int64_t rows = n.batch * n.steps;
  const int heads = static_cast<int>(n.query_heads + n.key_heads), queries = static_cast<int>(n.query_heads);
  const float over = n.norm == FFTMV_NORM_RMS ? 1.0f / dim : 1.0f;
  float wq[2][kNormPairs], wk[2][kNormPairs], gq[2][kNormPairs] = {}, gk[2][kNormPairs] = {};
#pragma unroll
  for (int e = 0; e < kNormPairs; ++e) {
    const int p = kNormPairs * l + e, i = pair_first(p, turned, halves), j = pair_second(p, turned, halves);
    wq[0][e] = n.q_weight && i < dim ? n.q_weight[i] : 1.0f;
    wq[1][e] = n.q_weight && j < dim ? n.q_weight[j] : 1.0f;
    wk[0][e] = n.k_weight && i < dim ? n.k_weight[i] : 1.0f;
    wk[1][e] = n.k_weight && j < dim ? n.k_weight[j] : 1.0f;
  }
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * plan.rows; first < rows;
       first += static_cast<int64_t>(gridDim.x) * plan.rows) {
    const int count = static_cast<int>(min(static_cast<int64_t>(plan.rows), rows - first));
    if (turned) {
      __syncthreads();
      for (int i = threadIdx.x; i < count * turned; i += kBlock) {
        const int64_t row = first + i / turned, b = row / n.steps, t = row - b * n.steps;
        const double position = n.positions ? n.positions[b * n.position_batch + t] : static_cast<double>(t);
        double turn = position * n.frequency[i % turned] * 0.15915494309189533577;  // 1 / (2 pi)
        turn -= rint(turn);
        float sn, cs;
        sincospif(2.0f * static_cast<float>(turn), &sn, &cs);
        turns[i] = make_float2(cs, sn);
      }
      __syncthreads();
    }
    for (int i = group; i < count * heads; i += GROUPS) {
      const int r = i / heads, h = i - r * heads;
      const int64_t row = first + r, b = row / n.steps, t = row - b * n.steps;
      const bool query = h < queries;
      const int64_t head = query ? h : h - queries;
      const bool held = !n.lengths || t < n.lengths[b];
      float a[kNormPairs] = {}, c[kNormPairs] = {};
      if (held) load_pairs(row_of<const T>(query ? n.q : n.k, b, t, head), at, l, turned, halves, dim, a, c);
      float dy[2][kNormPairs] = {};
      if constexpr (BACK) {
        if (held) load_pairs(row_of<const T>(query ? n.dqy : n.dky, b, t, head), at, l, turned, halves, dim, dy[0], dy[1]);
      }
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < kNormPairs; ++e) sum = fmaf(a[e], a[e], fmaf(c[e], c[e], sum));
      const float inverse = held ? inverse_root<T>(fmaf(across<LANES>(sum), over, n.eps)) : 0.0f;
      if constexpr (!BACK) {
#pragma unroll
        for (int e = 0; e < kNormPairs; ++e) {
          const int p = kNormPairs * l + e;
          const float u = a[e] * inverse * (query ? wq[0][e] : wk[0][e]), v = c[e] * inverse * (query ? wq[1][e] : wk[1][e]);
          const float2 w = p < turned ? turns[r * turned + p] : make_float2(1.0f, 0.0f);
          a[e] = held ? fmaf(u, w.x, -(v * w.y)) : 0.0f;
          c[e] = held ? fmaf(v, w.x, u * w.y) : 0.0f;
        }
        store_pairs(row_of<T>(query ? n.qy : n.ky, b, t, head), at, l, turned, halves, dim, a, c);
      } else {
        float inner = 0.0f;
#pragma unroll
        for (int e = 0; e < kNormPairs; ++e) {
          const int p = kNormPairs * l + e;
          const float2 w = p < turned ? turns[r * turned + p] : make_float2(1.0f, 0.0f);
          const float u = fmaf(dy[0][e], w.x, dy[1][e] * w.y), v = fmaf(dy[1][e], w.x, -(dy[0][e] * w.y));
          a[e] *= inverse;  // x / n
          c[e] *= inverse;
          (query ? gq[0][e] : gk[0][e]) += u * a[e];
          (query ? gq[1][e] : gk[1][e]) += v * c[e];
          dy[0][e] = u * (query ? wq[0][e] : wk[0][e]);
          dy[1][e] = v * (query ? wq[1][e] : wk[1][e]);
          inner = fmaf(dy[0][e], a[e], fmaf(dy[1][e], c[e], inner));
        }
        inner = across<LANES>(inner) * over;
#pragma unroll
        for (int e = 0; e < kNormPairs; ++e) {
          a[e] = held ? inverse * fmaf(-a[e], inner, dy[0][e]) : 0.0f;
          c[e] = held ? inverse * fmaf(-c[e], inner, dy[1][e]) : 0.0f;
        }
        store_pairs(row_of<T>(query ? n.dq : n.dk, b, t, head), at, l, turned, halves, dim, a, c);
      }
    }
  }
  if constexpr (BACK) {
    if (!partials) return;
    // the groups' sums, joined in a fixed order: one weight and half of the pairs after the other
    float *sums = reinterpret_cast<float *>(turns);
    static_assert(sizeof(turns) >= kBlock * kNormPairs * sizeof(float), "one sum of each thread");
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kNormPairs; ++e)
        sums[group * (LANES * kNormPairs) + l * kNormPairs + e] = v < 2 ? gq[v][e] : gk[v - 2][e];
      __syncthreads();
      for (int p = threadIdx.x; p < LANES * kNormPairs; p += kBlock) {
        const int i = v % 2 ? pair_second(p, turned, halves) : pair_first(p, turned, halves);
        if (i >= dim) continue;
        float s = 0.0f;
#pragma unroll 4
        for (int q = 0; q < GROUPS; ++q) s += sums[q * (LANES * kNormPairs) + p];
        partials[(static_cast<int64_t>(blockIdx.x) * 2 + v / 2) * dim + i] = s;
      }
    }
  }
}

// The workgroups' sums for one element of one weight each: a wave's lanes take
// every 64th, and add up across.
__global__ __launch_bounds__(kWave) void qk_norm_sums_kernel(const float *partials, int blocks, int dim, float *dq, float *dk) {
  const int i = blockIdx.x % dim, which = blockIdx.x / dim;
  float *to = which ? dk : dq;
  if (!to) return;
  float s = 0.0f;
  for (int b = threadIdx.x; b < blocks; b += kWave) s += partials[(static_cast<int64_t>(b) * 2 + which) * dim + i];
  s = across<kWave>(s);
  if (threadIdx.x == 0) to[i] = s;
}

template <typename F>
hipError_t by_lanes(int64_t dim, F f) {
  if (dim <= 64) return f(Const<8>{});
  if (dim <= 128) return f(Const<16>{});
  if (dim <= 256) return f(Const<32>{});
  return f(Const<64>{});
}

}  // namespace

hipError_t launch_qk_norm_forward(const fftmv_qk_norm_t &n, hipStream_t s) {
  const int64_t rows = n.batch * n.steps;
  if (rows == 0) return hipSuccess;
  const NormPlan plan = qk_norm_plan(rows, n.frequencies, false);
  return by_dtype(n.dtype, [&](auto t) {
    return by_lanes(n.dim, [&](auto lanes) {
      qk_norm_kernel<decltype(t), decltype(lanes)::value, false><<<plan.blocks, kBlock, 0, s>>>(n, plan, nullptr);
      return hipGetLastError();
    });
  });
}

hipError_t launch_qk_norm_backward(const fftmv_qk_norm_t &n, hipStream_t s) {
  const int64_t rows = n.batch * n.steps;
  const NormPlan plan = qk_norm_plan(rows, n.frequencies, true);
  float *partials = n.dq_weight || n.dk_weight ? static_cast<float *>(n.workspace) : nullptr;
  if (rows > 0) {
    const hipError_t e = by_dtype(n.dtype, [&](auto t) {
      return by_lanes(n.dim, [&](auto lanes) {
        qk_norm_kernel<decltype(t), decltype(lanes)::value, true><<<plan.blocks, kBlock, 0, s>>>(n, plan, partials);
        return hipGetLastError();
      });
    });
    if (e != hipSuccess) return e;
  }
  if (!n.dq_weight && !n.dk_weight) return hipSuccess;
  const int blocks = rows ? plan.blocks : 0, dim = static_cast<int>(n.dim);
  qk_norm_sums_kernel<<<2 * dim, kWave, 0, s>>>(partials, blocks, dim, n.dq_weight, n.dk_weight);
  return hipGetLastError();
}

}  // namespace fftmv
