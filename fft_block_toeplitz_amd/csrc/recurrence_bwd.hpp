// Backward kernel of the gated linear recurrence.
//
// With s_t = a_t r_t, the gradient that a step hands to the one before it,
//   r_t = dh_t + s_{t+1},   s_t = a_t s_{t+1} + a_t dh_t
// is the same scan from the end. dgate needs h_{t-1} as well: it is recomputed
// in FP32 from the state that entered the chunk (the forward's carries), so
// that x, gate and dh are read once each, dx and dgate written once, and no
// rounded h is read at all.
#pragma once

#include "recurrence.hpp"

namespace fftmv {

template <int W>
struct BackwardLds {
  static constexpr int G = kThreads / W;
  // maps of the segments, forward A h + H and backward A s + S; then what
  // enters them, in H and S
  float A[kSegs][W], H[kSegs][W], S[kSegs][W];
  float gA[G][W], gH[G][W], gS[G][W];  // maps of the groups
  float enter[W];                      // what the chunk behind hands over
  __align__(8) uint8_t front_bits[kWaves], back_bits[kWaves];
  uint32_t ticket, order;
};

// The chunk's join: from the segments' maps (written, not yet synchronised)
// to the state that enters each segment from the front, in lds.H, and the
// gradient that enters it from behind, in lds.S.
template <int W, int VEC>
__device__ __forceinline__ void backward_join(const fftmv_recurrence_t &r, const ScanAxis &axis, const Chunk &c,
                                              const ScanChain &s, int64_t order, float carry, uint32_t early,
                                              BackwardLds<W> &lds) {
  constexpr int G = BackwardLds<W>::G, SG = kSegs / G;
  constexpr uint32_t kGroup = ~0u >> (32 - SG);
  const int tid = threadIdx.x, col = tid % W, grp = tid / W;
  __syncthreads();
  const uint32_t fronts = read_segment_bits(lds.front_bits), backs = read_segment_bits(lds.back_bits);

  // maps of groups of segments: one thread per column and group
  float mA[SG], mH[SG], mS[SG], cA = 1.0f, cH = 0.0f, cS = 0.0f;
#pragma unroll
  for (int i = 0; i < SG; ++i) {
    mA[i] = lds.A[grp * SG + i][col];
    mH[i] = lds.H[grp * SG + i][col];
    mS[i] = lds.S[grp * SG + i][col];
    cH = through(fronts >> (grp * SG + i) & 1u, mA[i], mH[i], cH);
    cA *= mA[i];
  }
#pragma unroll
  for (int i = SG - 1; i >= 0; --i) cS = through(backs >> (grp * SG + i) & 1u, mA[i], mS[i], cS);
  lds.gA[grp][col] = cA;
  lds.gH[grp][col] = cH;
  lds.gS[grp][col] = cS;
  __syncthreads();

  if (tid < W) {  // what the chunk behind hands over
    float in = 0.0f;
    if (axis.joined()) {
      float A = 1.0f, S = 0.0f;
#pragma unroll
      for (int j = G - 1; j >= 0; --j) {
        S = through(backs >> (j * SG) & kGroup, lds.gA[j][col], lds.gS[j][col], S);
        A *= lds.gA[j][col];
      }
      in = meet_chain<W>(s, order, col, A, S, backs, !c.tail, early);
    }
    lds.enter[col] = in;
  }
  // meanwhile, the state that enters each segment
  {
    float h = carry;
    for (int j = 0; j < grp; ++j) h = through(fronts >> (j * SG) & kGroup, lds.gA[j][col], lds.gH[j][col], h);
#pragma unroll
    for (int i = 0; i < SG; ++i) {
      lds.H[grp * SG + i][col] = h;
      h = through(fronts >> (grp * SG + i) & 1u, mA[i], mH[i], h);
    }
  }
  __syncthreads();
  float v = lds.enter[col];
  for (int j = G - 1; j > grp; --j) v = through(backs >> (j * SG) & kGroup, lds.gA[j][col], lds.gS[j][col], v);
#pragma unroll
  for (int i = SG - 1; i >= 0; --i) {
    lds.S[grp * SG + i][col] = v;
    v = through(backs >> (grp * SG + i) & 1u, mA[i], mS[i], v);
  }
  __syncthreads();
}

template <typename T, int VEC, int DECAY, int DRIVE>
__global__ __launch_bounds__(kThreads, 4) void recurrence_backward_kernel(fftmv_recurrence_t r, ScanAxis axis) {
  constexpr int W = kLanes * VEC;
  __shared__ BackwardLds<W> lds;
  const int tid = threadIdx.x, seg = tid / kLanes, lane = tid % kLanes;
  const int64_t chains = axis.chains * axis.blocks, chain = blockIdx.x % chains;
  const int64_t block = chain % axis.blocks;
  const int64_t ch = column_channel<VEC>(r.channels, block * W + lane * VEC);
  const ScanChain s = scan_chain<W>(r.workspace, axis, chain);

  // as in the forward kernel, but places count from the end of the time axis
  int64_t order = blockIdx.x / chains;
  Chunk c = chunk_at(r, axis, chain / axis.blocks, axis.places - 1 - order);
  uint32_t ticket = 0;
  if (axis.joined() && tid == 0) ticket = draw_place(s);
  Vec<T, VEC> x[kRows], g[kRows], d[kRows];
  auto load = [&]() {
    const Rows q = ordinary_rows(r, c, seg);
    load_rows<true>(r, q, r.gate, r.gate_batch, r.gate_step, ch, g);
    load_rows<true>(r, q, r.x, r.x_batch, r.x_step, ch, x);
    load_rows<true>(r, q, r.dh, r.dh_batch, r.dh_step, ch, d);
  };
  if (c.ordinary) load();
  uint32_t early = 0;
  float carry = 0.0f;
  if (axis.joined()) {
    if (tid == 0) lds.ticket = ticket;
    __syncthreads();
    const int64_t drawn = __builtin_amdgcn_readfirstlane(lds.ticket);
    if (drawn >= axis.places) return;  // a workspace that was not zero
    if (drawn != order) {
      order = drawn;
      c = chunk_at(r, axis, c.chain, axis.places - 1 - order);
      if (c.ordinary) load();
    }
    if (!c.tail && tid < W) early = peek_state(s, (order - 1) * W + tid);
    // the state that enters the chunk (unused where a sequence starts)
    const int64_t cc = column_channel<VEC>(r.channels, block * W + tid % W);
    if (!c.head)
      carry = r.carries[(c.chain * axis.places + c.place) * r.channels + cc];
    else if (c.ordinary && r.h0)
      carry = r.h0[c.seq * r.channels + cc];
  }

  float A[VEC], H[VEC], S[VEC], h[VEC], b[VEC], w[kRows][VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) A[e] = 1.0f, H[e] = 0.0f, S[e] = 0.0f;
  uint32_t left = 0;
  auto join = [&](uint32_t front, uint32_t back) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      lds.A[seg][lane * VEC + e] = A[e];
      lds.H[seg][lane * VEC + e] = H[e];
      lds.S[seg][lane * VEC + e] = S[e];
    }
    const uint64_t fb = __ballot(front != 0), bb = __ballot(back != 0);
    if (tid % kWave == 0) lds.front_bits[tid / kWave] = segment_bits(fb), lds.back_bits[tid / kWave] = segment_bits(bb);
    backward_join<W, VEC>(r, axis, c, s, order, carry, early, lds);
    if (axis.joined() && tid == 0) left = leave_chain(s);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      h[e] = lds.H[seg][lane * VEC + e];
      b[e] = lds.S[seg][lane * VEC + e];
    }
  };
  // one step forward: w = h_{t-1} (- x_t), the factor of dgate
  auto ahead = [&](int i) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const Terms t = decay_terms<T, DECAY>(g[i][e]);
      w[i][e] = DRIVE == FFTMV_DRIVE_COMPLEMENT ? h[e] - x[i][e] : h[e];
      h[e] = fmaf(t.a, h[e], drive_of<DRIVE>(t, x[i][e]));
    }
  };
  // one step back: b becomes s_t
  auto behind = [&](int i, bool dead, float (&du)[VEC], float (&dv)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const Terms t = decay_terms<T, DECAY>(g[i][e]);
      const float rt = d[i][e] + b[e];
      b[e] = dead ? 0.0f : t.a * rt;
      du[e] = dead ? 0.0f : DRIVE == FFTMV_DRIVE_COMPLEMENT ? rt * t.rest : rt;
      dv[e] = dead ? 0.0f : rt * w[i][e] * t.slope;
    }
  };

  if (c.ordinary) {
    const Rows q = ordinary_rows(r, c, seg);
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const Terms t = decay_terms<T, DECAY>(g[i][e]);
        H[e] = fmaf(t.a, H[e], drive_of<DRIVE>(t, x[i][e]));
        A[e] *= t.a;
        S[e] = fmaf(A[e], d[i][e], S[e]);  // a_0 .. a_i dh_i
      }
    join(0, 0);
    forget(g);
    forget(x);
    forget(d);
#pragma unroll
    for (int i = 0; i < kRows; ++i) ahead(i);
    forget(g);
#pragma unroll
    for (int i = kRows - 1; i >= 0; --i) {
      float du[VEC], dv[VEC];
      behind(i, false, du, dv);
      store_row<true, T, VEC>(r, q, i, r.dx, r.dx_batch, r.dx_step, ch, du);
      store_row<true, T, VEC>(r, q, i, r.dgate, r.dgate_batch, r.dgate_step, ch, dv);
    }
    if (c.head && seg == 0) store_state(r.dh0, c.seq, r.channels, ch, b);
  } else {
    const Rows q = special_rows(r, axis, c, seg);
    load_rows<false>(r, q, r.gate, r.gate_batch, r.gate_step, ch, g);
    load_rows<false>(r, q, r.x, r.x_batch, r.x_step, ch, x);
    load_rows<false>(r, q, r.dh, r.dh_batch, r.dh_step, ch, d);
    bool closed = false;  // a later row's gradient no longer reaches the segment's first
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const bool dead = q.dead >> i & 1u, start = q.start >> i & 1u, last = q.last >> i & 1u;
      closed |= dead;
      float h0[VEC] = {}, dl[VEC] = {};
      if (start) load_state(r.h0, q.seq[i], r.channels, ch, h0);
      if (last) load_state(r.dh_last, q.seq[i], r.channels, ch, dl);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const Terms t = decay_terms<T, DECAY>(g[i][e]);
        const float before = start ? h0[e] : H[e];
        H[e] = dead ? 0.0f : fmaf(t.a, before, drive_of<DRIVE>(t, x[i][e]));
        A[e] *= t.a;
        if (!closed) S[e] = fmaf(A[e], d[i][e] + dl[e], S[e]);
      }
      closed |= last;
    }
    join(q.start | q.dead, q.last | q.dead);
    forget(g);
    forget(x);
    forget(d);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (q.start >> i & 1u) load_state(r.h0, q.seq[i], r.channels, ch, h);
      ahead(i);
    }
    forget(g);
#pragma unroll
    for (int i = kRows - 1; i >= 0; --i) {
      if (q.last >> i & 1u) load_state(r.dh_last, q.seq[i], r.channels, ch, b);
      float du[VEC], dv[VEC];
      behind(i, q.dead >> i & 1u, du, dv);
      store_row<false, T, VEC>(r, q, i, r.dx, r.dx_batch, r.dx_step, ch, du);
      store_row<false, T, VEC>(r, q, i, r.dgate, r.dgate_batch, r.dgate_step, ch, dv);
      if (q.start >> i & 1u) store_state(r.dh0, q.seq[i], r.channels, ch, b);
      if (q.empty >> i & 1u) {
        float dl[VEC];
        load_state(r.dh_last, q.seq[i], r.channels, ch, dl);
        store_state(r.dh0, q.seq[i], r.channels, ch, dl);
      }
    }
  }
  if ((r.offsets || r.steps == 0) && c.place == 0) pass_empty<VEC>(r, seg, ch, r.dh_last, r.dh0);
  if (axis.joined()) {
    if (tid == 0) lds.order = left;
    __syncthreads();
    if (lds.order == static_cast<uint32_t>(axis.places - 1)) clear_chain<W>(s, axis.places);
  }
}

template <typename T, int VEC>
hipError_t launch_recurrence_backward_vec(const fftmv_recurrence_t &r, hipStream_t s) {
  const ScanAxis axis = scan_axis(r.batch, r.steps, r.offsets != nullptr, r.channels, kLanes * VEC);
  if (!grid_fits(axis.workgroups(), kThreads)) return hipErrorInvalidConfiguration;
  return by_recurrence_kind(r.decay, r.drive, [&](auto d, auto u) {
    recurrence_backward_kernel<T, VEC, decltype(d)::value, decltype(u)::value>
        <<<static_cast<unsigned>(axis.workgroups()), kThreads, 0, s>>>(r, axis);
    return hipGetLastError();
  });
}

// As the forward: rows shorter than one vector take one channel a lane.
template <typename T>
hipError_t launch_recurrence_backward_as(const fftmv_recurrence_t &r, hipStream_t s) {
  return r.channels >= kVec<T> ? launch_recurrence_backward_vec<T, kVec<T>>(r, s)
                               : launch_recurrence_backward_vec<T, 1>(r, s);
}

}  // namespace fftmv
