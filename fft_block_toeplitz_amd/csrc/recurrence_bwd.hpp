// Backward kernel of the gated linear recurrence.
//
// With s_t = a_t r_t, the gradient that a step hands to the one before it,
//   r_t = dh_t + s_{t+1},   s_t = a_t s_{t+1} + a_t dh_t
// is the same scan from the end. dgate needs h_{t-1} as well: it is recomputed
// in FP32 from the state that entered the chunk (the forward's carries), so
// that x, gate and dh are read once each, dx and dgate written once, and no
// rounded h is read at all.
//
// Memory traffic bounds it, and at this many workgroups the chunks' joins: 4 x
// 4096 x 4096 bf16 take 212 us (3.2 TB/s of five fields; 145 with the joins left
// out, which gives wrong values), 8 x 2000 x 5000 261 us, 8 x 1000 x 5000 FP32
// 183 us (4.4 TB/s).
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
  uint32_t ticket;
  uint32_t over;  // a group's product of decays is out of range
};

// The chunk's join: from the segments' maps (written, not yet synchronised)
// to the state that enters each segment from the front, in lds.H, and the
// gradient that enters it from behind, in lds.S.
template <int W, int VEC>
__device__ __forceinline__ void backward_join(const fftmv_recurrence_t &r, const ScanAxis &axis, const Chunk &c,
                                              const ScanChain &s, int order, float carry, uint64_t early,
                                              BackwardLds<W> &lds) {
  constexpr int G = BackwardLds<W>::G, SG = kSegs / G;
  constexpr uint32_t kGroup = ~0u >> (32 - SG);
  const int tid = threadIdx.x, col = tid % W, grp = tid / W;
  if (tid == 0) lds.over = 0;
  __syncthreads();
  const uint32_t fronts = read_segment_bits(lds.front_bits), backs = read_segment_bits(lds.back_bits);

  // maps of groups of segments: one thread per column and group
  float cA = 1.0f, cH = 0.0f, cS = 0.0f;
#pragma unroll
  for (int i = 0; i < SG; ++i) {
    const float A = lds.A[grp * SG + i][col];
    cH = through(fronts >> (grp * SG + i) & 1u, A, lds.H[grp * SG + i][col], cH);
    cA *= A;
  }
#pragma unroll
  for (int i = SG - 1; i >= 0; --i)
    cS = through(backs >> (grp * SG + i) & 1u, lds.A[grp * SG + i][col], lds.S[grp * SG + i][col], cS);
  lds.gA[grp][col] = cA;
  lds.gH[grp][col] = cH;
  lds.gS[grp][col] = cS;
  if (!in_range(cA)) lds.over = 1;
  __syncthreads();
  auto walk_back = [&](float v, int from) {  // through the groups behind `from`, the last one first
#pragma unroll 1
    for (int j = G - 1; j > from; --j) v = through_group<true, SG, W>(lds.A, lds.S, lds.gA, lds.gS, backs, j, col, v);
    return v;
  };

  if (tid < W) {  // what the chunk behind hands over
    float in = 0.0f;
    if (axis.joined()) {
      float A = 1.0f, S = 0.0f;
#pragma unroll
      for (int j = G - 1; j >= 0; --j) {
        S = through(backs >> (j * SG) & kGroup, lds.gA[j][col], lds.gS[j][col], S);
        A *= lds.gA[j][col];
      }
      const bool mapped = in_range(A), all = __ballot(!mapped) == 0;
      if (!all && !mapped) S = walk_back(0.0f, -1);  // (a group's product out of range makes A infinite or NaN)
      in = meet_chain<W>(s, order, col, A, S, backs, mapped, !c.tail, early, [&](float v) {
        float u = fmaf(A, v, S);
        if (!all && !mapped) u = walk_back(v, -1);
        return u;
      });
    }
    lds.enter[col] = in;
  }
  // meanwhile, the state that enters each segment
  const bool over = __builtin_amdgcn_readfirstlane(lds.over);
  {
    float h = carry;
    if (over) {
#pragma unroll 1
      for (int j = 0; j < grp; ++j) h = through_group<false, SG, W>(lds.A, lds.H, lds.gA, lds.gH, fronts, j, col, h);
      __syncthreads();  // the segments' maps are overwritten below
    } else {
      for (int j = 0; j < grp; ++j) h = through(fronts >> (j * SG) & kGroup, lds.gA[j][col], lds.gH[j][col], h);
    }
#pragma unroll
    for (int i = 0; i < SG; ++i) {
      float &H = lds.H[grp * SG + i][col];
      const float next = through(fronts >> (grp * SG + i) & 1u, lds.A[grp * SG + i][col], H, h);
      H = h;
      h = next;
    }
  }
  __syncthreads();
  float v = lds.enter[col];
  if (over) {
    v = walk_back(v, grp);
    __syncthreads();
  } else {
    for (int j = G - 1; j > grp; --j) v = through(backs >> (j * SG) & kGroup, lds.gA[j][col], lds.gS[j][col], v);
  }
#pragma unroll
  for (int i = SG - 1; i >= 0; --i) {
    float &S = lds.S[grp * SG + i][col];
    const float next = through(backs >> (grp * SG + i) & 1u, lds.A[grp * SG + i][col], S, v);
    S = v;
    v = next;
  }
  __syncthreads();
}

template <typename T, int VEC, int DECAY, int DRIVE>
__global__ __launch_bounds__(kThreads, 4) void recurrence_backward_kernel(fftmv_recurrence_t r, ScanAxis axis,
                                                                          bool streamed) {
  constexpr int W = kLanes * VEC;
  __shared__ BackwardLds<W> lds;
  const int tid = threadIdx.x, seg = tid / kLanes, lane = tid % kLanes;
  // chains of all blocks of channels: block by block of one sequence, then the
  // next. Neighbours share the lines at their edges, and so an XCD.
  const uint32_t chains = static_cast<uint32_t>(axis.chains) * axis.blocks;
  const uint32_t chain = static_cast<uint32_t>(xcd_contiguous_block(blockIdx.x % chains, chains));
  const int block = chain % static_cast<uint32_t>(axis.blocks), over_batch = chain / static_cast<uint32_t>(axis.blocks);
  const int64_t ch = column_channel<VEC>(r.channels, static_cast<int64_t>(block) * W + lane * VEC);
  const ScanChain s = scan_chain<W>(r, axis, chain);

  // as in the forward kernel, but places count from the end of the time axis
  int order = blockIdx.x / chains;
  uint32_t ticket = 0;
  bool drawn = !axis.joined();
  if (!drawn && tid == 0) ticket = draw_place(s);
  Chunk c;
  Rows q;
  Vec<T, VEC> x[kRows], g[kRows], d[kRows];
  for (;;) {
    c = chunk_at(r, axis, over_batch, axis.places - 1 - order);
    q = rows_of(r, axis, c, seg);
    load_rows(r, axis, c, q, r.gate, r.gate_batch, r.gate_step, ch, g);
    load_rows(r, axis, c, q, r.x, r.x_batch, r.x_step, ch, x);
    load_rows(r, axis, c, q, r.dh, r.dh_batch, r.dh_step, ch, d);
    if (drawn) break;
    drawn = true;
    if (tid == 0) lds.ticket = settle_ticket(s, ticket, axis.places);
    __syncthreads();
    const uint32_t t = __builtin_amdgcn_readfirstlane(lds.ticket);
    if (t >= static_cast<uint32_t>(axis.places)) return;  // a workspace or number that the call may not have
    if (t == static_cast<uint32_t>(order)) break;
    order = static_cast<int>(t);
  }
  // The maps' terms are held through the join; what the gradients need besides
  // is evaluated again behind it. (Holding that too would pass 128 registers;
  // evaluating everything in each of the three passes took 202 instead of 194
  // us at 8 x 1000 x 5000 FP32. FP32 inputs beside both a and u would, too:
  // there the complement's terms are evaluated in all three.)
  constexpr bool kHold = sizeof(T) == 2 || DRIVE == FFTMV_DRIVE_PLAIN;
  float A[VEC], h[VEC], b[VEC], a[kRows][VEC], u[kRows][VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) A[e] = 1.0f, h[e] = 0.0f, b[e] = 0.0f;
  bool open = true;  // a later row's gradient reaches the segment's first
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float dl[VEC] = {};
    if (!c.ordinary) {
      open = open && !q.dead(i);
      if (q.start(i)) load_state(r.h0, q.seq[i], r.channels, ch, h);
      if (q.last(i)) load_state(r.dh_last, q.seq[i], r.channels, ch, dl);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const Terms t = decay_terms<T, DECAY>(g[i][e]);
      a[i][e] = t.a;
      u[i][e] = drive_of<DRIVE>(t, x[i][e]);
      h[e] = fmaf(t.a, h[e], u[i][e]);
      A[e] *= t.a;
      b[e] = open ? fmaf(A[e], d[i][e] + dl[e], b[e]) : b[e];  // a_0 .. a_i dh_i
    }
    if (!c.ordinary) {
      open = open && !q.last(i);
      if (q.dead(i)) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = 0.0f;
      }
    }
    row_done();
  }
  uint64_t early = 0;
  float carry = 0.0f;
  if (axis.joined()) {
    if (!c.tail && tid < W) early = peek<W>(s, order - 1, 2, tid);
    // the state that enters the chunk (unused where a sequence starts)
    const int64_t cc = column_channel<VEC>(r.channels, static_cast<int64_t>(block) * W + tid % W);
    if (!c.head)
      carry = r.carries[(static_cast<int64_t>(c.chain) * axis.places + c.place) * r.channels + cc];
    else if (c.ordinary && r.h0)
      carry = r.h0[c.seq * r.channels + cc];
  }

#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    lds.A[seg][lane * VEC + e] = A[e];
    lds.H[seg][lane * VEC + e] = h[e];
    lds.S[seg][lane * VEC + e] = b[e];
  }
  const uint64_t front = __ballot(q.closed_front()), back = __ballot(q.closed_back());
  if (tid % kWave == 0) {
    lds.front_bits[tid / kWave] = segment_bits(front);
    lds.back_bits[tid / kWave] = segment_bits(back);
  }
  backward_join<W, VEC>(r, axis, c, s, order, carry, early, lds);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    h[e] = lds.H[seg][lane * VEC + e];
    b[e] = lds.S[seg][lane * VEC + e];
  }

  // forward to w = h_{t-1} (- x_t), the factor of dgate
  if constexpr (!kHold) forget(g);
  float w[kRows][VEC];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (!c.ordinary && q.start(i)) load_state(r.h0, q.seq[i], r.channels, ch, h);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[i][e] = DRIVE == FFTMV_DRIVE_COMPLEMENT ? h[e] - x[i][e] : h[e];
      if constexpr (kHold) {
        h[e] = fmaf(a[i][e], h[e], u[i][e]);
      } else {
        const Terms t = decay_terms<T, DECAY>(g[i][e]);
        h[e] = fmaf(t.a, h[e], drive_of<DRIVE>(t, x[i][e]));
      }
    }
  }
  // and back: b becomes s_t
  forget(g);
#pragma unroll
  for (int i = kRows - 1; i >= 0; --i) {
    if (!c.ordinary && q.last(i)) load_state(r.dh_last, q.seq[i], r.channels, ch, b);
    float du[VEC], dv[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const Terms t = decay_terms<T, DECAY>(g[i][e]);
      const float rt = d[i][e] + b[e];
      b[e] = t.a * rt;
      du[e] = DRIVE == FFTMV_DRIVE_COMPLEMENT ? rt * t.rest : rt;
      dv[e] = rt * w[i][e] * t.slope;
    }
    if (!c.ordinary && q.dead(i)) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) b[e] = du[e] = dv[e] = 0.0f;
    }
    store_row<T, VEC>(r, axis, c, q, i, r.dx, r.dx_batch, r.dx_step, ch, du, streamed);
    store_row<T, VEC>(r, axis, c, q, i, r.dgate, r.dgate_batch, r.dgate_step, ch, dv, streamed);
    if (!c.ordinary) {
      if (q.start(i)) store_state(r.dh0, q.seq[i], r.channels, ch, b);
      if (q.empty(i)) {
        float dl[VEC];
        load_state(r.dh_last, q.seq[i], r.channels, ch, dl);
        store_state(r.dh0, q.seq[i], r.channels, ch, dl);
      }
    }
    row_done();
  }
  // an ordinary chunk at the front of its sequence
  if (c.ordinary && c.head && seg == 0) store_state(r.dh0, c.seq, r.channels, ch, b);
  if ((r.offsets || r.steps == 0) && c.place == 0) pass_empty<VEC>(r, seg, ch, r.dh_last, r.dh0);
}

// All rows of a field start on a line of memory.
template <typename T>
bool on_lines(const fftmv_recurrence_t &r, const void *p, int64_t batch, int64_t step) {
  const int64_t strides = (r.offsets ? 0 : batch) | step;
  return (reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(strides * static_cast<int64_t>(sizeof(T)))) % 128 == 0;
}

template <typename T, int VEC>
hipError_t launch_recurrence_backward_vec(const fftmv_recurrence_t &r, hipStream_t s) {
  // Where rows start inside a line, two blocks of channels write parts of one:
  // through the caches these leave as one write (8 x 2000 x 5000 bf16 260 us,
  // streamed 280; 4 x 4096 x 4096, on lines, 211 and 206).
  const bool streamed = on_lines<T>(r, r.dx, r.dx_batch, r.dx_step) &&
                        on_lines<T>(r, r.dgate, r.dgate_batch, r.dgate_step);
  const ScanAxis axis = scan_axis(r.batch, r.steps, r.offsets != nullptr, r.channels, kLanes * VEC);
  if (!grid_fits(axis.workgroups(), kThreads)) return hipErrorInvalidConfiguration;
  return by_recurrence_kind(r.decay, r.drive, [&](auto d, auto u) {
    recurrence_backward_kernel<T, VEC, decltype(d)::value, decltype(u)::value>
        <<<static_cast<unsigned>(axis.workgroups()), kThreads, 0, s>>>(r, axis, streamed);
    return hipGetLastError();
  });
}

// Four channels a lane in every type: three inputs of eight 16-bit ones would
// not fit the registers of two workgroups a CU. Rows shorter than that take
// one channel a lane.
template <typename T>
hipError_t launch_recurrence_backward_as(const fftmv_recurrence_t &r, hipStream_t s) {
  return r.channels >= 4 ? launch_recurrence_backward_vec<T, 4>(r, s) : launch_recurrence_backward_vec<T, 1>(r, s);
}

}  // namespace fftmv
