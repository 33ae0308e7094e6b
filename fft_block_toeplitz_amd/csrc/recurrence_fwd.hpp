// Forward kernel of the gated linear recurrence.
//
// x and gate are read once, h written once, and memory traffic bounds it as far
// as the chunks' joins let it: 4 x 4096 x 4096 bf16 take 116 us (3.5 TB/s of
// three fields; 86 with the joins left out, which gives wrong values), 8 x 2000
// x 5000 143 us, 8 x 1000 x 5000 FP32 122 us (3.9 TB/s). A series of one
// chunk joins nothing.
#pragma once

#include "recurrence.hpp"

namespace fftmv {

template <int W>
struct ForwardLds {
  static constexpr int G = kThreads / W;  // groups of segments in the join
  float A[kSegs][W], H[kSegs][W];         // maps of the segments; then, in H, the states that enter them
  float gA[G][W], gH[G][W];               // maps of the groups
  float enter[W];                         // the state that enters the chunk
  __align__(8) uint8_t bits[kWaves];
  uint32_t ticket;
  uint32_t over;  // a group's product of decays is out of range
};

// The chunk's join: from the segments' maps in lds.A, lds.H (written, not yet
// synchronised) to the state that enters each segment, in lds.H.
template <int W, int VEC>
__device__ __forceinline__ void forward_join(const fftmv_recurrence_t &r, const ScanAxis &axis, const Chunk &c,
                                             const ScanChain &s, int block, uint64_t early,
                                             ForwardLds<W> &lds) {
  constexpr int G = ForwardLds<W>::G, SG = kSegs / G;
  constexpr uint32_t kGroup = ~0u >> (32 - SG);
  static_assert(G * SG == kSegs, "whole groups");
  const int tid = threadIdx.x, col = tid % W, grp = tid / W;
  if (tid == 0) lds.over = 0;
  __syncthreads();
  const uint32_t constants = read_segment_bits(lds.bits);

  // maps of groups of segments: one thread per column and group
  float cA = 1.0f, cH = 0.0f;
#pragma unroll
  for (int i = 0; i < SG; ++i) {
    const float A = lds.A[grp * SG + i][col];
    cH = through(constants >> (grp * SG + i) & 1u, A, lds.H[grp * SG + i][col], cH);
    cA *= A;
  }
  lds.gA[grp][col] = cA;
  lds.gH[grp][col] = cH;
  if (!in_range(cA)) lds.over = 1;
  __syncthreads();
  auto walk = [&](float h, int groups) {
#pragma unroll 1
    for (int j = 0; j < groups; ++j) h = through_group<false, SG, W>(lds.A, lds.H, lds.gA, lds.gH, constants, j, col, h);
    return h;
  };

  if (tid < W) {  // the state that enters the chunk
    const int64_t ch = column_channel<VEC>(r.channels, static_cast<int64_t>(block) * W + col);
    float in = 0.0f;
    // an ordinary chunk at the front of its sequence; a special one has it in a segment's map
    const bool first = c.ordinary && c.head;
    if (first && r.h0) in = r.h0[c.seq * r.channels + ch];
    if (axis.joined()) {
      float A = 1.0f, H = 0.0f;
#pragma unroll
      for (int j = 0; j < G; ++j) {
        H = through(constants >> (j * SG) & kGroup, lds.gA[j][col], lds.gH[j][col], H);
        A *= lds.gA[j][col];
      }
      const bool mapped = in_range(A), all = __ballot(!mapped) == 0;
      if (!all && !mapped) H = walk(0.0f, G);  // (a group's product out of range makes A infinite or NaN)
      auto behind = [&](float h) {
        float v = fmaf(A, h, H);
        if (!all && !mapped) v = walk(h, G);
        return v;
      };
      if (first) H = behind(in);
      const float from = meet_chain<W>(s, c.place, col, A, H, first || constants, mapped, !c.head, early, behind);
      if (!first) in = from;
      if (r.carries) r.carries[(static_cast<int64_t>(c.chain) * axis.places + c.place) * r.channels + ch] = in;
    }
    lds.enter[col] = in;
  }
  __syncthreads();

  float h = lds.enter[col];
  if (__builtin_amdgcn_readfirstlane(lds.over)) {
    h = walk(h, grp);
    __syncthreads();  // the segments' maps are overwritten below
  } else {
    for (int j = 0; j < grp; ++j) h = through(constants >> (j * SG) & kGroup, lds.gA[j][col], lds.gH[j][col], h);
  }
#pragma unroll
  for (int i = 0; i < SG; ++i) {
    float &H = lds.H[grp * SG + i][col];
    const float next = through(constants >> (grp * SG + i) & 1u, lds.A[grp * SG + i][col], H, h);
    H = h;
    h = next;
  }
  __syncthreads();
}

template <typename T, int VEC, int DECAY, int DRIVE>
__global__ __launch_bounds__(kThreads, 4) void recurrence_forward_kernel(fftmv_recurrence_t r, ScanAxis axis) {
  constexpr int W = kLanes * VEC;  // columns of the workgroup
  __shared__ ForwardLds<W> lds;
  const int tid = threadIdx.x, seg = tid / kLanes, lane = tid % kLanes;
  // chains of all blocks of channels: block by block of one sequence, then the
  // next. Neighbours share the lines at their edges, and so an XCD.
  const uint32_t chains = static_cast<uint32_t>(axis.chains) * axis.blocks;
  const uint32_t chain = static_cast<uint32_t>(xcd_contiguous_block(blockIdx.x % chains, chains));
  const int block = chain % static_cast<uint32_t>(axis.blocks), over_batch = chain / static_cast<uint32_t>(axis.blocks);
  const int64_t ch = column_channel<VEC>(r.channels, static_cast<int64_t>(block) * W + lane * VEC);
  const ScanChain s = scan_chain<W>(r, axis, chain);

  // Loads for the place that blockIdx suggests while the ticket is drawn; a
  // second time in the rare case that it says another.
  int place = blockIdx.x / chains;
  uint32_t ticket = 0;
  bool drawn = !axis.joined();
  if (!drawn && tid == 0) ticket = draw_place(s);
  Chunk c;
  Rows q;
  Vec<T, VEC> x[kRows], g[kRows];
  for (;;) {
    c = chunk_at(r, axis, over_batch, place);
    q = rows_of(r, axis, c, seg);
    load_rows(r, axis, c, q, r.gate, r.gate_batch, r.gate_step, ch, g);
    load_rows(r, axis, c, q, r.x, r.x_batch, r.x_step, ch, x);
    if (drawn) break;
    drawn = true;
    if (tid == 0) lds.ticket = settle_ticket(s, ticket, axis.places);
    __syncthreads();
    const uint32_t t = __builtin_amdgcn_readfirstlane(lds.ticket);
    if (t >= static_cast<uint32_t>(axis.places)) return;  // a workspace or number that the call may not have
    if (t == static_cast<uint32_t>(place)) break;
    place = static_cast<int>(t);
  }
  uint64_t early = 0;
  if (axis.joined() && !c.head && tid < W) early = peek<W>(s, place - 1, 2, tid);

  // one row: v becomes its state
  auto step = [&](int i, float (&v)[VEC]) {
    if (!c.ordinary && q.start(i)) load_state(r.h0, q.seq[i], r.channels, ch, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const Terms t = decay_terms<T, DECAY>(g[i][e]);
      v[e] = fmaf(t.a, v[e], drive_of<DRIVE>(t, x[i][e]));
    }
    if (!c.ordinary && q.dead(i)) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = 0.0f;
    }
  };

  float A[VEC], h[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) A[e] = 1.0f, h[e] = 0.0f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    step(i, h);
#pragma unroll
    for (int e = 0; e < VEC; ++e) A[e] *= decay_terms<T, DECAY>(g[i][e]).a;
    row_done();
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    lds.A[seg][lane * VEC + e] = A[e];
    lds.H[seg][lane * VEC + e] = h[e];
  }
  const uint64_t front = __ballot(q.closed_front());
  if (tid % kWave == 0) lds.bits[tid / kWave] = segment_bits(front);
  forward_join<W, VEC>(r, axis, c, s, block, early, lds);
#pragma unroll
  for (int e = 0; e < VEC; ++e) h[e] = lds.H[seg][lane * VEC + e];

  // The rows once more, now from the state that enters them: the inputs are
  // held through the join as they came, and their terms computed again.
  forget(g);
  forget(x);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    step(i, h);
    store_row<T, VEC>(r, axis, c, q, i, r.h, r.h_batch, r.h_step, ch, h);
    if (!c.ordinary) {
      if (q.last(i)) store_state(r.h_last, q.seq[i], r.channels, ch, h);
      if (q.empty(i)) {
        float h0[VEC];
        load_state(r.h0, q.seq[i], r.channels, ch, h0);
        store_state(r.h_last, q.seq[i], r.channels, ch, h0);
      }
    }
    row_done();
  }
  if ((r.offsets || r.steps == 0) && c.place == 0) pass_empty<VEC>(r, seg, ch, r.h0, r.h_last);
}

template <typename T, int VEC>
hipError_t launch_recurrence_forward_vec(const fftmv_recurrence_t &r, hipStream_t s) {
  const ScanAxis axis = scan_axis(r.batch, r.steps, r.offsets != nullptr, r.channels, kLanes * VEC);
  if (!grid_fits(axis.workgroups(), kThreads)) return hipErrorInvalidConfiguration;
  return by_recurrence_kind(r.decay, r.drive, [&](auto d, auto u) {
    recurrence_forward_kernel<T, VEC, decltype(d)::value, decltype(u)::value>
        <<<static_cast<unsigned>(axis.workgroups()), kThreads, 0, s>>>(r, axis);
    return hipGetLastError();
  });
}

// Rows shorter than one 16-byte vector (C < VEC) take one channel a lane.
template <typename T>
hipError_t launch_recurrence_forward_as(const fftmv_recurrence_t &r, hipStream_t s) {
  return r.channels >= kVec<T> ? launch_recurrence_forward_vec<T, kVec<T>>(r, s)
                               : launch_recurrence_forward_vec<T, 1>(r, s);
}

}  // namespace fftmv
