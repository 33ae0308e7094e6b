// Forward kernel of the gated linear recurrence.
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
  uint32_t ticket, order;
};

// The chunk's join: from the segments' maps in lds.A, lds.H (written, not yet
// synchronised) to the state that enters each segment, in lds.H.
template <int W, int VEC>
__device__ __forceinline__ void forward_join(const fftmv_recurrence_t &r, const ScanAxis &axis, const Chunk &c,
                                             const ScanChain &s, int64_t block, uint32_t early,
                                             ForwardLds<W> &lds) {
  constexpr int G = ForwardLds<W>::G, SG = kSegs / G;
  constexpr uint32_t kGroup = ~0u >> (32 - SG);
  static_assert(G * SG == kSegs, "whole groups");
  const int tid = threadIdx.x, col = tid % W, grp = tid / W;
  __syncthreads();
  const uint32_t constants = read_segment_bits(lds.bits);

  // maps of groups of segments: one thread per column and group
  float mA[SG], mH[SG], cA = 1.0f, cH = 0.0f;
#pragma unroll
  for (int i = 0; i < SG; ++i) {
    mA[i] = lds.A[grp * SG + i][col];
    mH[i] = lds.H[grp * SG + i][col];
    cH = through(constants >> (grp * SG + i) & 1u, mA[i], mH[i], cH);
    cA *= mA[i];
  }
  lds.gA[grp][col] = cA;
  lds.gH[grp][col] = cH;
  __syncthreads();

  if (tid < W) {  // the state that enters the chunk
    const int64_t ch = column_channel<VEC>(r.channels, block * W + col);
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
      if (first) H = fmaf(A, in, H);
      const float from = meet_chain<W>(s, c.place, col, A, H, first || constants, !c.head, early);
      if (!first) in = from;
      if (r.carries) r.carries[(c.chain * axis.places + c.place) * r.channels + ch] = in;
    }
    lds.enter[col] = in;
  }
  __syncthreads();

  float h = lds.enter[col];
  for (int j = 0; j < grp; ++j) h = through(constants >> (j * SG) & kGroup, lds.gA[j][col], lds.gH[j][col], h);
#pragma unroll
  for (int i = 0; i < SG; ++i) {
    lds.H[grp * SG + i][col] = h;
    h = through(constants >> (grp * SG + i) & 1u, mA[i], mH[i], h);
  }
  __syncthreads();
}

template <typename T, int VEC, int DECAY, int DRIVE>
__global__ __launch_bounds__(kThreads, 4) void recurrence_forward_kernel(fftmv_recurrence_t r, ScanAxis axis) {
  constexpr int W = kLanes * VEC;  // columns of the workgroup
  __shared__ ForwardLds<W> lds;
  const int tid = threadIdx.x, seg = tid / kLanes, lane = tid % kLanes;
  const int64_t chains = axis.chains * axis.blocks, chain = blockIdx.x % chains;
  const int64_t block = chain % axis.blocks;
  const int64_t ch = column_channel<VEC>(r.channels, block * W + lane * VEC);
  const ScanChain s = scan_chain<W>(r.workspace, axis, chain);

  // Loads for the place that blockIdx suggests while the ticket is drawn;
  // once more in the rare case that it says another.
  Chunk c = chunk_at(r, axis, chain / axis.blocks, blockIdx.x / chains);
  uint32_t ticket = 0;
  if (axis.joined() && tid == 0) ticket = draw_place(s);
  Vec<T, VEC> x[kRows], g[kRows];
  auto load = [&]() {
    const Rows q = ordinary_rows(r, c, seg);
    load_rows<true>(r, q, r.gate, r.gate_batch, r.gate_step, ch, g);
    load_rows<true>(r, q, r.x, r.x_batch, r.x_step, ch, x);
  };
  if (c.ordinary) load();
  uint32_t early = 0;
  if (axis.joined()) {
    if (tid == 0) lds.ticket = ticket;
    __syncthreads();
    const int64_t place = __builtin_amdgcn_readfirstlane(lds.ticket);
    if (place >= axis.places) return;  // a workspace that was not zero
    if (place != c.place) {
      c = chunk_at(r, axis, c.chain, place);
      if (c.ordinary) load();
    }
    if (!c.head && tid < W) early = peek_state(s, (place - 1) * W + tid);
  }

  float A[VEC], H[VEC], h[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) A[e] = 1.0f, H[e] = 0.0f;
  uint32_t order = 0;
  auto to_lds = [&](uint32_t reset) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      lds.A[seg][lane * VEC + e] = A[e];
      lds.H[seg][lane * VEC + e] = H[e];
    }
    const uint64_t b = __ballot(reset != 0);
    if (tid % kWave == 0) lds.bits[tid / kWave] = segment_bits(b);
    forward_join<W, VEC>(r, axis, c, s, block, early, lds);
    if (axis.joined() && tid == 0) order = leave_chain(s);
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = lds.H[seg][lane * VEC + e];
  };
  // 16-bit inputs are held through the join as they are and their terms
  // computed twice; FP32 ones as the terms, which take no more room.
  constexpr bool kAgain = sizeof(T) == 2;
  auto again = [&]() {
    if constexpr (kAgain) {
      forget(g);
      forget(x);
    }
  };
  auto step = [&](int i, int e, float before) {
    const Terms t = decay_terms<T, DECAY>(g[i][e]);
    return fmaf(t.a, before, drive_of<DRIVE>(t, x[i][e]));
  };
  if (c.ordinary) {
    const Rows q = ordinary_rows(r, c, seg);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        H[e] = step(i, e, H[e]);
        A[e] *= decay_terms<T, DECAY>(g[i][e]).a;
      }
      row_done();
    }
    to_lds(0);
    again();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] = step(i, e, h[e]);
      store_row<true, T, VEC>(r, q, i, r.h, r.h_batch, r.h_step, ch, h);
      row_done();
    }
  } else {
    const Rows q = special_rows(r, axis, c, seg);
    load_rows<false>(r, q, r.gate, r.gate_batch, r.gate_step, ch, g);
    load_rows<false>(r, q, r.x, r.x_batch, r.x_step, ch, x);
    auto special_step = [&](int i, float (&v)[VEC]) {
      if (q.start >> i & 1u) load_state(r.h0, q.seq[i], r.channels, ch, v);
      const bool dead = q.dead >> i & 1u;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = dead ? 0.0f : step(i, e, v[e]);
    };
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      special_step(i, H);
#pragma unroll
      for (int e = 0; e < VEC; ++e) A[e] *= decay_terms<T, DECAY>(g[i][e]).a;
      row_done();
    }
    to_lds(q.start | q.dead);
    again();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      special_step(i, h);
      store_row<false, T, VEC>(r, q, i, r.h, r.h_batch, r.h_step, ch, h);
      if (q.last >> i & 1u) store_state(r.h_last, q.seq[i], r.channels, ch, h);
      if (q.empty >> i & 1u) {
        float h0[VEC];
        load_state(r.h0, q.seq[i], r.channels, ch, h0);
        store_state(r.h_last, q.seq[i], r.channels, ch, h0);
      }
      row_done();
    }
  }
  if ((r.offsets || r.steps == 0) && c.place == 0) pass_empty<VEC>(r, seg, ch, r.h0, r.h_last);
  if (axis.joined()) {
    if (tid == 0) lds.order = order;
    __syncthreads();
    if (lds.order == static_cast<uint32_t>(axis.places - 1)) clear_chain<W>(s, axis.places);
  }
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
