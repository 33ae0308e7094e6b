// Forward kernel of the gated linear recurrence.
#pragma once

#include "recurrence.hpp"

namespace fftmv {

template <typename T, int VEC, int DECAY, int DRIVE>
__global__ __launch_bounds__(kThreads, 2) void recurrence_forward_kernel(fftmv_recurrence_t r, int64_t rows,
                                                                    int64_t chunks, int64_t blocks, bool joined) {
  constexpr int W = kLanes * VEC;        // channels of the workgroup
  constexpr int G = kThreads / W;          // groups of segments in the join
  constexpr int SG = kSegs / G;          // segments of a group
  static_assert(G * SG == kSegs, "whole groups");
  __shared__ float sA[kSegs][W], sH[kSegs][W], gA[G][W], gH[G][W], enter[W];
  __shared__ __align__(8) uint8_t bits[kThreads / kWave];

  const Place place = take_place(joined ? r.workspace : nullptr, blocks);
  const int64_t k = place.chunk;
  if (k >= chunks) return;  // a workspace that was not zero
  const int tid = threadIdx.x, seg = tid / kLanes, lane = tid % kLanes;
  const int64_t ch = column_channel<VEC>(r.channels, place.block * W + lane * VEC);

  const Rows q = rows_at(r, rows, k * kChunk + seg * kRows);
  const bool special = __ballot(q.special()) != 0;
  Vec<T, VEC> x[kRows], g[kRows];
  load_rows<T, VEC>(r, q, special, r.gate, r.gate_batch, r.gate_step, ch, g);
  load_rows<T, VEC>(r, q, special, r.x, r.x_batch, r.x_step, ch, x);

  // the map of the segment
  const uint32_t reset = q.start | q.dead;
  float a[kRows][VEC], u[kRows][VEC], A[VEC], H[VEC];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const Terms t = decay_terms<T, DECAY>(g[i][e]);
      a[i][e] = t.a;
      u[i][e] = drive_of<DRIVE>(t, x[i][e]);
    }
#pragma unroll
  for (int e = 0; e < VEC; ++e) A[e] = 1.0f, H[e] = 0.0f;
  if (!special) {
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        H[e] = fmaf(a[i][e], H[e], u[i][e]);
        A[e] *= a[i][e];
      }
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const bool dead = q.dead >> i & 1u, constant = reset >> i & 1u;
      const float *h0 = nullptr;
      if ((q.start >> i & 1u) && r.h0) h0 = r.h0 + sequence_of(r, q.row0 + i) * r.channels + ch;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (h0) u[i][e] = fmaf(a[i][e], h0[e], u[i][e]);
        if (dead) u[i][e] = 0.0f;
        H[e] = constant ? u[i][e] : fmaf(a[i][e], H[e], u[i][e]);
        A[e] *= a[i][e];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    sA[seg][lane * VEC + e] = A[e];
    sH[seg][lane * VEC + e] = H[e];
  }
  {
    const uint64_t b = __ballot(reset != 0);
    if (tid % kWave == 0) bits[tid / kWave] = segment_bits(b);
  }
  __syncthreads();
  const SegmentBits constants = read_segment_bits(bits);

  // the maps of groups of segments: one thread per channel and group
  const int col = tid % W, grp = tid / W;
  float mA[SG], mH[SG];
  {
    float cA = 1.0f, cH = 0.0f;
#pragma unroll
    for (int i = 0; i < SG; ++i) {
      mA[i] = sA[grp * SG + i][col];
      mH[i] = sH[grp * SG + i][col];
      cH = constants >> (grp * SG + i) & 1u ? mH[i] : fmaf(mA[i], cH, mH[i]);
      cA *= mA[i];
    }
    gA[grp][col] = cA;
    gH[grp][col] = cH;
  }
  __syncthreads();
  constexpr SegmentBits kGroup = ~SegmentBits(0) >> (8 * sizeof(SegmentBits) - SG);

  // the state that enters the chunk
  if (tid < W) {
    float in = 0.0f;
    if (joined) {
      const ScanBlock s = scan_block<W>(r.workspace, blocks, chunks, place.block);
      const Rows head = rows_at(r, rows, k * kChunk);
      float cA = 1.0f, cH = 0.0f;
#pragma unroll
      for (int j = 0; j < G; ++j) {
        cH = constants >> (j * SG) & kGroup ? gH[j][col] : fmaf(gA[j][col], cH, gH[j][col]);
        cA *= gA[j][col];
      }
      if (constants)
        publish_state(s, k * W + col, cH);
      else
        publish_map(s, k * W + col, cA, cH);
      if (!((head.start | head.dead) & 1u)) in = state_before<W>(s, k, col);
      if (!constants) publish_state(s, k * W + col, fmaf(cA, in, nonzero(cH)));
    }
    if (r.carries) r.carries[k * r.channels + column_channel<VEC>(r.channels, place.block * W + col)] = in;
    enter[col] = in;
  }
  __syncthreads();

  // the state that enters each segment, in the place of its map
  {
    float h = enter[col];
    for (int j = 0; j < grp; ++j)
      h = constants >> (j * SG) & kGroup ? gH[j][col] : fmaf(gA[j][col], h, gH[j][col]);
#pragma unroll
    for (int i = 0; i < SG; ++i) {
      sH[grp * SG + i][col] = h;
      h = constants >> (grp * SG + i) & 1u ? mH[i] : fmaf(mA[i], h, mH[i]);
    }
  }
  __syncthreads();
  float h[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) h[e] = sH[seg][lane * VEC + e];

  T *out = static_cast<T *>(r.h) + ch;
  if (!special) {
    out += row_offset(r, q.row0, r.h_batch, r.h_step);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] = fmaf(a[i][e], h[e], u[i][e]);
      store_vec<T, VEC>(out + i * r.h_step, h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const bool constant = reset >> i & 1u;
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] = constant ? u[i][e] : fmaf(a[i][e], h[e], u[i][e]);
      if (i < static_cast<int>(q.n))
        store_vec<T, VEC>(out + row_offset(r, q.row0 + i, r.h_batch, r.h_step), h);
      if ((q.last >> i & 1u) && r.h_last) {
        float *to = r.h_last + sequence_of(r, q.row0 + i) * r.channels + ch;
#pragma unroll
        for (int e = 0; e < VEC; ++e) to[e] = h[e];
      }
    }
  }
  // empty sequences hand their first state on
  if (k == 0 && r.h_last && (r.offsets || r.lengths || rows == 0)) {
    for (int64_t b = seg; b < r.batch; b += kSegs) {
      const bool empty = r.offsets ? r.offsets[b + 1] <= r.offsets[b] : held_steps(r, static_cast<uint32_t>(b)) == 0;
      if (empty)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          r.h_last[b * r.channels + ch + e] = r.h0 ? r.h0[b * r.channels + ch + e] : 0.0f;
    }
  }
  if (joined) leave_place<W>(scan_block<W>(r.workspace, blocks, chunks, place.block), chunks);
}

template <typename T, int VEC>
hipError_t launch_recurrence_forward_vec(const fftmv_recurrence_t &r, hipStream_t s) {
  const ScanGrid<T, VEC> grid(r);
  if (!grid.fits()) return hipErrorInvalidConfiguration;
  return by_recurrence_kind(r.decay, r.drive, [&](auto d, auto u) {
    recurrence_forward_kernel<T, VEC, decltype(d)::value, decltype(u)::value>
        <<<static_cast<unsigned>(grid.chunks * grid.blocks), kThreads, 0, s>>>(r, grid.rows, grid.chunks, grid.blocks,
                                                                            chunks_joined(r, grid.chunks));
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
