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

// Hides where a value came from, so that what was computed from it before is
// computed again instead of kept: the decays of a thread's elements take 64
// registers each time they are kept, an exponential when they are not.
template <typename T, int VEC>
__device__ __forceinline__ void forget(Vec<T, VEC> (&v)[kRows]) {
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if constexpr (VEC * sizeof(T) == 16) {
      u32x4_any w = __builtin_bit_cast(u32x4_any, v[i]);
      asm volatile("" : "+v"(w));
      v[i] = __builtin_bit_cast(Vec<T, VEC>, w);
    }
  }
}

template <typename T, int VEC, int DECAY, int DRIVE>
__global__ __launch_bounds__(kThreads, 4) void recurrence_backward_kernel(fftmv_recurrence_t r, int64_t rows,
                                                                        int64_t chunks, int64_t blocks,
                                                                        bool joined) {
  constexpr int W = kLanes * VEC, G = kThreads / W, SG = kSegs / G;
  constexpr SegmentBits kGroup = ~SegmentBits(0) >> (8 * sizeof(SegmentBits) - SG);
  // maps of the segments and of groups of them: forward A h + H, backward A s + S
  __shared__ float sA[kSegs][W], sH[kSegs][W], sS[kSegs][W], gA[G][W], gH[G][W], gS[G][W], enter[W];
  __shared__ __align__(8) uint8_t front_bits[kThreads / kWave], back_bits[kThreads / kWave];

  const Place place = take_place(joined ? r.workspace : nullptr, blocks);
  if (place.chunk >= chunks) return;  // a workspace that was not zero
  const int64_t k = chunks - 1 - place.chunk;
  const int tid = threadIdx.x, seg = tid / kLanes, lane = tid % kLanes;
  const int64_t ch = column_channel<VEC>(r.channels, place.block * W + lane * VEC);
  const int col = tid % W, grp = tid / W;

  const Rows q = rows_at(r, rows, k * kChunk + seg * kRows);
  const bool special = __ballot(q.special()) != 0;
  Vec<T, VEC> x[kRows], g[kRows], d[kRows];
  load_rows<T, VEC>(r, q, special, r.gate, r.gate_batch, r.gate_step, ch, g);
  load_rows<T, VEC>(r, q, special, r.x, r.x_batch, r.x_step, ch, x);
  load_rows<T, VEC>(r, q, special, r.dh, r.dh_batch, r.dh_step, ch, d);
  // the state that enters the chunk; the forward left 0 where none does
  float carry = 0.0f;
  if (rows > 0) carry = r.carries[k * r.channels + column_channel<VEC>(r.channels, place.block * W + col)];

  const uint32_t front = q.start | q.dead, back = q.last | q.dead;
  float A[VEC], H[VEC], S[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) A[e] = 1.0f, H[e] = 0.0f, S[e] = 0.0f;
  if (!special) {
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const Terms t = decay_terms<T, DECAY>(g[i][e]);
        H[e] = fmaf(t.a, H[e], drive_of<DRIVE>(t, x[i][e]));
        A[e] *= t.a;
        S[e] = fmaf(A[e], d[i][e], S[e]);  // a_0 .. a_i dh_i
      }
  } else {
    bool closed = false;  // a later row's gradient no longer reaches the segment's first
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const bool dead = q.dead >> i & 1u, start = q.start >> i & 1u, last = q.last >> i & 1u;
      closed |= dead;
      const float *h0 = nullptr, *dl = nullptr;
      if (start && r.h0) h0 = r.h0 + sequence_of(r, q.row0 + i) * r.channels + ch;
      if (last && r.dh_last) dl = r.dh_last + sequence_of(r, q.row0 + i) * r.channels + ch;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const Terms t = decay_terms<T, DECAY>(g[i][e]);
        float u = drive_of<DRIVE>(t, x[i][e]);
        if (h0) u = fmaf(t.a, h0[e], u);
        if (dead) u = 0.0f;
        H[e] = start || dead ? u : fmaf(t.a, H[e], u);
        A[e] *= t.a;
        const float dv = dl ? d[i][e] + dl[e] : d[i][e];
        if (!closed) S[e] = fmaf(A[e], dv, S[e]);
      }
      closed |= last;
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    sA[seg][lane * VEC + e] = A[e];
    sH[seg][lane * VEC + e] = H[e];
    sS[seg][lane * VEC + e] = S[e];
  }
  {
    const uint64_t f = __ballot(front != 0), b = __ballot(back != 0);
    if (tid % kWave == 0) front_bits[tid / kWave] = segment_bits(f), back_bits[tid / kWave] = segment_bits(b);
  }
  __syncthreads();
  const SegmentBits fronts = read_segment_bits(front_bits), backs = read_segment_bits(back_bits);

  // the maps of groups of segments: one thread per channel and group
  float mA[SG], mH[SG], mS[SG];
  {
    float cA = 1.0f, cH = 0.0f, cS = 0.0f;
#pragma unroll
    for (int i = 0; i < SG; ++i) {
      mA[i] = sA[grp * SG + i][col];
      mH[i] = sH[grp * SG + i][col];
      mS[i] = sS[grp * SG + i][col];
      cH = fronts >> (grp * SG + i) & 1u ? mH[i] : fmaf(mA[i], cH, mH[i]);
      cA *= mA[i];
    }
#pragma unroll
    for (int i = SG - 1; i >= 0; --i) cS = backs >> (grp * SG + i) & 1u ? mS[i] : fmaf(mA[i], cS, mS[i]);
    gA[grp][col] = cA;
    gH[grp][col] = cH;
    gS[grp][col] = cS;
  }
  __syncthreads();

  // what the chunk behind hands over
  if (tid < W) {
    float in = 0.0f;
    if (joined) {
      const ScanBlock s = scan_block<W>(r.workspace, blocks, chunks, place.block);
      const int64_t end = rows - 1 - k * kChunk < kChunk - 1 ? rows - 1 : k * kChunk + kChunk - 1;  // last row
      const Rows tail = rows_at(r, rows, end);
      float cA = 1.0f, cS = 0.0f;
#pragma unroll
      for (int j = G - 1; j >= 0; --j) {
        cS = backs >> (j * SG) & kGroup ? gS[j][col] : fmaf(gA[j][col], cS, gS[j][col]);
        cA *= gA[j][col];
      }
      const int64_t word = place.chunk * W + col;
      if (backs)
        publish_state(s, word, cS);
      else
        publish_map(s, word, cA, cS);
      if (!((tail.last | tail.dead) & 1u)) in = state_before<W>(s, place.chunk, col);
      if (!backs) publish_state(s, word, fmaf(cA, in, nonzero(cS)));
    }
    enter[col] = in;
  }
  // meanwhile, the state that enters each segment, in the place of its map
  {
    float h = carry;
    for (int j = 0; j < grp; ++j)
      h = fronts >> (j * SG) & kGroup ? gH[j][col] : fmaf(gA[j][col], h, gH[j][col]);
#pragma unroll
    for (int i = 0; i < SG; ++i) {
      sH[grp * SG + i][col] = h;
      h = fronts >> (grp * SG + i) & 1u ? mH[i] : fmaf(mA[i], h, mH[i]);
    }
  }
  __syncthreads();
  {
    float s = enter[col];
    for (int j = G - 1; j > grp; --j)
      s = backs >> (j * SG) & kGroup ? gS[j][col] : fmaf(gA[j][col], s, gS[j][col]);
#pragma unroll
    for (int i = SG - 1; i >= 0; --i) {
      sS[grp * SG + i][col] = s;
      s = backs >> (grp * SG + i) & 1u ? mS[i] : fmaf(mA[i], s, mS[i]);
    }
  }
  __syncthreads();

  forget(g);
  forget(x);
  forget(d);
  // forward over the segment: w = h_{t-1} (- x_t), the factor of dgate
  float h[VEC], s[VEC], w[kRows][VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    h[e] = sH[seg][lane * VEC + e];
    s[e] = sS[seg][lane * VEC + e];
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (special && (q.start >> i & 1u)) {
      const float *h0 = r.h0 ? r.h0 + sequence_of(r, q.row0 + i) * r.channels + ch : nullptr;
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] = h0 ? h0[e] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const Terms t = decay_terms<T, DECAY>(g[i][e]);
      w[i][e] = DRIVE == FFTMV_DRIVE_COMPLEMENT ? h[e] - x[i][e] : h[e];
      h[e] = fmaf(t.a, h[e], drive_of<DRIVE>(t, x[i][e]));
    }
  }
  forget(g);
  // backward over it
  T *dx = static_cast<T *>(r.dx) + ch, *dg = static_cast<T *>(r.dgate) + ch;
#pragma unroll
  for (int i = kRows - 1; i >= 0; --i) {
    const bool dead = special && (q.dead >> i & 1u);
    if (special && (q.last >> i & 1u)) {
      const float *dl = r.dh_last ? r.dh_last + sequence_of(r, q.row0 + i) * r.channels + ch : nullptr;
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[e] = dl ? dl[e] : 0.0f;
    }
    float du[VEC], dv[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const Terms t = decay_terms<T, DECAY>(g[i][e]);
      const float rt = d[i][e] + s[e];
      s[e] = dead ? 0.0f : t.a * rt;
      du[e] = dead ? 0.0f : DRIVE == FFTMV_DRIVE_COMPLEMENT ? rt * t.rest : rt;
      dv[e] = dead ? 0.0f : rt * w[i][e] * t.slope;
    }
    if (!special) {
      store_vec<T, VEC>(dx + row_offset(r, q.row0, r.dx_batch, r.dx_step) + i * r.dx_step, du);
      store_vec<T, VEC>(dg + row_offset(r, q.row0, r.dgate_batch, r.dgate_step) + i * r.dgate_step, dv);
    } else if (i < static_cast<int>(q.n)) {
      store_vec<T, VEC>(dx + row_offset(r, q.row0 + i, r.dx_batch, r.dx_step), du);
      store_vec<T, VEC>(dg + row_offset(r, q.row0 + i, r.dgate_batch, r.dgate_step), dv);
    }
    if (special && (q.start >> i & 1u) && r.dh0) {
      float *to = r.dh0 + sequence_of(r, q.row0 + i) * r.channels + ch;
#pragma unroll
      for (int e = 0; e < VEC; ++e) to[e] = s[e];
    }
  }
  // empty sequences hand their last state's gradient on
  if (k == 0 && r.dh0 && (r.offsets || r.lengths || rows == 0)) {
    for (int64_t b = seg; b < r.batch; b += kSegs) {
      const bool empty = r.offsets ? r.offsets[b + 1] <= r.offsets[b] : held_steps(r, static_cast<uint32_t>(b)) == 0;
      if (empty)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          r.dh0[b * r.channels + ch + e] = r.dh_last ? r.dh_last[b * r.channels + ch + e] : 0.0f;
    }
  }
  if (joined) leave_place<W>(scan_block<W>(r.workspace, blocks, chunks, place.block), chunks);
}

template <typename T, int VEC>
hipError_t launch_recurrence_backward_vec(const fftmv_recurrence_t &r, hipStream_t s) {
  const ScanGrid<T, VEC> grid(r);
  if (!grid.fits()) return hipErrorInvalidConfiguration;
  return by_recurrence_kind(r.decay, r.drive, [&](auto d, auto u) {
    recurrence_backward_kernel<T, VEC, decltype(d)::value, decltype(u)::value>
        <<<static_cast<unsigned>(grid.chunks * grid.blocks), kThreads, 0, s>>>(r, grid.rows, grid.chunks, grid.blocks,
                                                                            chunks_joined(r, grid.chunks));
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
