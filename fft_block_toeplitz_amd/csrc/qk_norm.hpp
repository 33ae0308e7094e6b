// Norms of queries and keys for each head with a rotation by position, forward
// and backward.
//
// Memory traffic bounds both: x (and dy) in, y (or dx) out, once each. A few
// lanes have one head of one row, four pairs of elements a lane, so that the
// rotation needs no other lane; LANES of them add up the squares. The pairs'
// sines and cosines are the same for all heads of a row: a workgroup computes
// them once for its rows, in LDS. Angles are reduced to a turn in FP64: half a
// million positions along, FP32 would leave two digits of them.
#pragma once

#include "common.hpp"
#include "internal.hpp"
#include "sequence.hpp"

namespace fftmv {

hipError_t launch_qk_norm_forward(const fftmv_qk_norm_t &n, hipStream_t s);
hipError_t launch_qk_norm_backward(const fftmv_qk_norm_t &n, hipStream_t s);

constexpr int kNormPairs = 4;     // pairs of elements a lane
constexpr int kNormTurns = 1024;  // sines and cosines a workgroup keeps
constexpr int kNormRows = 8;      // rows a workgroup takes at once, at most
constexpr int kNormMost = 1024;   // workgroups of a backward call, each with a row of partial sums

struct NormPlan {
  int rows;    // rows that a workgroup takes at once
  int blocks;  // workgroups
};
inline NormPlan qk_norm_plan(int64_t rows, int64_t frequencies, bool back) {
  NormPlan p;
  const int64_t fit = frequencies ? kNormTurns / frequencies : kNormRows;
  // few rows: one a workgroup, so that all of the card takes part
  p.rows = static_cast<int>(rows <= 2048 ? 1 : fit < kNormRows ? fit : kNormRows);
  const int64_t blocks = (rows + p.rows - 1) / p.rows;
  p.blocks = static_cast<int>(back && blocks > kNormMost ? kNormMost : blocks > (1 << 20) ? 1 << 20 : blocks);
  return p;
}
inline size_t qk_norm_workspace(int64_t rows, int64_t dim) {
  return size_t{2} * (rows < kNormMost ? rows : kNormMost) * dim * sizeof(float);
}

}  // namespace fftmv
