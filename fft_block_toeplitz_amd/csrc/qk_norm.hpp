// Norms of queries and keys for each head with a rotation by position, forward
// and backward.
//
// Memory traffic bounds both: x (and dy) in, y (or dx) out, once each. A few
// lanes have one head of one row, eight elements a lane, four pairs where they
// are rotated, so that the rotation needs no other lane; LANES of them add up
// the squares. A workgroup has some rows of the queries or of the keys: one
// set of weights and of their gradients stays in registers, and each group of
// lanes fetches its next head while it works on this one. The pairs' sines and
// cosines are the same for all heads of a row: a workgroup computes them once
// for its rows, in LDS. Angles are reduced to a turn in FP64: half a million
// positions along, FP32 would leave two digits of them.
// 16384 rows of 40 heads of 128 bf16: 58 us, 5.8 TB/s (out of memory 73, a copy's
// rate); with results through the caches 90. Gradients of as many rows of 32
// heads: 78 us. 9995 rows of 10 heads of 75 FP32 take 29 and 24 us, for 12 and
// 19 of bytes: rows that are not aligned, a third of the lanes idle, and the
// card filled once.
#pragma once

#include <algorithm>

#include "common.hpp"
#include "internal.hpp"
#include "sequence.hpp"

namespace fftmv {

hipError_t launch_qk_norm_forward(const fftmv_qk_norm_t &n, hipStream_t s);
hipError_t launch_qk_norm_backward(const fftmv_qk_norm_t &n, hipStream_t s);

constexpr int kNormElements = 8;           // elements a lane
constexpr int kNormPairs = 4;              // pairs of elements a lane
constexpr int kNormTurns = 2048;           // cosines a workgroup keeps, and as many sines: 16 KB of LDS
constexpr int kNormRows = 32;              // rows a workgroup takes at once, at most
constexpr int kNormUnits = 256;            // heads of rows that it takes at once, about
// Workgroups that fill the card, four on each CU. (Gradients of 8 x 2048 rows of
// 32 heads of 128 bf16, before later steps: 1024 88 us, 2048 96, 512 122.)
constexpr int kNormWide = 1024;

// How the elements of a head lie on the lanes. Apart: first the rotated pairs,
// four a lane, then the rest, eight a lane; the last lane of either goes back
// until it has four or eight, and what it shares with the lane before counts
// for sums there alone. Where a part is shorter than a lane, or the lanes do
// not suffice, pairs follow each other through all of the head, and lanes with
// an end in them take their elements one by one. (All heads that way: 9995 rows
// of 10 heads of 75 FP32 with gradients 73 us instead of 54, 16384 rows of 40 heads
// of 128 bf16 63 instead of 57.)
struct NormPlan {
  int turned, dim;    // pairs that are rotated, elements
  int apart;          // 0: pairs follow each other
  int turned_lanes;   // lanes with rotated pairs
  int lanes;          // lanes with elements
  int turns;          // cosines of a row, one more lane's for what is not rotated
  int rows[2];        // rows that a workgroup takes at once: queries, keys
  int blocks[2];      // workgroups
};

// Workgroups of a backward call for the queries or the keys, at most: each leaves a row of partial sums.
inline int64_t norm_share(int64_t heads, int64_t all) { return std::max<int64_t>(kNormWide * heads / all, 1); }

inline NormPlan qk_norm_plan(int64_t rows, int64_t query_heads, int64_t key_heads, int64_t dim, int64_t frequencies,
                             bool back) {
  NormPlan p;
  p.turned = static_cast<int>(frequencies);
  p.dim = static_cast<int>(dim);
  const int rest = p.dim - 2 * p.turned;
  p.turned_lanes = (p.turned + kNormPairs - 1) / kNormPairs;
  p.lanes = p.turned_lanes + (rest + kNormElements - 1) / kNormElements;
  p.apart = (p.turned == 0 || p.turned >= kNormPairs) && (rest == 0 || rest >= kNormElements) && p.lanes <= kWave;
  if (!p.apart) p.lanes = (p.dim + kNormElements - 1) / kNormElements;
  p.turns = (p.turned_lanes + 1) * kNormPairs;
  const int64_t heads[2] = {query_heads, key_heads};
  for (int i = 0; i < 2; ++i) {
    // few rows: so few at a time that all of the card takes part (64 rows of 40 heads of 128: 4.2 us, six at a
    // time 12.9; 2048 rows 10 and 16)
    const int64_t each = std::max<int64_t>(heads[i], 1), spread = rows * (query_heads + key_heads) / (kNormWide * each);
    const int64_t fit = p.turned ? kNormTurns / p.turns : kNormRows;
    const int64_t r = std::min({kNormUnits / each, spread, fit, int64_t{kNormRows}});
    p.rows[i] = static_cast<int>(r < 1 ? 1 : r);
    const int64_t blocks = heads[i] ? (rows + p.rows[i] - 1) / p.rows[i] : 0;
    p.blocks[i] = static_cast<int>(std::min<int64_t>(blocks, back ? norm_share(heads[i], query_heads + key_heads) : 1 << 20));
  }
  return p;
}
// Bytes of the partial sums of the weights' gradients, of any number of rotated pairs.
inline size_t qk_norm_workspace(int64_t rows, int64_t query_heads, int64_t key_heads, int64_t dim) {
  int64_t blocks = 0;
  for (const int64_t heads : {query_heads, key_heads})
    if (heads) blocks += std::min(rows, norm_share(heads, query_heads + key_heads));
  return static_cast<size_t>(blocks) * dim * sizeof(float);
}

}  // namespace fftmv
