// The scan of the gated linear recurrence h_t = a_t h_{t-1} + u_t, shared by
// its forward and backward kernels.
//
// A workgroup takes one chunk of kChunk rows of the flattened time axis (the
// sequences one after the other) for kLanes * VEC channels: 128 bytes of
// every row. Its threads are kSegs segments of kRows rows by kLanes
// lanes of 16 bytes, so that a wave's load covers eight whole cache lines and
// a thread keeps its kRows x VEC elements in registers: each input is read
// once.
//
// A run of steps maps the state that enters it, h, to A h + H with A the
// product of its decays. Three levels join these maps, each in a fixed order
// (results are bitwise reproducible):
//   - the rows of a segment, by one thread per VEC channels;
//   - the segments of the chunk, in LDS, by one thread per channel and group
//     of segments;
//   - the chunks, through the workspace: a workgroup publishes its chunk's
//     (A, H) before it waits for anything, then folds the maps in front of it
//     onto the nearest published state: the same sequence of operations
//     whatever state it found, since the state behind a chunk is itself
//     defined as fma(A, state before, H).
// A chunk's number is drawn from a counter, not taken from blockIdx: every
// lower chunk has then been started by a running workgroup, which publishes
// without waiting, so all waits end in whatever order workgroups run.
//
// Where a sequence starts, or in rows that no sequence holds, the map is a
// constant: those rows select instead of multiplying (a non-finite state of
// one sequence never meets the next).
#pragma once

#include <type_traits>

#include "common.hpp"
#include "internal.hpp"
#include "sequence.hpp"

namespace fftmv {

constexpr int kChunk = FFTMV_RECURRENCE_CHUNK;
constexpr int kLanes = 8;                  // threads across a row
constexpr int kRows = 4;                   // rows of a segment
constexpr int kSegs = kChunk / kRows;      // segments of a chunk
constexpr int kThreads = kSegs * kLanes;
constexpr int kSegsPerWave = kWave / kLanes;
static_assert(kThreads <= 512 && kThreads % kWave == 0, "a chunk is one workgroup");

// ------------------------------------------------------------- workspace
// Per block of channels: a counter line, then per chunk and channel the map
// (A, H) as one 64-bit word and the state behind the chunk as one 32-bit
// word. A word is written once, whole, and zero stands for "not there yet"
// (the value +0 is written as -0), so no word needs a flag or a fence.
struct ScanCounters {
  uint32_t ticket, done;
  uint32_t pad[30];  // a 128-byte line for each block of channels
};

inline int64_t scan_chunks(int64_t rows) { return (rows + kChunk - 1) / kChunk; }

// Host: enough for blocks of 32 and of 64 channels.
inline size_t scan_workspace_bytes(int64_t rows, int64_t channels) {
  const int64_t chunks = scan_chunks(rows);
  if (chunks <= 1) return 0;
  const int64_t pairs = (channels + 63) / 64;
  return static_cast<size_t>(2 * pairs) * sizeof(ScanCounters) + static_cast<size_t>(chunks * pairs) * 64 * 12;
}

struct ScanBlock {  // the workspace of one block of channels
  ScanCounters *count;
  uint64_t *map;    // [chunks][W]
  uint32_t *state;  // [chunks][W]
};

template <int W>
__device__ __forceinline__ ScanBlock scan_block(void *ws, int64_t blocks, int64_t chunks, int64_t block) {
  ScanBlock s;
  unsigned char *p = static_cast<unsigned char *>(ws);
  s.count = reinterpret_cast<ScanCounters *>(p) + block;
  p += blocks * static_cast<int64_t>(sizeof(ScanCounters));
  s.map = reinterpret_cast<uint64_t *>(p) + block * chunks * W;
  s.state = reinterpret_cast<uint32_t *>(p + blocks * chunks * W * 8) + block * chunks * W;
  return s;
}

__device__ __forceinline__ float nonzero(float v) {
  return __builtin_bit_cast(uint32_t, v) == 0u ? -0.0f : v;
}

__device__ __forceinline__ void publish_map(const ScanBlock &s, int64_t i, float A, float H) {
  const uint64_t w = static_cast<uint64_t>(__builtin_bit_cast(uint32_t, nonzero(H))) << 32 |
                     __builtin_bit_cast(uint32_t, A);
  __hip_atomic_store(s.map + i, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_state(const ScanBlock &s, int64_t i, float h) {
  __hip_atomic_store(s.state + i, __builtin_bit_cast(uint32_t, nonzero(h)), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}

// The state behind chunk k - 1 in column c. Looks at the kWindow chunks
// before k together; a state is there sooner or later, since each of them
// publishes its own. The bound on the polls ends the wait if the workspace
// was not what the call requires (not zero on entry): the result is NaN.
template <int W>
__device__ float state_before(const ScanBlock &s, int64_t k, int c) {
  constexpr int kWindow = 8;
  for (int poll = 0; poll < (1 << 20); ++poll) {
    uint32_t st[kWindow];
    uint64_t mp[kWindow];
#pragma unroll
    for (int j = 0; j < kWindow; ++j) {
      const int64_t i = k - 1 - j;
      st[j] = 0;
      mp[j] = 0;
      if (i >= 0) {
        st[j] = __hip_atomic_load(s.state + i * W + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        mp[j] = __hip_atomic_load(s.map + i * W + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    // the nearest state with every map behind it
    int found = kWindow;
    bool open = true;
#pragma unroll
    for (int j = 0; j < kWindow; ++j) {
      if (open && st[j]) found = j, open = false;
      if (open && !mp[j]) open = false;
    }
    if (found < kWindow) {
      float h = 0.0f;
#pragma unroll
      for (int j = kWindow - 1; j >= 0; --j) {
        if (j == found) h = __builtin_bit_cast(float, st[j]);
        if (j < found)
          h = nonzero(fmaf(__builtin_bit_cast(float, static_cast<uint32_t>(mp[j])), h,
                           __builtin_bit_cast(float, static_cast<uint32_t>(mp[j] >> 32))));
      }
      return h;
    }
    __builtin_amdgcn_s_sleep(1);
  }
  return __builtin_nanf("");
}

// This workgroup's place: a block of channels from blockIdx, and the next
// chunk of it that nobody took. Ends with a barrier. Chunks count from the
// front of the time axis (forward) or from its end (backward).
struct Place {
  int64_t block, chunk;
};
__device__ __forceinline__ Place take_place(void *ws, int64_t blocks) {
  __shared__ uint32_t ticket;
  Place p;
  p.block = blockIdx.x % blocks;
  p.chunk = blockIdx.x / blocks;
  if (ws) {
    if (threadIdx.x == 0)
      ticket = __hip_atomic_fetch_add(&(static_cast<ScanCounters *>(ws) + p.block)->ticket, 1u, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    p.chunk = ticket;
  }
  return p;
}

// Leaves the workspace of a block of channels zero: done by its last
// workgroup to get here, when no other can still read or write it. (The words
// that a workgroup published have arrived before it counts itself: they come
// from the wave of thread 0, which waits for its stores.)
template <int W>
__device__ __forceinline__ void leave_place(const ScanBlock &s, int64_t chunks) {
  __shared__ uint32_t order;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    order = __hip_atomic_fetch_add(&s.count->done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (order != static_cast<uint32_t>(chunks - 1)) return;
  for (int64_t i = threadIdx.x; i < chunks * W; i += kThreads) {
    __hip_atomic_store(s.map + i, uint64_t(0), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(s.state + i, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (threadIdx.x == 0) {
    __hip_atomic_store(&s.count->ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(&s.count->done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

// ------------------------------------------------------------------ rows
// Which of a thread's rows start a sequence, end one, belong to none.
struct Rows {
  uint32_t row0;               // first row on the flattened axis
  uint32_t n;                  // how many of the kRows rows exist
  uint32_t start, last, dead;  // one bit a row; dead: in no sequence, or not there
  __device__ __forceinline__ bool special() const { return start | last | dead; }
};

// The sequence that holds `row` when packed: the last one that starts at or
// before it (-1: none does; batch: behind the last one's end).
__device__ __forceinline__ int packed_sequence(const fftmv_recurrence_t &r, uint32_t row) {
  int lo = 0, hi = static_cast<int>(r.batch) + 1;  // offsets[0..lo) <= row < offsets[hi..]
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (r.offsets[mid] <= static_cast<int64_t>(row)) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

__device__ __forceinline__ int sequence_of(const fftmv_recurrence_t &r, uint32_t row) {
  return r.offsets ? packed_sequence(r, row) : static_cast<int>(row / static_cast<uint32_t>(r.steps));
}

__device__ __forceinline__ uint32_t held_steps(const fftmv_recurrence_t &r, uint32_t b) {
  const int T = static_cast<int>(r.steps);
  if (!r.lengths) return T;
  const int l = r.lengths[b];
  return l < 0 ? 0 : l > T ? T : l;
}

__device__ __forceinline__ Rows rows_at(const fftmv_recurrence_t &r, int64_t rows, int64_t row0) {
  Rows q;
  q.row0 = static_cast<uint32_t>(row0);
  const int64_t left = rows - row0;
  q.n = left <= 0 ? 0 : left < kRows ? static_cast<uint32_t>(left) : kRows;
  q.start = q.last = 0;
  q.dead = q.n < kRows ? ~0u << q.n & ((1u << kRows) - 1u) : 0u;
  if (q.n == 0) return q;
  if (r.offsets) {
    int s = packed_sequence(r, q.row0);
    const int S = static_cast<int>(r.batch);
    int64_t from = s >= 0 ? r.offsets[s] : -1, to = s < S ? r.offsets[s + 1] : INT64_MAX;
    for (uint32_t i = 0; i < q.n; ++i) {
      const int64_t row = row0 + i;
      while (row >= to) {  // on to the next sequence that holds a row
        ++s;
        from = to;
        to = s < S ? r.offsets[s + 1] : INT64_MAX;
      }
      if (s < 0 || s >= S) {
        q.dead |= 1u << i;
      } else {
        if (row == from) q.start |= 1u << i;
        if (row + 1 == to) q.last |= 1u << i;
      }
    }
  } else {
    const uint32_t T = static_cast<uint32_t>(r.steps);
    uint32_t b = q.row0 / T, t = q.row0 - b * T;
    // the common segment lies inside one sequence, away from its ends
    if (!r.lengths && t > 0 && t + q.n < T) return q;
    uint32_t held = held_steps(r, b);
    for (uint32_t i = 0; i < q.n; ++i) {
      if (t == T) t = 0, ++b, held = held_steps(r, b);
      if (t >= held) {
        q.dead |= 1u << i;
      } else {
        if (t == 0) q.start |= 1u << i;
        if (t + 1 == held) q.last |= 1u << i;
      }
      ++t;
    }
  }
  return q;
}

// Where the row starts in a field, in elements.
__device__ __forceinline__ int64_t row_offset(const fftmv_recurrence_t &r, uint32_t row, int64_t sb, int64_t st) {
  if (r.offsets) return static_cast<int64_t>(row) * st;
  const uint32_t T = static_cast<uint32_t>(r.steps), b = row / T;
  return static_cast<int64_t>(b) * sb + static_cast<int64_t>(row - b * T) * st;
}

// One field's rows of this thread. wave_special (the same in the whole wave):
// some lane's rows are not kRows ordinary neighbours.
template <typename T, int VEC>
__device__ __forceinline__ void load_rows(const fftmv_recurrence_t &r, const Rows &q, bool wave_special,
                                          const void *field, int64_t sb, int64_t st, int64_t ch,
                                          Vec<T, VEC> (&v)[kRows]) {
  const T *p = static_cast<const T *>(field) + ch;
  if (!wave_special) {
    p += row_offset(r, q.row0, sb, st);
#pragma unroll
    for (int i = 0; i < kRows; ++i) v[i] = load_vec<T, VEC>(p + i * st);
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (q.dead >> i & 1u)
        v[i] = Vec<T, VEC>{};
      else
        v[i] = load_vec<T, VEC>(p + row_offset(r, q.row0 + i, sb, st));
    }
  }
}

// The channel of a column of the blocks. Columns beyond the last channel step
// back by whole vectors to the row's last VEC channels: they repeat another
// column's work, bit for bit, and store the same values, so that every load
// and store is a whole vector inside its row.
template <int VEC>
__device__ __forceinline__ int64_t column_channel(int64_t channels, int64_t column) {
  const int64_t e = column % VEC, c0 = column - e;
  return (c0 + VEC <= channels ? c0 : channels - VEC) + e;
}

// ------------------------------------------------------------ small helpers
// One bit for each of a wave's kSegsPerWave segments from a ballot over its
// lanes (all lanes of a segment agree): the lowest bit of byte i becomes bit i.
__device__ __forceinline__ uint8_t segment_bits(uint64_t ballot) {
  static_assert(kLanes == 8 && kSegsPerWave == 8, "a segment is a byte of the ballot");
  return static_cast<uint8_t>((ballot & 0x0101010101010101ull) * 0x0102040810204080ull >> 56);
}
// The chunk's segments with a constant map: the waves' bits in one word.
using SegmentBits = typename std::conditional<kThreads / kWave == 8, uint64_t, uint32_t>::type;
static_assert(sizeof(SegmentBits) * kWave == kThreads, "a byte for each wave");
__device__ __forceinline__ SegmentBits read_segment_bits(const uint8_t *bits) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(bits);
  SegmentBits b = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(w[0]));
  if constexpr (sizeof(SegmentBits) == 8)
    b |= static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(w[1]))) << 32;
  return b;
}

// Forward or backward launch over all chunks and blocks of channels.
template <typename T, int VEC>
struct ScanGrid {
  static constexpr int W = kLanes * VEC;
  int64_t rows, chunks, blocks;
  explicit ScanGrid(const fftmv_recurrence_t &r) {
    rows = r.offsets ? r.steps : r.batch * r.steps;
    chunks = rows > 0 ? scan_chunks(rows) : 1;
    blocks = (r.channels + W - 1) / W;
  }
  bool fits() const { return grid_fits(chunks * blocks, kThreads); }
};

// Chunks that all begin with a sequence need nothing from each other.
inline bool chunks_joined(const fftmv_recurrence_t &r, int64_t chunks) {
  return chunks > 1 && (r.offsets || kChunk % r.steps != 0);
}

template <typename F>
hipError_t by_recurrence_kind(int decay, int drive, F f) {
  return by_three(decay, [&](auto d) { return by_two(drive, [&](auto u) { return f(d, u); }); });
}

}  // namespace fftmv
