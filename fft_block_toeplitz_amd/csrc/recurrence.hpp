// The scan of the gated linear recurrence h_t = a_t h_{t-1} + u_t, shared by
// its forward and backward kernels.
//
// A workgroup takes one chunk of kChunk rows (time steps) of kLanes * VEC
// channels: kSegs segments of kRows rows, by kLanes lanes of 16 bytes, so a
// row of the chunk is 256 bytes and a thread keeps its kRows x VEC elements
// in registers: each input is read once. (128-byte rows, half a wave each,
// measured 10-25% slower: the memory system serves whole lines, and rows
// rarely start on one.)
//
// A run of steps maps the state that enters it, h, to A h + H with A the
// product of its decays. Three levels join these maps, each in a fixed order
// (results are bitwise reproducible):
//   - the rows of a segment, by one thread per VEC channels;
//   - the segments of the chunk, in LDS, by one thread per channel and group
//     of segments;
//   - the chunks of a chain (one sequence, or the whole packed axis), through
//     the workspace: a workgroup publishes its chunk's (A, H) before it waits
//     for anything, then folds the maps in front of it onto the nearest
//     published state: the same sequence of operations whatever state it
//     found, since the state behind a chunk is itself defined as
//     fma(A, state before, H).
// A chunk's place in its chain is drawn from a counter, not taken from
// blockIdx: every chunk in front has then been started by a running
// workgroup, which publishes without waiting, so all waits end in whatever
// order workgroups run. Workgroups go through all chains place by place: with
// many chains the state in front is usually there before it is asked for.
//
// Where a sequence starts, or in rows that no sequence holds, the map is a
// constant: those rows select instead of multiplying (a non-finite state of
// one sequence never meets the next).
#pragma once

#include "common.hpp"
#include "internal.hpp"
#include "sequence.hpp"

namespace fftmv {

constexpr int kChunk = FFTMV_RECURRENCE_CHUNK;
constexpr int kLanes = 16;              // threads across a row
constexpr int kRows = 4;                // rows of a segment
constexpr int kSegs = kChunk / kRows;   // segments of a chunk
constexpr int kThreads = kSegs * kLanes;
constexpr int kSegsPerWave = kWave / kLanes;
constexpr int kWaves = kThreads / kWave;
static_assert(kSegs == 32 && kSegsPerWave == 4 && kWaves == 8, "one bit of a word for each segment");

// How the rows are cut: chains of `places` chunks, `blocks` of channels.
struct ScanAxis {
  int64_t places;   // chunks of a chain
  int64_t chains;   // chains over the batch (1 when packed)
  int64_t blocks;   // blocks of W channels
  int64_t per;      // sequences of one chunk, where whole ones fit (else 1)
  __host__ __device__ bool joined() const { return places > 1; }
  int64_t workgroups() const { return places * chains * blocks; }
};

inline ScanAxis scan_axis(int64_t batch, int64_t steps, bool packed, int64_t channels, int64_t width) {
  ScanAxis a;
  a.blocks = (channels + width - 1) / width;
  a.per = 1;
  if (steps == 0) {  // only first and last states, by one workgroup per block
    a.places = a.chains = 1;
  } else if (packed) {
    a.places = (steps + kChunk - 1) / kChunk;
    a.chains = 1;
  } else if (steps > kChunk / 2) {
    a.places = (steps + kChunk - 1) / kChunk;
    a.chains = batch;
  } else {
    a.places = 1;
    a.per = kChunk / steps;
    a.chains = (batch + a.per - 1) / a.per;
  }
  return a;
}

// Rows of `carries`: one for every chunk, none where no chunk follows another.
inline int64_t scan_carries(int64_t batch, int64_t steps, bool packed) {
  const ScanAxis a = scan_axis(batch, steps, packed, 1, 1);
  return a.joined() ? a.places * a.chains : 0;
}

// ------------------------------------------------------------- workspace
// A counter line for every chain and block; then for every chunk and column
// the map (A, H) as one 64-bit word and the state behind the chunk as one
// 32-bit word. A word is written once, whole, and zero stands for "not there
// yet" (the value +0 is written as -0), so no word needs a flag or a fence.
struct ScanCounters {
  uint32_t ticket, done;
  uint32_t pad[30];  // 128 bytes
};

// Host: enough for every block width.
inline size_t scan_workspace_bytes(int64_t batch, int64_t steps, bool packed, int64_t channels) {
  const int64_t widest = 8 * kLanes;
  const ScanAxis a = scan_axis(batch, steps, packed, channels, widest);
  if (!a.joined()) return 0;
  const int64_t pairs = a.chains * a.blocks;  // blocks half as wide: twice as many counters
  return static_cast<size_t>(2 * pairs) * sizeof(ScanCounters) + static_cast<size_t>(a.places * pairs) * widest * 12;
}

struct ScanChain {  // the workspace of one chain and block of channels
  ScanCounters *count;
  uint64_t *map;    // [places][W]
  uint32_t *state;  // [places][W]
};

template <int W>
__device__ __forceinline__ ScanChain scan_chain(void *ws, const ScanAxis &a, int64_t chain) {
  ScanChain s;
  const int64_t all = a.chains * a.blocks;
  unsigned char *p = static_cast<unsigned char *>(ws);
  s.count = reinterpret_cast<ScanCounters *>(p) + chain;
  p += all * static_cast<int64_t>(sizeof(ScanCounters));
  s.map = reinterpret_cast<uint64_t *>(p) + chain * a.places * W;
  s.state = reinterpret_cast<uint32_t *>(p + all * a.places * W * 8) + chain * a.places * W;
  return s;
}

__device__ __forceinline__ float nonzero(float v) { return __builtin_bit_cast(uint32_t, v) == 0u ? -0.0f : v; }

__device__ __forceinline__ void publish_map(const ScanChain &s, int64_t i, float A, float H) {
  const uint64_t w = static_cast<uint64_t>(__builtin_bit_cast(uint32_t, nonzero(H))) << 32 |
                     __builtin_bit_cast(uint32_t, A);
  __hip_atomic_store(s.map + i, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_state(const ScanChain &s, int64_t i, float h) {
  __hip_atomic_store(s.state + i, __builtin_bit_cast(uint32_t, nonzero(h)), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t peek_state(const ScanChain &s, int64_t i) {
  return __hip_atomic_load(s.state + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state behind place p - 1 in column c. Looks at the kWindow chunks in
// front of p together; a state is there sooner or later, since each of them
// publishes its own. The bound on the polls ends the wait if the workspace
// was not what the call requires (not zero on entry): the result is NaN.
template <int W>
__device__ float state_before(const ScanChain &s, int64_t p, int c) {
  constexpr int kWindow = 8;
  for (int poll = 0; poll < (1 << 20); ++poll) {
    uint32_t st[kWindow];
    uint64_t mp[kWindow];
#pragma unroll
    for (int j = 0; j < kWindow; ++j) {
      const int64_t i = p - 1 - j;
      st[j] = 0;
      mp[j] = 0;
      if (i >= 0) {
        st[j] = peek_state(s, i * W + c);
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

// What a chunk does with the states of its chain, by one thread per column:
// publishes its map (A, H), or, when it is `closed` (nothing that enters it
// leaves it), its state H; returns the state that enters it, where `needed`.
// `early`: what peek_state saw in front some time ago, 0 for nothing. All its
// words have arrived when it returns.
template <int W>
__device__ __forceinline__ float meet_chain(const ScanChain &s, int64_t p, int col, float A, float H, bool closed,
                                            bool needed, uint32_t early) {
  float in = 0.0f;
  if (closed)
    publish_state(s, p * W + col, H);
  else if (!early)
    publish_map(s, p * W + col, A, H);
  if (needed) in = early ? __builtin_bit_cast(float, early) : state_before<W>(s, p, col);
  if (!closed) publish_state(s, p * W + col, fmaf(A, in, nonzero(H)));
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  return in;
}

// Draws the next place of the chain, in the thread that gets the ticket.
__device__ __forceinline__ uint32_t draw_place(const ScanChain &s) {
  return __hip_atomic_fetch_add(&s.count->ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Counts a workgroup that will not touch the chain's words again.
__device__ __forceinline__ uint32_t leave_chain(const ScanChain &s) {
  return __hip_atomic_fetch_add(&s.count->done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Leaves the workspace of a chain zero: by the last workgroup that left it.
template <int W>
__device__ __forceinline__ void clear_chain(const ScanChain &s, int64_t places) {
  for (int64_t i = threadIdx.x; i < places * W; i += kThreads) {
    s.map[i] = 0;
    s.state[i] = 0;
  }
  if (threadIdx.x == 0) s.count->ticket = s.count->done = 0;
}

// ------------------------------------------------------------------ rows
// Which of a thread's rows start a sequence, end one, belong to none. In an
// ordinary chunk (below) all that is known and only seq[0] and t[0] are set.
struct Rows {
  uint32_t present, start, last, dead;  // a bit a row; dead: in no sequence, or not present
  uint32_t empty;                       // dead, and stands for an empty sequence of a padded batch
  uint32_t seq[kRows], t[kRows];        // sequence, and step within its strides (packed: the row)
};

// The sequence that holds `row` when packed: the last one that starts at or
// before it (-1: none does; batch: behind the last one's end).
__device__ __forceinline__ int packed_sequence(const fftmv_recurrence_t &r, int64_t row) {
  int lo = 0, hi = static_cast<int>(r.batch) + 1;  // offsets[0..lo) <= row < offsets[hi..]
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (r.offsets[mid] <= row) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

__device__ __forceinline__ int64_t held_steps(const fftmv_recurrence_t &r, int64_t b) {
  if (!r.lengths) return r.steps;
  const int64_t l = r.lengths[b];
  return l < 0 ? 0 : l > r.steps ? r.steps : l;
}

// One chunk, as the whole workgroup sees it.
struct Chunk {
  int64_t chain, place;  // over the batch; along the time axis
  int64_t seq;           // sequence of the first row (of all rows if ordinary)
  bool ordinary;         // all rows are steps of one sequence, none its last
  bool head, tail;       // nothing enters from the chunk in front / from the one behind
};

__device__ __forceinline__ Chunk chunk_at(const fftmv_recurrence_t &r, const ScanAxis &a, int64_t chain,
                                          int64_t place) {
  Chunk c;
  c.chain = chain;
  c.place = place;
  const int64_t t0 = place * kChunk, end = t0 + kChunk;
  if (r.offsets) {
    const int s = packed_sequence(r, t0);
    const bool held = s >= 0 && s < r.batch && t0 < r.steps;
    c.seq = s;
    c.head = place == 0 || !held || r.offsets[s] == t0;
    c.ordinary = held && end < r.offsets[s + 1] && end < r.steps;
    const int64_t back = end < r.steps ? end : r.steps;  // behind the chunk's last row
    const int e = packed_sequence(r, back - 1);
    c.tail = back >= r.steps || e < 0 || e >= r.batch || r.offsets[e + 1] == back;
  } else {
    c.seq = chain * a.per;
    const int64_t held = a.per > 1 || r.steps == 0 ? 0 : held_steps(r, c.seq);
    c.ordinary = end < held;
    c.head = place == 0 || t0 >= held;
    c.tail = end >= held;
  }
  return c;
}

__device__ __forceinline__ Rows ordinary_rows(const fftmv_recurrence_t &r, const Chunk &c, int seg) {
  Rows q;
  q.start = q.last = q.dead = q.empty = 0;
  q.present = (1u << kRows) - 1u;
  q.seq[0] = static_cast<uint32_t>(c.seq);
  q.t[0] = static_cast<uint32_t>(c.place * kChunk + seg * kRows);
  return q;
}

__device__ __forceinline__ Rows special_rows(const fftmv_recurrence_t &r, const ScanAxis &a, const Chunk &c, int seg) {
  Rows q;
  q.present = q.start = q.last = q.empty = 0;
  const int64_t row0 = c.place * kChunk + seg * kRows;
  if (r.offsets) {
    int s = packed_sequence(r, row0);
    const int S = static_cast<int>(r.batch);
    int64_t from = s >= 0 ? r.offsets[s] : -1, to = s < S ? r.offsets[s + 1] : INT64_MAX;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t row = row0 + i;
      while (row >= to && s < S) {  // on to the next sequence that holds a row
        ++s;
        from = to;
        to = s < S ? r.offsets[s + 1] : INT64_MAX;
      }
      q.seq[i] = static_cast<uint32_t>(s < 0 || s >= S ? 0 : s);
      q.t[i] = static_cast<uint32_t>(row);
      if (row < r.steps) {
        q.present |= 1u << i;
        if (s >= 0 && s < S) {
          if (row == from) q.start |= 1u << i;
          if (row + 1 == to) q.last |= 1u << i;
        }
      }
      if (row >= r.steps || s < 0 || s >= S) q.empty |= 1u << i;  // for now: dead
    }
    q.dead = q.empty;
    q.empty = 0;
  } else {
    q.dead = 0;
    const uint32_t T = static_cast<uint32_t>(r.steps), local = static_cast<uint32_t>(seg * kRows);
    uint32_t b = static_cast<uint32_t>(c.seq), t = static_cast<uint32_t>(row0);
    if (a.per > 1) b += local / T, t = local % T;
    const int64_t end = (c.chain + 1) * a.per < r.batch ? (c.chain + 1) * a.per : r.batch;  // first sequence not here
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (a.per > 1 && t == T) t = 0, ++b;
      const bool here = t < T && b < end;
      q.seq[i] = here ? b : 0;
      q.t[i] = t;
      int64_t held = 0;
      if (here) {
        held = held_steps(r, b);
        q.present |= 1u << i;
        if (held == 0 && t == 0) q.empty |= 1u << i;
      }
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

// Where row i of a thread starts in a field, in elements.
__device__ __forceinline__ int64_t row_offset(const fftmv_recurrence_t &r, const Rows &q, int i, int64_t sb,
                                              int64_t st) {
  const int64_t t = static_cast<int64_t>(q.t[i]) * st;
  return r.offsets ? t : static_cast<int64_t>(q.seq[i]) * sb + t;
}

// One field's rows of this thread.
template <bool ORDINARY, typename T, int VEC>
__device__ __forceinline__ void load_rows(const fftmv_recurrence_t &r, const Rows &q, const void *field, int64_t sb,
                                          int64_t st, int64_t ch, Vec<T, VEC> (&v)[kRows]) {
  const T *p = static_cast<const T *>(field) + ch;
  if constexpr (ORDINARY) {
    p += row_offset(r, q, 0, sb, st);
#pragma unroll
    for (int i = 0; i < kRows; ++i) v[i] = load_vec<T, VEC>(p + i * st);
  } else {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      v[i] = Vec<T, VEC>{};
      if (!(q.dead >> i & 1u)) v[i] = load_vec<T, VEC>(p + row_offset(r, q, i, sb, st));
    }
  }
}
template <bool ORDINARY, typename T, int VEC>
__device__ __forceinline__ void store_row(const fftmv_recurrence_t &r, const Rows &q, int i, void *field, int64_t sb,
                                          int64_t st, int64_t ch, const float (&f)[VEC]) {
  T *p = static_cast<T *>(field) + ch;
  if constexpr (ORDINARY)
    store_vec<T, VEC>(p + row_offset(r, q, 0, sb, st) + i * st, f);
  else if (q.present >> i & 1u)
    store_vec<T, VEC>(p + row_offset(r, q, i, sb, st), f);
}

// Hides where a value came from, so that what was computed from it before is
// computed again instead of kept: the decays of a thread's elements take 32
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

// Keeps the compiler from starting on further rows' exponentials before a row
// is done: it would hold them all, and spill.
__device__ __forceinline__ void row_done() { __builtin_amdgcn_sched_barrier(0); }

// VEC channels of a [batch][channels] state, zeros where there is none.
template <int VEC>
__device__ __forceinline__ void load_state(const float *p, int64_t seq, int64_t channels, int64_t ch,
                                           float (&v)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = p ? p[seq * channels + ch + e] : 0.0f;
}
template <int VEC>
__device__ __forceinline__ void store_state(float *p, int64_t seq, int64_t channels, int64_t ch,
                                            const float (&v)[VEC]) {
  if (!p) return;
#pragma unroll
  for (int e = 0; e < VEC; ++e) p[seq * channels + ch + e] = v[e];
}

// Empty sequences that no row stands for (packed ones, and all where there
// are no steps): `to` gets what `from` has.
template <int VEC>
__device__ __forceinline__ void pass_empty(const fftmv_recurrence_t &r, int seg, int64_t ch, const float *from,
                                           float *to) {
  for (int64_t b = seg; b < r.batch; b += kSegs)
    if (r.offsets ? r.offsets[b + 1] <= r.offsets[b] : true) {
      float v[VEC];
      load_state(from, b, r.channels, ch, v);
      store_state(to, b, r.channels, ch, v);
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

// One bit for each of a wave's segments from a ballot over its lanes (all
// lanes of a segment agree).
__device__ __forceinline__ uint8_t segment_bits(uint64_t b) {
  return static_cast<uint8_t>((b & 1u) | (b >> 15 & 2u) | (b >> 30 & 4u) | (b >> 45 & 8u));
}
// All segments' bits from the waves' nibbles.
__device__ __forceinline__ uint32_t read_segment_bits(const uint8_t *bits) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(bits);
  uint32_t all = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v = __builtin_amdgcn_readfirstlane(w[i]);
    all |= ((v & 0xFu) | (v >> 4 & 0xF0u) | (v >> 8 & 0xF00u) | (v >> 12 & 0xF000u)) << 16 * i;
  }
  return all;
}

// Joins the maps of `n` segments in the order of the rows (or, backwards,
// from the last): h becomes the state behind them.
__device__ __forceinline__ float through(bool constant, float A, float H, float h) {
  return constant ? H : fmaf(A, h, H);
}

template <typename F>
hipError_t by_recurrence_kind(int decay, int drive, F f) {
  return by_three(decay, [&](auto d) { return by_two(drive, [&](auto u) { return f(d, u); }); });
}

}  // namespace fftmv
