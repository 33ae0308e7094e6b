// The scan of the gated linear recurrence h_t = a_t h_{t-1} + u_t, shared by
// its forward and backward kernels.
//
// A workgroup takes one chunk of kChunk rows (time steps) of kLanes * VEC
// channels: kSegs segments of kRows rows, by kLanes lanes, and a thread keeps
// its kRows x VEC elements in registers: each input is read once. A lane has 16
// bytes of a row, so that a chunk's row is 256 bytes (128-byte rows measured
// 10-25% slower: the memory system serves whole lines, and rows rarely start
// on one); in the 16-bit backward pass, whose three inputs would not fit the
// registers at that width, 8 bytes, and the row 128.
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
//     fma(A, state before, H). (A chunk whose A is out of FP32's range publishes
//     no map, only its state, which went through its segments one by one.)
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
  int places;  // chunks of a chain
  int chains;  // chains over the batch (1 when packed)
  int blocks;  // blocks of W channels
  int per;     // sequences of one chunk, where whole ones fit (else 1)
  __host__ __device__ bool joined() const { return places > 1; }
  int64_t pairs() const { return static_cast<int64_t>(chains) * blocks; }
  int64_t workgroups() const { return pairs() * places; }
};

inline ScanAxis scan_axis(int64_t batch, int64_t steps, bool packed, int64_t channels, int64_t width) {
  ScanAxis a;
  a.blocks = static_cast<int>((channels + width - 1) / width);
  a.per = 1;
  if (steps == 0) {  // only first and last states, by one workgroup per block
    a.places = a.chains = 1;
  } else if (packed || steps > kChunk / 2) {
    a.places = static_cast<int>((steps + kChunk - 1) / kChunk);
    a.chains = packed ? 1 : static_cast<int>(batch);
  } else {
    a.places = 1;
    a.per = static_cast<int>(kChunk / steps);
    a.chains = static_cast<int>((batch + a.per - 1) / a.per);
  }
  return a;
}

// Rows of `carries`: one for every chunk, none where no chunk follows another.
inline int64_t scan_carries(int64_t batch, int64_t steps, bool packed) {
  const ScanAxis a = scan_axis(batch, steps, packed, 1, 1);
  return a.joined() ? static_cast<int64_t>(a.places) * a.chains : 0;
}

// ------------------------------------------------------------- workspace
// Counters, one for every chain and block of channels, in a buffer of their
// own that every call leaves zero. And for every chunk and column three 64-bit
// words: the two halves of its map (A, H) and the state behind it, each below
// the number of the call in its upper half. A word is written once, whole,
// and is there when it carries this call's number: no flag, no fence, and
// nothing to clear for the next call, whatever its shape (the owner of the
// workspace counts the calls). With 12 bytes a column, cleared by the last
// workgroup of a chain, every workgroup had to wait for its words' arrival
// before counting itself: 235 instead of 207 us backward at 4 x 4096 x 4096
// bf16; cleared by a second launch, small calls took 3 us more.
struct ScanCounter {
  uint32_t ticket;
  uint32_t pad[31];  // a line of its own
};

// Host: enough for every block width.
struct ScanWorkspace {
  size_t counters = 0, words = 0;
};
inline ScanWorkspace scan_workspace_bytes(int64_t batch, int64_t steps, bool packed, int64_t channels) {
  const int64_t widest = 8 * kLanes;
  const ScanAxis a = scan_axis(batch, steps, packed, channels, widest);
  ScanWorkspace w;
  if (!a.joined()) return w;
  const int64_t pairs = a.pairs();  // blocks half as wide: twice as many chains
  w.counters = static_cast<size_t>(2 * pairs) * sizeof(ScanCounter);
  w.words = static_cast<size_t>(a.places * pairs) * widest * 24;
  return w;
}

struct ScanChain {  // the workspace of one chain and block of channels
  uint32_t *ticket;
  uint64_t *words;  // [places][3][W]
  uint32_t call;
  bool deep;        // many chunks of the chain run at once
};

template <int W>
__device__ __forceinline__ ScanChain scan_chain(const fftmv_recurrence_t &r, const ScanAxis &a, int chain) {
  ScanChain s;
  s.ticket = &(static_cast<ScanCounter *>(r.counters) + chain)->ticket;
  s.words = static_cast<uint64_t *>(r.workspace) + static_cast<int64_t>(chain) * a.places * (3 * W);
  s.call = r.call;
  s.deep = a.chains * a.blocks < 24;
  return s;
}

// Words of column c of a place: 0 and 1 its map (A, H), 2 the state behind it.
template <int W>
__device__ __forceinline__ void publish(const ScanChain &s, int place, int word, int c, float v) {
  __hip_atomic_store(s.words + static_cast<int64_t>(place) * (3 * W) + (word * W + c),
                     static_cast<uint64_t>(s.call) << 32 | __builtin_bit_cast(uint32_t, v), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
template <int W>
__device__ __forceinline__ uint64_t peek(const ScanChain &s, int place, int word, int c) {
  return __hip_atomic_load(s.words + static_cast<int64_t>(place) * (3 * W) + (word * W + c), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool is_there(const ScanChain &s, uint64_t word) {
  return static_cast<uint32_t>(word >> 32) == s.call;
}
__device__ __forceinline__ float value_of(uint64_t word) {
  return __builtin_bit_cast(float, static_cast<uint32_t>(word));
}

// The state behind place p - 1 in column c. Looks at the words of the two
// chunks in front of p together, and of two more where a chain has over twenty
// chunks running at once (some 500 workgroups run together): every word that
// is looked at delays all loads, every chunk less makes more of the chain wait
// in a row. Two | four chunks, us, one series of 61e6 bf16 or 31e6 FP32 elements
// in so many chains (blocks of channels):
//                    8           12          16          20          24          32
//   bf16 forward     157 | 112   130 | 117   109 | 106   115 | 114   102 | 102   101.6 | 102.0
//   bf16 backward    228 | 217   211 | 206   201 | 201   196 | 196   193 | 193   189.1 | 189.4
//   FP32 forward     150 | 102   123 |  99    90 |  85    99 |  97    83 |  82    79.9 |  80.8
//   FP32 backward    197 | 158   173 | 156   153 | 148   156 | 152   143 | 141   141.1 | 141.7
//   fp16, 45 packed  172 | 167   179 | 176   161 | 159   175 | 174   161 | 161   155   | 155
// A state is there sooner or later, since each chunk publishes its own. The
// bound on the polls ends the wait if the workspace
// was not what the call requires: the result is NaN.
template <int W>
__device__ __forceinline__ float state_before(const ScanChain &s, int p, int c) {
#pragma unroll 1
  for (int poll = 0; poll < (1 << 20); ++poll) {
    const int i0 = p - 1, i1 = p < 2 ? 0 : p - 2;
    const uint64_t s0 = peek<W>(s, i0, 2, c), s1 = peek<W>(s, i1, 2, c);
    const uint64_t A0 = peek<W>(s, i0, 0, c), H0 = peek<W>(s, i0, 1, c);
    if (is_there(s, s0)) return value_of(s0);
    if (is_there(s, A0) && is_there(s, H0)) {
      if (is_there(s, s1)) return fmaf(value_of(A0), value_of(s1), value_of(H0));
      if (s.deep) {
        const int i2 = p < 3 ? 0 : p - 3, i3 = p < 4 ? 0 : p - 4;
        const uint64_t s2 = peek<W>(s, i2, 2, c), s3 = peek<W>(s, i3, 2, c);
        const uint64_t A1 = peek<W>(s, i1, 0, c), H1 = peek<W>(s, i1, 1, c);
        const uint64_t A2 = peek<W>(s, i2, 0, c), H2 = peek<W>(s, i2, 1, c);
        if (is_there(s, A1) && is_there(s, H1)) {
          float h = 0.0f;
          bool found = is_there(s, s2);
          if (found) {
            h = value_of(s2);
          } else if (is_there(s, A2) && is_there(s, H2) && is_there(s, s3)) {
            found = true;
            h = fmaf(value_of(A2), value_of(s3), value_of(H2));
          }
          if (found) return fmaf(value_of(A0), fmaf(value_of(A1), h, value_of(H1)), value_of(H0));
        }
      }
    }
    __builtin_amdgcn_s_sleep(1);
  }
  return __builtin_nanf("");
}

// What a chunk does with the states of its chain, by one thread per column:
// publishes its map (A, H), where it has one, or, when it is `closed` (nothing
// that enters it leaves it), its state H; returns the state that enters it,
// where `needed`. behind(h): the state behind the chunk for h in front.
// `early`: what peek saw as the state in front some time ago.
template <int W, typename F>
__device__ __forceinline__ float meet_chain(const ScanChain &s, int p, int col, float A, float H, bool closed,
                                            bool mapped, bool needed, uint64_t early, F behind) {
  // the columns of a wave wait together
  const bool ready = needed && __ballot(!is_there(s, early)) == 0;
  float in = 0.0f;
  if (closed) {
    publish<W>(s, p, 2, col, H);
  } else if (!ready && mapped) {
    publish<W>(s, p, 0, col, A);
    publish<W>(s, p, 1, col, H);
  }
  if (needed) in = ready ? value_of(early) : state_before<W>(s, p, col);
  if (!closed) {
    publish<W>(s, p, 2, col, behind(in));
  }
  return in;
}

// The next place of a chain is the count before this call's addition; the
// thread that drew the last one leaves the counter zero.
__device__ __forceinline__ uint32_t draw_place(const ScanChain &s) {
  return __hip_atomic_fetch_add(s.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t settle_ticket(const ScanChain &s, uint32_t ticket, int places) {
  if (ticket == static_cast<uint32_t>(places - 1))
    __hip_atomic_store(s.ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return ticket;
}

// ------------------------------------------------------------------ rows
// Which of a thread's rows start a sequence, end one, belong to none. In an
// ordinary chunk (below) none does, and seq[0] alone is set.
struct Rows {
  uint32_t bits;   // kRows bits each, from bit 0: dead (in no sequence, or not present), start, last, and from
                   // bit 16: not present, empty (a row that stands for an empty sequence of a padded batch)
  int row0;        // step of row 0 in the sequence c.seq (packed: the row)
  int seq[kRows];
  __device__ __forceinline__ bool dead(int i) const { return bits >> i & 1u; }
  __device__ __forceinline__ bool start(int i) const { return bits >> (4 + i) & 1u; }
  __device__ __forceinline__ bool last(int i) const { return bits >> (8 + i) & 1u; }
  __device__ __forceinline__ bool absent(int i) const { return bits >> (16 + i) & 1u; }
  __device__ __forceinline__ bool empty(int i) const { return bits >> (20 + i) & 1u; }
  __device__ __forceinline__ bool closed_front() const { return bits & 0x0FFu; }
  __device__ __forceinline__ bool closed_back() const { return bits & 0xF0Fu; }
};
static_assert(kRows == 4, "nibbles");

// Where packed sequence i starts, clamped to the axis as lengths are.
__device__ __forceinline__ int packed_start(const fftmv_recurrence_t &r, int i) {
  const int T = static_cast<int>(r.steps), o = r.offsets[i];
  return o < 0 ? 0 : o > T ? T : o;
}

// The sequence that holds `row` when packed: the last one that starts at or
// before it (-1: none does; batch: behind the last one's end).
__device__ __forceinline__ int packed_sequence(const fftmv_recurrence_t &r, int row) {
  int lo = 0, hi = static_cast<int>(r.batch) + 1;  // offsets[0..lo) <= row < offsets[hi..]
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (r.offsets[mid] <= row) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

__device__ __forceinline__ int held_steps(const fftmv_recurrence_t &r, int b) {
  const int T = static_cast<int>(r.steps);
  if (!r.lengths) return T;
  const int l = r.lengths[b];
  return l < 0 ? 0 : l > T ? T : l;
}

// One chunk, as the whole workgroup sees it.
struct Chunk {
  int chain, place;  // over the batch; along the time axis
  int seq;           // sequence of the first row (of all rows if ordinary)
  bool ordinary;     // all rows are steps of one sequence, none its last
  bool head, tail;   // nothing enters from the chunk in front / from the one behind
};

__device__ __forceinline__ Chunk chunk_at(const fftmv_recurrence_t &r, const ScanAxis &a, int chain, int place) {
  const int T = static_cast<int>(r.steps), S = static_cast<int>(r.batch);
  const int t0 = place * kChunk, end = T - t0 > kChunk ? t0 + kChunk : T;  // behind the last row
  Chunk c;
  c.chain = chain;
  c.place = place;
  int seq;
  bool ordinary, head, tail;
  if (r.offsets) {
    seq = packed_sequence(r, t0);
    const bool held = seq >= 0 && seq < S && t0 < T;
    head = place == 0 || !held || packed_start(r, seq) == t0;
    ordinary = held && T - t0 > kChunk && end < packed_start(r, seq + 1);
    const int e = ordinary ? seq : packed_sequence(r, end - 1);
    tail = end >= T || e < 0 || e >= S || packed_start(r, e + 1) == end;
  } else {
    seq = chain * a.per;
    const int held = a.per > 1 || T == 0 ? 0 : held_steps(r, seq);
    ordinary = held - t0 > kChunk;
    head = place == 0 || t0 >= held;
    tail = held - t0 <= kChunk;
  }
  // the same in every lane: kept in scalar registers
  c.seq = __builtin_amdgcn_readfirstlane(seq);
  const uint32_t bits = __builtin_amdgcn_readfirstlane((ordinary ? 1 : 0) | (head ? 2 : 0) | (tail ? 4 : 0));
  c.ordinary = bits & 1u;
  c.head = bits & 2u;
  c.tail = bits & 4u;
  return c;
}

__device__ __forceinline__ Rows rows_of(const fftmv_recurrence_t &r, const ScanAxis &a, const Chunk &c, int seg) {
  Rows q;
  q.bits = 0;
  q.seq[0] = c.seq;
  q.row0 = c.place * kChunk + seg * kRows;
  if (c.ordinary) return q;
  const int T = static_cast<int>(r.steps), S = static_cast<int>(r.batch);
  const int left = T - c.place * kChunk - seg * kRows;  // rows of the axis from here on, where one sequence has it
  if (r.offsets) {
    int s = left > 0 ? packed_sequence(r, q.row0) : S;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const bool here = i < left;
      const int row = q.row0 + i;
      while (here && s < S && row >= packed_start(r, s + 1)) ++s;  // on to the next sequence that holds a row
      const bool held = here && s >= 0 && s < S;
      q.seq[i] = held ? s : 0;
      if (!here) q.bits |= 1u << (16 + i);
      if (!held) q.bits |= 1u << i;
      if (held && row == packed_start(r, s)) q.bits |= 1u << (4 + i);
      if (held && row + 1 == packed_start(r, s + 1)) q.bits |= 1u << (8 + i);
    }
  } else {
    const bool many = a.per > 1;
    const int end = a.per < S - c.seq ? c.seq + a.per : S;  // first sequence not here
    int b = c.seq, t = q.row0;
    if (many) b += t / T, t %= T;
    else if (left <= 0) b = end;
    int held = b < end ? held_steps(r, b) : 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (many ? t == T : i == left) {
        t = 0, ++b;
        if (!many) b = end;
        held = b < end ? held_steps(r, b) : 0;
      }
      const bool here = b < end;
      q.seq[i] = here ? b : c.seq;
      if (!here) q.bits |= 1u << (16 + i);
      if (here && held == 0 && t == 0) q.bits |= 1u << (20 + i);
      if (!here || t >= held) q.bits |= 1u << i;
      else if (t == 0) q.bits |= 1u << (4 + i);
      if (here && t + 1 == held) q.bits |= 1u << (8 + i);
      ++t;
    }
  }
  return q;
}

// Where row i of a thread starts in a field, in elements.
__device__ __forceinline__ int64_t row_offset(const fftmv_recurrence_t &r, const ScanAxis &a, const Chunk &c,
                                              const Rows &q, int i, int64_t sb, int64_t st) {
  const int seq = c.ordinary ? c.seq : q.seq[i];
  int64_t t = static_cast<int64_t>(q.row0) + i;
  if (a.per > 1) t -= static_cast<int64_t>(seq - c.seq) * r.steps;
  return (r.offsets ? 0 : static_cast<int64_t>(seq) * sb) + t * st;
}

// One field's rows of this thread. In the place of a dead row comes the first
// row of the chunk's sequence (or of the axis): always there, in cache, and
// not used.
template <typename T, int VEC>
__device__ __forceinline__ void load_rows(const fftmv_recurrence_t &r, const ScanAxis &a, const Chunk &c,
                                          const Rows &q, const void *field, int64_t sb, int64_t st, int64_t ch,
                                          Vec<T, VEC> (&v)[kRows]) {
  const T *p = static_cast<const T *>(field) + ch;
  if (c.ordinary) {
    p += row_offset(r, a, c, q, 0, sb, st);
#pragma unroll
    for (int i = 0; i < kRows; ++i) v[i] = load_vec<T, VEC>(p + i * st);
  } else if (r.steps > 0) {
    const int64_t instead = r.offsets ? 0 : c.seq * sb;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t at = row_offset(r, a, c, q, i, sb, st);
      v[i] = load_vec<T, VEC>(p + (q.dead(i) ? instead : at));
    }
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_row(const fftmv_recurrence_t &r, const ScanAxis &a, const Chunk &c,
                                          const Rows &q, int i, void *field, int64_t sb, int64_t st, int64_t ch,
                                          const float (&f)[VEC], bool streamed = true) {
  T *p = static_cast<T *>(field) + ch;
  if (c.ordinary)
    store_vec<T, VEC>(p + row_offset(r, a, c, q, 0, sb, st) + i * st, f, streamed);
  else if (!q.absent(i))
    store_vec<T, VEC>(p + row_offset(r, a, c, q, i, sb, st), f, streamed);
}

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
#pragma unroll 1
  for (int64_t b = seg; b < r.batch; b += kSegs)
    if (!r.offsets || packed_start(r, static_cast<int>(b) + 1) <= packed_start(r, static_cast<int>(b))) {
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

// A product of decays that FP32 holds. Decays above one can pass its range
// within a chunk while the states that they act on are zero or tiny: such a
// product is used nowhere, and the states go through the single segments (of
// kRows decays each) instead.
__device__ __forceinline__ bool in_range(float A) { return fabsf(A) <= 3.402823466e38f; }

// The same through group j of SG segments, whose maps are A, H and whose joined
// map is gA, gH; BACK from the last segment.
template <bool BACK, int SG, int W>
__device__ __forceinline__ float through_group(const float (*A)[W], const float (*H)[W], const float (*gA)[W],
                                               const float (*gH)[W], uint32_t constants, int j, int col, float h) {
  constexpr uint32_t kGroup = ~0u >> (32 - SG);
  if (constants >> (j * SG) & kGroup) return gH[j][col];
  const float a = gA[j][col];
  if (in_range(a)) return fmaf(a, h, gH[j][col]);
#pragma unroll 1
  for (int i = 0; i < SG; ++i) {
    const int seg = j * SG + (BACK ? SG - 1 - i : i);
    h = fmaf(A[seg][col], h, H[seg][col]);
  }
  return h;
}

template <typename F>
hipError_t by_recurrence_kind(int decay, int drive, F f) {
  return by_three(decay, [&](auto d) { return by_two(drive, [&](auto u) { return f(d, u); }); });
}

}  // namespace fftmv
