// Group normalisation: which kernels a call takes, and the sums of the
// parameters' gradients.
#include "group_norm.hpp"

namespace fftmv {
namespace {

__global__ __launch_bounds__(kBlock) void param_sums_kernel(fftmv_group_norm_t g, int64_t rows) {
  __shared__ float lds[2 * kBlock];
  param_sums(g, rows, blockIdx.x, lds);
}

int round64(int64_t n) { return static_cast<int>((n + 63) / 64 * 64); }

// Groups of the widest slabs over at most `lanes` lanes of `vec` channels,
// every slab at least one vector wide; 0 where there are none. As few slabs as
// that gives, of about the same width.
int widest_slab(int D, int G, int vec, int lanes) {
  constexpr int kMostGroups = 256;  // whose statistics lie in LDS
  const int64_t fit = static_cast<int64_t>(lanes) * vec / D;
  const int most = static_cast<int>(std::min<int64_t>({fit, G, kMostGroups}));
  auto wide = [&](int gs) {
    return static_cast<int64_t>(gs) * D >= vec && static_cast<int64_t>((G - 1) % gs + 1) * D >= vec;
  };
  if (most > 0) {
    const int slabs = (G + most - 1) / most, even = (G + slabs - 1) / slabs;
    if (wide(even)) return even;
  }
  for (int gs = most; gs >= 1; --gs)
    if (wide(gs)) return gs;
  return 0;
}

// Pieces of one group wider than the lanes of a workgroup: as few as 256 lanes
// allow, of about the same width, in whole vectors; the last one at least one
// vector wide.
void cut_group(NormShape &s, int vec) {
  const int64_t D = s.D, most = 256 * static_cast<int64_t>(vec), pieces = (D + most - 1) / most;
  int64_t width = ((D + pieces - 1) / pieces + vec - 1) / vec * vec;
  while ((D - 1) % width + 1 < vec) width -= vec;
  s.width = static_cast<int>(width);
  s.cut = static_cast<int>((D + width - 1) / width);
  s.gs = 1;
  s.slabs = s.G * s.cut;
  s.lx = s.width / vec;
  s.threads = 256;
  s.ty = s.threads / s.lx;
  s.sub = 1;
}

void take_slab(NormShape &s, int gs, int vec, int threads) {
  s.gs = gs;
  s.slabs = (s.G + gs - 1) / gs;
  s.lx = (gs * s.D + vec - 1) / vec;
  s.ty = threads / s.lx;
  s.sub = 1;
  s.threads = threads;
}

void take_team(NormShape &s, int sums) {
  s.team = 64;
  while (s.team > 1 && s.team * sums > s.threads) s.team /= 2;
}

}  // namespace

hipError_t launch_param_sums(const fftmv_group_norm_t &g, int64_t rows, hipStream_t s) {
  param_sums_kernel<<<static_cast<unsigned>((g.channels + kSumChannels - 1) / kSumChannels), kBlock, 0,
                      s>>>(g, rows);
  return hipGetLastError();
}

NormPlan norm_plan(int64_t samples, int64_t rows, int64_t channels, int64_t groups, int dtype, bool backward) {
  NormPlan p;
  NormShape &s = p.s;
  s.N = samples;
  s.S = static_cast<int>(rows);
  s.G = static_cast<int>(groups);
  s.D = static_cast<int>(channels / groups);
  const int es = dtype == FFTMV_F32 ? 4 : 2;
  p.vec = 16 / es;
  s.cut = 1;
  const bool wide = s.D > 1024 * p.vec;  // one group is more than a workgroup's lanes
  if (!wide && widest_slab(s.D, s.G, p.vec, 1024) == 0) p.vec = 1;
  const int v = p.vec, alone = static_cast<int>((static_cast<int64_t>(s.D) + v - 1) / v);  // lanes of one group
  const bool split = wide || rows == 0;
  // A row or two of many samples: one workgroup for each group. Us forward and
  // backward, so | cut and split as below: 2000 tokens of 9000 bf16 channels 43
  // and 99 | 104 and 186, 300 of them 19 and 39 | 23 and 43, 64 of them 16.5 and 28
  // | 14.7 and 20; 2000 samples of two rows 81 and 173 | 110 and 193, 300 of them 34
  // and 63 | 24 and 43; 2000 of three 118 and 258 | 114 and 203.
  if (wide && rows > 0 && rows <= 2 && samples * groups >= 256 * rows * rows) {
    p.kind = NormPlan::kWide;
    p.rows = samples;
    p.workspace = backward ? static_cast<size_t>(samples * channels) * 8 : 0;
    return p;
  }
  p.whole = s.D % v == 0;
  const int64_t bytes = samples * std::max<int64_t>(rows, 1) * channels * es;
  const int Q = backward ? 2 : 4;

  // Single rows, or a few: Q samples at a time in a thread's registers, so
  // that a barrier serves all of them, and narrow ones side by side (forward
  // and backward, bf16: 16000 x 5000 in 25 groups 82 and 180 us against 134 and
  // 206 one by one, 20522 x 246 in 2 groups 15 and 29 against 26 and 78);
  // where that leaves too few workgroups for the CUs, the form below takes
  // them one by one.
  if (!split && rows <= 8) {
    const int R = std::max(1, s.S);
    const int64_t least = static_cast<int64_t>(alone) * R;
    const int threads = least <= 256 ? 256 : least <= 512 ? 512 : 0;
    const int gs = threads ? widest_slab(s.D, s.G, v, threads / R) : 0;
    if (gs > 0 && (threads == 256 || p.whole)) {
      take_slab(s, gs, v, threads);
      constexpr int kMostSums = 512;  // of a thread's sample, whose statistics lie in LDS
      s.sub = std::min(s.ty / R, std::max(1, kMostSums / s.gs));
      s.ty = R;
      s.threads = round64(static_cast<int64_t>(s.lx) * s.ty * s.sub);
      while (s.sub > 1 && (samples + Q * s.sub - 1) / (Q * s.sub) * s.slabs < 512) s.sub /= 2;
      s.threads = round64(static_cast<int64_t>(s.lx) * s.ty * s.sub);
      const int64_t turns = (samples + Q * s.sub - 1) / (Q * s.sub);
      if (turns * s.slabs >= 256) {
        p.kind = NormPlan::kTokens;
        s.across = static_cast<int>(std::min<int64_t>(turns, std::max(1, (backward ? 1024 : 2048) / s.slabs)));
      }
    }
  }
  // A sample's slab in registers: one row a thread, or up to eight (backward,
  // with twice the inputs: four). 400 samples of 100 rows of 8 x 64 bf16 take
  // 30 and 56 us, split 42 and 64.
  const int several = backward ? 4 : 8;
  for (int P = 1; !split && P <= several && p.kind == NormPlan::kSplit; P *= several) {
    const int most = P == 1 ? kNormThreads : kHeldThreads;
    for (int threads = 256; threads <= most && p.kind == NormPlan::kSplit; threads *= 2) {
      for (int lanes = std::min(threads, 256); lanes >= 1; lanes /= 2) {
        const int gs = widest_slab(s.D, s.G, v, std::max(lanes, alone));
        if (gs == 0) continue;
        take_slab(s, gs, v, threads);
        if (s.lx > threads || s.S > P * s.ty) continue;
        // one row a thread: for few rows, or where one takes most of the threads
        if (P == 1 && s.lx * s.S > 256 && alone <= 256) continue;
        // rows of less than 64 bytes waste the lines that they touch (200
        // samples of 256 rows of 64 x 8 bf16: 112 and 197 us instead of 31 and 67)
        if (s.lx * v * es < 64 && s.slabs > 1) break;
        // narrower while workgroups are fewer than CUs, down to 128 bytes a row:
        // 4 samples of 64 rows of 16 x 64 bf16 6.6 us forward, whole slabs 7.6;
        // going on to twice the CUs, 16 of 64 rows of 32 x 64 15.0 instead of
        // 12.5 backward
        while (samples * s.slabs < 256 && s.gs > 1) {
          const int half = widest_slab(s.D, s.G, v, s.lx / 2);
          if (half == 0 || half * s.D * es < 128) break;
          take_slab(s, half, v, threads);
        }
        s.ty = std::min(s.ty, std::max(1, s.S));
        s.threads = std::min(threads, round64(static_cast<int64_t>(s.lx) * s.ty));
        // One row a thread is the quickest to answer, and cuts large inputs
        // into rows of little more than a line: 400 samples of 16 rows of 8 x 64
        // bf16 take 9.7 and 16 us, 13 and 20 with several rows a thread; 1000
        // of 12 rows of 16 x 64, 25 and 38 against 17 and 35.
        if (P == 1 && alone <= 256 && samples * s.slabs > 4096) continue;
        // Sums by channel (groups that cut vectors) on too few CUs take longer
        // than a second launch: 1 x 256 rows of 50 x 100 bf16 22 us forward,
        // split 16; with whole vectors, 40 x 128, 10.5 against 15.
        if (!p.whole && samples * s.slabs < 64 && bytes > (int64_t(1) << 20)) break;
        p.kind = P == 1 ? NormPlan::kRow : NormPlan::kResident;
        s.across = static_cast<int>(std::min<int64_t>(samples, std::max(1, (backward ? 1024 : 8192) / s.slabs)));
        break;
      }
    }
  }
  if (p.kind != NormPlan::kSplit) {
    const int q = p.kind == NormPlan::kTokens ? Q : 1, sets = backward ? 2 * q : q;
    take_team(s, sets * s.sub * s.gs);
    const size_t flat = static_cast<size_t>(s.sub) * s.ty * s.lx;
    size_t floats = sets * flat * (p.whole ? 1 : v) + (backward ? 4 : 2) * static_cast<size_t>(q) * s.sub * s.gs;
    if (backward) floats = std::max(floats, flat * v);
    p.lds = floats * 4;
    p.rows = s.across;
    p.workspace = backward && s.across > 1 ? static_cast<size_t>(s.across) * channels * 8 : 0;
    return p;
  }
  // Split: ranges of rows over many workgroups. Groups wider than a workgroup's
  // lanes as well, cut into pieces: 4000 rows of 5000 FP32 channels in one group
  // take 52 us forward and 62 backward, 70 and 51 thousand by one workgroup.
  if (wide) {
    cut_group(s, v);
  } else {
    int gs = widest_slab(s.D, s.G, v, std::max(alone, 32));  // 512 bytes of a row, or one group
    if (gs == 0) gs = widest_slab(s.D, s.G, v, 1024);
    take_slab(s, gs, v, 256);
    if (s.lx > 256) take_slab(s, s.gs, v, round64(s.lx));
  }
  take_team(s, s.gs);
  const int64_t tile = 8 * static_cast<int64_t>(s.ty);
  const int64_t want = std::max<int64_t>(1, 2048 / std::max<int64_t>(1, samples * s.slabs));
  const int64_t tiles = std::max<int64_t>(1, (rows + tile - 1) / tile);
  const int64_t per = (tiles + want - 1) / want;  // tiles of a range
  s.range = static_cast<int>(std::min<int64_t>(per * tile, INT32_MAX));
  s.across = static_cast<int>(std::max<int64_t>(1, (rows + s.range - 1) / s.range));
  p.lds = (static_cast<size_t>(s.ty) * s.lx * v + s.gs) * 4;
  p.rows = samples * s.across;
  p.workspace = static_cast<size_t>(p.rows) * ((backward ? channels : 0) + (wide ? s.slabs : groups)) * 8;
  return p;
}

}  // namespace fftmv
