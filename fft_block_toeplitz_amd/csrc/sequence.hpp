// Interface between the C entry points of the sequence operators
// (sequence.cpp) and their kernels (recurrence*.hip, group_norm*.hip), and
// the element arithmetic that the kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fftmv.h"

namespace fftmv {

// one translation unit per direction and element type
hipError_t launch_recurrence_forward_f32(const fftmv_recurrence_t &r, hipStream_t s);
hipError_t launch_recurrence_forward_bf16(const fftmv_recurrence_t &r, hipStream_t s);
hipError_t launch_recurrence_forward_f16(const fftmv_recurrence_t &r, hipStream_t s);
hipError_t launch_recurrence_backward_f32(const fftmv_recurrence_t &r, hipStream_t s);
hipError_t launch_recurrence_backward_bf16(const fftmv_recurrence_t &r, hipStream_t s);
hipError_t launch_recurrence_backward_f16(const fftmv_recurrence_t &r, hipStream_t s);
hipError_t launch_recurrence_step(const fftmv_recurrence_step_t &r, hipStream_t s);
hipError_t launch_group_norm_forward_f32(const fftmv_group_norm_t &g, hipStream_t s);
hipError_t launch_group_norm_forward_bf16(const fftmv_group_norm_t &g, hipStream_t s);
hipError_t launch_group_norm_forward_f16(const fftmv_group_norm_t &g, hipStream_t s);
hipError_t launch_group_norm_backward_f32(const fftmv_group_norm_t &g, hipStream_t s);
hipError_t launch_group_norm_backward_bf16(const fftmv_group_norm_t &g, hipStream_t s);
hipError_t launch_group_norm_backward_f16(const fftmv_group_norm_t &g, hipStream_t s);

using bf16 = __bf16;
using f16 = _Float16;

// --------------------------------------------------------- vectors of 16 bytes
// VEC neighbouring channels of one row. A row starts at any element address;
// gfx950 takes 16-byte global accesses at any alignment, so odd channel
// counts and strides keep the wide loads.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
// VEC elements as words, for the widths that one access moves whole
template <int BYTES>
struct Words {
  using type = u32x4_any;
};
template <>
struct Words<8> {
  using type = u32x2_any;
};

template <typename T, int VEC>
struct Vec {
  T v[VEC];
  __device__ __forceinline__ float operator[](int e) const { return static_cast<float>(v[e]); }
};

template <typename T>
constexpr int kVec = 16 / sizeof(T);

template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> load_vec(const T *p) {
  if constexpr (VEC * sizeof(T) >= 8) {
    return __builtin_bit_cast(Vec<T, VEC>, *reinterpret_cast<const typename Words<VEC * sizeof(T)>::type *>(p));
  } else {
    Vec<T, VEC> r;
#pragma unroll
    for (int e = 0; e < VEC; ++e) r.v[e] = p[e];
    return r;
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[VEC], bool streamed = true) {
  Vec<T, VEC> r;
#pragma unroll
  for (int e = 0; e < VEC; ++e) r.v[e] = static_cast<T>(f[e]);
  if constexpr (VEC * sizeof(T) >= 8) {
    // streamed past the caches: no kernel here reads its own output, and the
    // inputs' lines that two blocks of channels share stay longer (8192 x 4096
    // bf16 normalised in 36 us, through the caches 39)
    using W = typename Words<VEC * sizeof(T)>::type;
    if (streamed)
      __builtin_nontemporal_store(__builtin_bit_cast(W, r), reinterpret_cast<W *>(p));
    else
      *reinterpret_cast<W *>(p) = __builtin_bit_cast(W, r);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) p[e] = r.v[e];
  }
}

// Hides where a value came from, so that what was computed from it before is
// computed again instead of kept: what a thread's 32 elements became takes 32
// registers, an exponential more where it is computed again.
template <typename T, int VEC, int N>
__device__ __forceinline__ void forget(Vec<T, VEC> (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (VEC * sizeof(T) >= 8) {
      auto w = __builtin_bit_cast(typename Words<VEC * sizeof(T)>::type, v[i]);
      asm volatile("" : "+v"(w));
      v[i] = __builtin_bit_cast(Vec<T, VEC>, w);
    }
  }
}

// Keeps the compiler from starting on further rows' exponentials before a row
// is done: it would hold them all, and spill.
__device__ __forceinline__ void row_done() { __builtin_amdgcn_sched_barrier(0); }

// ------------------------------------------------ terms of the recurrence
// a = the decay, rest = 1 - a, slope = da/dg, each to a few ulp of FP32.
// sigmoid: with t = exp(-|g|) <= 1 nothing overflows, 1 - a comes from t
// without cancellation (a gate of 10 leaves 1 - a = 4.5e-5, which 1.0f - a
// would hold to 3 digits only), and a NaN stays one.
struct Terms {
  float a, rest, slope;
};

// exp(v). FP32 elements take the library's (1 ulp); for 16-bit ones, whose
// v is known to 2^-11 of itself at best, the hardware's exp2 of the once
// rounded v log2(e), off by |v| 2^-24 relative, costs a quarter as much.
template <typename T>
__device__ __forceinline__ float exp_of(float v) {
  if constexpr (sizeof(T) == 4) return expf(v);
  return __builtin_amdgcn_exp2f(1.44269504088896341f * v);
}

// 1 / v, v in [1, 1e38]. For 16-bit elements the hardware's reciprocal (1 ulp). FP32
// ones take a step of Newton's iteration behind it, which leaves half an ulp,
// the quotient's own rounding: a decay's error enters once a step, and with the
// bare reciprocal the gradient of h0 over 1000 steps was off by 3.2e-7 instead
// of 2.4e-7. (8 x 1000 x 5000 FP32 forward: 119 us bare, 122 so, 135 with the
// division.)
template <typename T>
__device__ __forceinline__ float inverse_of(float v) {
  const float r = __builtin_amdgcn_rcpf(v);
  if constexpr (sizeof(T) == 4) return fmaf(r, fmaf(-v, r, 1.0f), r);
  return r;
}

template <typename T, int DECAY>
__device__ __forceinline__ Terms decay_terms(float g) {
  Terms r;
  if constexpr (DECAY == FFTMV_DECAY_SIGMOID) {
    const float t = exp_of<T>(-fabsf(g));
    const float big = inverse_of<T>(1.0f + t), small = t * big;
    r.a = g >= 0.0f ? big : small;
    r.rest = g >= 0.0f ? small : big;
    r.slope = big * small;
  } else if constexpr (DECAY == FFTMV_DECAY_EXP) {
    r.a = exp_of<T>(g);
    r.rest = -expm1f(g);
    r.slope = r.a;
  } else {
    r.a = g;
    r.rest = 1.0f - g;
    r.slope = 1.0f;
  }
  return r;
}

// u, the drive of one step.
template <int DRIVE>
__device__ __forceinline__ float drive_of(const Terms &t, float x) {
  return DRIVE == FFTMV_DRIVE_COMPLEMENT ? t.rest * x : x;
}

// ------------------------------------------------------------- activations
// exp(v), -128 <= v <= 87, to an ulp and a half (0 below -87): the hardware's exp2 of the rounded
// v log2(e), made good for what that rounding left off. (16000 tokens of
// 5000 channels FP32 with SiLU: 138 us forward, 144 with the library's expf.)
__device__ __forceinline__ float exp_near(float v) {
  constexpr float kLog2e = 1.44269502162933349609375f, kRest = 1.92596298909109e-8f;  // their sum is log2(e)
  const float w = kLog2e * v, off = fmaf(kRest, v, fmaf(kLog2e, v, -w));
  const float e = __builtin_amdgcn_exp2f(w);
  return fmaf(e, 0.693147180559945309f * off, e);
}

// Phi(z), the normal distribution's integral, and exp(-z^2 / 2) beside it:
//   Phi(-|z|) = erfc(x) / 2,  x = |z| / sqrt(2),  erfc(x) = exp(-x^2) t R(t),  t = 1 / (1 + k x),
// R a polynomial fitted to exp(x^2) erfc(x) / t with the least relative error.
// 16-bit elements: k = 0.33, x in [0, 10], 1.2e-7; in FP32 arithmetic 6e-7 up to
// |z| = 3, and beyond it -z^2 / 2, rounded before exp2, makes that grow as z^2, to
// 8e-6 at 12.5, all far below their type's rounding. (The library's erfc costs
// three times as much: a GELU forward of 32768 x 320 fp16 was bound by it.)
// FP32 elements: up to |z| = 1 Phi = 1/2 + z P(z^2), 5.3e-8, which loses nothing
// to 1 - Phi(-|z|); from there k = 0.4, 1.3e-7, with the rounding of z^2 made good
// in the exponential. (2 x 16384 x 320: 43 us forward, 61 backward; with the library's
// erfc 48 and 71; by the 16-bit elements' way 41 and 58, dx 1.05e-7 off, not 8.3e-8.)
constexpr float kTail16[] = {0.18635779619216919f,  0.18295612931251526f, 0.20122270286083221f,  0.047224629670381546f,
                             0.40849229693412781f, -0.35114115476608276f, 0.46023201942443848f, -0.13534443080425262f};
constexpr float kTail32[] = {0.2256411910057068f,   0.22646473348140717f, 0.2002403885126114f,  0.2082897424697876f,
                             0.01665278896689415f, 0.23601338267326355f, -0.11349567770957947f};
constexpr float kCentre32[] = {0.3989422619342804f, -0.06648958474397659f, 0.009967196732759476f,
                               -0.001169353723526001f, 9.423524170415476e-05f};
template <int N>
__device__ __forceinline__ float polynomial(const float (&c)[N], float t) {
  float p = c[N - 1];
#pragma unroll
  for (int i = N - 2; i >= 0; --i) p = fmaf(p, t, c[i]);
  return p;
}

struct Normal {
  float phi, bell;
};
template <typename T>
__device__ __forceinline__ Normal normal_of(float z) {
  Normal r;
  if constexpr (sizeof(T) == 4) {
    const float a = fminf(fabsf(z), 16.0f);  // Phi has reached its ends before
    const float w = a * a, e = exp_near(-0.5f * w);
    r.bell = fmaf(e, -0.5f * fmaf(a, a, -w), e);
    const float t = inverse_of<T>(fmaf(0.28284271247461901f, a, 1.0f));
    const float half = 0.5f * r.bell * (polynomial(kTail32, t) * t);
    float centre = fmaf(z, polynomial(kCentre32, w), 0.5f), side = z < 0.0f ? half : 1.0f - half;
    asm volatile("" : "+v"(centre), "+v"(side));  // both and no branch: a wave has lanes on either side
    r.phi = a < 1.0f ? centre : side;
  } else {
    const float x = 0.70710678118654752f * fabsf(z);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.33f, x, 1.0f));
    r.bell = __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);
    const float half = 0.5f * r.bell * polynomial(kTail16, t) * t;
    r.phi = z < 0.0f ? half : 1.0f - half;
  }
  return r;
}

// The logistic function of z and its complement. 16-bit elements take the
// hardware's exp2 of the once rounded argument, |z| 2^-24 off relative. For FP32
// ones e = exp(-z) is right to 3 2^-24, and p = 1 / (1 + e) to 5, whatever z. The
// complement is 1 - p, exact as far as p is, or, where that cancels, e p. (Beyond
// |z| = 87, where FP32 ends, p stays what it is there: 1, or 1.6e-38.)
struct Logistic {
  float p, rest;
};
template <typename T>
__device__ __forceinline__ Logistic logistic(float z) {
  Logistic r;
  if constexpr (sizeof(T) == 4) {
    const float e = exp_near(-__builtin_amdgcn_fmed3f(z, -87.0f, 87.0f));
    r.p = inverse_of<T>(1.0f + e);
    r.rest = z > 2.0f ? e * r.p : 1.0f - r.p;
  } else {
    r.p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896341f * z));
    r.rest = 1.0f - r.p;
  }
  return r;
}

// act(z) and act'(z), z of elements of type T.
template <typename T, int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == FFTMV_ACT_SILU) {
    return z * logistic<T>(z).p;
  } else if constexpr (ACT == FFTMV_ACT_GELU) {
    return z * normal_of<T>(z).phi;
  } else {
    return z;
  }
}
template <typename T, int ACT>
__device__ __forceinline__ float activate_slope(float z) {
  if constexpr (ACT == FFTMV_ACT_SILU) {
    const Logistic l = logistic<T>(z);
    return fmaf(l.p * z, l.rest, l.p);
  } else if constexpr (ACT == FFTMV_ACT_GELU) {
    const Normal n = normal_of<T>(z);
    return fmaf(0.39894228040143268f * z, n.bell, n.phi);
  } else {
    return 1.0f;
  }
}

// ------------------------------------------------------------ type dispatch
template <typename F>
hipError_t by_dtype(int dtype, F f) {
  if (dtype == FFTMV_BF16) return f(bf16{});
  if (dtype == FFTMV_F16) return f(f16{});
  return f(float{});
}
template <int V>
struct Const {
  static constexpr int value = V;
};
template <typename F>
hipError_t by_three(int v, F f) {
  if (v == 0) return f(Const<0>{});
  if (v == 1) return f(Const<1>{});
  return f(Const<2>{});
}
template <typename F>
hipError_t by_two(int v, F f) {
  return v == 0 ? f(Const<0>{}) : f(Const<1>{});
}

}  // namespace fftmv
