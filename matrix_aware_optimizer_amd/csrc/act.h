// Activations of a gated block and where the block's outputs go.
//
//   silu       a(x) = x s(x)              s(x) = 1 / (1 + exp(-x))
//   gelu       a(x) = x P(x)              P(x) = erfc(-x / sqrt 2) / 2, the normal distribution
//   gelu_tanh  a(x) = x s(2 z)            z = sqrt(2 / pi) (x + 0.044715 x^3); (1 + tanh z) / 2 = s(2 z)
//   relu       a(x) = max(x, 0)
// in fp32 throughout.  Written with s and erfc and not with 1 + tanh or 1 + erf, whose sum
// loses its digits for negative x.
#pragma once

#include "common.h"

namespace muon {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2_t x = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2_t));
}

// 16 bytes at p; PASSING: past the caches' order of keeping.  The outputs of products on large tiles
// pass, so that the operands' panels stay in L2 (measured then: 2048 x 14336 x 4096 int8 gated 253 -> 245 us, 1999
// x 4096 x 14336 140 -> 134, weight gradients 857 -> 849).  Not what the next kernel reads (dg, du),
// and not rows that end inside a cache line, whose halves would pass one by one (weight gradients
// of 14335 x 4095 from 64 tokens 190 -> 235).  A choice of the type: as a branch in the store it costs
// more than it gains (136 against 129 us for the second).
template <bool PASSING, typename T>
__device__ __forceinline__ void store16_as(T* p, const uint4& v) {
  typename Unaligned<T>::x4 w;
  w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  if constexpr (PASSING) __builtin_nontemporal_store(w, reinterpret_cast<typename Unaligned<T>::x4*>(p));
  else *reinterpret_cast<typename Unaligned<T>::x4*>(p) = w;
}
inline bool whole_lines(const void* p, int64_t pitch_bytes) { return (reinterpret_cast<uintptr_t>(p) | uintptr_t(pitch_bytes)) % 128 == 0; }
// N consecutive outputs at p, rounded once to the stored type
template <int N, bool PASSING>
__device__ __forceinline__ void store_n(bf16_t* p, const float (&v)[N]) {
  if constexpr (N == 8)
    store16_as<PASSING>(p, make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])));
  else if constexpr (N == 4) store8(p, make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])));
  else p[0] = f32_to_bf16(v[0]);
}
template <int N, bool PASSING>
__device__ __forceinline__ void store_n(float* p, const float (&v)[N]) {
  if constexpr (N == 1) p[0] = v[0];
  else
#pragma unroll
    for (int k = 0; k < N; k += 4)
      store16_as<PASSING>(p + k, make_uint4(__float_as_uint(v[k]), __float_as_uint(v[k + 1]), __float_as_uint(v[k + 2]), __float_as_uint(v[k + 3])));
}
template <int N>
__device__ __forceinline__ void load_n(const bf16_t* p, float (&v)[N]) {
  if constexpr (N == 8) {
    const uint4 r = load16(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float((k & 1) ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
  } else if constexpr (N == 4) {
    const uint2 r = load8(p);
    v[0] = __uint_as_float(r.x << 16); v[1] = __uint_as_float(r.x & 0xffff0000u);
    v[2] = __uint_as_float(r.y << 16); v[3] = __uint_as_float(r.y & 0xffff0000u);
  } else {
    v[0] = bf16_to_f32(p[0]);
  }
}
template <int N>
__device__ __forceinline__ void load_n(const float* p, float (&v)[N]) {
  if constexpr (N == 1) v[0] = p[0];
  else
#pragma unroll
    for (int k = 0; k < N; k += 4) {
      const uint4 r = load16(p + k);
      v[k] = __uint_as_float(r.x); v[k + 1] = __uint_as_float(r.y); v[k + 2] = __uint_as_float(r.z); v[k + 3] = __uint_as_float(r.w);
    }
}

// The logistic function; 1 / (1 + inf) = 0 for large negative x.  exp(-x) = 2^t with t = -x log2 e rounded
// is off by up to 1.5 |x| 2^-24 of itself, 2^-17 at -80, which the 2^-8 of a bf16 output covers.  FULL, for what is
// stored in fp32: r = -x - t ln 2 is what the rounding left, and s moves by -s (1 - s) r (its square is under
// 2^-34); |x| is cut at 200, where s is 0 or 1.
// silu of gates down to -80 into fp32: 3.2 units of 2^-24 instead of 61, for 2 to 4% of int8 gated 2048 x 14336 x 4096 into
// fp32 (239 to 248 -> 245 to 252 us).
template <bool FULL>
__device__ __forceinline__ float logistic(float x) {
  constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147182f, kLn2Rest = -1.90465421e-9f;   // ln 2 in two parts
  if (!FULL) return __builtin_amdgcn_rcpf(1.0f + __expf(-x));
  const float n = __builtin_amdgcn_fmed3f(-x, -200.0f, 200.0f), t = n * kLog2e;
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
  const float r = fmaf(t, -kLn2Rest, fmaf(t, -kLn2, n));
  return fmaf(fmaf(s, s, -s), r, s);
}

constexpr float kTanhA = 0.044715f, kTanh2C = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kRsqrt2 = 0.70710678118654752f, kRsqrt2Pi = 0.39894228040143268f;

// a(x); SLOPE: a'(x) too
template <bool SLOPE, bool FULL>
__device__ __forceinline__ float activate(int act, float x, float& slope) {
  switch (act) {
    case MUON_ACT_SILU: {
      const float s = logistic<FULL>(x);
      if (SLOPE) slope = s * fmaf(x, 1.0f - s, 1.0f);
      return x * s;
    }
    case MUON_ACT_GELU: {
      const float p = 0.5f * erfcf(-kRsqrt2 * x);
      if (SLOPE) slope = fmaf(x * kRsqrt2Pi, __expf(-0.5f * x * x), p);
      return x * p;
    }
    case MUON_ACT_GELU_TANH: {
      // the square is cut so that the slope of a saturated gate is 0 times a number, not 0 times infinity
      const float x2 = fminf(x * x, 1e30f), s = logistic<FULL>(kTanh2C * x * fmaf(kTanhA, x2, 1.0f));
      if (SLOPE) slope = fmaf(x * s * (1.0f - s), kTanh2C * fmaf(3.0f * kTanhA, x2, 1.0f), s);
      return x * s;
    }
    default:   // max(x, 0), with NaN staying NaN; the slope at 0 is 0
      if (SLOPE) slope = x > 0.0f ? 1.0f : 0.0f;
      return x <= 0.0f ? 0.0f : x;
  }
}

inline bool valid_act(int a) { return a >= MUON_ACT_SILU && a <= MUON_ACT_RELU; }

// h = act(g) u of two sums, in H and (for the backward) g and u in G and U.  SCALED: the sums
// are of int8 codes, g = float(sum) (sa sg), with one rounding of the integer, one of the
// product of the scales and one of theirs.
template <typename TC, bool SCALED, bool PASSING = false>
struct GluOut {
  using sum_t = std::conditional_t<SCALED, int, float>;
  static constexpr int E = 16 / int(sizeof(TC));
  TC* H;
  bf16_t *G, *U;
  int64_t ldh, ldg, width;
  int act;
  const float *sa, *sg, *su;

  template <int N> struct Cols { float g[SCALED ? N : 1], u[SCALED ? N : 1]; };
  template <int N> struct Pre { float a; };
  GluOut<TC, SCALED, SCALED> passing() const { return {H, G, U, ldh, ldg, width, act, sa, sg, su}; }
  bool lines() const { return whole_lines(H, ldh * int64_t(sizeof(TC))); }
  __device__ __forceinline__ GluOut at(int) const { return *this; }
  template <int N> __device__ __forceinline__ Cols<N> cols(int64_t col) const {
    Cols<N> c;
    if constexpr (SCALED)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        c.g[k] = sg[min(col + k, width - 1)];
        c.u[k] = su[min(col + k, width - 1)];
      }
    return c;
  }
  template <int N> __device__ __forceinline__ Pre<N> pre(int64_t row, int64_t) const { return {SCALED ? sa[row] : 0.0f}; }
  template <int N>
  __device__ __forceinline__ void store(int64_t row, int64_t col, const sum_t (&v)[2][N], const Cols<N>& c, const Pre<N>& p) const {
    float g[N], u[N], h[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if constexpr (SCALED) {
        g[k] = float(v[0][k]) * (p.a * c.g[k]);
        u[k] = float(v[1][k]) * (p.a * c.u[k]);
      } else {
        g[k] = v[0][k];
        u[k] = v[1][k];
      }
    }
    float none;
    switch (act) {   // outside the loop: one uniform branch
#define MUON_ACT_CASE(A)                                                      \
  case A:                                                                     \
    _Pragma("unroll") for (int k = 0; k < N; ++k) h[k] = activate<false, std::is_same_v<TC, float>>(A, g[k], none) * u[k]; \
    break;
      MUON_ACT_CASE(MUON_ACT_SILU)
      MUON_ACT_CASE(MUON_ACT_GELU)
      MUON_ACT_CASE(MUON_ACT_GELU_TANH)
      default:
        MUON_ACT_CASE(MUON_ACT_RELU)
#undef MUON_ACT_CASE
    }
    store_n<N, PASSING>(H + row * ldh + col, h);
    if (!SCALED && G != nullptr) {
      store_n<N, false>(G + row * ldg + col, g);
      store_n<N, false>(U + row * ldg + col, u);
    }
  }
};

}  // namespace muon
