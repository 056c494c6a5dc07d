// 8-bit floating point matrices with a power-of-two scale for each row's group
// of 128 columns: the quantiser and the product C = beta C + alpha A B^T.
//
// Format.  A matrix [rows][cols] is held as codes q [rows][ldq] (one byte, OCP
// e4m3 or e5m2, zero from cols up to the next multiple of 128) and scale bytes
// (E8M0: byte s stands for 2^(s - 127)).  The scale bytes of four consecutive
// groups of one row form a 32-bit word, and the words lie group-major:
// byte (row, group g) at ((g / 4) * R4 + row) * 4 + g % 4, R4 = rows rounded up
// to 4.  A tile of a product then reads the words of its rows as one contiguous
// run per 512 columns, and the matrix instruction takes the byte as it is.
#include <algorithm>

#include "common.h"
#include "gemm.h"

namespace muon {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// 32 bytes of a matrix operand from two 16-byte reads
__device__ __forceinline__ i32x8_t join(const u32x4_t (&v)[2]) {
  i32x8_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = int(v[0][i]);
    r[4 + i] = int(v[1][i]);
  }
  return r;
}

constexpr int kGroup = MUON_FP8_GROUP;   // columns under one scale

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t scale_rows(int64_t rows) { return ceil_div(rows, 4) * 4; }

// ---------------------------------------------------------------------------
// Quantiser
// ---------------------------------------------------------------------------
// amax = m 2^E (1 <= m < 2): the smallest e with amax <= MAX 2^e, MAX = 1.75 2^8
// (e4m3) or 1.75 2^15 (e5m2), is E - 8 (or 15), plus one when m > 1.75.  In bits:
// the biased exponent field less that, plus one when the fraction is over 0x600000.
// The byte is at least 1, so that 2^e is a normal fp32.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  constexpr int drop = FMT == MUON_FP8_E4M3 ? 8 : 15;
  if (amax_bits == 0) return 127;
  const int b = int(amax_bits >> 23) - drop + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return uint32_t(b < 1 ? 1 : b);
}
// 2^e as the scaled conversions take it
__device__ __forceinline__ float scale_float(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}

// maximum over the 16 lanes of a DPP row, in every lane (rotations by 8, 4, 2, 1)
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max_u32(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x128, 0xf, 0xf, true)));
  v = max_u32(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x124, 0xf, 0xf, true)));
  v = max_u32(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x122, 0xf, 0xf, true)));
  v = max_u32(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x121, 0xf, 0xf, true)));
  return v;
}

// A thread's 8 x 8 entries.  Maxima are of |x| as bits (of the fp32 value); with FINITE
// infinities and NaN count as 0, without it they show as 0x7f800000 or more.  The codes
// come from the scaled conversions, x 2^-e rounded once to nearest even; e4m3 has no
// infinity: an infinite entry becomes NaN there, as NaN does.
typedef short s16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

template <typename T> struct Cells;

// bf16 stays packed: two columns per register
template <> struct Cells<bf16_t> {
  uint32_t w[8][4];
  static constexpr int COLS = 4;   // registers of column maxima

  __device__ __forceinline__ void load(int p, const bf16_t* src, int64_t left) {
    if (left >= 8) {
      const uint4 r = load16(src);
      w[p][0] = r.x; w[p][1] = r.y; w[p][2] = r.z; w[p][3] = r.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = 2 * j < left ? src[2 * j] : 0u, hi = 2 * j + 1 < left ? src[2 * j + 1] : 0u;
        w[p][j] = lo | (hi << 16);
      }
    }
  }
  template <bool FINITE> __device__ __forceinline__ uint32_t abs2(int p, int j) const {
    uint32_t a = w[p][j] & 0x7fff7fffu;
    if (FINITE) {
      if ((a & 0xffffu) >= 0x7f80u) a &= 0xffff0000u;
      if (a >= 0x7f800000u) a &= 0xffffu;
    }
    return a;
  }
  template <bool FINITE> __device__ __forceinline__ uint32_t row(int p) const {
    const uint32_t m = max_u16x2(max_u16x2(abs2<FINITE>(p, 0), abs2<FINITE>(p, 1)),
                                 max_u16x2(abs2<FINITE>(p, 2), abs2<FINITE>(p, 3)));
    return max_u32(m << 16, m & 0xffff0000u);
  }
  template <bool FINITE> __device__ __forceinline__ uint32_t col(int c) const {
    uint32_t m = abs2<FINITE>(0, c);
#pragma unroll
    for (int p = 1; p < 8; ++p) m = max_u16x2(m, abs2<FINITE>(p, c));
    return m;
  }
  __device__ __forceinline__ static uint32_t join(uint32_t a, uint32_t b) { return max_u16x2(a, b); }
  // maximum of column j from the registers of column maxima
  __device__ __forceinline__ static uint32_t of_column(const uint32_t (&m)[4], int j) {
    return (j & 1) ? m[j >> 1] & 0xffff0000u : m[j >> 1] << 16;
  }
  template <int FMT> __device__ __forceinline__ static uint32_t codes(uint32_t a, uint32_t b, float scale) {
    s16x2_t r = {0, 0};
    if constexpr (FMT == MUON_FP8_E4M3) {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, a), scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, b), scale, true);
    } else {
      r = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(r, __builtin_bit_cast(bf16x2_t, a), scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(r, __builtin_bit_cast(bf16x2_t, b), scale, true);
    }
    return __builtin_bit_cast(uint32_t, r);
  }
  template <int FMT> __device__ __forceinline__ uint2 row_codes(int p, float s) const {
    return make_uint2(codes<FMT>(w[p][0], w[p][1], s), codes<FMT>(w[p][2], w[p][3], s));
  }
  template <int FMT> __device__ __forceinline__ uint2 col_codes(int j, float s) const {
    uint32_t v[4];   // rows 2 q, 2 q + 1 of column j
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v[q] = (j & 1) ? __builtin_amdgcn_perm(w[2 * q + 1][j >> 1], w[2 * q][j >> 1], 0x07060302u)
                     : __builtin_amdgcn_perm(w[2 * q + 1][j >> 1], w[2 * q][j >> 1], 0x05040100u);
    return make_uint2(codes<FMT>(v[0], v[1], s), codes<FMT>(v[2], v[3], s));
  }
};

template <> struct Cells<float> {
  float v[8][8];
  static constexpr int COLS = 8;

  __device__ __forceinline__ void load(int p, const float* src, int64_t left) {
    if (left >= 8) {
      const uint4 a = load16(src), b = load16(src + 4);
      v[p][0] = __uint_as_float(a.x); v[p][1] = __uint_as_float(a.y); v[p][2] = __uint_as_float(a.z); v[p][3] = __uint_as_float(a.w);
      v[p][4] = __uint_as_float(b.x); v[p][5] = __uint_as_float(b.y); v[p][6] = __uint_as_float(b.z); v[p][7] = __uint_as_float(b.w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[p][j] = j < left ? src[j] : 0.0f;
    }
  }
  template <bool FINITE> __device__ __forceinline__ uint32_t abs1(int p, int j) const {
    const uint32_t a = __float_as_uint(v[p][j]) & 0x7fffffffu;
    return FINITE && a >= 0x7f800000u ? 0u : a;
  }
  template <bool FINITE> __device__ __forceinline__ uint32_t row(int p) const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max_u32(m, abs1<FINITE>(p, j));
    return m;
  }
  template <bool FINITE> __device__ __forceinline__ uint32_t col(int j) const {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) m = max_u32(m, abs1<FINITE>(p, j));
    return m;
  }
  __device__ __forceinline__ static uint32_t join(uint32_t a, uint32_t b) { return max_u32(a, b); }
  __device__ __forceinline__ static uint32_t of_column(const uint32_t (&m)[8], int j) { return m[j]; }
  template <int FMT> __device__ __forceinline__ static uint32_t codes(float a, float b, float c, float d, float scale) {
    s16x2_t r = {0, 0};
    if constexpr (FMT == MUON_FP8_E4M3) {
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, true);
    } else {
      r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, a, b, scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, c, d, scale, true);
    }
    return __builtin_bit_cast(uint32_t, r);
  }
  template <int FMT> __device__ __forceinline__ uint2 row_codes(int p, float s) const {
    return make_uint2(codes<FMT>(v[p][0], v[p][1], v[p][2], v[p][3], s), codes<FMT>(v[p][4], v[p][5], v[p][6], v[p][7], s));
  }
  template <int FMT> __device__ __forceinline__ uint2 col_codes(int j, float s) const {
    return make_uint2(codes<FMT>(v[0][j], v[1][j], v[2][j], v[3][j], s), codes<FMT>(v[4][j], v[5][j], v[6][j], v[7][j], s));
  }
};

struct QuantArgs {
  const void* x;
  int64_t rows, cols, ldx;
  uint8_t *q, *s, *qt, *st;   // q/s or qt/st may be null
  int64_t ldq, ldqt;
};

// One workgroup per 128 x 128 tile, read once: each thread holds an 8 x 8 block
// (rows 8 (t / 16) .., columns 8 (t % 16) ..), so that row groups, column groups
// and the whole tile's maximum all come from registers (16 lanes of one wave share
// a row; columns meet in LDS), and the transposed codes leave through a 16 KB tile of
// LDS whose 8-byte chunks are XOR-swizzled.  Bound by memory: 2 (bf16) or 4 bytes read
// and 1 or 2 written per entry.  4096 x 14336 bf16 to both orientations, inputs from
// memory: 54 us, 4.3 TB/s against 4.9 of a large copy (with unpacked maxima and separate
// multiplications 63 us); 2305 x 4096 fp32 in blocks: 12 us.
template <typename T, int FMT, bool BLOCK>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(QuantArgs g) {
  using C_ = Cells<T>;
  constexpr int NC = C_::COLS;
  __shared__ __attribute__((aligned(16))) char tile[128 * 128];
  __shared__ uint32_t colmax[4][16 * NC];
  const int t = threadIdx.x, cg = t & 15, rg = t >> 4, wave = t >> 6;
  const int64_t kb = blockIdx.x, rb = blockIdx.y;
  const int64_t c0 = kb * 128 + 8 * cg, r0 = rb * 128 + 8 * rg;
  C_ x;
#pragma unroll
  for (int p = 0; p < 8; ++p)
    x.load(p, static_cast<const T*>(g.x) + (r0 + p) * g.ldx + c0, r0 + p < g.rows ? g.cols - c0 : 0);
  const bool rows_out = g.q != nullptr, cols_out = g.qt != nullptr;
  uint32_t rm[8], cm[NC], all = 0;
  auto maxima = [&](auto finite) __attribute__((always_inline)) {
    constexpr bool FINITE = decltype(finite)::value;
    all = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      rm[p] = x.template row<FINITE>(p);
      all = max_u32(all, rm[p]);
    }
    if (!BLOCK && cols_out)
#pragma unroll
      for (int c = 0; c < NC; ++c) cm[c] = x.template col<FINITE>(c);
  };
  maxima(std::false_type{});
  if (__any(all >= 0x7f800000u)) maxima(std::true_type{});   // infinities or NaN: leave them out
  if (BLOCK) {
    all = row16_max(all);
    all = max_u32(all, uint32_t(__shfl_xor(int(all), 16, kWave)));
    all = max_u32(all, uint32_t(__shfl_xor(int(all), 32, kWave)));
    if ((t & 63) == 0) colmax[wave][0] = all;
    __syncthreads();
    all = max_u32(max_u32(colmax[0][0], colmax[1][0]), max_u32(colmax[2][0], colmax[3][0]));
  }
  const int64_t kbs = (g.cols + 127) / 128, rbs = (g.rows + 127) / 128;
  if (rows_out) {
    const int64_t R4 = (g.rows + 3) / 4 * 4;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const uint32_t byte = scale_byte<FMT>(BLOCK ? all : row16_max(rm[p]));
      const int64_t r = r0 + p;
      if (r < g.rows) *reinterpret_cast<uint2*>(g.q + r * g.ldq + c0) = x.template row_codes<FMT>(p, scale_float(byte));
      if (cg == 0 && r < R4) {
        uint8_t* dst = g.s + ((kb >> 2) * R4 + r) * 4;
        dst[kb & 3] = r < g.rows ? byte : 127;
        if (kb == kbs - 1)   // the last word's unused bytes
          for (int64_t f = (kb & 3) + 1; f < 4; ++f) dst[f] = 127;
      }
    }
  }
  if (!cols_out) return;
  if (!BLOCK) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      cm[c] = C_::join(cm[c], uint32_t(__shfl_xor(int(cm[c]), 16, kWave)));
      cm[c] = C_::join(cm[c], uint32_t(__shfl_xor(int(cm[c]), 32, kWave)));
      if ((t & 63) < 16) colmax[wave][NC * cg + c] = cm[c];
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; ++c)
      cm[c] = C_::join(C_::join(colmax[0][NC * cg + c], colmax[1][NC * cg + c]),
                       C_::join(colmax[2][NC * cg + c], colmax[3][NC * cg + c]));
  }
  const int64_t C4 = (g.cols + 3) / 4 * 4;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t byte = scale_byte<FMT>(BLOCK ? all : C_::of_column(cm, j));
    *reinterpret_cast<uint2*>(tile + (8 * cg + j) * 128 + ((rg ^ cg) << 3)) = x.template col_codes<FMT>(j, scale_float(byte));
    const int64_t c = c0 + j;
    if (rg == 0 && c < C4) {
      uint8_t* dst = g.st + ((rb >> 2) * C4 + c) * 4;
      dst[rb & 3] = c < g.cols ? byte : 127;
      if (rb == rbs - 1)
        for (int64_t f = (rb & 3) + 1; f < 4; ++f) dst[f] = 127;
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int c = (t >> 3) + 32 * h, ch = 2 * (t & 7), sw = (c >> 3) & 15;
    if (kb * 128 + c < g.cols) {
      const uint2 a = *reinterpret_cast<const uint2*>(tile + c * 128 + ((ch ^ sw) << 3));
      const uint2 b = *reinterpret_cast<const uint2*>(tile + c * 128 + (((ch + 1) ^ sw) << 3));
      *reinterpret_cast<uint4*>(g.qt + (kb * 128 + c) * g.ldqt + rb * 128 + 8 * ch) = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
}

// ---------------------------------------------------------------------------
// Product
// ---------------------------------------------------------------------------
struct Fp8GemmArgs {
  const uint8_t *A, *B;     // codes: A [m][lda], B [n][ldb]
  const uint8_t *sa, *sb;   // scale words
  void* C;
  int64_t m, n, K, lda, ldb, ldc;
  int64_t ra4, rb4;         // rows of the scale arrays
  float alpha, beta;
  int splits;               // parts of a split contraction (tile kernels): > 1 writes fp32 partial products
  float* partials;          // [splits][m][ldp]
  int64_t ldp;
};

// C[row][col .. col + 3] <- beta C + alpha acc, one rounding to the stored type
template <typename TC>
__device__ __forceinline__ void store4(const Fp8GemmArgs& g, int64_t row, int64_t col, const float acc[4]) {
  TC* dst = static_cast<TC*>(g.C) + row * g.ldc + col;
  if (col + 4 <= g.n) {
    float o[4];
    if constexpr (sizeof(TC) == 2) {
      if (g.beta != 0.0f) {
        const uint2 z = load8(dst);
        o[0] = fmaf(g.beta, __uint_as_float(z.x << 16), g.alpha * acc[0]);
        o[1] = fmaf(g.beta, __uint_as_float(z.x & 0xffff0000u), g.alpha * acc[1]);
        o[2] = fmaf(g.beta, __uint_as_float(z.y << 16), g.alpha * acc[2]);
        o[3] = fmaf(g.beta, __uint_as_float(z.y & 0xffff0000u), g.alpha * acc[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = g.alpha * acc[i];
      }
      store8(dst, make_uint2(uint32_t(f32_to_bf16(o[0])) | (uint32_t(f32_to_bf16(o[1])) << 16),
                             uint32_t(f32_to_bf16(o[2])) | (uint32_t(f32_to_bf16(o[3])) << 16)));
    } else {
      if (g.beta != 0.0f) {
        const uint4 z = load16(dst);
        o[0] = fmaf(g.beta, __uint_as_float(z.x), g.alpha * acc[0]);
        o[1] = fmaf(g.beta, __uint_as_float(z.y), g.alpha * acc[1]);
        o[2] = fmaf(g.beta, __uint_as_float(z.z), g.alpha * acc[2]);
        o[3] = fmaf(g.beta, __uint_as_float(z.w), g.alpha * acc[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = g.alpha * acc[i];
      }
      store16(dst, make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3])));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < g.n) {
        float o = g.alpha * acc[i];
        if (g.beta != 0.0f) o = fmaf(g.beta, to_f32(dst[i]), o);
        dst[i] = from_f32<TC>(o);
      }
  }
}

// Two ways to multiply.  The fp8 matrix instructions (scaled or not) line up the
// eight products of eight neighbouring k-values at the largest of them and drop
// what lies more than 13 bits below it, before anything is added in fp32: measured
// on MI355X, a Gaussian product is off by 1.5e-5 of its norm, against 2.5e-7 for
// the bf16 instructions.  For a bf16 C that is a hundredth of its own rounding
// (2^-9), and the fp8 instructions run at twice the bf16 rate, so they are used.  An
// fp32 C (a momentum that gradients are summed into) keeps what fp32 holds: its
// codes are widened to bf16 with their scale (v_cvt_scalef32_pk_bf16_*, exact) and
// multiplied on the bf16 instructions.

// eight codes times their scale, as bf16 (exact: at most four significant bits)
template <int FMT>
__device__ __forceinline__ bf16x8_t widen8(uint32_t lo, uint32_t hi, float scale) {
  uint32_t w[4];
  if constexpr (FMT == MUON_FP8_E4M3) {
    w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
    w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
    w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
    w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
  } else {
    w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, false));
    w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, true));
    w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, false));
    w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, true));
  }
  return __builtin_bit_cast(bf16x8_t, make_uint4(w[0], w[1], w[2], w[3]));
}
// 2^(s - 127) for the scale byte in the low bits of `word`
__device__ __forceinline__ float scale_value(uint32_t word) { return __uint_as_float((word & 255u) << 23); }

// Products straight from memory: no tile is staged, each wave reads 32 bytes per
// lane of 16 rows of B and of MT x 16 rows of A and multiplies them on
// v_mfma_scale_f32_16x16x128 (one instruction spans a whole group of 128, so the
// group's scales go in with it), or widened on four v_mfma_f32_16x16x32_bf16.  Bound by
// reading B: 1 x 14336 x 4096 15 us, 3.9 TB/s.  The waves of a workgroup take the groups of the
// contraction in turn and their sums meet in LDS, added in the order of the waves.
// B is the first operand: a lane holds four consecutive columns of one row of C.
template <int FA, typename TC, int MT>
__global__ __launch_bounds__(1024) void fp8_gemm_direct_kernel(Fp8GemmArgs g) {
  constexpr bool EXACT = sizeof(TC) == 4;
  extern __shared__ __attribute__((aligned(16))) float red[];   // [waves][MT * 4][64]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int r = lane & 15, kq = lane >> 4;
  const int64_t n0 = int64_t(blockIdx.x) * 16, m0 = int64_t(blockIdx.y) * (16 * MT);
  const int64_t brow = min(n0 + r, g.n - 1);
  // 16 bytes at 16 kq and at 64 + 16 kq of the group: whole 64-byte runs of a row per
  // load, the same k-values for both operands
  const uint8_t* pb = g.B + brow * g.ldb + 16 * kq;
  const uint8_t* psb = g.sb + brow * 4;
  const uint8_t* pa[MT];
  const uint8_t* psa[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t arow = min(m0 + 16 * i + r, g.m - 1);
    pa[i] = g.A + arow * g.lda + 16 * kq;
    psa[i] = g.sa + arow * 4;
  }
  f32x4_t acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t groups = g.K / kGroup;
  constexpr int U = MT == 1 ? 4 : 2;   // groups whose loads are in flight together
  for (int64_t kb0 = wave; kb0 < groups; kb0 += U * waves) {
    u32x4_t fb[U][2], fa[U][MT][2];
    int sb[U], sa[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t kb = min(kb0 + u * waves, groups - 1);   // past the end: read again, not used
      sb[u] = psb[(kb >> 2) * g.rb4 * 4 + (kb & 3)];
#pragma unroll
      for (int c = 0; c < 2; ++c) fb[u][c] = *reinterpret_cast<const u32x4_t*>(pb + kb * kGroup + 64 * c);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        sa[u][i] = psa[i][(kb >> 2) * g.ra4 * 4 + (kb & 3)];
#pragma unroll
        for (int c = 0; c < 2; ++c) fa[u][i][c] = *reinterpret_cast<const u32x4_t*>(pa[i] + kb * kGroup + 64 * c);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb0 + u * waves >= groups) break;
      bf16x8_t wb[4];
      if constexpr (EXACT) {
#pragma unroll
        for (int p = 0; p < 4; ++p)
          wb[p] = widen8<MUON_FP8_E4M3>(fb[u][p >> 1][2 * (p & 1)], fb[u][p >> 1][2 * (p & 1) + 1], scale_value(sb[u]));
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if constexpr (EXACT) {
#pragma unroll
          for (int p = 0; p < 4; ++p)
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                wb[p], widen8<FA>(fa[u][i][p >> 1][2 * (p & 1)], fa[u][i][p >> 1][2 * (p & 1) + 1], scale_value(sa[u][i])),
                acc[i], 0, 0, 0);
        } else {
          acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(fb[u]), join(fa[u][i]), acc[i], 0, FA, 0, sb[u], 0,
                                                                    sa[u][i]);
        }
      }
    }
  }
  if (waves > 1) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[((wave * MT + i) * 4 + v) * 64 + lane] = acc[i][v];
    __syncthreads();
    if (wave >= MT) return;
  }
  // wave i finishes row block i (a single wave finishes all)
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (waves > 1 && i % waves != wave) continue;
    float o[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) o[v] = acc[i][v];
    if (waves > 1) {
#pragma unroll
      for (int v = 0; v < 4; ++v) o[v] = 0.0f;
      for (int w = 0; w < waves; ++w)
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] += red[((w * MT + i) * 4 + v) * 64 + lane];
    }
    const int64_t row = m0 + 16 * i + r, col = n0 + 4 * kq;
    if (row < g.m && col < g.n) store4<TC>(g, row, col, o);
  }
}

template <int FA, typename TC, int MT>
int launch_direct(const Fp8GemmArgs& g, hipStream_t st) {
  const int64_t groups = g.K / kGroup;
  const int waves = int(std::max<int64_t>(1, std::min<int64_t>(groups / 8, 8)));   // eight groups each, up to eight waves
  const uint32_t lds = waves > 1 ? uint32_t(waves) * MT * 4 * 64 * 4 : 0;
  const dim3 grid(ceil_div(g.n, 16), ceil_div(g.m, 16 * MT));
  launch_kernel(fp8_gemm_direct_kernel<FA, TC, MT>, grid, dim3(64 * waves), lds, st, g);
  return launch_status();
}

// Tiled product.  A workgroup of four waves computes BM x BN of C.  Both operands
// come through a ring of S stages in LDS, each 64 k-values (half a group) of every
// row: 64-byte rows of four 16-byte chunks, chunk c of row r at slot
// c ^ ((r / 4) % 4), filled by global -> LDS DMA (16 bytes per lane), followed by the
// rows' scale words (4 bytes per lane).  A lane's operand is 32 bytes of one row: chunks
// h and 2 + h for half-wave h, the same k-values for both operands, so their order
// does not matter.  Per step: wait until this wave's copies of the next stage have
// landed, s_barrier (everybody's have, and everybody is done with the stage before),
// start the copy S - 1 steps ahead, read the next operands, multiply the current ones.
// Four waves of 128 x 128 (one per SIMD) read 64 KB of LDS per step of a 256 x 256 tile,
// where eight of 64 x 128 would read 96 KB: with the 34 KB written, 76% instead of all of
// what LDS moves in the step's 1024 matrix cycles.
template <int BM_, int BN_, int WM_, int WN_, int S_>
struct Fp8Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_;
  static constexpr int W = (BM / WM) * (BN / WN), NT = W * kWave;
  static constexpr int FM = WM / 32, FN = WN / 32;
  static constexpr int A_BYTES = BM * 64, B_BYTES = BN * 64;
  static constexpr int STAGE = A_BYTES + B_BYTES + (BM + BN) * 4;
  static constexpr int LDS_BYTES = S * STAGE;
  static constexpr int A_DMA = A_BYTES / 1024 / W, B_DMA = B_BYTES / 1024 / W, S_ALL = (BM + BN) / 64;
  static constexpr int S_DMA = (S_ALL + W - 1) / W;   // past the last, a wave copies the last rows again
  static constexpr int D = A_DMA + B_DMA + S_DMA;   // DMA instructions per wave and stage
  static_assert(A_BYTES % (1024 * W) == 0 && B_BYTES % (1024 * W) == 0, "DMA split");
  static_assert(BM % 64 == 0, "one DMA of scale words lies in one operand");
  static_assert(S >= 3 && D * (S - 2) <= 63 && LDS_BYTES <= 160 * 1024, "ring");
};

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 (or 4) bytes per lane from base + off to LDS bytes [lds_addr + 16 (4) * lane), as gemm::dma16
// (with the wait state between the write of M0 and the load)
__device__ __forceinline__ void dma16_at(const uint8_t* base, uint32_t off, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base),
               "s"(__builtin_amdgcn_readfirstlane(lds_addr))
               : "memory", "m0");
}
__device__ __forceinline__ void dma4_at(const uint8_t* base, uint32_t off, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base),
               "s"(__builtin_amdgcn_readfirstlane(lds_addr))
               : "memory", "m0");
}
#pragma clang diagnostic pop

// This wave's copies but the last N have landed and all its LDS reads are done (those
// were issued a whole step earlier), then all waves meet: what lands next may
// overwrite the stage that was read before.
template <int N>
__device__ __forceinline__ void ring_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

constexpr int kGroupRows = 8;   // tile rows walked together, column by column

// Where a unit's result goes: C <- beta C + alpha acc for an m x width matrix of row pitch ld
template <typename TS>
struct TileOut {
  TS* C;
  int64_t ld, width;
  float alpha, beta;
};

// One BM x BN tile at rows m0, columns n0 over 64-value steps [kt0, kt0 + nk) (both even)
template <int FA, bool EXACT, typename TS, int BM, int BN, int WM, int WN, int S>
__device__ __forceinline__ void fp8_tile_unit(const Fp8GemmArgs& g, int64_t m0, int64_t n0, int kt0, int nk,
                                              const TileOut<TS>& out, char* lds) {
  using C_ = Fp8Tile<BM, BN, WM, WN, S>;
  constexpr int FM = C_::FM, FN = C_::FN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 31, h = lane >> 5;
  const int wm0 = (wave / (BN / WN)) * WM, wn0 = (wave % (BN / WN)) * WN;
  // rows past the matrix read its last row; what they compute is not stored
  const int mlast = int(min(g.m - 1 - m0, int64_t(BM - 1))), nlast = int(min(g.n - 1 - n0, int64_t(BN - 1)));
  const uint8_t* At = g.A + m0 * g.lda;
  const uint8_t* Bt = g.B + n0 * g.ldb;
  uint32_t a_off[C_::A_DMA], b_off[C_::B_DMA];
#pragma unroll
  for (int i = 0; i < C_::A_DMA; ++i) {
    const int r = 16 * (wave * C_::A_DMA + i) + (lane >> 2);
    a_off[i] = uint32_t(min(r, mlast)) * uint32_t(g.lda) + (((lane & 3) ^ ((r >> 2) & 3)) << 4);
  }
#pragma unroll
  for (int i = 0; i < C_::B_DMA; ++i) {
    const int r = 16 * (wave * C_::B_DMA + i) + (lane >> 2);
    b_off[i] = uint32_t(min(r, nlast)) * uint32_t(g.ldb) + (((lane & 3) ^ ((r >> 2) & 3)) << 4);
  }
  // scale words: 64 rows per DMA, of A for the first BM / 64 of them
  const uint8_t* s_src[C_::S_DMA];
  int64_t s_step[C_::S_DMA];
  uint32_t s_off[C_::S_DMA];
#pragma unroll
  for (int i = 0; i < C_::S_DMA; ++i) {
    const int r = 64 * min(wave * C_::S_DMA + i, C_::S_ALL - 1);
    const bool of_a = r < BM;
    s_off[i] = uint32_t(of_a ? min(r + lane, mlast) : min(r - BM + lane, nlast)) * 4;
    s_src[i] = of_a ? g.sa + m0 * 4 : g.sb + n0 * 4;
    s_step[i] = (of_a ? g.ra4 : g.rb4) * 4;
  }
  const uint32_t lds_base =
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds));
  // copy q (0 .. D - 1) of stage kt to ring offset `off`
  auto issue_one = [&](int q, int kt, uint32_t off) __attribute__((always_inline)) {
    const uint32_t st = lds_base + off;
    if (q < C_::A_DMA) {
      dma16_at(At + int64_t(kt) * 64, a_off[q], st + (wave * C_::A_DMA + q) * 1024);
    } else if (q < C_::A_DMA + C_::B_DMA) {
      const int b = q - C_::A_DMA;
      dma16_at(Bt + int64_t(kt) * 64, b_off[b], st + C_::A_BYTES + (wave * C_::B_DMA + b) * 1024);
    } else {
      const int s = q - C_::A_DMA - C_::B_DMA;
      dma4_at(s_src[s] + (kt >> 3) * s_step[s], s_off[s], st + C_::A_BYTES + C_::B_BYTES + min(wave * C_::S_DMA + s, C_::S_ALL - 1) * 256);
    }
  };
  auto ring_next = [](uint32_t o) {
    o += C_::STAGE;
    return o == uint32_t(S * C_::STAGE) ? 0u : o;
  };
  struct Frags {
    u32x4_t a[FM][2], b[FN][2];
    uint32_t sa[FM], sb[FN];
  };
  // LDS read q (0 .. READS - 1) of a step's operands: the scale words, then B's and A's blocks
  constexpr int READS = 3 * (FM + FN);
  const int a_at[2] = {gemm::krow_off(wm0 + fr, h), gemm::krow_off(wm0 + fr, 2 + h)};
  const int b_at[2] = {C_::A_BYTES + gemm::krow_off(wn0 + fr, h), C_::A_BYTES + gemm::krow_off(wn0 + fr, 2 + h)};
  const int sa_at = C_::A_BYTES + C_::B_BYTES + (wm0 + fr) * 4, sb_at = C_::A_BYTES + C_::B_BYTES + (BM + wn0 + fr) * 4;
  auto read_one = [&](int q, const char* st, Frags& f) __attribute__((always_inline)) {
    if (q < FN) {
      f.sb[q] = *reinterpret_cast<const uint32_t*>(st + sb_at + 128 * q);
    } else if (q < FN + FM) {
      f.sa[q - FN] = *reinterpret_cast<const uint32_t*>(st + sa_at + 128 * (q - FN));
    } else if (q < FM + 3 * FN) {
      const int b = q - FN - FM;
      f.b[b >> 1][b & 1] = *reinterpret_cast<const u32x4_t*>(st + b_at[b & 1] + 2048 * (b >> 1));
    } else {
      const int a = q - FM - 3 * FN;
      f.a[a >> 1][a & 1] = *reinterpret_cast<const u32x4_t*>(st + a_at[a & 1] + 2048 * (a >> 1));
    }
  };
  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  // One step's products, in MFMAs 0 .. N - 1; `between(n)` is what the wave issues after
  // MFMA n, while the matrix unit works (a wave issues in order, so copies and reads
  // have to stand between the products, not in front of them).
  constexpr int PHASES = EXACT ? 4 : 1, N = PHASES * FM * FN;
  auto mma = [&](int kt, const Frags& f, auto&& between) __attribute__((always_inline)) {
    const int sh = 8 * ((kt >> 1) & 3);   // this group's byte of the scale words
    if constexpr (EXACT) {
      float va[FM], vb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) va[i] = scale_value(f.sa[i] >> sh);
#pragma unroll
      for (int j = 0; j < FN; ++j) vb[j] = scale_value(f.sb[j] >> sh);
      // operand w (A's blocks, then B's) of phase p, widened while phase p - 1 multiplies
      bf16x8_t w[2][FM + FN];
      auto widen = [&](int p, int k) __attribute__((always_inline)) {
        const int c = p >> 1, e = 2 * (p & 1);
        w[p & 1][k] = k < FM ? widen8<FA>(f.a[k][c][e], f.a[k][c][e + 1], va[k])
                             : widen8<MUON_FP8_E4M3>(f.b[k - FM][c][e], f.b[k - FM][c][e + 1], vb[k - FM]);
      };
#pragma unroll
      for (int k = 0; k < FM + FN; ++k) widen(0, k);
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int t = 0; t < FM * FN; ++t) {
          const int i = t / FN, j = t % FN;
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[p & 1][FM + j], w[p & 1][i], acc[i][j], 0, 0, 0);
          if (p < 3) {
#pragma unroll
            for (int k = t; k < FM + FN; k += FM * FN) widen(p + 1, k);
          }
          between(p * FM * FN + t);
          __builtin_amdgcn_sched_barrier(0);
        }
    } else {
      uint32_t va[FM], vb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) va[i] = f.sa[i] >> sh;
#pragma unroll
      for (int j = 0; j < FN; ++j) vb[j] = f.sb[j] >> sh;
#pragma unroll
      for (int t = 0; t < FM * FN; ++t) {
        const int i = t / FN, j = t % FN;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(f.b[j]), join(f.a[i]), acc[i][j], 0, FA, 0,
                                                                    int(vb[j]), 0, int(va[i]));
        between(t);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (s < nk)
#pragma unroll
      for (int q = 0; q < C_::D; ++q) issue_one(q, kt0 + s, uint32_t(s) * C_::STAGE);
  if (nk >= S - 1) ring_barrier<C_::D * (S - 2)>();
  else ring_barrier<0>();
  Frags f0, f1;
#pragma unroll
  for (int q = 0; q < READS; ++q) read_one(q, lds, f0);
  uint32_t o_cur = 0, o_iss = uint32_t(S - 1) * C_::STAGE;
  int it = 0;
  constexpr int RPM = (READS + N * 3 / 4 - 1) / (N * 3 / 4);   // reads per MFMA, done after three quarters of them
  auto steady = [&](Frags& cur, Frags& nxt) __attribute__((always_inline)) {
    const char* st = lds + ring_next(o_cur);
    ring_barrier<C_::D * (S - 3)>();
    mma(kt0 + it, cur, [&](int n) __attribute__((always_inline)) {
#pragma unroll
      for (int r = 0; r < RPM; ++r)
        if (RPM * n + r < READS) read_one(RPM * n + r, st, nxt);
#pragma unroll
      for (int q = 0; q < C_::D; ++q)
        if (q * N / C_::D == n) issue_one(q, kt0 + it + S - 1, o_iss);
    });
    o_cur = ring_next(o_cur);
    o_iss = ring_next(o_iss);
    ++it;
  };
  auto drain = [&](Frags& cur, Frags& nxt) __attribute__((always_inline)) {
    const bool more = it + 1 < nk;
    if (more) {
      ring_barrier<0>();
      const char* st = lds + ring_next(o_cur);
#pragma unroll
      for (int q = 0; q < READS; ++q) read_one(q, st, nxt);
    }
    mma(kt0 + it, cur, [](int) {});
    o_cur = ring_next(o_cur);
    ++it;
  };
  while (it + S < nk) {   // two steps that both still copy a stage
    steady(f0, f1);
    steady(f1, f0);
  }
  if (it + S - 1 < nk) {
    // one more copy is due: this step and the one after it
    steady(f0, f1);
    drain(f1, f0);
  }
  while (it < nk) {
    drain(f0, f1);
    drain(f1, f0);
  }
  // The tile leaves through LDS, 32 rows at a time and each wave through its own part of
  // the ring, so that rows are read (beta) and written 16 bytes per lane and whole lines
  // at a time.  Accumulator v of a lane: column 8 (v / 4) + 4 h + v % 4 of B's block, row
  // fr of A's.
  ring_barrier<0>();
  constexpr int LDW = WN + 4, E = 16 / int(sizeof(TS)), LPR = WN / E, RPP = 64 / LPR, PASSES = 32 / RPP;
  static_assert(C_::W * 32 * LDW * 4 <= C_::LDS_BYTES, "the slabs fit the ring");
  float* slab = reinterpret_cast<float*>(lds) + wave * 32 * LDW;
  const int pr = lane / LPR, pc = (lane % LPR) * E;
  const int64_t col = n0 + wn0 + pc;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4_t*>(slab + fr * LDW + 32 * j + 8 * q + 4 * h) =
            f32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    const int64_t row0 = m0 + wm0 + 32 * i + pr;
    if (col + E <= out.width) {
      uint4 was[PASSES];
      if (out.beta != 0.0f) {
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          was[p] = make_uint4(0, 0, 0, 0);
          if (row0 + RPP * p < g.m) was[p] = load16(out.C + (row0 + RPP * p) * out.ld + col);
        }
      }
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        float o[E];
#pragma unroll
        for (int k = 0; k < E; k += 4) {
          const f32x4_t x = *reinterpret_cast<const f32x4_t*>(slab + (pr + RPP * p) * LDW + pc + k);
#pragma unroll
          for (int v = 0; v < 4; ++v) o[k + v] = out.alpha * x[v];
        }
        if (out.beta != 0.0f) {
          const uint32_t w[4] = {was[p].x, was[p].y, was[p].z, was[p].w};
#pragma unroll
          for (int k = 0; k < E; ++k) {
            float c;
            if constexpr (sizeof(TS) == 2) c = __uint_as_float((k & 1) ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
            else c = __uint_as_float(w[k]);
            o[k] = fmaf(out.beta, c, o[k]);
          }
        }
        if (row0 + RPP * p < g.m) {
          TS* dst = out.C + (row0 + RPP * p) * out.ld + col;
          if constexpr (sizeof(TS) == 2) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const f32x2_t x = {o[2 * k], o[2 * k + 1]};
              w[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2_t));
            }
            store16(dst, make_uint4(w[0], w[1], w[2], w[3]));
          } else {
            store16(dst, make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3])));
          }
        }
      }
    } else {
      for (int p = 0; p < PASSES; ++p)
        if (row0 + RPP * p < g.m)
          for (int k = 0; k < E; ++k)
            if (col + k < out.width) {
              TS* dst = out.C + (row0 + RPP * p) * out.ld + col + k;
              float o = out.alpha * slab[(pr + RPP * p) * LDW + pc + k];
              if (out.beta != 0.0f) o = fmaf(out.beta, to_f32(*dst), o);
              *dst = from_f32<TS>(o);
            }
    }
  }
}

// tile t of the grid of TM x TN tiles: groups of kGroupRows tile rows, column by column
__device__ __forceinline__ void tile_at(int64_t t, int64_t TM, int64_t TN, int64_t& tm, int64_t& tn) {
  const int64_t per = int64_t(kGroupRows) * TN, first = (t / per) * kGroupRows;
  const int64_t size = min(TM - first, int64_t(kGroupRows)), r = t % per;
  tm = __builtin_amdgcn_readfirstlane(int(first + r % size));
  tn = __builtin_amdgcn_readfirstlane(int(r / size));
}

template <typename TC>
__device__ __forceinline__ TileOut<TC> whole_out(const Fp8GemmArgs& g) {
  return TileOut<TC>{static_cast<TC*>(g.C), g.ldc, g.n, g.alpha, g.beta};
}

// All tiles of one size; with SPLIT each is g.splits units along the contraction, whose
// fp32 results lie one after another in g.partials.  777 x 2304 x 768: 7.5 us; 48 x 4096 x
// 14336 in 16 splits of 64 x 128 tiles: 14 us, 4.3 TB/s of B, and 5.5 us to join them.
template <int FA, typename TC, int BM, int BN, int WM, int WN, int S, bool SPLIT>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void fp8_gemm_tile_kernel(Fp8GemmArgs g) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  constexpr bool EXACT = sizeof(TC) == 4;
  const int64_t TM = (g.m + BM - 1) / BM, TN = (g.n + BN - 1) / BN;
  int64_t u = gemm::xcd_remap(blockIdx.x, gridDim.x), tm, tn;
  if constexpr (SPLIT) {
    // a split's tiles are neighbours, and the splits of 128-value groups as even as they come
    const int64_t tiles = TM * TN, part = u / tiles, groups = g.K / kGroup;
    tile_at(u % tiles, TM, TN, tm, tn);
    const int g0 = __builtin_amdgcn_readfirstlane(int(part * groups / g.splits));
    const int g1 = __builtin_amdgcn_readfirstlane(int((part + 1) * groups / g.splits));
    const TileOut<float> out{g.partials + part * g.m * g.ldp, g.ldp, g.ldp, 1.0f, 0.0f};
    fp8_tile_unit<FA, EXACT, float, BM, BN, WM, WN, S>(g, tm * BM, tn * BN, 2 * g0, 2 * (g1 - g0), out, lds);
  } else {
    tile_at(u, TM, TN, tm, tn);
    fp8_tile_unit<FA, EXACT, TC, BM, BN, WM, WN, S>(g, tm * BM, tn * BN, 0, __builtin_amdgcn_readfirstlane(int(g.K / 64)),
                                                    whole_out<TC>(g), lds);
  }
}

// 256 x 256 tiles in rounds of one per CU; those of the last, partial round come in
// `parts` (2: 128 x 256, 4: 128 x 128) so that they fill the CUs.  Workgroups [0, whole)
// take whole tiles.  Bound by the matrix unit at the clock that the chip holds (1.75 GHz;
// busy 57% of the cycles at 4096 x 14336 x 4096, the rest waits for stages and the ends of
// tiles): bf16 C 8192^3 425 us, 2.6 PFLOP/s (a library product with one scale: 2.8),
// 4096 x 14336 x 4096 206 - 235 us from box to box; its fp32 C with beta 408 - 456 us,
// 1.1 - 1.2 PFLOP/s on the bf16 instructions (library 1.25).
template <int FA, typename TC>
__global__ __launch_bounds__(256) void fp8_gemm_mixed_kernel(Fp8GemmArgs g, int64_t whole, int parts) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  constexpr bool EXACT = sizeof(TC) == 4;
  const int64_t TM = (g.m + 255) / 256, TN = (g.n + 255) / 256;
  const int nk = __builtin_amdgcn_readfirstlane(int(g.K / 64));
  const int64_t b = blockIdx.x;
  int64_t tm, tn;
  if (b < whole) {
    tile_at(gemm::xcd_remap(b, whole), TM, TN, tm, tn);
    fp8_tile_unit<FA, EXACT, TC, 256, 256, 128, 128, 4>(g, tm * 256, tn * 256, 0, nk, whole_out<TC>(g), lds);
    return;
  }
  const int64_t u = gemm::xcd_remap(b - whole, int64_t(gridDim.x) - whole), part = u % parts;
  tile_at(whole + u / parts, TM, TN, tm, tn);
  const int64_t m0 = tm * 256 + 128 * (part & 1), n0 = tn * 256 + 128 * (part >> 1);
  if (m0 >= g.m || n0 >= g.n) return;
  if (parts == 2) fp8_tile_unit<FA, EXACT, TC, 128, 256, 64, 128, 4>(g, m0, n0, 0, nk, whole_out<TC>(g), lds);
  else fp8_tile_unit<FA, EXACT, TC, 128, 128, 64, 64, 4>(g, m0, n0, 0, nk, whole_out<TC>(g), lds);
}

// C <- beta C + alpha sum of the splits' partial products, added in their order
template <typename TC>
__global__ __launch_bounds__(256) void fp8_gemm_join_kernel(Fp8GemmArgs g) {
  const int64_t per = g.ldp / 4, t = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (t >= g.m * per) return;
  const int64_t row = t / per, col = (t % per) * 4;
  const float* src = g.partials + row * g.ldp + col;
  f32x4_t sum = *reinterpret_cast<const f32x4_t*>(src);
  for (int p = 1; p < g.splits; ++p) sum += *reinterpret_cast<const f32x4_t*>(src + p * g.m * g.ldp);
  const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
  store4<TC>(g, row, col, v);
}

template <int FA, typename TC, int BM, int BN, int WM, int WN, int S, bool SPLIT>
int launch_tile(const Fp8GemmArgs& g, hipStream_t st) {
  using C_ = Fp8Tile<BM, BN, WM, WN, S>;
  auto kern = fp8_gemm_tile_kernel<FA, TC, BM, BN, WM, WN, S, SPLIT>;
  static std::atomic<uint64_t> configured{0};   // devices with the LDS limit set
  if (gemm::set_lds_limit(kern, C_::LDS_BYTES, configured) != MUON_OK) return MUON_ELAUNCH;
  const int64_t tiles = ceil_div(g.m, BM) * ceil_div(g.n, BN) * (SPLIT ? g.splits : 1);
  if (tiles > INT32_MAX) return MUON_EINVAL;
  launch_kernel(kern, dim3(tiles), dim3(C_::NT), C_::LDS_BYTES, st, g);
  return launch_status();
}

template <int FA, typename TC>
int launch_mixed(const Fp8GemmArgs& g, int64_t whole, int64_t rest, int parts, hipStream_t st) {
  auto kern = fp8_gemm_mixed_kernel<FA, TC>;
  constexpr int LDS = Fp8Tile<256, 256, 128, 128, 4>::LDS_BYTES;
  static std::atomic<uint64_t> configured{0};
  if (gemm::set_lds_limit(kern, LDS, configured) != MUON_OK) return MUON_ELAUNCH;
  if (whole + rest * parts > INT32_MAX) return MUON_EINVAL;
  launch_kernel(kern, dim3(whole + rest * parts), dim3(256), LDS, st, g, whole, parts);
  return launch_status();
}

// How a product is cut, by its sizes alone (kCus: one 256 x 256 tile each).
//  direct  up to 16 rows: bound by reading B once, straight from memory
//  split   fewer 128-wide tiles than half the CUs: along the contraction into units of at
//          least 512 k-values, about two per CU, joined by a second kernel; up to 64 rows
//          on 64 x 128 tiles
//  small   128 x 128 tiles where 256 x 256 ones would leave more than half the CUs idle
//  mixed   256 x 256 tiles, the last round in halves or quarters
constexpr int64_t kCus = 256;
enum ProductKind { kDirect, kSplit, kSmall, kMixed };
struct ProductPlan {
  ProductKind kind;
  int splits;
};
inline ProductPlan plan_product(int64_t m, int64_t n, int64_t K) {
  if (m <= 16 || K == 0) return {kDirect, 1};
  const int64_t tiles = ceil_div(m, m <= 64 ? 64 : 128) * ceil_div(n, 128);
  const int64_t splits = std::min<int64_t>(std::min<int64_t>(16, K / 512), ceil_div(2 * kCus, tiles));
  if (2 * tiles <= kCus && splits > 1) return {kSplit, int(splits)};
  if (m <= 64) return {kDirect, 1};
  if (2 * ceil_div(m, 256) * ceil_div(n, 256) < kCus) return {kSmall, 1};
  return {kMixed, 1};
}

template <int FA, typename TC>
int launch_product(const Fp8GemmArgs& g, const ProductPlan& plan, hipStream_t st) {
  switch (plan.kind) {
    case kDirect:
      if (g.m <= 16) return launch_direct<FA, TC, 1>(g, st);
      if (g.m <= 32) return launch_direct<FA, TC, 2>(g, st);
      return launch_direct<FA, TC, 4>(g, st);
    case kSplit: {
      const int status = g.m <= 64 ? launch_tile<FA, TC, 64, 128, 32, 64, 4, true>(g, st)
                                   : launch_tile<FA, TC, 128, 128, 64, 64, 4, true>(g, st);
      if (status != MUON_OK) return status;
      launch_kernel(fp8_gemm_join_kernel<TC>, dim3(ceil_div(g.m * (g.ldp / 4), 256)), dim3(256), 0, st, g);
      return launch_status();
    }
    case kSmall:
      return launch_tile<FA, TC, 128, 128, 64, 64, 4, false>(g, st);
    default: {
      const int64_t tiles = ceil_div(g.m, 256) * ceil_div(g.n, 256), rest = tiles % kCus;
      const int parts = rest * 4 <= kCus ? 4 : rest * 2 <= kCus ? 2 : 1;
      if (rest == 0 || parts == 1) return launch_mixed<FA, TC>(g, tiles, 0, 1, st);
      return launch_mixed<FA, TC>(g, tiles - rest, rest, parts, st);
    }
  }
}

// the tiles address their 256 rows with 32-bit offsets
constexpr int64_t kMaxPitch = (int64_t(1) << 24) - 16;

bool valid_fmt(int f) { return f == MUON_FP8_E4M3 || f == MUON_FP8_E5M2; }

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t fp8_scale_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > MUON_FP8_MAX_SIDE || cols > MUON_FP8_MAX_SIDE) return 0;
  return size_t(ceil_div(ceil_div(cols, kGroup), 4)) * size_t(scale_rows(rows)) * 4;
}

int fp8_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, int fmt, int block_rows,
                 void* q, int64_t ldq, void* s, void* qt, int64_t ldqt, void* st, void* stream) {
  if (rows < 0 || cols < 0 || rows > MUON_FP8_MAX_SIDE || cols > MUON_FP8_MAX_SIDE) return MUON_EINVAL;
  if (block_rows != 1 && block_rows != kGroup) return MUON_EINVAL;
  if (!valid_dtype(x_dtype) || !valid_fmt(fmt)) return MUON_EDTYPE;
  if ((q == nullptr) != (s == nullptr) || (qt == nullptr) != (st == nullptr)) return MUON_EINVAL;
  if (rows == 0 || cols == 0) return MUON_OK;
  if (x == nullptr || (q == nullptr && qt == nullptr) || ldx < cols) return MUON_EINVAL;
  if (q != nullptr && (ldq < ceil_div(cols, kGroup) * kGroup || ldq % 16 != 0)) return MUON_EINVAL;
  if (qt != nullptr && (ldqt < ceil_div(rows, kGroup) * kGroup || ldqt % 16 != 0)) return MUON_EINVAL;
  if (!aligned16(x) || !aligned16(q) || !aligned16(s) || !aligned16(qt) || !aligned16(st)) return MUON_EALIGN;
  QuantArgs g{};
  g.x = x; g.rows = rows; g.cols = cols; g.ldx = ldx;
  g.q = static_cast<uint8_t*>(q); g.s = static_cast<uint8_t*>(s);
  g.qt = static_cast<uint8_t*>(qt); g.st = static_cast<uint8_t*>(st);
  g.ldq = ldq; g.ldqt = ldqt;
  const dim3 grid(ceil_div(cols, 128), ceil_div(rows, 128));
  hipStream_t hs = static_cast<hipStream_t>(stream);
  auto go = [&](auto t_c, auto f_c) {
    using T = decltype(t_c);
    constexpr int F = decltype(f_c)::value;
    if (block_rows == 1) launch_kernel(fp8_quantize_kernel<T, F, false>, grid, dim3(256), 0, hs, g);
    else launch_kernel(fp8_quantize_kernel<T, F, true>, grid, dim3(256), 0, hs, g);
  };
  using E4 = std::integral_constant<int, MUON_FP8_E4M3>;
  using E5 = std::integral_constant<int, MUON_FP8_E5M2>;
  if (x_dtype == MUON_F32) fmt == MUON_FP8_E4M3 ? go(float{}, E4{}) : go(float{}, E5{});
  else fmt == MUON_FP8_E4M3 ? go(bf16_t{}, E4{}) : go(bf16_t{}, E5{});
  return launch_status();
}

size_t fp8_gemm_workspace_bytes(int64_t m, int64_t n, int64_t K) {
  if (m <= 0 || n <= 0 || K <= 0 || m > MUON_FP8_MAX_SIDE || n > MUON_FP8_MAX_SIDE || K > MUON_FP8_MAX_SIDE) return 0;
  const ProductPlan p = plan_product(m, n, K);
  return p.kind == kSplit ? size_t(p.splits) * size_t(m) * size_t(ceil_div(n, 4) * 4) * 4 : 0;
}

int fp8_gemm(const void* A, int a_fmt, int64_t lda, const void* sa, const void* B, int b_fmt, int64_t ldb,
             const void* sb, void* C, int c_dtype, int64_t ldc, int64_t m, int64_t n, int64_t K, float alpha,
             float beta, void* workspace, size_t ws_bytes, void* stream) {
  if (m < 0 || n < 0 || K < 0 || m > MUON_FP8_MAX_SIDE || n > MUON_FP8_MAX_SIDE || K > MUON_FP8_MAX_SIDE)
    return MUON_EINVAL;
  if (K % kGroup != 0) return MUON_EINVAL;
  if (!valid_fmt(a_fmt) || b_fmt != MUON_FP8_E4M3 || !valid_dtype(c_dtype)) return MUON_EDTYPE;
  if (m == 0 || n == 0) return MUON_OK;
  if (C == nullptr || ldc < n) return MUON_EINVAL;
  if (K > 0 && (A == nullptr || B == nullptr || sa == nullptr || sb == nullptr)) return MUON_EINVAL;
  if (lda < K || ldb < K || lda % 16 != 0 || ldb % 16 != 0 || lda > kMaxPitch || ldb > kMaxPitch) return MUON_EINVAL;
  if (!aligned16(A) || !aligned16(B) || !aligned16(sa) || !aligned16(sb) || !aligned16(C)) return MUON_EALIGN;
  const size_t need = fp8_gemm_workspace_bytes(m, n, K);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return MUON_EWORKSPACE;
  if (need > 0 && !aligned16(workspace)) return MUON_EALIGN;
  Fp8GemmArgs g{};
  g.A = static_cast<const uint8_t*>(A); g.B = static_cast<const uint8_t*>(B);
  g.sa = static_cast<const uint8_t*>(sa); g.sb = static_cast<const uint8_t*>(sb);
  g.C = C; g.m = m; g.n = n; g.K = K; g.lda = lda; g.ldb = ldb; g.ldc = ldc;
  g.ra4 = scale_rows(m); g.rb4 = scale_rows(n);
  g.alpha = alpha; g.beta = beta;
  const ProductPlan plan = plan_product(m, n, K);
  g.splits = plan.splits;
  g.partials = static_cast<float*>(workspace);
  g.ldp = ceil_div(n, 4) * 4;
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (a_fmt == MUON_FP8_E4M3)
    return c_dtype == MUON_F32 ? launch_product<0, float>(g, plan, hs) : launch_product<0, bf16_t>(g, plan, hs);
  return c_dtype == MUON_F32 ? launch_product<1, float>(g, plan, hs) : launch_product<1, bf16_t>(g, plan, hs);
}

}  // extern "C"
