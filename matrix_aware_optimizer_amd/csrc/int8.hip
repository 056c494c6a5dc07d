// 8-bit integer matrices with one scale for each row: the quantiser, the product
// C = sa sb (A B^T), and the gated block on such operands.
//
// Format.  A matrix [rows][cols] is held as codes q [rows][ldq] (int8, zero from cols up to the
// next multiple of 64) and scales s [rows] (fp32); entry (i, j) stands for q[i][j] s[i].
#include <algorithm>

#include "act.h"
#include "common.h"
#include "tile.h"

namespace muon {
namespace {

using tile::ceil_div;

constexpr int kStep = MUON_INT8_STEP;

// ---------------------------------------------------------------------------
// Quantiser
// ---------------------------------------------------------------------------
struct QuantArgs {
  const void* x;
  int64_t rows, cols, ldx;
  int8_t* q;
  int64_t ldq;
  float* s;
};

// rint(x / s) of the exact quotient, ties to even: r = x * (1 / s) is within 2^-22 |r| of it,
// so rint(r) is it or its neighbour, and the sign of the remainder x - k s (exact in one fma)
// says which, its double (exact too; half of a scale under 2^-125 need not be) against s.
__device__ __forceinline__ int quotient(float x, float s, float inv) {
  float k = rintf(x * inv);
  const float rem = fmaf(-k, s, x), twice = 2.0f * fabsf(rem);
  if (twice >= s) {
    // on or past the half: the neighbour on the remainder's side, where it is nearer, or even
    const bool past = twice > s, odd = (int(k) & 1) != 0;
    if (past || odd) k += copysignf(1.0f, rem);
  }
  return int(k);
}

// Eight codes.  x * inv + 3 * 2^22 rounds x * inv to an integer, ties to even, and its low byte
// is the code in two's complement.  inv is off by 2^-24 of itself, so the integer is that of
// the exact quotient unless x * inv lies within 127 * 2^-24 of a half; a wave that holds such
// an entry (one in a hundred, by chance) takes the remainders.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s, float inv) {
  constexpr float kShift = 12582912.0f;
  float k[8], far = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    k[i] = fmaf(x[i], inv, kShift);
    far = fmaxf(far, fabsf(fmaf(x[i], inv, kShift - k[i])));
  }
  if (__any(far > 0.49999f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = kShift + float(quotient(x[i], s, inv));
  }
  uint32_t w[4];   // bytes 0 of neighbours
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_perm(__float_as_uint(k[2 * i + 1]), __float_as_uint(k[2 * i]), 0x0c0c0400u);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Eight neighbouring columns of a row as loaded.  top(): the largest magnitude as fp32 bits (NaN
// and infinity are the largest).
template <typename T> struct Eight;
template <> struct Eight<bf16_t> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const bf16_t* p, int64_t left) {
    if (left >= 8) {
      const uint4 r = load16(p);
      w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = 2 * j < left ? p[2 * j] : 0u, hi = 2 * j + 1 < left ? p[2 * j + 1] : 0u;
        w[j] = lo | (hi << 16);
      }
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
    u16x2_t m = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w[j] & 0x7fff7fffu));
    return uint32_t(m[0] > m[1] ? m[0] : m[1]) << 16;
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float((k & 1) ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
  }
};
template <> struct Eight<float> {
  float x[8];
  __device__ __forceinline__ void load(const float* p, int64_t left) {
    if (left >= 8) load_n<8>(p, x);
    else
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = k < left ? p[k] : 0.0f;
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t a = __float_as_uint(x[k]) & 0x7fffffffu;
      m = a > m ? a : m;
    }
    return m;
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = x[k];
  }
};

// Bound by memory: 4096 x 14336 bf16 34.6 us, 5.1 TB/s, a large copy's rate (read twice, with a
// division for each entry, it was 111 us; read once, with the remainders for all, 43).
// Rows of W waves, four waves to a workgroup, eight neighbouring columns per thread and chunk.
// Up to 512 W CH columns a row is read once and stays in registers (CH chunks of a thread);
// longer rows (CH = 0) are read twice, the second time from the caches.
template <typename T, int W, int CH>
__global__ __launch_bounds__(256) void int8_quantize_kernel(QuantArgs g) {
  constexpr int NT = 64 * W, N = CH > 0 ? CH : 1;
  __shared__ float part[4];
  const int lane = threadIdx.x & 63, t = threadIdx.x % NT;
  const int64_t row = int64_t(blockIdx.x) * (4 / W) + threadIdx.x / NT;
  if (W == 1 && row >= g.rows) return;
  const T* x = static_cast<const T*>(g.x) + row * g.ldx;
  uint32_t bits = 0;
  Eight<T> v[N];
  if constexpr (CH > 0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) v[i].load(x + (t + i * NT) * 8, g.cols - (t + i * NT) * 8);
#pragma unroll
    for (int i = 0; i < CH; ++i) bits = max(bits, v[i].top());
  } else {
    for (int64_t c = int64_t(t) * 8; c < g.cols; c += NT * 8) {
      v[0].load(x + c, g.cols - c);
      bits = max(bits, v[0].top());
    }
  }
  float m = __uint_as_float(min(bits, 0x7f800000u));   // infinite or NaN: infinity
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
  if constexpr (W > 1) {
    if (lane == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  }
  const bool finite = m < INFINITY;
  const float s = fmaxf(m * (1.0f / 127.0f), 0x1p-126f), inv = 1.0f / s;
  const int64_t padded = ceil_div(g.cols, kStep) * kStep;
  int8_t* q = g.q + row * g.ldq;
  auto write = [&](int64_t c, const Eight<T>& e) __attribute__((always_inline)) {
    float r[8];
    e.values(r);
    const uint2 w = codes8(r, s, inv);
    if (c < padded) *reinterpret_cast<uint2*>(q + c) = finite ? w : make_uint2(0, 0);
  };
  if constexpr (CH > 0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) write((t + i * NT) * 8, v[i]);
  } else {
    for (int64_t c = int64_t(t) * 8; c < padded; c += NT * 8) {
      v[0].load(x + c, g.cols - c);
      write(c, v[0]);
    }
  }
  if (t == 0) g.s[row] = finite ? s : NAN;
}

template <typename T, int W, int CH>
int launch_quantize(const QuantArgs& g, hipStream_t st) {
  launch_kernel(int8_quantize_kernel<T, W, CH>, dim3(ceil_div(g.rows, 4 / W)), dim3(256), 0, st, g);
  return launch_status();
}
template <typename T>
int quantize(const QuantArgs& g, hipStream_t st) {
  if (g.cols <= 512) return launch_quantize<T, 1, 1>(g, st);
  if (g.cols <= 2048) return launch_quantize<T, 4, 1>(g, st);
  if (g.cols <= 4096) return launch_quantize<T, 4, 2>(g, st);
  if (g.cols <= 8192) return launch_quantize<T, 4, 4>(g, st);
  if (g.cols <= 16384) return launch_quantize<T, 4, 8>(g, st);
  return launch_quantize<T, 4, 0>(g, st);
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
// C = float(sum) (sa sb): one rounding of the integer, one of the product of the scales, one of
// theirs, and one to C
template <typename TC, bool PASSING = false>
struct ScaleOut {
  using sum_t = int;
  static constexpr int E = 16 / int(sizeof(TC));
  TC* C;
  int64_t ldc, width;
  const float *sa, *sb;

  template <int N> struct Cols { float b[N]; };
  template <int N> struct Pre { float a; };
  ScaleOut<TC, true> passing() const { return {C, ldc, width, sa, sb}; }
  bool lines() const { return whole_lines(C, ldc * int64_t(sizeof(TC))); }
  __device__ __forceinline__ ScaleOut at(int) const { return *this; }
  template <int N> __device__ __forceinline__ Cols<N> cols(int64_t col) const {
    Cols<N> c;
#pragma unroll
    for (int k = 0; k < N; ++k) c.b[k] = sb[min(col + k, width - 1)];
    return c;
  }
  template <int N> __device__ __forceinline__ Pre<N> pre(int64_t row, int64_t) const { return {sa[row]}; }
  template <int N>
  __device__ __forceinline__ void store(int64_t row, int64_t col, const int (&v)[1][N], const Cols<N>& c, const Pre<N>& p) const {
    float o[N];
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = float(v[0][k]) * (p.a * c.b[k]);
    store_n<N, PASSING>(C + row * ldc + col, o);
  }
};

// An empty contraction: zeros whatever the scales hold, as the quantiser gives a matrix without columns none.
template <typename TC>
__global__ __launch_bounds__(256) void zeros_kernel(TC* C, int64_t m, int64_t n, int64_t ldc) {
  for (int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x; t < m * n; t += int64_t(gridDim.x) * 256) C[t / n * ldc + t % n] = TC(0);
}
template <typename TC>
int launch_zeros(void* C, int64_t m, int64_t n, int64_t ldc, hipStream_t st) {
  launch_kernel(zeros_kernel<TC>, tile::grid_of(m * n), dim3(256), 0, st, static_cast<TC*>(C), m, n, ldc);
  return launch_status();
}

template <bool DUAL, class Out>
int launch_product(const tile::Source& g, const Out& out, const tile::Plan& plan, void* workspace, hipStream_t st) {
  using tile::kI8;
  const tile::Split sp{plan.parts, 1, workspace, ceil_div(g.n, 4) * 4};
  if constexpr (!DUAL)
    if (plan.kind == tile::kDirect) return tile::launch_direct(g, out, st);
  switch (plan.kind) {
    case tile::kNarrow:
      return tile::launch_sized<tile::Config<kI8, 64, 64, 32, 64, 9, false, false, DUAL>, false>(g, out, sp, st);
    case tile::kSmall:
      return tile::launch_sized<tile::Config<kI8, 128, 128, 64, 64, 5, false, false, DUAL>, false>(g, out, sp, st);
    default:
      return tile::launch_large<kI8, false, false, DUAL>(g, out, sp, st);
  }
}

bool side_ok(int64_t v) { return v >= 0 && v <= MUON_GLU_MAX_SIDE; }

size_t workspace_bytes(int64_t m, int64_t n, int64_t K, int mats) {
  if (m <= 0 || n <= 0 || K <= 0 || !side_ok(m) || !side_ok(n) || K > MUON_INT8_MAX_K) return 0;
  return tile::sum_bytes(tile::plan_product(m, n, K / kStep, mats, 1, true, true), m, n, mats, 1);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int int8_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, void* q, int64_t ldq, float* s,
                  void* stream) {
  if (!side_ok(rows) || !side_ok(cols)) return MUON_EINVAL;
  if (!valid_dtype(x_dtype)) return MUON_EDTYPE;
  if (rows == 0 || cols == 0) return MUON_OK;
  if (x == nullptr || q == nullptr || s == nullptr || ldx < cols) return MUON_EINVAL;
  if (ldq < ceil_div(cols, kStep) * kStep || ldq % 16 != 0) return MUON_EINVAL;
  if (!aligned16(x) || !aligned16(q) || !aligned16(s)) return MUON_EALIGN;
  const QuantArgs g{x, rows, cols, ldx, static_cast<int8_t*>(q), ldq, s};
  hipStream_t hs = static_cast<hipStream_t>(stream);
  return x_dtype == MUON_F32 ? quantize<float>(g, hs) : quantize<bf16_t>(g, hs);
}

size_t int8_gemm_workspace_bytes(int64_t m, int64_t n, int64_t K) { return workspace_bytes(m, n, K, 1); }
size_t int8_glu_workspace_bytes(int64_t m, int64_t n, int64_t K) { return workspace_bytes(m, n, K, 2); }

int int8_gemm(const void* A, int64_t lda, const float* sa, const void* B, int64_t ldb, const float* sb, void* C,
              int c_dtype, int64_t ldc, int64_t m, int64_t n, int64_t K, void* workspace, size_t ws_bytes, void* stream) {
  if (!side_ok(m) || !side_ok(n) || K < 0 || K > MUON_INT8_MAX_K || K % kStep != 0) return MUON_EINVAL;
  if (!valid_dtype(c_dtype)) return MUON_EDTYPE;
  if (m == 0 || n == 0) return MUON_OK;
  if (!numel_ok(m * n)) return MUON_EINVAL;
  if (sa == nullptr || sb == nullptr || C == nullptr || ldc < n || (K > 0 && (A == nullptr || B == nullptr))) return MUON_EINVAL;
  if (lda < K || ldb < K || lda % 16 != 0 || ldb % 16 != 0 || lda > tile::kMaxPitch || ldb > tile::kMaxPitch) return MUON_EINVAL;
  if (!aligned16(A) || !aligned16(sa) || !aligned16(B) || !aligned16(sb) || !aligned16(C)) return MUON_EALIGN;
  const size_t need = int8_gemm_workspace_bytes(m, n, K);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return MUON_EWORKSPACE;
  if (need > 0 && !aligned16(workspace)) return MUON_EALIGN;
  const char *a = static_cast<const char*>(A), *b = static_cast<const char*>(B);
  const tile::Source g{{a, a}, {b, b}, lda, ldb, m, n, K, 1};
  const tile::Plan plan = tile::plan_product(m, n, K / kStep, 1, 1, true, true);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (K == 0) return c_dtype == MUON_F32 ? launch_zeros<float>(C, m, n, ldc, hs) : launch_zeros<bf16_t>(C, m, n, ldc, hs);
  if (c_dtype == MUON_F32) return launch_product<false>(g, ScaleOut<float>{static_cast<float*>(C), ldc, n, sa, sb}, plan, workspace, hs);
  return launch_product<false>(g, ScaleOut<bf16_t>{static_cast<bf16_t*>(C), ldc, n, sa, sb}, plan, workspace, hs);
}

int int8_glu(const void* A, int64_t lda, const float* sa, const void* Bg, const float* sg, const void* Bu, const float* su,
             int64_t ldb, int act, void* H, int h_dtype, int64_t ldh, int64_t m, int64_t n, int64_t K, void* workspace,
             size_t ws_bytes, void* stream) {
  if (!side_ok(m) || !side_ok(n) || K < 0 || K > MUON_INT8_MAX_K || K % kStep != 0 || !valid_act(act)) return MUON_EINVAL;
  if (!valid_dtype(h_dtype)) return MUON_EDTYPE;
  if (m == 0 || n == 0) return MUON_OK;
  if (!numel_ok(m * n)) return MUON_EINVAL;
  if (sa == nullptr || sg == nullptr || su == nullptr || H == nullptr || ldh < n) return MUON_EINVAL;
  if (K > 0 && (A == nullptr || Bg == nullptr || Bu == nullptr)) return MUON_EINVAL;
  if (lda < K || ldb < K || lda % 16 != 0 || ldb % 16 != 0 || lda > tile::kMaxPitch || ldb > tile::kMaxPitch) return MUON_EINVAL;
  if (!aligned16(A) || !aligned16(sa) || !aligned16(Bg) || !aligned16(sg) || !aligned16(Bu) || !aligned16(su) || !aligned16(H))
    return MUON_EALIGN;
  const size_t need = int8_glu_workspace_bytes(m, n, K);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return MUON_EWORKSPACE;
  if (need > 0 && !aligned16(workspace)) return MUON_EALIGN;
  const char* a = static_cast<const char*>(A);
  const tile::Source g{{a, a}, {static_cast<const char*>(Bg), static_cast<const char*>(Bu)}, lda, ldb, m, n, K, 1};
  const tile::Plan plan = tile::plan_product(m, n, K / kStep, 2, 1, true, true);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (K == 0) return h_dtype == MUON_F32 ? launch_zeros<float>(H, m, n, ldh, hs) : launch_zeros<bf16_t>(H, m, n, ldh, hs);
  if (h_dtype == MUON_F32)
    return launch_product<true>(g, GluOut<float, true>{static_cast<float*>(H), nullptr, nullptr, ldh, 0, n, act, sa, sg, su}, plan, workspace, hs);
  return launch_product<true>(g, GluOut<bf16_t, true>{static_cast<bf16_t*>(H), nullptr, nullptr, ldh, 0, n, act, sa, sg, su}, plan, workspace, hs);
}

}  // extern "C"
