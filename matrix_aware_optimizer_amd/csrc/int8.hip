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
// against s / 2 says which.
__device__ __forceinline__ int quotient(float x, float s, float inv) {
  float k = rintf(x * inv);
  const float rem = fmaf(-k, s, x), half = 0.5f * s;
  if (fabsf(rem) >= half) {
    // on or past the half: the neighbour on the remainder's side, where it is nearer, or even
    const bool past = fabsf(rem) > half, odd = (int(k) & 1) != 0;
    if (past || odd) k += copysignf(1.0f, rem);
  }
  return int(k);
}

template <typename T>
__global__ __launch_bounds__(256) void int8_quantize_kernel(QuantArgs g) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __shared__ float part[4];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(g.x) + row * g.ldx;
  float m = 0.0f;
  bool bad = false;
  for (int64_t c = threadIdx.x; c < g.cols; c += 256) {
    const float v = fabsf(to_f32(x[c]));
    bad |= !(v < INFINITY);
    m = fmaxf(m, v);
  }
  if (bad) m = INFINITY;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
  if (lane == 0) part[wave] = m;
  __syncthreads();
  m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const bool finite = m < INFINITY;
  const float s = fmaxf(m * (1.0f / 127.0f), 0x1p-126f), inv = 1.0f / s;
  const int64_t padded = ceil_div(g.cols, kStep) * kStep;
  for (int64_t c = threadIdx.x; c < padded; c += 256)
    g.q[row * g.ldq + c] = finite && c < g.cols ? int8_t(quotient(to_f32(x[c]), s, inv)) : int8_t(0);
  if (threadIdx.x == 0) g.s[row] = finite ? s : NAN;
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
// C = float(sum) (sa sb): one rounding of the integer, one of the product of the scales, one of
// theirs, and one to C
template <typename TC>
struct ScaleOut {
  using sum_t = int;
  static constexpr int E = 16 / int(sizeof(TC));
  TC* C;
  int64_t ldc, width;
  const float *sa, *sb;

  template <int N> struct Cols { float b[N]; };
  template <int N> struct Pre { float a; };
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
    store_n<N>(C + row * ldc + col, o);
  }
};

template <bool DUAL, class Out>
int launch_product(const tile::Source& g, const Out& out, const tile::Plan& plan, void* workspace, hipStream_t st) {
  constexpr int NB = DUAL ? 2 : 1;
  using tile::kI8;
  const tile::Split sp{plan.parts, 1, workspace, ceil_div(g.n, 4) * 4};
  switch (plan.kind) {
    case tile::kDirect:
      return tile::launch_direct<kI8, NB>(g, out, st);
    case tile::kNarrow:
      return tile::launch_sized<tile::Config<kI8, 64, 128, 32, 64, 4, false, false, DUAL>, false>(g, out, sp, st);
    case tile::kSmall:
      return tile::launch_sized<tile::Config<kI8, 128, 128, 64, 64, 4, false, false, DUAL>, false>(g, out, sp, st);
    default:
      return tile::launch_tiles<tile::Config<kI8, 256, 256, 128, 128, 4, false, false, DUAL>, false, false>(g, out, sp, st);
  }
}

bool side_ok(int64_t v) { return v >= 0 && v <= MUON_GLU_MAX_SIDE; }

size_t workspace_bytes(int64_t m, int64_t n, int64_t K, int mats) {
  if (m <= 0 || n <= 0 || K <= 0 || !side_ok(m) || !side_ok(n) || K > MUON_INT8_MAX_K) return 0;
  return tile::sum_bytes(tile::plan_product(m, n, K / kStep, mats, 1, true), m, n, mats, 1);
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
  if (x_dtype == MUON_F32) launch_kernel(int8_quantize_kernel<float>, dim3(rows), dim3(256), 0, hs, g);
  else launch_kernel(int8_quantize_kernel<bf16_t>, dim3(rows), dim3(256), 0, hs, g);
  return launch_status();
}

size_t int8_gemm_workspace_bytes(int64_t m, int64_t n, int64_t K) { return workspace_bytes(m, n, K, 1); }
size_t int8_glu_workspace_bytes(int64_t m, int64_t n, int64_t K) { return workspace_bytes(m, n, K, 2); }

int int8_gemm(const void* A, int64_t lda, const float* sa, const void* B, int64_t ldb, const float* sb, void* C,
              int c_dtype, int64_t ldc, int64_t m, int64_t n, int64_t K, void* workspace, size_t ws_bytes, void* stream) {
  if (!side_ok(m) || !side_ok(n) || K < 0 || K > MUON_INT8_MAX_K || K % kStep != 0) return MUON_EINVAL;
  if (!valid_dtype(c_dtype)) return MUON_EDTYPE;
  if (m == 0 || n == 0) return MUON_OK;
  if (sa == nullptr || sb == nullptr || C == nullptr || ldc < n || (K > 0 && (A == nullptr || B == nullptr))) return MUON_EINVAL;
  if (lda < K || ldb < K || lda % 16 != 0 || ldb % 16 != 0 || lda > tile::kMaxPitch || ldb > tile::kMaxPitch) return MUON_EINVAL;
  if (!aligned16(A) || !aligned16(sa) || !aligned16(B) || !aligned16(sb) || !aligned16(C)) return MUON_EALIGN;
  const size_t need = int8_gemm_workspace_bytes(m, n, K);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return MUON_EWORKSPACE;
  if (need > 0 && !aligned16(workspace)) return MUON_EALIGN;
  const char *a = static_cast<const char*>(A), *b = static_cast<const char*>(B);
  const tile::Source g{{a, a}, {b, b}, lda, ldb, m, n, K, 1};
  const tile::Plan plan = tile::plan_product(m, n, K / kStep, 1, 1, true);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (c_dtype == MUON_F32) return launch_product<false>(g, ScaleOut<float>{static_cast<float*>(C), ldc, n, sa, sb}, plan, workspace, hs);
  return launch_product<false>(g, ScaleOut<bf16_t>{static_cast<bf16_t*>(C), ldc, n, sa, sb}, plan, workspace, hs);
}

int int8_glu(const void* A, int64_t lda, const float* sa, const void* Bg, const float* sg, const void* Bu, const float* su,
             int64_t ldb, int act, void* H, int h_dtype, int64_t ldh, int64_t m, int64_t n, int64_t K, void* workspace,
             size_t ws_bytes, void* stream) {
  if (!side_ok(m) || !side_ok(n) || K < 0 || K > MUON_INT8_MAX_K || K % kStep != 0 || !valid_act(act)) return MUON_EINVAL;
  if (!valid_dtype(h_dtype)) return MUON_EDTYPE;
  if (m == 0 || n == 0) return MUON_OK;
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
  const tile::Plan plan = tile::plan_product(m, n, K / kStep, 2, 1, true);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (h_dtype == MUON_F32)
    return launch_product<true>(g, GluOut<float, true>{static_cast<float*>(H), nullptr, nullptr, ldh, 0, n, act, sa, sg, su}, plan, workspace, hs);
  return launch_product<true>(g, GluOut<bf16_t, true>{static_cast<bf16_t*>(H), nullptr, nullptr, ldh, 0, n, act, sa, sg, su}, plan, workspace, hs);
}

}  // extern "C"
