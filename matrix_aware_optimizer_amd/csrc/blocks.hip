// Newton-Schulz orthogonalisation of many small blocks (the heads of attention
// projections): short side s <= 128, any long side, any row pitch.
//
// One iteration is X' = (a I + b A + c A A) X with A = X X^T on the short side.
// With X = T X0, T starts as I and stays a polynomial of A0 = X0 X0^T, and so does
// every later A; polynomials of one symmetric matrix are symmetric and commute:
//     P = a I + b A + c A A,   T' = P T,   A' = X' X'^T = P (P A).
// The long side is therefore touched twice only: once for A0, once for U = T X0.
// All iterations between work on s x s matrices, one workgroup per block.  A is made
// symmetric again in every iteration: what rounding leaves in it that is not symmetric
// would grow sevenfold per iteration where A has converged, while symmetric errors
// shrink there.
// X0 = M / |M|_F, and |M|_F^2 is the trace of M M^T.  Three launches serve every block
// of a call:
//   gram   partial M M^T over chunks of the long side (lower 32 x 32 tiles only)
//   poly   sums the chunks in order, scales by the trace, iterates, writes T / |M|_F
//   apply  U = T M, or W <- (1 - eta decay) W - eta scale U
//
// Rounding.  A relative error d of A0 grows by at most a^2 per iteration where A is
// small, so A and T are held in fp32 and multiplied as such: every s x s product takes
// its operands as sums of three bf16 parts (24 bits and the range of fp32), the six
// products of parts that reach 2^-24, added in fp32: six matrix instructions where
// fp32 ones would take the time of sixteen.  (Two fp16 parts, three products, were half
// as exact as fp32: square blocks with small singular values showed it.)  An fp32 M is
// split in the same way, a bf16 M is taken as it is.  T enters the last product in two
// bf16 parts (2^-17 of U, far under half a step of a bf16 output) or three (fp32
// outputs), M there in as many at most; products of parts beyond the last one kept are
// left out.
#include <algorithm>

#include "common.h"
#include "gemm.h"

namespace muon {
namespace {

constexpr int kMaxRuns = 24;       // problems of one launch (by-value kernel argument)

// One problem: `count` blocks of rows x cols, seen as s x l with s <= l (tall: transposed)
struct Run {
  const void* M;
  void* out;
  int64_t ld_m, stride_m, ld_out, stride_out;
  int64_t partials, parts;   // byte offsets of its partial Grams and its T in the workspace
  int32_t s, l, count, chunk, chunks, slabs, units;   // chunk: k-values per gram unit; slabs per apply unit
  int32_t kind;   // kTall | kF32 | kBig
  int32_t out_f32;
};
enum { kTall = 1, kF32 = 2, kBig = 4 };   // kBig: a short side over 64
template <typename T, bool TALL, bool BIG>
constexpr int kind_of() {
  return (TALL ? kTall : 0) | (sizeof(T) == 4 ? kF32 : 0) | (BIG ? kBig : 0);
}

struct Runs {
  Run r[kMaxRuns];
  int n;
};

struct Epilogue {
  float c1, c2;   // W <- c1 W - c2 U
  int update;
};

__host__ __device__ constexpr int tiles_of(int nt) { return nt * (nt + 1) / 2; }

// lower tile t -> (row, column)
__device__ __forceinline__ void tile_rc(int t, int& i, int& j) {
  i = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0;
  j = t - i * (i + 1) / 2;
}

// unit `u` of a launch -> its run and the index within it (uniform)
__device__ __forceinline__ const Run& find_run(const Runs& runs, int& u, int units_per_count) {
  int k = 0;
  for (; k < runs.n - 1; ++k) {
    const int units = units_per_count == 0 ? runs.r[k].count * runs.r[k].chunks
                                           : units_per_count == 1 ? runs.r[k].count : runs.r[k].count * runs.r[k].units;
    if (u < units) break;
    u -= units;
  }
  return runs.r[k];
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// the bf16 values nearest to x, packed; x becomes what they leave (exact)
__device__ __forceinline__ uint32_t leading_part(f32x2_t& x) {
  const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2_t));
  x[0] -= __uint_as_float(w << 16);
  x[1] -= __uint_as_float(w & 0xffff0000u);
  return w;
}

// A region of a row-major matrix on its way from memory to LDS: rows [r0, r0 + NR),
// columns [c0, c0 + NC), entries outside rows x cols as zeros.  fetch() leaves it in
// registers (LD 16-byte pieces per thread, 256 threads), so that it is under way while
// the region before is multiplied; store() writes it as bf16 planes: a bf16 entry as it
// is, an fp32 entry as its NP leading bf16 parts.
template <typename T, int LD>
struct Region {
  static constexpr int E = 16 / sizeof(T);
  uint4 w[LD];

  __device__ __forceinline__ void fetch(const T* src, int64_t ld, int rows, int cols, int r0, int c0, int NR, int NC) {
    const int per = NC / E, n = NR * per;
#pragma unroll
    for (int q = 0; q < LD; ++q) {
      const int t = threadIdx.x + 256 * q;
      w[q] = make_uint4(0, 0, 0, 0);
      if (t < n) {
        const int r = t / per, c = (t % per) * E;
        const T* p = src + int64_t(r0 + r) * ld + c0 + c;
        if (r0 + r < rows) {
          if (c0 + c + E <= cols) {
            w[q] = load16(p);
          } else {
            uint32_t e[E];
#pragma unroll
            for (int k = 0; k < E; ++k) {
              e[k] = 0;
              if (c0 + c + k < cols) {
                if constexpr (sizeof(T) == 2) e[k] = p[k];
                else e[k] = __float_as_uint(p[k]);
              }
            }
            if constexpr (sizeof(T) == 2)
              w[q] = make_uint4(e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6] | (e[7] << 16));
            else
              w[q] = make_uint4(e[0], e[1], e[2], e[3]);
          }
        }
      }
    }
  }

  // tile holds U for the region: dst = U, or c1 (what fetch() got) - c2 U
  __device__ __forceinline__ void finish(const float* tile, int tile_ld, T* dst, int64_t ld, int rows, int cols, int r0,
                                         int c0, int NR, int NC, const Epilogue& e) const {
    const int per = NC / E, n = NR * per;
#pragma unroll
    for (int q = 0; q < LD; ++q) {
      const int t = threadIdx.x + 256 * q;
      if (t < n) {
        const int r = t / per, c = (t % per) * E;
        if (r0 + r >= rows || c0 + c >= cols) continue;
        float v[E];
#pragma unroll
        for (int k = 0; k < E; k += 4) {
          const f32x4_t x = *reinterpret_cast<const f32x4_t*>(tile + r * tile_ld + c + k);
#pragma unroll
          for (int m = 0; m < 4; ++m) v[k + m] = x[m];
        }
        const uint32_t was[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
        if (e.update) {
#pragma unroll
          for (int k = 0; k < E; ++k) {
            float o;
            if constexpr (sizeof(T) == 2) o = __uint_as_float((k & 1) ? was[k >> 1] & 0xffff0000u : was[k >> 1] << 16);
            else o = __uint_as_float(was[k]);
            v[k] = fmaf(e.c1, o, -e.c2 * v[k]);
          }
        }
        T* p = dst + int64_t(r0 + r) * ld + c0 + c;
        if (c0 + c + E <= cols) {
          uint4 o;
          if constexpr (sizeof(T) == 2) {
            f32x2_t a = {v[0], v[1]}, b = {v[2], v[3]}, g = {v[4], v[5]}, h = {v[6], v[7]};
            o = make_uint4(__builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2_t)),
                           __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2_t)),
                           __builtin_bit_cast(uint32_t, __builtin_convertvector(g, bf16x2_t)),
                           __builtin_bit_cast(uint32_t, __builtin_convertvector(h, bf16x2_t)));
          } else {
            o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
          }
          store16(p, o);
        } else {
#pragma unroll
          for (int k = 0; k < E; ++k)
            if (c0 + c + k < cols) p[k] = from_f32<T>(v[k]);
        }
      }
    }
  }

  template <int NP>
  __device__ __forceinline__ void store(char* lds, int pitch, int plane, int NR, int NC) const {
    const int per = NC / E, n = NR * per;
#pragma unroll
    for (int q = 0; q < LD; ++q) {
      const int t = threadIdx.x + 256 * q;
      if (t < n) {
        const int r = t / per, c = (t % per) * E;
        char* dst = lds + r * pitch + c * 2;
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<uint4*>(dst) = w[q];
        } else {
          f32x2_t lo = {__uint_as_float(w[q].x), __uint_as_float(w[q].y)};
          f32x2_t hi = {__uint_as_float(w[q].z), __uint_as_float(w[q].w)};
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const uint32_t a = leading_part(lo), b = leading_part(hi);
            *reinterpret_cast<uint2*>(dst + p * plane) = make_uint2(a, b);
          }
        }
      }
    }
  }
};

// LDS pitches (bytes), so that one access spreads over the 64 banks.  Rows read 16
// bytes per lane along themselves: an odd multiple of 16.  Rows read transposed, four
// at a time: 64 over a multiple of 128 (the four rows start in four different quarters
// of the banks).
constexpr int row_pitch(int bytes) { return bytes + 16; }
constexpr int tr_pitch(int bytes) { return bytes + 64; }

// An operand's 32 x 16 fragment of one plane, the 32 index values along the rows
// (contiguous k) or along the columns (k-major, transposed on the way)
template <bool KMAJOR>
__device__ __forceinline__ u32x4_t fragment(const char* plane, int pitch, int first, int ks, int lane) {
  if constexpr (KMAJOR) {
    const int gi = lane & 15, G = lane >> 4;
    const char* base = plane + (ks * 16 + 8 * (G >> 1) + (gi >> 2)) * pitch + (first + 16 * (G & 1) + 4 * (gi & 3)) * 2;
    return gemm::read_tr_pair(base, base + 4 * pitch);
  } else {
    return *reinterpret_cast<const u32x4_t*>(plane + (first + (lane & 31)) * pitch + (2 * ks + (lane >> 5)) * 16);
  }
}

// ---------------------------------------------------------------------------
// gram: tile t of M M^T over one chunk, as it lies in the accumulators: [t][16][64].
// Bound by reading M (and, for an fp32 M, by its six products and its splitting): 144
// blocks 768 x 64 bf16 8.5 us; 32 blocks 128 x 4096 11 us in bf16 (3.0 TB/s), 26 in fp32
// (2.6); 50 blocks 80 x 2309 fp32 18 us.
// ---------------------------------------------------------------------------
template <typename T> constexpr int gram_slab() { return 128 / sizeof(T); }   // k-values staged at a time

template <typename T, bool TALL, bool BIG>
__global__ __launch_bounds__(256) void blocks_gram_kernel(Runs runs, char* ws) {
  constexpr int SLAB = gram_slab<T>(), NP = sizeof(T) == 2 ? 1 : 3, SIDE = BIG ? 128 : 64;
  constexpr int PITCH = TALL ? tr_pitch(2 * SIDE) : row_pitch(2 * SLAB);   // tall [SLAB][s], wide [s][SLAB]
  constexpr int PLANE = (TALL ? SLAB : SIDE) * PITCH;
  constexpr int NA = BIG ? 3 : 1;   // lower tiles of a wave
  __shared__ __attribute__((aligned(16))) char lds[NP * PLANE];
  int u = blockIdx.x;
  const Run& run = find_run(runs, u, 0);
  const int b = u / run.chunks, chunk = u % run.chunks;
  const int s = run.s, l = run.l, nt = (s + 31) / 32, sp = nt * 32;
  const T* M = static_cast<const T*>(run.M) + b * run.stride_m;
  const int64_t ld = run.ld_m;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nlow = tiles_of(nt);
  const int k0 = chunk * run.chunk, k1 = min(l, k0 + run.chunk);
  f32x16_t acc[NA];
#pragma unroll
  for (int q = 0; q < NA; ++q)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[q][v] = 0.0f;
  Region<T, BIG ? 4 : 2> reg;
  auto fetch = [&](int k) __attribute__((always_inline)) {
    if (TALL) reg.fetch(M, ld, k1, s, k, 0, SLAB, sp);
    else reg.fetch(M, ld, s, k1, 0, k, sp, SLAB);
  };
  fetch(k0);
  for (int k = k0; k < k1; k += SLAB) {
    __syncthreads();
    if (TALL) reg.template store<NP>(lds, PITCH, PLANE, SLAB, sp);
    else reg.template store<NP>(lds, PITCH, PLANE, sp, SLAB);
    __syncthreads();
    if (k + SLAB < k1) fetch(k + SLAB);
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      const int t = wave + 4 * q;
      if (t < nlow) {
        int ti, tj;
        tile_rc(t, ti, tj);
#pragma unroll
        for (int ks = 0; ks < SLAB / 16; ++ks) {
          u32x4_t fa[NP], fb[NP];
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            fa[p] = fragment<TALL>(lds + p * PLANE, PITCH, ti * 32, ks, lane);
            fb[p] = fragment<TALL>(lds + p * PLANE, PITCH, tj * 32, ks, lane);
          }
#pragma unroll
          for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int r = 0; p + r < NP; ++r) gemm::Mfma<bf16_t>::mma(fa[p], fb[r], acc[q]);
        }
      }
    }
  }
  float* dst = reinterpret_cast<float*>(ws + run.partials) + int64_t(u) * nlow * 1024;
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const int t = wave + 4 * q;
    if (t < nlow)
#pragma unroll
      for (int v = 0; v < 16; ++v) dst[t * 1024 + v * 64 + lane] = acc[q][v];
  }
}

// ---------------------------------------------------------------------------
// poly: one workgroup per block, one wave per strip of 16 columns
// ---------------------------------------------------------------------------
// A wave holds its strip of A, T and P as it comes out of v_mfma_f32_16x16x32_bf16:
// lane (r, g = lane / 16) has rows 16 y + 4 g .. + 3 of column r of the strip, for every
// y.  All matrices are symmetric, so that is also row r of the strip, and two of these
// groups of four (y = 2 t, 2 t + 1) are eight of the 32 k-values of one matrix
// instruction: a strip is its own second operand without leaving the registers, if the
// first operand takes the k-values in the same order.  Only A (for A A) and P (for
// P T, P A and P (P A)) are first operands, and go through LDS as rows.  17 products of
// a block in five steps, one after another on one CU: 21 us at s = 64, 48 at 80 and 96, 95
// at 128 (five steps, up to 256 blocks); there matrix instructions take 46% of the cycles,
// splitting operands and moving accumulators most of the others.
constexpr int kParts = 3;

template <int NY>
struct SymOperand {
  bf16x8_t p[kParts][NY / 2];
};

template <int NY>
__device__ __forceinline__ void split_strip(const f32x4_t (&v)[NY], SymOperand<NY>& o) {
#pragma unroll
  for (int t = 0; t < NY / 2; ++t) {
    uint32_t w[kParts][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f32x2_t x = {v[2 * t + (q >> 1)][2 * (q & 1)], v[2 * t + (q >> 1)][2 * (q & 1) + 1]};
#pragma unroll
      for (int p = 0; p < kParts; ++p) w[p][q] = leading_part(x);
    }
#pragma unroll
    for (int p = 0; p < kParts; ++p)
      o.p[p][t] = __builtin_bit_cast(bf16x8_t, make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]));
  }
}

template <int NY>
struct SymLds {
  static constexpr int PITCH = NY * 32 + 16;        // bytes per row: an odd multiple of 16
  static constexpr int PLANE = NY * 16 * PITCH;
  static constexpr int BYTES = kParts * PLANE;
  static constexpr int BUFFERS = 2 * BYTES <= 150 * 1024 ? 2 : 1;   // two take turns, or one serves all
};

template <int NY>
__device__ __forceinline__ void put_strip(char* buf, int wave, int lane, const SymOperand<NY>& o) {
  char* row = buf + (16 * wave + (lane & 15)) * SymLds<NY>::PITCH + 16 * (lane >> 4);
#pragma unroll
  for (int p = 0; p < kParts; ++p)
#pragma unroll
    for (int t = 0; t < NY / 2; ++t) *reinterpret_cast<bf16x8_t*>(row + 64 * t + p * SymLds<NY>::PLANE) = o.p[p][t];
}

// out = S o for the wave's strips, S in LDS.  The parts of the pieces of S are read DEPTH
// pieces (16 x 32) ahead of their products.
template <int NY, int NS>
__device__ __forceinline__ void sym_product(const char* buf, int lane, const SymOperand<NY> (&o)[NS],
                                            f32x4_t (&out)[NS][NY]) {
  constexpr int NT = NY / 2, PIECES = NY * NT, DEPTH = PIECES < 4 ? 1 : 3;
  const char* row = buf + (lane & 15) * SymLds<NY>::PITCH + 16 * (lane >> 4);
  bf16x8_t f[DEPTH + 1][kParts];
  auto read = [&](int k) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < kParts; ++p)
      f[k % (DEPTH + 1)][p] = *reinterpret_cast<const bf16x8_t*>(row + (k / NT) * 16 * SymLds<NY>::PITCH + (k % NT) * 64 +
                                                                 p * SymLds<NY>::PLANE);
  };
#pragma unroll
  for (int k = 0; k < DEPTH; ++k) read(k);
#pragma unroll
  for (int y = 0; y < NY; ++y) {
    f32x4_t acc[2][NS];   // two sums per strip, neither waiting for the other
#pragma unroll
    for (int i = 0; i < NS; ++i) acc[0][i] = acc[1][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int k = y * NT + t;
      if (k + DEPTH < PIECES) read(k + DEPTH);
      const bf16x8_t(&s)[kParts] = f[k % (DEPTH + 1)];
#pragma unroll
      for (int p = 0; p < kParts; ++p)
#pragma unroll
        for (int r = 0; p + r < kParts; ++r)
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            f32x4_t& to = acc[(p + r) == 2 ? 1 : 0][i];
            to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(s[p], o[i].p[r][t], to, 0, 0, 0);
          }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) out[i][y] = acc[0][i] + acc[1][i];
  }
}

// Strips of a wave.  One gives the most waves; at s > 96 eight waves would each read all
// of S for every product, as long as their matrix instructions take, so four waves take
// two strips each.
template <int NY> constexpr int strips() { return NY == 8 ? 2 : 1; }

template <int NY>
__global__ __launch_bounds__(64 * NY / strips<NY>()) void blocks_poly_kernel(Runs runs, char* ws, float a, float b, float c,
                                                                             int steps) {
  extern __shared__ __attribute__((aligned(16))) char sm[];
  constexpr int NS = strips<NY>(), W = NY / NS;
  constexpr bool SHARED = SymLds<NY>::BUFFERS == 1;
  char* buf = sm;                                        // what is written next
  char* other = SHARED ? sm : sm + SymLds<NY>::BYTES;
  int u = blockIdx.x;
  const Run& run = find_run(runs, u, 1);
  constexpr int nlow = tiles_of(NY / 2), sp = 16 * NY;
  constexpr int LD = sp + 4;   // floats per row of a whole fp32 matrix in LDS: rows four apart start a quarter of the banks apart
  static_assert(sp * LD * 4 <= SymLds<NY>::BYTES, "the matrix fits a buffer");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  f32x4_t A[NS][NY], T[NS][NY];
  double total = 0.0;                                    // |M|_F^2
  // f(i, y): the wave's strip i (strip NS wave + i of the matrix, column 16 strip + r of this
  // lane), rows 16 y + 4 g .. + 3
  auto each = [&](auto&& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int y = 0; y < NY; ++y) f(i, y);
  };
  auto column = [&](int i) { return 16 * (NS * wave + i) + r; };
  // the identity's entries in a tile on the diagonal (y == strip)
  float unit[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) unit[v] = 4 * g + v == r ? 1.0f : 0.0f;
  {
    // The partial Grams are lower 32 x 32 tiles as they lay in the accumulators: float4 q of
    // a tile is value v = q / 16 of lanes 4 (q % 16) .., row 8 (v / 4) + 4 (lane / 32) + v % 4,
    // columns lane % 32 ... All threads add them up, chunk after chunk (four in flight), and
    // lay the whole matrix out in LDS.
    constexpr int THREADS = 64 * W, Q = nlow * 256 / THREADS;   // float4 per thread
    static_assert(nlow * 256 % THREADS == 0, "whole float4 per thread");
    const int chunks = run.chunks;
    const f32x4_t* src = reinterpret_cast<const f32x4_t*>(ws + run.partials) + int64_t(u) * chunks * nlow * 256 + threadIdx.x;
    f32x4_t sum[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) sum[q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    int k = 0;
    for (; k + 4 <= chunks; k += 4, src += 4 * nlow * 256) {
      f32x4_t w[4][Q];
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int q = 0; q < Q; ++q) w[e][q] = src[e * nlow * 256 + q * THREADS];
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int q = 0; q < Q; ++q) sum[q] += w[e][q];
    }
    for (; k < chunks; ++k, src += nlow * 256)
#pragma unroll
      for (int q = 0; q < Q; ++q) sum[q] += src[q * THREADS];
    float* full = reinterpret_cast<float*>(sm);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int at = threadIdx.x + q * THREADS, tile = at >> 8, v = (at & 255) >> 4, l4 = 4 * (at & 15);
      int ti, tj;
      tile_rc(tile, ti, tj);
      const int row = 32 * ti + 8 * (v >> 2) + 4 * (l4 >> 5) + (v & 3), col = 32 * tj + (l4 & 31);
      *reinterpret_cast<f32x4_t*>(full + row * LD + col) = sum[q];
      if (ti != tj)
#pragma unroll
        for (int e = 0; e < 4; ++e) full[(col + e) * LD + row] = sum[q][e];
    }
    __syncthreads();
    each([&](int i, int y) __attribute__((always_inline)) {
      A[i][y] = *reinterpret_cast<const f32x4_t*>(full + column(i) * LD + 16 * y + 4 * g);
    });
#pragma unroll
    for (int d = 0; d < sp; d += 64)
      if (d + lane < sp) total += double(full[(d + lane) * LD + d + lane]);
    total = wave_sum(total);          // every wave adds the same entries in the same order
    __syncthreads();
  }
  // a block of zeros gives U = 0
  const float inv = total == 0.0 ? 0.0f : float(1.0 / total);
  const float root = total == 0.0 ? 0.0f : float(1.0 / sqrt(total));
  each([&](int i, int y) __attribute__((always_inline)) {
    A[i][y] *= inv;
#pragma unroll
    for (int v = 0; v < 4; ++v) T[i][y][v] = y == NS * wave + i ? unit[v] : 0.0f;
  });
  auto split = [&](const f32x4_t (&v)[NS][NY], SymOperand<NY> (&o)[NS]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NS; ++i) split_strip<NY>(v[i], o[i]);
  };
  // one buffer: everybody is done reading before it is written; two: the one written now
  // was read before the last barrier
  auto put = [&](const SymOperand<NY> (&o)[NS]) __attribute__((always_inline)) {
    if (SHARED) __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) put_strip<NY>(buf, NS * wave + i, lane, o[i]);
    __syncthreads();
    char* const w = buf;
    buf = other;
    other = w;
  };
  for (int it = 0; it < steps; ++it) {
    const bool last = it == steps - 1;
    SymOperand<NY> oA[NS];
    f32x4_t P[NS][NY];
    if (it > 0) {
      // (A + A^T) / 2: strips as rows in, their rows out
      if (SHARED) __syncthreads();
      float* full = reinterpret_cast<float*>(buf);
      each([&](int i, int y) __attribute__((always_inline)) {
        *reinterpret_cast<f32x4_t*>(full + column(i) * LD + 16 * y + 4 * g) = A[i][y];
      });
      __syncthreads();
      each([&](int i, int y) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < 4; ++v) A[i][y][v] = 0.5f * (A[i][y][v] + full[(16 * y + 4 * g + v) * LD + column(i)]);
      });
      char* const w = buf;
      buf = other;
      other = w;
    }
    split(A, oA);
    if (c != 0.0f) {
      put(oA);
      sym_product<NY, NS>(other, lane, oA, P);               // A A
    } else {
      each([&](int i, int y) __attribute__((always_inline)) { P[i][y] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}; });
    }
    each([&](int i, int y) __attribute__((always_inline)) {
      const float on = y == NS * wave + i ? a : 0.0f;        // this tile lies on the diagonal
#pragma unroll
      for (int v = 0; v < 4; ++v) P[i][y][v] = fmaf(c, P[i][y][v], fmaf(b, A[i][y][v], on * unit[v]));
    });
    SymOperand<NY> o[NS];
    split(P, o);
    if (it == 0) {
      each([&](int i, int y) __attribute__((always_inline)) { T[i][y] = P[i][y]; });
      if (last) break;
      put(o);
    } else {
      put(o);
      split(T, o);
      sym_product<NY, NS>(other, lane, o, T);                // T' = P T
      if (last) break;
    }
    sym_product<NY, NS>(other, lane, oA, P);                 // P A
    split(P, o);
    sym_product<NY, NS>(other, lane, o, A);                  // A' = P (P A)
  }
  // T / |M|_F in three bf16 parts, rows of [part][sp][sp]
  bf16_t* dst = reinterpret_cast<bf16_t*>(ws + run.parts) + int64_t(u) * 3 * sp * sp + 4 * g;
  each([&](int i, int y) __attribute__((always_inline)) {
    f32x2_t lo = {T[i][y][0] * root, T[i][y][1] * root}, hi = {T[i][y][2] * root, T[i][y][3] * root};
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      uint2 w;
      w.x = leading_part(lo);
      w.y = leading_part(hi);
      *reinterpret_cast<uint2*>(dst + p * sp * sp + column(i) * sp + 16 * y) = w;
    }
  });
}

// ---------------------------------------------------------------------------
// apply: U = T M.  A wave keeps 32 rows of T in registers and multiplies them with its
// share of a slab of the long side.  The results meet in LDS in the output's own layout
// (over the slab's operand planes, which are done with), so that the output is read (for
// an update; fetched while the slab is multiplied) and written in whole rows, 16 bytes
// per lane.  Bound by memory: 32 blocks 128 x 4096, fp32 M, bf16 W updated: 37 us, 3.6 TB/s
// (50 us with rows written 8 bytes per lane); 144 blocks 768 x 64 bf16 updated: 15.5 us.
// ---------------------------------------------------------------------------
// entries of the long side at a time: 64 keep two waves per SIMD in registers
constexpr int apply_slab(bool all_bf16, bool big) { return all_bf16 && !big ? 128 : 64; }
template <typename T, typename TO, bool TALL, bool BIG>
struct ApplyTile {
  static constexpr int LS = apply_slab(sizeof(T) == 2 && sizeof(TO) == 2, BIG), SIDE = BIG ? 128 : 64, NQ = SIDE / 16;
  static constexpr int NPT = sizeof(TO) == 2 ? 2 : 3;                 // bf16 parts of T
  static constexpr int NPM = sizeof(T) == 2 ? 1 : NPT;                // and of M
  static constexpr int PITCH = TALL ? row_pitch(2 * SIDE) : tr_pitch(2 * LS);   // tall [LS][s], wide [s][LS]
  static constexpr int PLANE = (TALL ? LS : SIDE) * PITCH;
  static constexpr int ROWS = TALL ? LS : SIDE, COLS = TALL ? SIDE : LS;        // of the output's tile
  static constexpr int OUT_LD = COLS + 4;
  static constexpr int LDS_BYTES = NPM * PLANE > ROWS * OUT_LD * 4 ? NPM * PLANE : ROWS * OUT_LD * 4;
  static constexpr int M_LOADS = SIDE * LS * int(sizeof(T)) / 16 / 256, OUT_LOADS = SIDE * LS * int(sizeof(TO)) / 16 / 256;
};

template <typename T, typename TO, bool TALL, bool BIG>
__global__ __launch_bounds__(256, 2) void blocks_apply_kernel(Runs runs, const char* ws, Epilogue e) {
  using C_ = ApplyTile<T, TO, TALL, BIG>;
  constexpr int LS = C_::LS, NQ = C_::NQ, NPT = C_::NPT, NPM = C_::NPM, PITCH = C_::PITCH, PLANE = C_::PLANE;
  constexpr int TILES = BIG ? LS / 32 : LS / 64;               // 32 x 32 tiles of a wave and slab (a short side over 32)
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int u = blockIdx.x;
  const Run& run = find_run(runs, u, 2);
  const int b = u / run.units, unit = u % run.units;
  const int s = run.s, l = run.l, nt = (s + 31) / 32, sp = nt * 32;
  const T* M = static_cast<const T*>(run.M) + b * run.stride_m;
  TO* out = static_cast<TO*>(run.out) + b * run.stride_out;
  const int64_t ld = run.ld_m, ld_out = run.ld_out;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 31, h = lane >> 5;
  // 4 waves: row tile ti, and every groups-th 32 entries of the long side
  const int groups = 4 / nt, ti = wave % nt, grp = wave / nt;
  const bool busy = grp < groups;
  const int l0 = unit * run.slabs * LS, l1 = min(l, l0 + run.slabs * LS);
  Region<T, C_::M_LOADS> reg;
  Region<TO, C_::OUT_LOADS> old;
  auto fetch = [&](int x) __attribute__((always_inline)) {
    if (TALL) reg.fetch(M, ld, l, s, x, 0, LS, sp);
    else reg.fetch(M, ld, s, l, 0, x, sp, LS);
  };
  fetch(l0);
  u32x4_t tf[NPT][NQ];
#pragma unroll
  for (int p = 0; p < NPT; ++p)
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      tf[p][q] = u32x4_t{0, 0, 0, 0};
      if (16 * q < sp && busy)
        tf[p][q] = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const bf16_t*>(ws + run.parts) +
                                                     (int64_t(b) * 3 + p) * sp * sp + (ti * 32 + fr) * sp + 16 * q + 8 * h);
    }
  for (int x = l0; x < l1; x += LS) {
    __syncthreads();
    if (TALL) reg.template store<NPM>(lds, PITCH, PLANE, LS, sp);
    else reg.template store<NPM>(lds, PITCH, PLANE, sp, LS);
    __syncthreads();
    if (e.update) {
      if (TALL) old.fetch(out, ld_out, l, s, x, 0, LS, sp);
      else old.fetch(out, ld_out, s, l, 0, x, sp, LS);
    }
    if (x + LS < l1) fetch(x + LS);
    f32x16_t acc[TILES];
#pragma unroll
    for (int k = 0; k < TILES; ++k) {
      const int j = grp + k * groups;   // this tile's 32 entries of the slab
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[k][v] = 0.0f;
      if (busy && 32 * j < LS) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          if (16 * q < sp) {
#pragma unroll
            for (int p = 0; p < NPM; ++p) {
              const u32x4_t fm = fragment<!TALL>(lds + p * PLANE, PITCH, 32 * j, q, lane);
#pragma unroll
              for (int r = 0; p + r < NPT; ++r) {
                // the index that is contiguous in the output first: four of its entries per lane
                if (TALL) gemm::Mfma<bf16_t>::mma(tf[r][q], fm, acc[k]);
                else gemm::Mfma<bf16_t>::mma(fm, tf[r][q], acc[k]);
              }
            }
          }
        }
      }
    }
    __syncthreads();
    float* tile = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int k = 0; k < TILES; ++k) {
      const int j = grp + k * groups;
      if (busy && 32 * j < LS) {
        // accumulator v of this lane: first operand's row 8 (v / 4) + 4 h + v % 4, second's row fr
        const int row = (TALL ? 32 * j : 32 * ti) + fr, col = (TALL ? 32 * ti : 32 * j) + 4 * h;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<f32x4_t*>(tile + row * C_::OUT_LD + col + 8 * q) =
              f32x4_t{acc[k][4 * q], acc[k][4 * q + 1], acc[k][4 * q + 2], acc[k][4 * q + 3]};
      }
    }
    __syncthreads();
    if (TALL) old.finish(tile, C_::OUT_LD, out, ld_out, l, s, x, 0, LS, sp, e);
    else old.finish(tile, C_::OUT_LD, out, ld_out, s, l, 0, x, sp, LS, e);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool valid_shape(const muon_block_problem& p) {
  if (p.rows < 0 || p.cols < 0 || p.count < 0) return false;
  if (p.rows > MUON_BLOCKS_MAX_LONG || p.cols > MUON_BLOCKS_MAX_LONG || p.count > MUON_BLOCKS_MAX_COUNT) return false;
  return std::min(p.rows, p.cols) <= MUON_BLOCKS_MAX_SHORT;
}
bool empty(const muon_block_problem& p) { return p.rows == 0 || p.cols == 0 || p.count == 0; }

// How a problem is cut: chunks of the long side for the Gram, slabs per unit of the
// last product, chosen so that all blocks of the call together give the 256 CUs
// about four workgroups each (two over a short side of 64, which need twice the
// registers), but a chunk is never shorter than 256 entries: each one writes a whole
// partial Gram, and the one CU that iterates reads them all.
void cut(Run& r, int64_t total_blocks) {
  const int64_t want = std::max<int64_t>(1, ceil_div((r.kind & kBig) ? 512 : 1024, std::max<int64_t>(total_blocks, 1)));
  const int64_t slab = (r.kind & kF32) ? gram_slab<float>() : gram_slab<bf16_t>();
  int64_t chunks = std::min<int64_t>(want, ceil_div(r.l, 256));
  r.chunk = int(ceil_div(ceil_div(r.l, chunks), slab) * slab);
  r.chunks = int(ceil_div(r.l, r.chunk));
  const int64_t ls = apply_slab(!(r.kind & kF32) && !r.out_f32, (r.kind & kBig) != 0);
  const int64_t slabs = ceil_div(r.l, ls);
  r.slabs = int(ceil_div(slabs, std::min<int64_t>(slabs, want)));
  r.units = int(ceil_div(slabs, r.slabs));
}

// Fills the run of one problem and moves `bytes` past its workspace.
Run make_run(const muon_block_problem& p, int64_t total_blocks, size_t& bytes) {
  Run r{};
  const bool tall = p.rows > p.cols;
  r.M = p.M; r.out = p.out;
  r.ld_m = p.ld_m; r.stride_m = p.stride_m; r.ld_out = p.ld_out; r.stride_out = p.stride_out;
  r.s = int(std::min(p.rows, p.cols)); r.l = int(std::max(p.rows, p.cols)); r.count = int(p.count);
  r.kind = (tall ? kTall : 0) | (p.m_dtype == MUON_F32 ? kF32 : 0) | (r.s > 64 ? kBig : 0);
  r.out_f32 = p.out_dtype == MUON_F32;
  cut(r, total_blocks);
  const int64_t nt = ceil_div(r.s, 32), sp = nt * 32;
  r.partials = int64_t(bytes);
  bytes += round_up(size_t(r.count) * r.chunks * tiles_of(int(nt)) * 4096, 256);
  r.parts = int64_t(bytes);
  bytes += round_up(size_t(r.count) * sp * sp * 6, 256);
  return r;
}

int64_t count_blocks(const muon_block_problem* probs, int n) {
  int64_t total = 0;
  for (int i = 0; i < n; ++i)
    if (!empty(probs[i])) total += probs[i].count;
  return total;
}

template <typename T, typename TO, bool TALL, bool BIG>
int launch_apply(const Runs& runs, const char* ws, const Epilogue& e, hipStream_t st) {
  int64_t units = 0;
  for (int i = 0; i < runs.n; ++i) units += int64_t(runs.r[i].count) * runs.r[i].units;
  constexpr int LDS = ApplyTile<T, TO, TALL, BIG>::LDS_BYTES;
  static std::atomic<uint64_t> configured{0};
  if (gemm::set_lds_limit(blocks_apply_kernel<T, TO, TALL, BIG>, LDS, configured) != MUON_OK) return MUON_ELAUNCH;
  launch_kernel(blocks_apply_kernel<T, TO, TALL, BIG>, dim3(units), dim3(256), LDS, st, runs, ws, e);
  return launch_status();
}

template <typename T, bool TALL, bool BIG>
int launch_gram(const Runs& runs, char* ws, hipStream_t st) {
  int64_t units = 0;
  for (int i = 0; i < runs.n; ++i) units += int64_t(runs.r[i].count) * runs.r[i].chunks;
  launch_kernel(blocks_gram_kernel<T, TALL, BIG>, dim3(units), dim3(256), 0, st, runs, ws);
  return launch_status();
}

// calls f on the runs of `all` that `pick` chooses, kMaxRuns at a time
template <typename Pick, typename F>
int for_runs(const Run* all, int n, Pick pick, F f) {
  Runs runs;
  runs.n = 0;
  for (int i = 0; i <= n; ++i) {
    if (i < n && pick(all[i])) runs.r[runs.n++] = all[i];
    if (runs.n == kMaxRuns || (i == n && runs.n > 0)) {
      const int status = f(runs);
      if (status != MUON_OK) return status;
      runs.n = 0;
    }
  }
  return MUON_OK;
}

int run_blocks(const muon_block_problem* probs, int nprobs, float a, float b, float c, int steps, const Epilogue& e,
               void* workspace, size_t ws_bytes, hipStream_t st) {
  if (nprobs < 0 || steps < 0 || (nprobs > 0 && probs == nullptr) || nprobs > MUON_BLOCKS_MAX_PROBLEMS) return MUON_EINVAL;
  int64_t units = 0;
  for (int i = 0; i < nprobs; ++i) {
    const muon_block_problem& p = probs[i];
    if (!valid_shape(p)) return MUON_EINVAL;
    if (!valid_dtype(p.m_dtype) || !valid_dtype(p.out_dtype)) return MUON_EDTYPE;
    if (empty(p)) continue;
    if (p.M == nullptr || p.out == nullptr || p.ld_m < p.cols || p.ld_out < p.cols) return MUON_EINVAL;
    if (p.count > 1 && (p.stride_m <= 0 || p.stride_out <= 0)) return MUON_EINVAL;
    if (!aligned16(p.M) || !aligned16(p.out)) return MUON_EALIGN;
    units += p.count * ceil_div(std::max(p.rows, p.cols), 64);
  }
  if (units > INT32_MAX) return MUON_EINVAL;
  const int64_t total = count_blocks(probs, nprobs);
  if (total == 0) return MUON_OK;
  const size_t need = ns_blocks_workspace_bytes(probs, nprobs);
  if (workspace == nullptr || ws_bytes < need) return MUON_EWORKSPACE;
  if (!aligned16(workspace)) return MUON_EALIGN;
  char* ws = static_cast<char*>(workspace);
  Run all[MUON_BLOCKS_MAX_PROBLEMS];
  int n = 0;
  size_t bytes = 0;
  for (int i = 0; i < nprobs; ++i)
    if (!empty(probs[i])) all[n++] = make_run(probs[i], total, bytes);
  // gram and apply: one launch per type, orientation and half of the range of short sides
  const auto gram = [&](auto t_c, auto tall_c, auto big_c) {
    using T = decltype(t_c);
    constexpr bool TALL = decltype(tall_c)::value, BIG = decltype(big_c)::value;
    return for_runs(all, n, [](const Run& r) { return r.kind == kind_of<T, TALL, BIG>(); },
                    [&](const Runs& runs) { return launch_gram<T, TALL, BIG>(runs, ws, st); });
  };
  const auto apply = [&](auto t_c, auto tall_c, auto big_c) {
    using T = decltype(t_c);
    constexpr bool TALL = decltype(tall_c)::value, BIG = decltype(big_c)::value;
    const int status = for_runs(all, n, [](const Run& r) { return r.kind == kind_of<T, TALL, BIG>() && !r.out_f32; },
                                [&](const Runs& runs) { return launch_apply<T, bf16_t, TALL, BIG>(runs, ws, e, st); });
    if (status != MUON_OK) return status;
    return for_runs(all, n, [](const Run& r) { return r.kind == kind_of<T, TALL, BIG>() && r.out_f32; },
                    [&](const Runs& runs) { return launch_apply<T, float, TALL, BIG>(runs, ws, e, st); });
  };
  const auto every_kind = [&](const auto& f) {
    using Yes = std::true_type;
    using No = std::false_type;
    int status = f(bf16_t{}, No{}, No{});
    if (status == MUON_OK) status = f(bf16_t{}, No{}, Yes{});
    if (status == MUON_OK) status = f(bf16_t{}, Yes{}, No{});
    if (status == MUON_OK) status = f(bf16_t{}, Yes{}, Yes{});
    if (status == MUON_OK) status = f(float{}, No{}, No{});
    if (status == MUON_OK) status = f(float{}, No{}, Yes{});
    if (status == MUON_OK) status = f(float{}, Yes{}, No{});
    if (status == MUON_OK) status = f(float{}, Yes{}, Yes{});
    return status;
  };
  int status = every_kind(gram);
  if (status != MUON_OK) return status;
  const auto poly = [&](auto ny) {
    constexpr int NY = decltype(ny)::value;
    return for_runs(all, n, [](const Run& r) { return (r.s + 31) / 32 * 2 == NY; }, [&](const Runs& runs) {
      int64_t blocks = 0;
      for (int i = 0; i < runs.n; ++i) blocks += runs.r[i].count;
      constexpr int LDS = SymLds<NY>::BUFFERS * SymLds<NY>::BYTES;
      static std::atomic<uint64_t> configured{0};
      if (gemm::set_lds_limit(blocks_poly_kernel<NY>, LDS, configured) != MUON_OK) return int(MUON_ELAUNCH);
      launch_kernel(blocks_poly_kernel<NY>, dim3(blocks), dim3(64 * NY / strips<NY>()), LDS, st, runs, ws, a, b, c, steps);
      return launch_status();
    });
  };
  status = poly(std::integral_constant<int, 2>{});
  if (status == MUON_OK) status = poly(std::integral_constant<int, 4>{});
  if (status == MUON_OK) status = poly(std::integral_constant<int, 6>{});
  if (status == MUON_OK) status = poly(std::integral_constant<int, 8>{});
  if (status != MUON_OK) return status;
  return every_kind(apply);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t ns_blocks_workspace_bytes(const muon_block_problem* probs, int nprobs) {
  if (probs == nullptr || nprobs <= 0 || nprobs > MUON_BLOCKS_MAX_PROBLEMS) return 0;
  for (int i = 0; i < nprobs; ++i)
    if (!valid_shape(probs[i])) return 0;
  const int64_t total = count_blocks(probs, nprobs);
  size_t bytes = 0;
  for (int i = 0; i < nprobs; ++i)
    if (!empty(probs[i])) make_run(probs[i], total, bytes);
  return bytes;
}

int ns_blocks(const muon_block_problem* probs, int nprobs, float a, float b, float c, int steps, void* workspace,
              size_t ws_bytes, void* stream) {
  return run_blocks(probs, nprobs, a, b, c, steps, Epilogue{0.0f, 0.0f, 0}, workspace, ws_bytes,
                    static_cast<hipStream_t>(stream));
}

int ns_blocks_update(const muon_block_problem* probs, int nprobs, float a, float b, float c, int steps, float eta,
                     float decay, float scale, void* workspace, size_t ws_bytes, void* stream) {
  const Epilogue e{float(1.0 - double(eta) * double(decay)), float(double(eta) * double(scale)), 1};
  return run_blocks(probs, nprobs, a, b, c, steps, e, workspace, ws_bytes, static_cast<hipStream_t>(stream));
}

}  // extern "C"
