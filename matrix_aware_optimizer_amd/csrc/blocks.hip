// Newton-Schulz orthogonalisation of many small blocks (the heads of attention
// projections): short side s <= 128, any long side, any row pitch.
//
// One iteration is X' = (a I + b A + c A A) X with A = X X^T on the short side.
// With X = T X0, T starts as I and stays a polynomial of A0 = X0 X0^T, and so does
// every later A; polynomials of one symmetric matrix are symmetric and commute:
//     P = a I + b A + c A A,   T' = P T,   A' = X' X'^T = P A P.
// The long side is therefore touched twice only: once for A0, once for U = T X0.
// All iterations between work on s x s matrices, in fp32 on matrix cores, one
// workgroup per block with everything in LDS.  X0 = M / |M|_F, and |M|_F^2 is the
// trace of M M^T.  Three launches serve every block of a call:
//   gram   partial M M^T over chunks of the long side (lower 32 x 32 tiles only)
//   poly   sums the chunks in order, scales by the trace, iterates, writes T / |M|_F
//   apply  U = T M, or W <- (1 - eta decay) W - eta scale U
//
// Rounding.  A relative error d of A0 grows by at most a^2 per iteration where A is
// small, so A and T are held and multiplied in fp32 (products of bf16 splits would
// not do: 2^-17 a^8 is 0.15 for a = 3.4445).  The products with a bf16 M are exact
// in bf16 matrix instructions; T enters the last one as the sum of two bf16 parts
// (error 2^-17, under half a step of a bf16 U or W) or three (fp32 outputs: 2^-25).
#include <algorithm>

#include "common.h"
#include "gemm.h"

namespace muon {
namespace {

constexpr int kMaxRuns = 24;       // problems of one launch (by-value kernel argument)
constexpr int kTile = 32;
constexpr int kTilePitch = 33;     // floats per row of a tile in LDS
constexpr int kTileFloats = kTile * kTilePitch;
constexpr int kMaxTiles = 10;      // lower 32 x 32 tiles of a 128 x 128 matrix

// One problem: `count` blocks of rows x cols, seen as s x l with s <= l (tall: transposed)
struct Run {
  const void* M;
  void* out;
  int64_t ld_m, stride_m, ld_out, stride_out;
  int64_t partials, parts;   // byte offsets of its partial Grams and its T in the workspace
  int32_t s, l, count, chunk, chunks, slabs, units;   // chunk: k-values per gram unit; slabs per apply unit
  int32_t vec_m, vec_out, kind;   // kind: kTall | kF32
  int32_t out_f32;
};
enum { kTall = 1, kF32 = 2 };

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

// Rows [r0, r0 + NR) and columns [c0, c0 + NC) of a row-major matrix into LDS rows of
// `pitch` bytes; entries outside rows x cols become zero.
template <typename T>
__device__ __forceinline__ void load_region(const T* src, int64_t ld, int rows, int cols, int r0, int c0, int NR, int NC,
                                            char* lds, int pitch, bool vec) {
  constexpr int E = 16 / sizeof(T);
  const int per = NC / E, n = NR * per;
  for (int t = threadIdx.x; t < n; t += 256) {
    const int r = t / per, c = (t % per) * E;
    const T* p = src + int64_t(r0 + r) * ld + c0 + c;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (r0 + r < rows) {
      if (vec && c0 + c + E <= cols) {
        w = *reinterpret_cast<const uint4*>(p);
      } else {
        T e[E];
#pragma unroll
        for (int q = 0; q < E; ++q) e[q] = c0 + c + q < cols ? p[q] : T(0);
        w = *reinterpret_cast<const uint4*>(e);
      }
    }
    *reinterpret_cast<uint4*>(lds + r * pitch + c * int(sizeof(T))) = w;
  }
}

// LDS pitches (bytes), so that one access spreads over the 64 banks.  Rows read 16
// bytes per lane along themselves: 16 over a multiple of 128 (eight rows start in
// eight different groups of four banks).  bf16 rows read transposed, four rows at a
// time: 64 over a multiple of 256.  fp32 rows read across by the two half-waves, four
// rows apart: 32 over a multiple of 64 (four rows are half the banks).
constexpr int kRowPitchTr = 320;

// ---------------------------------------------------------------------------
// gram: tile t of M M^T over one chunk, as it lies in the accumulators: [t][16][64]
// ---------------------------------------------------------------------------
template <typename T, bool TALL>
__global__ __launch_bounds__(256) void blocks_gram_kernel(Runs runs, char* ws) {
  constexpr int SLAB = 128 / sizeof(T);            // k-values staged at a time
  constexpr int PITCH_W = 128 + 16;                // wide: [s][SLAB]
  constexpr int PITCH_T = sizeof(T) == 2 ? kRowPitchTr : 544;   // tall: [SLAB][s]
  __shared__ __attribute__((aligned(16))) char lds[TALL ? SLAB * PITCH_T : 128 * PITCH_W];
  int u = blockIdx.x;
  const Run& run = find_run(runs, u, 0);
  const int b = u / run.chunks, chunk = u % run.chunks;
  const int s = run.s, l = run.l, nt = (s + 31) / 32, sp = nt * 32;
  const T* M = static_cast<const T*>(run.M) + b * run.stride_m;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 31, h = lane >> 5;
  const int nlow = tiles_of(nt);
  const int k0 = chunk * run.chunk, k1 = min(l, k0 + run.chunk);
  f32x16_t acc[3];
#pragma unroll
  for (int q = 0; q < 3; ++q)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[q][v] = 0.0f;
  for (int k = k0; k < k1; k += SLAB) {
    __syncthreads();
    if (TALL) load_region<T>(M, run.ld_m, k1, s, k, 0, SLAB, sp, lds, PITCH_T, run.vec_m);
    else load_region<T>(M, run.ld_m, s, k1, 0, k, sp, SLAB, lds, PITCH_W, run.vec_m);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const int t = wave + 4 * q;
      if (t < nlow) {
        int ti, tj;
        tile_rc(t, ti, tj);
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            u32x4_t fa, fb;
            if constexpr (TALL) {
              const int gi = lane & 15, G = lane >> 4;
              const char* base = lds + (ks * 16 + 8 * (G >> 1) + (gi >> 2)) * PITCH_T + (16 * (G & 1) + 4 * (gi & 3)) * 2;
              fa = gemm::read_tr_pair(base + ti * 64, base + ti * 64 + 4 * PITCH_T);
              fb = gemm::read_tr_pair(base + tj * 64, base + tj * 64 + 4 * PITCH_T);
            } else {
              fa = *reinterpret_cast<const u32x4_t*>(lds + (ti * 32 + fr) * PITCH_W + (2 * ks + h) * 16);
              fb = *reinterpret_cast<const u32x4_t*>(lds + (tj * 32 + fr) * PITCH_W + (2 * ks + h) * 16);
            }
            gemm::Mfma<bf16_t>::mma(fa, fb, acc[q]);
          }
        } else {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            f32x4_t fa, fb;
            if constexpr (TALL) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const char* row = lds + (8 * g + 4 * h + e) * PITCH_T + fr * 4;
                fa[e] = *reinterpret_cast<const float*>(row + ti * 128);
                fb[e] = *reinterpret_cast<const float*>(row + tj * 128);
              }
            } else {
              fa = *reinterpret_cast<const f32x4_t*>(lds + (ti * 32 + fr) * PITCH_W + (2 * g + h) * 16);
              fb = *reinterpret_cast<const f32x4_t*>(lds + (tj * 32 + fr) * PITCH_W + (2 * g + h) * 16);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[q] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[e], fb[e], acc[q], 0, 0, 0);
          }
        }
      }
    }
  }
  float* dst = reinterpret_cast<float*>(ws + run.partials) + int64_t(u) * nlow * 1024;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const int t = wave + 4 * q;
    if (t < nlow)
#pragma unroll
      for (int v = 0; v < 16; ++v) dst[t * 1024 + v * 64 + lane] = acc[q][v];
  }
}

// ---------------------------------------------------------------------------
// poly: one workgroup per block, one wave per lower tile
// ---------------------------------------------------------------------------
// Fragment of symmetric matrix S (lower tiles in LDS): entry (row 32 X + r, column
// 32 K + k), from the tile itself or, above the diagonal, from its mirror image.
struct TileReader {
  const float* p;
  int step;   // floats from one k to the next
};
__device__ __forceinline__ TileReader tile_reader(const float* S, int X, int K, int r, int h) {
  const bool low = X >= K;
  const int t = low ? X * (X + 1) / 2 + K : K * (K + 1) / 2 + X;
  const float* base = S + t * kTileFloats;
  return low ? TileReader{base + r * kTilePitch + h, 1} : TileReader{base + r + h * kTilePitch, kTilePitch};
}

// acc += tile (ti, tj) of L R, both symmetric
__device__ __forceinline__ void sym_product(const float* L, const float* R, int ti, int tj, int nt, int r, int h,
                                            f32x16_t& acc) {
  for (int K = 0; K < nt; ++K) {
    const TileReader a = tile_reader(L, ti, K, r, h), b = tile_reader(R, tj, K, r, h);
#pragma unroll
    for (int k = 0; k < 16; ++k)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.p[2 * k * a.step], b.p[2 * k * b.step], acc, 0, 0, 0);
  }
}

__device__ __forceinline__ void put_tile(float* S, int t, int r, int h, const f32x16_t& v) {
#pragma unroll
  for (int q = 0; q < 16; ++q) S[t * kTileFloats + (8 * (q >> 2) + 4 * h + (q & 3)) * kTilePitch + r] = v[q];
}

__global__ __launch_bounds__(64 * kMaxTiles) void blocks_poly_kernel(Runs runs, char* ws, float a, float b, float c,
                                                                     int steps) {
  extern __shared__ __attribute__((aligned(16))) float sm[];
  __shared__ double trace[4];
  int u = blockIdx.x;
  const Run& run = find_run(runs, u, 1);
  const int s = run.s, nt = (s + 31) / 32, nlow = tiles_of(nt), sp = nt * 32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  const bool busy = wave < nlow;
  float* SA = sm;
  float* ST = sm + nlow * kTileFloats;
  float* SP = sm + 2 * nlow * kTileFloats;
  int ti = 0, tj = 0;
  tile_rc(busy ? wave : 0, ti, tj);
  f32x16_t A, T, P;
#pragma unroll
  for (int v = 0; v < 16; ++v) A[v] = T[v] = P[v] = 0.0f;
  // entries of this lane on the matrix's diagonal
  auto diag = [&](int v) { return ti == tj && 8 * (v >> 2) + 4 * h + (v & 3) == r; };
  if (busy) {
    const float* src = reinterpret_cast<const float*>(ws + run.partials) + int64_t(u) * run.chunks * nlow * 1024 +
                       wave * 1024 + lane;
    for (int k = 0; k < run.chunks; ++k)
#pragma unroll
      for (int v = 0; v < 16; ++v) A[v] += src[int64_t(k) * nlow * 1024 + v * 64];
    if (ti == tj) {
      double t = 0.0;
#pragma unroll
      for (int v = 0; v < 16; ++v) t += diag(v) ? double(A[v]) : 0.0;
      t = wave_sum(t);
      if (lane == 0) trace[ti] = t;
    }
  }
  __syncthreads();
  double total = 0.0;
  for (int i = 0; i < nt; ++i) total += trace[i];
  // a block of zeros gives U = 0
  const float inv = total == 0.0 ? 0.0f : float(1.0 / total);
  const float root = total == 0.0 ? 0.0f : float(1.0 / sqrt(total));
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    A[v] *= inv;
    T[v] = diag(v) ? 1.0f : 0.0f;
  }
  if (busy && steps > 0) put_tile(SA, wave, r, h, A);
  for (int it = 0; it < steps; ++it) {
    __syncthreads();
    if (busy) {
#pragma unroll
      for (int v = 0; v < 16; ++v) P[v] = 0.0f;
      if (c != 0.0f) sym_product(SA, SA, ti, tj, nt, r, h, P);
#pragma unroll
      for (int v = 0; v < 16; ++v) P[v] = fmaf(c, P[v], fmaf(b, A[v], diag(v) ? a : 0.0f));
      put_tile(SP, wave, r, h, P);
      if (it == 0) {
        T = P;
        put_tile(ST, wave, r, h, T);
      }
    }
    __syncthreads();
    const bool last = it == steps - 1;
    f32x16_t Y, T2;
    if (busy) {
#pragma unroll
      for (int v = 0; v < 16; ++v) Y[v] = T2[v] = 0.0f;
      if (it > 0) {
        sym_product(SP, ST, ti, tj, nt, r, h, T2);
        T = T2;
      }
      if (!last) sym_product(SP, SA, ti, tj, nt, r, h, Y);
    }
    if (last) break;
    __syncthreads();
    if (busy) {
      put_tile(SA, wave, r, h, Y);
      if (it > 0) put_tile(ST, wave, r, h, T);
    }
    __syncthreads();
    if (busy) {
#pragma unroll
      for (int v = 0; v < 16; ++v) A[v] = 0.0f;
      sym_product(SA, SP, ti, tj, nt, r, h, A);
    }
    __syncthreads();
    if (busy) put_tile(SA, wave, r, h, A);
  }
  if (!busy) return;
  // T / |M|_F, both triangles: fp32 [sp][sp], or two or three bf16 parts of it
  char* base = ws + run.parts;
  if (run.kind & kF32) {
    float* dst = reinterpret_cast<float*>(base) + int64_t(u) * sp * sp;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int i = ti * 32 + 8 * (v >> 2) + 4 * h + (v & 3), j = tj * 32 + r;
      dst[i * sp + j] = T[v] * root;
      if (ti != tj) dst[j * sp + i] = T[v] * root;
    }
  } else {
    bf16_t* dst = reinterpret_cast<bf16_t*>(base) + int64_t(u) * 3 * sp * sp;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int i = ti * 32 + 8 * (v >> 2) + 4 * h + (v & 3), j = tj * 32 + r;
      float x = T[v] * root;
      for (int part = 0; part < 3; ++part) {
        const bf16_t p = f32_to_bf16(x);
        x -= bf16_to_f32(p);
        dst[part * sp * sp + i * sp + j] = p;
        if (ti != tj) dst[part * sp * sp + j * sp + i] = p;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// apply: U = T M.  A wave keeps 32 rows of T in registers and runs over the long
// side; the operand whose index is contiguous in the output comes first, so a lane
// holds four consecutive entries of an output row.
// ---------------------------------------------------------------------------
template <typename TO>
__device__ __forceinline__ void write4(TO* dst, const float v[4], int valid, bool vec, const Epilogue& e) {
  if (vec && valid >= 4) {
    float o[4];
    if constexpr (sizeof(TO) == 2) {
      if (e.update) {
        const uint2 w = *reinterpret_cast<const uint2*>(dst);
        o[0] = fmaf(e.c1, __uint_as_float(w.x << 16), -e.c2 * v[0]);
        o[1] = fmaf(e.c1, __uint_as_float(w.x & 0xffff0000u), -e.c2 * v[1]);
        o[2] = fmaf(e.c1, __uint_as_float(w.y << 16), -e.c2 * v[2]);
        o[3] = fmaf(e.c1, __uint_as_float(w.y & 0xffff0000u), -e.c2 * v[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = v[i];
      }
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(uint32_t(f32_to_bf16(o[0])) | (uint32_t(f32_to_bf16(o[1])) << 16),
                     uint32_t(f32_to_bf16(o[2])) | (uint32_t(f32_to_bf16(o[3])) << 16));
    } else {
      if (e.update) {
        const float4 w = *reinterpret_cast<const float4*>(dst);
        o[0] = fmaf(e.c1, w.x, -e.c2 * v[0]);
        o[1] = fmaf(e.c1, w.y, -e.c2 * v[1]);
        o[2] = fmaf(e.c1, w.z, -e.c2 * v[2]);
        o[3] = fmaf(e.c1, w.w, -e.c2 * v[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = v[i];
      }
      *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < valid) {
        float o = v[i];
        if (e.update) o = fmaf(e.c1, to_f32(dst[i]), -e.c2 * v[i]);
        dst[i] = from_f32<TO>(o);
      }
  }
}

template <typename T> constexpr int apply_slab() { return sizeof(T) == 2 ? 128 : 64; }   // long-side entries at a time

template <typename T, typename TO, bool TALL>
__global__ __launch_bounds__(256) void blocks_apply_kernel(Runs runs, const char* ws, Epilogue e) {
  constexpr int LS = apply_slab<T>();
  constexpr bool BF = sizeof(T) == 2;
  constexpr int NP = BF ? (sizeof(TO) == 2 ? 2 : 3) : 1;
  constexpr int PITCH = TALL ? 128 * int(sizeof(T)) + 16 : (BF ? kRowPitchTr : 288);   // tall [LS][s], wide [s][LS]
  constexpr int NF = BF ? 8 : 16;                    // 16-byte fragments of 128 k-values
  __shared__ __attribute__((aligned(16))) char lds[(TALL ? LS : 128) * PITCH];
  int u = blockIdx.x;
  const Run& run = find_run(runs, u, 2);
  const int b = u / run.units, unit = u % run.units;
  const int s = run.s, l = run.l, nt = (s + 31) / 32, sp = nt * 32;
  const T* M = static_cast<const T*>(run.M) + b * run.stride_m;
  TO* out = static_cast<TO*>(run.out) + b * run.stride_out;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 31, h = lane >> 5;
  // 4 waves: row tile ti, and every groups-th 32 entries of the long side
  const int groups = 4 / nt, ti = wave % nt, grp = wave / nt;
  const bool busy = grp < groups;
  u32x4_t tf[NP][NF];
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int q = 0; q < NF; ++q) {
      tf[p][q] = u32x4_t{0, 0, 0, 0};
      const int kq = BF ? 16 * q + 8 * h : 8 * q + 4 * h;   // first k of this lane's 16 bytes
      if (kq < sp && busy) {
        const char* base = ws + run.parts;
        const int64_t at = int64_t(ti * 32 + fr) * sp + kq;
        if constexpr (BF)
          tf[p][q] = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const bf16_t*>(base) +
                                                       (int64_t(b) * 3 + p) * sp * sp + at);
        else
          tf[p][q] = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const float*>(base) + int64_t(b) * sp * sp + at);
      }
    }
  const int l0 = unit * run.slabs * LS, l1 = min(l, l0 + run.slabs * LS);
  for (int x = l0; x < l1; x += LS) {
    __syncthreads();
    if (TALL) load_region<T>(M, run.ld_m, l, s, x, 0, LS, sp, lds, PITCH, run.vec_m);
    else load_region<T>(M, run.ld_m, s, l, 0, x, sp, LS, lds, PITCH, run.vec_m);
    __syncthreads();
    if (!busy) continue;
    for (int j = grp; j < LS / 32; j += groups) {
      if (x + 32 * j >= l1) break;
      f32x16_t acc;
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
#pragma unroll
      for (int q = 0; q < NF; ++q) {
        if ((BF ? 16 : 8) * q < sp) {
          if constexpr (BF) {
            u32x4_t fm;
            if constexpr (TALL) {
              fm = *reinterpret_cast<const u32x4_t*>(lds + (32 * j + fr) * PITCH + (2 * q + h) * 16);
            } else {
              const int gi = lane & 15, G = lane >> 4;
              const char* base = lds + (q * 16 + 8 * (G >> 1) + (gi >> 2)) * PITCH + (32 * j + 16 * (G & 1) + 4 * (gi & 3)) * 2;
              fm = gemm::read_tr_pair(base, base + 4 * PITCH);
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              if (TALL) gemm::Mfma<bf16_t>::mma(tf[p][q], fm, acc);
              else gemm::Mfma<bf16_t>::mma(fm, tf[p][q], acc);
            }
          } else {
            f32x4_t fm;
            if constexpr (TALL) {
              fm = *reinterpret_cast<const f32x4_t*>(lds + (32 * j + fr) * PITCH + (2 * q + h) * 16);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                fm[k] = *reinterpret_cast<const float*>(lds + (8 * q + 4 * h + k) * PITCH + (32 * j + fr) * 4);
            }
            const f32x4_t t = __builtin_bit_cast(f32x4_t, tf[0][q]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (TALL) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(t[k], fm[k], acc, 0, 0, 0);
              else acc = __builtin_amdgcn_mfma_f32_32x32x2f32(fm[k], t[k], acc, 0, 0, 0);
            }
          }
        }
      }
      // accumulator v of this lane: first operand's row 8 (v / 4) + 4 h + v % 4, second's row fr
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v[4] = {acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
        const int first = 8 * q + 4 * h;
        const int row = TALL ? x + 32 * j + fr : ti * 32 + fr;
        const int col = TALL ? ti * 32 + first : x + 32 * j + first;
        if (row < (TALL ? l : s)) write4<TO>(out + int64_t(row) * run.ld_out + col, v, (TALL ? s : l) - col, run.vec_out, e);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
  size_t bytes = 0;
  int64_t blocks = 0;
};

bool valid_shape(const muon_block_problem& p) {
  if (p.rows < 0 || p.cols < 0 || p.count < 0) return false;
  if (p.rows > MUON_BLOCKS_MAX_LONG || p.cols > MUON_BLOCKS_MAX_LONG || p.count > MUON_BLOCKS_MAX_COUNT) return false;
  return std::min(p.rows, p.cols) <= MUON_BLOCKS_MAX_SHORT;
}
bool empty(const muon_block_problem& p) { return p.rows == 0 || p.cols == 0 || p.count == 0; }

// How a problem is cut: chunks of the long side for the Gram, slabs per unit of the
// last product, chosen so that all blocks of the call together give the 256 CUs
// about four workgroups each (two or three fit one by their LDS), but a chunk is
// never shorter than 256 entries: each one writes and reads a whole partial Gram.
void cut(Run& r, int64_t total_blocks) {
  const int64_t want = std::max<int64_t>(1, ceil_div(1024, std::max<int64_t>(total_blocks, 1)));
  const int64_t slab = (r.kind & kF32) ? 32 : 64;
  int64_t chunks = std::min<int64_t>(want, ceil_div(r.l, 256));
  r.chunk = int(ceil_div(ceil_div(r.l, chunks), slab) * slab);
  r.chunks = int(ceil_div(r.l, r.chunk));
  const int64_t ls = (r.kind & kF32) ? apply_slab<float>() : apply_slab<bf16_t>();
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
  r.kind = (tall ? kTall : 0) | (p.m_dtype == MUON_F32 ? kF32 : 0);
  r.out_f32 = p.out_dtype == MUON_F32;
  const int64_t em = p.m_dtype == MUON_F32 ? 4 : 8;
  r.vec_m = p.ld_m % em == 0 && (p.count <= 1 || p.stride_m % em == 0);
  r.vec_out = p.ld_out % 4 == 0 && (p.count <= 1 || p.stride_out % 4 == 0);
  cut(r, total_blocks);
  const int64_t nt = ceil_div(r.s, 32), sp = nt * 32;
  r.partials = int64_t(bytes);
  bytes += round_up(size_t(r.count) * r.chunks * tiles_of(int(nt)) * 4096, 256);
  r.parts = int64_t(bytes);
  bytes += round_up(size_t(r.count) * sp * sp * ((r.kind & kF32) ? 4 : 6), 256);
  return r;
}

int64_t count_blocks(const muon_block_problem* probs, int n) {
  int64_t total = 0;
  for (int i = 0; i < n; ++i)
    if (!empty(probs[i])) total += probs[i].count;
  return total;
}

template <typename T, typename TO, bool TALL>
int launch_apply(const Runs& runs, const char* ws, const Epilogue& e, hipStream_t st) {
  int64_t units = 0;
  for (int i = 0; i < runs.n; ++i) units += int64_t(runs.r[i].count) * runs.r[i].units;
  launch_kernel(blocks_apply_kernel<T, TO, TALL>, dim3(units), dim3(256), 0, st, runs, ws, e);
  return launch_status();
}

template <typename T, bool TALL>
int launch_gram(const Runs& runs, char* ws, hipStream_t st) {
  int64_t units = 0;
  for (int i = 0; i < runs.n; ++i) units += int64_t(runs.r[i].count) * runs.r[i].chunks;
  launch_kernel(blocks_gram_kernel<T, TALL>, dim3(units), dim3(256), 0, st, runs, ws);
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
  int n = 0, max_tiles = 0;
  size_t bytes = 0;
  for (int i = 0; i < nprobs; ++i)
    if (!empty(probs[i])) {
      all[n] = make_run(probs[i], total, bytes);
      max_tiles = std::max(max_tiles, tiles_of((all[n].s + 31) / 32));
      ++n;
    }
  for (int kind = 0; kind < 4; ++kind) {
    const int status = for_runs(all, n, [&](const Run& r) { return r.kind == kind; }, [&](const Runs& runs) {
      switch (kind) {
        case 0: return launch_gram<bf16_t, false>(runs, ws, st);
        case kTall: return launch_gram<bf16_t, true>(runs, ws, st);
        case kF32: return launch_gram<float, false>(runs, ws, st);
        default: return launch_gram<float, true>(runs, ws, st);
      }
    });
    if (status != MUON_OK) return status;
  }
  const int lds = 3 * max_tiles * kTileFloats * 4;
  static std::atomic<uint64_t> configured{0};
  if (gemm::set_lds_limit(blocks_poly_kernel, 3 * kMaxTiles * kTileFloats * 4, configured) != MUON_OK) return MUON_ELAUNCH;
  int status = for_runs(all, n, [](const Run&) { return true; }, [&](const Runs& runs) {
    int64_t blocks = 0;
    for (int i = 0; i < runs.n; ++i) blocks += runs.r[i].count;
    launch_kernel(blocks_poly_kernel, dim3(blocks), dim3(64 * max_tiles), lds, st, runs, ws, a, b, c, steps);
    return launch_status();
  });
  if (status != MUON_OK) return status;
  for (int kind = 0; kind < 8; ++kind) {
    status = for_runs(all, n, [&](const Run& r) { return r.kind == (kind & 3) && r.out_f32 == (kind >> 2); }, [&](const Runs& runs) {
      switch (kind) {
        case 0: return launch_apply<bf16_t, bf16_t, false>(runs, ws, e, st);
        case 1: return launch_apply<bf16_t, bf16_t, true>(runs, ws, e, st);
        case 2: return launch_apply<float, bf16_t, false>(runs, ws, e, st);
        case 3: return launch_apply<float, bf16_t, true>(runs, ws, e, st);
        case 4: return launch_apply<bf16_t, float, false>(runs, ws, e, st);
        case 5: return launch_apply<bf16_t, float, true>(runs, ws, e, st);
        case 6: return launch_apply<float, float, false>(runs, ws, e, st);
        default: return launch_apply<float, float, true>(runs, ws, e, st);
      }
    });
    if (status != MUON_OK) return status;
  }
  return MUON_OK;
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
