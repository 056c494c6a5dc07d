// Newton-Schulz orthogonalisation of many small blocks (the heads of attention
// projections): short side s <= 128, any long side, any row pitch.
//
// One iteration is X' = (a I + b A + c A A) X with A = X X^T on the short side.
// With X = T X0, T starts as I and stays a polynomial of A0 = X0 X0^T, and so does
// every later A; polynomials of one symmetric matrix are symmetric and commute:
//     P = a I + b A + c A A,   T' = P T,   A' = X' X'^T = P (P A).
// The long side is therefore touched twice only: once for A0, once for U = T X0.
// All iterations between work on s x s matrices, one workgroup per block.
// X0 = M / |M|_F, and |M|_F^2 is the trace of M M^T.  Three launches serve every block
// of a call:
//   gram   partial M M^T over chunks of the long side (lower 16 x 16 tiles only)
//   poly   sums the chunks in order, scales by the trace, iterates, writes T / |M|_F
//   apply  U = T M, or W <- (1 - eta decay) W - eta scale U
//
// Rounding.  A holds the squares of the singular values, so what rounding leaves in it
// in a direction that M lacks (or nearly lacks) grows by up to a^2 per iteration, where an
// iteration on X would see it grow by a; and a negative leftover grows without end.  In
// fp32 that is up to 2^-24 11.9^5 = 1% of U after five quintic steps on a block of low
// rank, and nothing is left of U after ten.  Gram and iterations are therefore computed in fp64, on the fp64
// matrix instructions: the same leftover is 2^-53 11.9^5.
// T reaches a^steps in the directions that M lacks, where its products with M cancel.  Up
// to 512 (five quintic steps) T and an fp32 M enter the last product in three bf16 parts
// each, and the six products of parts that reach 2^-24 are added in fp32: 2^-24 512 of U
// at worst, half of what an iteration on X in fp32 leaves.  (Two parts cost a bf16 U of
// low rank as much as its own rounding.)  Beyond that the last product is fp64 too.
#include <algorithm>
#include <cmath>

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

__host__ __device__ constexpr int tiles_of(int ny) { return ny * (ny + 1) / 2; }

// lower tile t -> (row, column)
__device__ __forceinline__ void tile_rc(int t, int& i, int& j) {
  i = 0;
  while (tiles_of(i + 1) <= t) ++i;
  j = t - tiles_of(i);
}

// v_mfma_f64_16x16x4: lane 16 g + i gives row i of the first operand and column i of the
// second, both for k = g, and holds rows 4 v + g of column i of the result.
typedef double f64x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void mma64(double a, double b, f64x4_t& acc) {
  acc = __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, acc, 0, 0, 0);
}

typedef double f64x2_t __attribute__((ext_vector_type(2)));

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

constexpr int kParts = 3;   // bf16 parts of T

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
// registers (LD 16-byte pieces of each of THREADS threads), so that it is under way while the
// region before is multiplied.  Its loads have no branches of their own, in which they
// would have to be waited for: rows and columns past the end are read at the last place
// that exists, and put right by piece(), where the values are used.  Rows shorter than a
// piece are read there altogether.
// With ANEW the addresses are formed at every fetch, instead of a row's being kept in
// registers for each piece.
template <typename T, int LD, bool ANEW = false, int THREADS = 256>
struct Region {
  static constexpr int E = 16 / int(sizeof(T));
  u32x4_t w[LD];
  const T* src;
  int64_t ld;
  int rows, cols, r0, c0, per, n;

  __device__ __forceinline__ void fetch(const T* from, int64_t pitch, int nrows, int ncols, int row0, int col0, int NR, int NC) {
    src = from; ld = pitch; rows = nrows; cols = ncols; r0 = row0; c0 = col0;
    per = NC / E; n = NR * per;
    if (cols >= E) {
      int first = threadIdx.x;
      if (ANEW) asm volatile("" : "+v"(first));
#pragma unroll
      for (int q = 0; q < LD; ++q) {
        const int t = min(first + THREADS * q, n - 1);
        const uint4 v = load16(src + int64_t(min(r0 + t / per, rows - 1)) * ld + min(c0 + t % per * E, cols - E));
        w[q] = u32x4_t{v.x, v.y, v.z, v.w};
      }
    }
  }

  // what fetch() got for piece q: row r, columns c .. c + E - 1 of the matrix
  __device__ __forceinline__ u32x4_t piece(int q, int r, int c) const {
    u32x4_t v = {0, 0, 0, 0};
    if (r < rows && c < cols) {
      if (c + E <= cols) {
        v = w[q];
      } else if (cols >= E) {   // the last E columns, of which the first lie before c
        uint64_t lo = w[q][0] | uint64_t(w[q][1]) << 32, hi = w[q][2] | uint64_t(w[q][3]) << 32;
        const int bits = (c + E - cols) * int(sizeof(T)) * 8;
        if (bits >= 64) {
          lo = hi >> (bits - 64);
          hi = 0;
        } else {
          lo = lo >> bits | hi << (64 - bits);
          hi >>= bits;
        }
        v = u32x4_t{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
      } else {
        const T* p = src + int64_t(r) * ld + c;
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (c + k < cols) {
            if constexpr (sizeof(T) == 2) v[k >> 1] |= uint32_t(p[k]) << (16 * (k & 1));
            else v[k] = __float_as_uint(p[k]);
          }
      }
    }
    return v;
  }

  // tile holds U for the region: dst = U, or c1 (what fetch() got) - c2 U
  __device__ __forceinline__ void finish(const float* tile, int tile_ld, T* dst, int64_t pitch, int nrows, int ncols, int row0,
                                         int col0, int NR, int NC, const Epilogue& e) const {
    const int pieces = NC / E;
#pragma unroll
    for (int q = 0; q < LD; ++q) {
      const int t = threadIdx.x + THREADS * q;
      if (t < NR * pieces) {
        const int lr = t / pieces, lc = t % pieces * E, r = row0 + lr, c = col0 + lc;
        if (r >= nrows || c >= ncols) continue;
        float v[E];
#pragma unroll
        for (int k = 0; k < E; k += 4) {
          const f32x4_t x = *reinterpret_cast<const f32x4_t*>(tile + lr * tile_ld + lc + k);
#pragma unroll
          for (int m = 0; m < 4; ++m) v[k + m] = x[m];
        }
        if (e.update) {
          const u32x4_t was = piece(q, r, c);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            float o;
            if constexpr (sizeof(T) == 2) o = __uint_as_float((k & 1) ? was[k >> 1] & 0xffff0000u : was[k >> 1] << 16);
            else o = __uint_as_float(was[k]);
            v[k] = fmaf(e.c1, o, -e.c2 * v[k]);
          }
        }
        T* p = dst + int64_t(r) * pitch + c;
        if (c + E <= ncols) {
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
            if (c + k < ncols) p[k] = from_f32<T>(v[k]);
        }
      }
    }
  }

  // to LDS as fp64: converting takes the same units as the matrix instructions (13 cycles
  // of their 64), so it is done once for each entry
  __device__ __forceinline__ void store_f64(char* lds, int pitch) const {
#pragma unroll
    for (int q = 0; q < LD; ++q) {
      const int t = threadIdx.x + THREADS * q;
      if (t < n) {
        const int r = t / per, c = t % per * E;
        const u32x4_t x = piece(q, r0 + r, c0 + c);
        f64x2_t* dst = reinterpret_cast<f64x2_t*>(lds + r * pitch + c * 8);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          if constexpr (sizeof(T) == 2) dst[k] = f64x2_t{__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xffff0000u)};
          else dst[k] = f64x2_t{__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])};
        }
      }
    }
  }

  // to LDS as bf16 planes: a bf16 entry as it is, an fp32 entry as its NP leading bf16 parts
  template <int NP>
  __device__ __forceinline__ void store(char* lds, int pitch, int plane) const {
#pragma unroll
    for (int q = 0; q < LD; ++q) {
      const int t = threadIdx.x + THREADS * q;
      if (t < n) {
        const int r = t / per, c = t % per * E;
        const u32x4_t x = piece(q, r0 + r, c0 + c);
        char* dst = lds + r * pitch + c * 2;
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<u32x4_t*>(dst) = x;
        } else {
          f32x2_t lo = {__uint_as_float(x[0]), __uint_as_float(x[1])};
          f32x2_t hi = {__uint_as_float(x[2]), __uint_as_float(x[3])};
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
// gram: lower 16 x 16 tile t of M M^T over one chunk, in fp64, as it lies in the
// accumulators: [t][4][64].  Bound by the fp64 matrix instructions (64 cycles each; two
// thirds of them at most while the next slab is converted and laid out): 144 blocks 768 x 64
// bf16 21 us, 32 blocks 128 x 4096 fp32 53 us, 50 blocks 80 x 2309 fp32 27 us.
// ---------------------------------------------------------------------------
constexpr int gram_slab(bool big) { return big ? 32 : 64; }   // k-values staged at a time

template <typename T, bool TALL, bool BIG>
__global__ __launch_bounds__(256, 2) void blocks_gram_kernel(Runs runs, char* ws) {
  constexpr int SLAB = gram_slab(BIG), SIDE = BIG ? 128 : 64;
  // fp64; tall [SLAB][s]: 16 entries of two rows at once, so that rows start half the banks
  // apart; wide [s][SLAB]: 16 bytes of 16 rows at once
  constexpr int PITCH = 8 * (TALL ? SIDE : SLAB) + (TALL ? 128 : 16);
  constexpr int NA = BIG ? 9 : 3;   // lower tiles of a wave
  __shared__ __attribute__((aligned(16))) char lds[(TALL ? SLAB : SIDE) * PITCH];
  int u = blockIdx.x;
  const Run& run = find_run(runs, u, 0);
  const int b = u / run.chunks, chunk = u % run.chunks;
  const int s = run.s, l = run.l, ny = (s + 15) / 16, sp = 16 * ny;
  const T* M = static_cast<const T*>(run.M) + b * run.stride_m;
  const int64_t ld = run.ld_m;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int nlow = tiles_of(ny);
  const int k0 = chunk * run.chunk, k1 = min(l, k0 + run.chunk);   // chunks are whole slabs, but for the last
  f64x4_t acc[NA];
#pragma unroll
  for (int q = 0; q < NA; ++q) acc[q] = f64x4_t{0.0, 0.0, 0.0, 0.0};
  Region<T, SIDE * SLAB * int(sizeof(T)) / 16 / 256> reg;
  auto fetch = [&](int k) __attribute__((always_inline)) {
    if (TALL) reg.fetch(M, ld, l, s, k, 0, SLAB, sp);
    else reg.fetch(M, ld, s, l, 0, k, sp, SLAB);
  };
  fetch(k0);
  constexpr int STEPS = SLAB / 8;
  int at[NA][2];                    // where the operands of the wave's tiles begin
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    int ti, tj;
    tile_rc(min(wave + 4 * q, nlow - 1), ti, tj);
    at[q][0] = TALL ? g * PITCH + (16 * ti + i) * 8 : (16 * ti + i) * PITCH + 16 * g;
    at[q][1] = TALL ? g * PITCH + (16 * tj + i) * 8 : (16 * tj + i) * PITCH + 16 * g;
  }
  for (int k = k0; k < k1; k += SLAB) {
    __syncthreads();
    reg.store_f64(lds, PITCH);
    __syncthreads();
    if (k + SLAB < k1) fetch(k + SLAB);
    // Pairs of k-values (any order will do, as long as both operands have the same), each read
    // while the pair before is multiplied.
    f64x2_t f[2][2];
    auto read = [&](int n) __attribute__((always_inline)) {
      const int q = n / STEPS, h = n % STEPS;
      if constexpr (TALL) {
        const char *pa = lds + at[q][0] + 8 * h * PITCH, *pb = lds + at[q][1] + 8 * h * PITCH;
        f[n & 1][0] = f64x2_t{*reinterpret_cast<const double*>(pa), *reinterpret_cast<const double*>(pa + 4 * PITCH)};
        f[n & 1][1] = f64x2_t{*reinterpret_cast<const double*>(pb), *reinterpret_cast<const double*>(pb + 4 * PITCH)};
      } else {
        f[n & 1][0] = *reinterpret_cast<const f64x2_t*>(lds + at[q][0] + 64 * h);
        f[n & 1][1] = *reinterpret_cast<const f64x2_t*>(lds + at[q][1] + 64 * h);
      }
    };
    read(0);
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      if (wave + 4 * q < nlow) {
#pragma unroll
        for (int n = q * STEPS; n < (q + 1) * STEPS; ++n) {
          if (n + 1 < NA * STEPS) read(n + 1);
          __builtin_amdgcn_sched_barrier(0);   // the reads stay in front
          mma64(f[n & 1][0][0], f[n & 1][1][0], acc[q]);
          mma64(f[n & 1][0][1], f[n & 1][1][1], acc[q]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
  double* dst = reinterpret_cast<double*>(ws + run.partials) + int64_t(u) * nlow * 256;
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const int t = wave + 4 * q;
    if (t < nlow)
#pragma unroll
      for (int v = 0; v < 4; ++v) dst[t * 256 + v * 64 + lane] = acc[q][v];
  }
}

// ---------------------------------------------------------------------------
// poly: one workgroup per block, one wave per strip of 16 columns
// ---------------------------------------------------------------------------
// Every matrix here is symmetric, so of NY x NY tiles only those at most NY / 2 below the
// diagonal, counted cyclically, are computed: wave j computes tile rows j .. j + NY / 2 of
// strip j (at an even NY the last of them only for j < NY / 2), which is the same work for
// every SIMD and half of the products.  They go to LDS, where the others are read
// transposed.  Of the tiles on the diagonal only the lower half is kept, for both: what
// rounding leaves in A that is not symmetric would grow by a^3 per iteration instead of a^2.
// A wave holds its strip as it comes out of the matrix instruction, tile slot d being tile
// row (j + d) % NY: element v of lane 16 g + i is row 4 v + g, column i of the tile.  That is
// also the second operand of four instructions that contract the tile's 16 rows, so a strip
// is its own second operand without leaving the registers.  First operands are rows of S,
// by symmetry columns, and come from LDS in the same layout.
// 17 products of a block in five steps, one after another on one CU: 40 us at s = 64, 74 at
// 80, 171 at 128 (up to 256 blocks); the SIMDs multiply during 48%, 49% and 82% of it (at 80
// one of them has two of the five strips).
template <int NY>
struct SymTiles {
  static constexpr int H = NY / 2;                 // slots 0 .. H are computed
  static constexpr int LD = 17, TILE = 16 * LD;    // doubles; rows of 17, so that transposed reads spread over the banks
  static constexpr int BYTES = tiles_of(NY) * TILE * 8;
  static_assert(2 * BYTES <= 160 * 1024, "two matrices fit LDS");
  int j, i, g;                                     // strip of the wave, lane

  __device__ __forceinline__ bool own(int d) const { return 2 * d < NY || (2 * d == NY && j < H); }
  // where the computed tile `delta` rows below the diagonal of strip c lies
  __device__ __forceinline__ static int at(int delta, int c) { return (delta * NY + c) * TILE; }
  // What addresses are made of: the strip, and element v = 0 of the lane in a tile as it is
  // stored and transposed.  Unknown to the compiler anew for each operation, or it keeps the
  // addresses of all of them in registers at once.
  struct Origin {
    int j, direct, across;
  };
  __device__ __forceinline__ Origin origin() const {
    Origin o{j, g * LD + i, i * LD + g};
    asm volatile("" : "+s"(o.j), "+v"(o.direct), "+v"(o.across));
    return o;
  }
  // element v = 0 of this lane in tile (row, col), row = col + delta (mod NY), and the step to
  // the next v: in the stored tile itself or, transposed, in tile (col, row)
  __device__ __forceinline__ static int first(const Origin& o, int delta, int row, int col, int& step) {
    const bool direct = 2 * delta < NY || (2 * delta == NY && col < H);
    step = direct ? 4 * LD : 4;
    return direct ? at(delta, col) + o.direct : at(NY - delta, row) + o.across;
  }
  __device__ __forceinline__ int wrap(int t) const { return t >= NY ? t - NY : t; }

  __device__ __forceinline__ void put(double* buf, const f64x4_t (&x)[H + 1]) const {
    const Origin o = origin();
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (4 * v + g >= i) {
        buf[at(0, o.j) + o.direct + 4 * v * LD] = x[0][v];
        buf[at(0, o.j) + o.across + 4 * v] = x[0][v];
      }
#pragma unroll
    for (int d = 1; d <= H; ++d)
      if (own(d))
#pragma unroll
        for (int v = 0; v < 4; ++v) buf[at(d, o.j) + o.direct + 4 * v * LD] = x[d][v];
  }
  // the whole strip: what the wave computed off the diagonal (unless `all` is read), and the
  // rest from LDS
  __device__ __forceinline__ void complete(const double* buf, const f64x4_t (&x)[H + 1], f64x4_t (&to)[NY],
                                           bool all = false) const {
    const Origin o = origin();
#pragma unroll
    for (int d = 0; d < NY; ++d) {
      if (d > 0 && d <= H && own(d) && !all) {
        to[d] = x[d <= H ? d : 0];
      } else {
        int step;
        const double* p = buf + first(o, d, wrap(o.j + d), o.j, step);
#pragma unroll
        for (int v = 0; v < 4; ++v) to[d][v] = p[v * step];
      }
    }
  }
  // the computed tiles of S by, S in LDS; the next first operands are read while the
  // current ones multiply
  __device__ __forceinline__ void product(const double* buf, const f64x4_t (&by)[NY], f64x4_t (&out)[H + 1]) const {
    if (own(H)) multiply<H + 1>(buf, by, out);
    else multiply<H>(buf, by, out);
  }
  template <int N>
  __device__ __forceinline__ void multiply(const double* buf, const f64x4_t (&by)[NY], f64x4_t (&out)[H + 1]) const {
    const Origin o = origin();
    double f[2][N];
    auto read = [&](int k) __attribute__((always_inline)) {
      const int e = k >> 2, v = k & 3;
#pragma unroll
      for (int d = 0; d < N; ++d) {
        // S's tile (row j + d, column j + e), by symmetry (j + e, j + d)
        int step;
        const double* p = buf + first(o, (e - d + NY) % NY, wrap(o.j + e), wrap(o.j + d), step);
        f[k & 1][d] = p[v * step];
      }
    };
#pragma unroll
    for (int d = 0; d < N; ++d) out[d] = f64x4_t{0.0, 0.0, 0.0, 0.0};
    read(0);
#pragma unroll
    for (int k = 0; k < 4 * NY; ++k) {
      if (k + 1 < 4 * NY) read(k + 1);
      __builtin_amdgcn_sched_barrier(0);   // the reads stay in front
#pragma unroll
      for (int d = 0; d < N; ++d)
        mma64(f[k & 1][d], by[k >> 2][k & 3], out[d]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

template <int NY>
__global__ __launch_bounds__(64 * NY, 2) void blocks_poly_kernel(Runs runs, char* ws, double a, double b, double c, int steps,
                                                                    int exact) {
  extern __shared__ __attribute__((aligned(16))) char sm[];
  using S_ = SymTiles<NY>;
  constexpr int H = S_::H, LD = S_::LD, TILE = S_::TILE, NLOW = tiles_of(NY);
  double* const bufA = reinterpret_cast<double*>(sm);
  double* const bufP = reinterpret_cast<double*>(sm + S_::BYTES);
  int u = blockIdx.x;
  const Run& run = find_run(runs, u, 1);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const S_ sym{wave, lane & 15, lane >> 4};
  const int i = sym.i, g = sym.g;
  f64x4_t A[NY], T[NY], out[H + 1];
  double root;                                     // 1 / |M|_F
  {
    // The chunks' Grams, added in their order, pairs of columns by all threads (four chunks'
    // loads in flight).  Tile (ti, tj) is stored as it is or, where it lies more than half way
    // down, as the transposed tile of strip ti.
    constexpr int Q = NY + 1, THREADS = 64 * NY;   // pairs of a thread: 128 in each tile
    const int chunks = run.chunks;
    const f64x2_t* src = reinterpret_cast<const f64x2_t*>(ws + run.partials) + int64_t(u) * chunks * NLOW * 128 + threadIdx.x;
    f64x2_t sum[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) sum[q] = f64x2_t{0.0, 0.0};
    int k = 0;
    for (; k + 4 <= chunks; k += 4, src += 4 * NLOW * 128) {
      f64x2_t w[4][Q];
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int q = 0; q < Q; ++q) w[e][q] = src[e * NLOW * 128 + q * THREADS];
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int q = 0; q < Q; ++q) sum[q] += w[e][q];
    }
    for (; k < chunks; ++k, src += NLOW * 128)
#pragma unroll
      for (int q = 0; q < Q; ++q) sum[q] += src[q * THREADS];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int p = threadIdx.x + q * THREADS, row = (p & 127) >> 3, col = 2 * (p & 7);
      int ti, tj;
      tile_rc(__builtin_amdgcn_readfirstlane(p >> 7), ti, tj);
      const bool direct = 2 * (ti - tj) <= NY;
      double* at = bufA + (direct ? S_::at(ti - tj, tj) + row * LD + col : S_::at(NY - (ti - tj), ti) + col * LD + row);
      at[0] = sum[q][0];
      at[direct ? 1 : LD] = sum[q][1];
    }
    __syncthreads();
    sym.complete(bufA, out, A, true);
    double total = 0.0;                            // |M|_F^2, the diagonal of the tiles on the diagonal
#pragma unroll
    for (int d = 0; d < 16 * NY; d += 64)
      if (d + lane < 16 * NY) total += bufA[S_::at(0, (d + lane) >> 4) + ((d + lane) & 15) * (LD + 1)];
    total = wave_sum(total);                       // every wave adds the same entries in the same order
    // a block of zeros gives U = 0; infinities and NaN make everything NaN
    const double inv = total == 0.0 ? 0.0 : total - total == 0.0 ? 1.0 / total : __builtin_nan("");
    root = total == 0.0 ? 0.0 : total - total == 0.0 ? 1.0 / sqrt(total) : __builtin_nan("");
#pragma unroll
    for (int d = 0; d < NY; ++d)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        A[d][v] *= inv;
        if (d <= H) out[d <= H ? d : 0][v] = A[d][v];
        T[d][v] = d == 0 && 4 * v + g == i ? 1.0 : 0.0;
      }
    __syncthreads();
    sym.put(bufA, out);
    __syncthreads();
  }
  for (int it = 0; it < steps; ++it) {
    const bool last = it == steps - 1;
    if (c != 0.0) {
      sym.product(bufA, A, out);                   // A A
    } else {
#pragma unroll
      for (int d = 0; d <= H; ++d) out[d] = f64x4_t{0.0, 0.0, 0.0, 0.0};
    }
    int on = i - g;                                // a on the diagonal, found anew instead of kept in registers
    asm volatile("" : "+v"(on));
#pragma unroll
    for (int d = 0; d <= H; ++d)
#pragma unroll
      for (int v = 0; v < 4; ++v) out[d][v] = fma(c, out[d][v], fma(b, A[d][v], d == 0 && 4 * v == on ? a : 0.0));
    sym.put(bufP, out);                            // P; its readers of the step before have met since
    __syncthreads();
    if (it == 0) {
      sym.complete(bufP, out, T);                  // T = P
    } else {
      sym.product(bufP, T, out);                   // T' = P T, through the buffer that A A has left
      sym.put(bufA, out);
      __syncthreads();
      sym.complete(bufA, out, T);
    }
    if (last) break;
    sym.product(bufP, A, out);                     // P A
    __syncthreads();
    sym.put(bufA, out);
    __syncthreads();
    sym.complete(bufA, out, A);
    sym.product(bufP, A, out);                     // A' = P (P A)
    __syncthreads();
    sym.put(bufA, out);
    __syncthreads();
    sym.complete(bufA, out, A);
  }
  if (exact) {   // T / |M|_F, rows of [16 NY][16 NY]
    double* dst = reinterpret_cast<double*>(ws + run.parts) + int64_t(u) * (256 * NY * NY) + 16 * wave + i;
#pragma unroll
    for (int d = 0; d < NY; ++d)
#pragma unroll
      for (int v = 0; v < 4; ++v) dst[(16 * sym.wrap(wave + d) + 4 * v + g) * (16 * NY)] = T[d][v] * root;
    return;
  }
  // or in three bf16 parts, rows of [part][sp][sp] with zeros past the last strip
  constexpr int sp = (NY + 1) / 2 * 32;
  bf16_t* dst = reinterpret_cast<bf16_t*>(ws + run.parts) + int64_t(u) * kParts * sp * sp;
#pragma unroll
  for (int d = 0; d < NY; ++d)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      f32x2_t x = {float(T[d][v] * root), 0.0f};
      bf16_t* at = dst + (16 * sym.wrap(wave + d) + 4 * v + g) * sp + 16 * wave + i;
#pragma unroll
      for (int p = 0; p < kParts; ++p) at[p * sp * sp] = bf16_t(leading_part(x));
    }
  if (NY % 2 != 0)
    for (int t = threadIdx.x; t < kParts * 16 * sp; t += 64 * NY) {
      const int p = t / (16 * sp), row = t / sp % 16, col = t % sp;
      dst[p * sp * sp + (16 * NY + row) * sp + col] = 0;
      dst[p * sp * sp + col * sp + 16 * NY + row] = 0;
    }
}

// ---------------------------------------------------------------------------
// apply: U = T M.  A wave keeps 32 rows of T in registers and multiplies them with its
// share of a slab of the long side.  The results meet in LDS in the output's own layout
// (over the slab's operand planes, which are done with), so that the output is read (for
// an update; fetched while the slab is multiplied) and written in whole rows, 16 bytes
// per lane.  Bound by memory for a bf16 M: 144 blocks 768 x 64 updated 17.4 us; an fp32 M's
// splitting and six products take about as long: 32 blocks 128 x 4096, bf16 W updated, 44 us.
// ---------------------------------------------------------------------------
// entries of the long side at a time: 64 keep two waves per SIMD in registers
constexpr int apply_slab(bool all_bf16, bool big) { return all_bf16 && !big ? 128 : 64; }
template <typename T, typename TO, bool TALL, bool BIG>
struct ApplyTile {
  static constexpr int LS = apply_slab(sizeof(T) == 2 && sizeof(TO) == 2, BIG), SIDE = BIG ? 128 : 64, NQ = SIDE / 16;
  static constexpr int NPT = kParts;                       // bf16 parts of T
  static constexpr int NPM = sizeof(T) == 2 ? 1 : kParts;  // and of M
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
  Region<T, C_::M_LOADS, true> reg;
  Region<TO, C_::OUT_LOADS, true> old;
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
    reg.template store<NPM>(lds, PITCH, PLANE);
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
// apply in fp64, where T is too large for parts.  A wave keeps 16 rows of T in registers
// and multiplies them with its share of a slab: four waves, or eight over a short side of
// 64.  The results meet in LDS as fp32, as above.  32 blocks 128 x 4096, fp32 M, bf16 W
// updated: 114 us, 50 blocks 80 x 2309 fp32 55, half of it matrix instructions.
// ---------------------------------------------------------------------------
constexpr int kExactSlab = 64;   // entries of the long side at a time
template <typename T, typename TO, bool TALL, bool BIG>
struct ExactTile {
  static constexpr int THREADS = BIG ? 512 : 256;
  static constexpr int LS = kExactSlab, SIDE = BIG ? 128 : 64, NK = SIDE / 16;
  // fp64; tall [LS][s]: 16 bytes of 16 rows at once; wide [s][LS]: 16 entries of two rows four
  // apart, which start half the banks apart
  static constexpr int PITCH = TALL ? 8 * SIDE + 16 : 8 * LS + 32;
  static constexpr int ROWS = TALL ? LS : SIDE, COLS = TALL ? SIDE : LS;        // of the tiles of M and of the output
  static constexpr int M_BYTES = ROWS * PITCH;
  static constexpr int OUT_LD = COLS + 4;
  static constexpr int LDS_BYTES = M_BYTES + ROWS * OUT_LD * 4;
  static constexpr int M_LOADS = SIDE * LS * int(sizeof(T)) / 16 / THREADS, OUT_LOADS = SIDE * LS * int(sizeof(TO)) / 16 / THREADS;
};

template <typename T, typename TO, bool TALL, bool BIG>
__global__ __launch_bounds__(BIG ? 512 : 256, 2) void blocks_apply_exact_kernel(Runs runs, const char* ws, Epilogue e) {
  using C_ = ExactTile<T, TO, TALL, BIG>;
  constexpr int LS = C_::LS, NK = C_::NK, PITCH = C_::PITCH, CT = LS / 16;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  float* const tile = reinterpret_cast<float*>(lds + C_::M_BYTES);
  int u = blockIdx.x;
  const Run& run = find_run(runs, u, 2);
  const int b = u / run.units, unit = u % run.units;
  const int s = run.s, l = run.l, ny = (s + 15) / 16, sp = 16 * ny;
  const T* M = static_cast<const T*>(run.M) + b * run.stride_m;
  TO* out = static_cast<TO*>(run.out) + b * run.stride_out;
  const int64_t ld = run.ld_m, ld_out = run.ld_out;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  // The wave's row tile of T, and its 16-entry columns of the slab.  Up to four row tiles: a
  // wave each, the slab shared where there are fewer.  More: waves 0 - 3 take one each, and of
  // those left over one is cut in four, two in two, three or four are taken whole.
  int row, first, step, count;
  if (!BIG || wave < 4) {
    const int tiles = BIG ? 4 : ny, groups = 4 / tiles;
    row = wave % tiles; first = wave / tiles; step = groups;
    count = first < groups ? CT / groups : 0;
  } else {
    const int w = wave - 4, extra = ny - 4, groups = extra <= 2 ? 4 / extra : 1;
    row = 4 + w % (4 / groups); first = w / (4 / groups); step = groups;
    count = w < extra * groups ? CT / groups : 0;
  }
  const int l0 = unit * run.slabs * LS, l1 = min(l, l0 + run.slabs * LS);
  Region<T, C_::M_LOADS, true, C_::THREADS> reg;
  Region<TO, C_::OUT_LOADS, true, C_::THREADS> old;
  auto fetch = [&](int x) __attribute__((always_inline)) {
    if (TALL) reg.fetch(M, ld, l, s, x, 0, LS, sp);
    else reg.fetch(M, ld, s, l, 0, x, sp, LS);
  };
  fetch(l0);
  // lane 16 g + i: row i of the tile, k-values 16 q + 4 g .. + 3
  f64x4_t tf[NK];
#pragma unroll
  for (int q = 0; q < NK; ++q) {
    tf[q] = f64x4_t{0.0, 0.0, 0.0, 0.0};
    if (q < ny && count > 0)
      tf[q] = *reinterpret_cast<const f64x4_t*>(reinterpret_cast<const double*>(ws + run.parts) + int64_t(b) * sp * sp +
                                                (row * 16 + i) * sp + 16 * q + 4 * g);
  }
  for (int x = l0; x < l1; x += LS) {
    reg.store_f64(lds, PITCH);
    __syncthreads();   // the slab is here, and the tile before has been read
    if (e.update) {
      if (TALL) old.fetch(out, ld_out, l, s, x, 0, LS, sp);
      else old.fetch(out, ld_out, s, l, 0, x, sp, LS);
    }
    if (x + LS < l1) fetch(x + LS);
    for (int k = 0; k < count; ++k) {
      const int j = first + k * step;
      f64x4_t acc[2] = {f64x4_t{0.0, 0.0, 0.0, 0.0}, f64x4_t{0.0, 0.0, 0.0, 0.0}};   // neither waits for the other
      // M's four k-values, each read while the four before are multiplied
      f64x4_t m[2];
      auto read = [&](int q) __attribute__((always_inline)) {
        if constexpr (TALL) {
          const f64x2_t* p = reinterpret_cast<const f64x2_t*>(lds + (16 * j + i) * PITCH + (16 * q + 4 * g) * 8);
          const f64x2_t a = p[0], b = p[1];
          m[q & 1] = f64x4_t{a[0], a[1], b[0], b[1]};
        } else {
          const char* p = lds + (16 * q + 4 * g) * PITCH + (16 * j + i) * 8;
#pragma unroll
          for (int c = 0; c < 4; ++c) m[q & 1][c] = *reinterpret_cast<const double*>(p + c * PITCH);
        }
      };
      read(0);
#pragma unroll
      for (int q = 0; q < NK; ++q) {
        if (q < ny) {
          if (q + 1 < NK) read(q + 1);
          __builtin_amdgcn_sched_barrier(0);   // the reads stay in front
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // tall: the slab's rows first, as U's rows lie along the long side
            if (TALL) mma64(m[q & 1][c], tf[q][c], acc[c & 1]);
            else mma64(tf[q][c], m[q & 1][c], acc[c & 1]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      const int r = (TALL ? 16 * j : 16 * row) + g, c = (TALL ? 16 * row : 16 * j) + i;
#pragma unroll
      for (int v = 0; v < 4; ++v) tile[(r + 4 * v) * C_::OUT_LD + c] = float(acc[0][v] + acc[1][v]);
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

// How a problem is cut.  Chunks of the long side for the Gram, so that all blocks of the
// call together give the 256 CUs one workgroup each at most, or two over 128 blocks: it is
// bound by the matrix instructions, and a second, half filled round costs as much as a whole
// one.  A chunk is never shorter than twice the short side: each one writes a whole partial
// Gram, 4 s^2 bytes, and the one CU that iterates reads them all.  Slabs per unit of the
// last product: about four workgroups for each CU (two over a short side of 64, which need
// twice the registers).
void cut(Run& r, int64_t total_blocks, bool exact) {
  total_blocks = std::max<int64_t>(total_blocks, 1);
  const int64_t slab = gram_slab((r.kind & kBig) != 0);
  const int64_t chunks = std::min(std::max<int64_t>((total_blocks <= 128 ? 256 : 512) / total_blocks, 1), ceil_div(r.l, 2 * r.s));
  r.chunk = int(ceil_div(ceil_div(r.l, chunks), slab) * slab);
  r.chunks = int(ceil_div(r.l, r.chunk));
  const int64_t want = ceil_div((r.kind & kBig) ? 512 : 1024, total_blocks);
  const int64_t ls = exact ? kExactSlab : apply_slab(!(r.kind & kF32) && !r.out_f32, (r.kind & kBig) != 0);
  const int64_t slabs = ceil_div(r.l, ls);
  r.slabs = int(ceil_div(slabs, std::min<int64_t>(slabs, want)));
  r.units = int(ceil_div(slabs, r.slabs));
}

// Fills the run of one problem and moves `bytes` past its workspace.
Run make_run(const muon_block_problem& p, int64_t total_blocks, bool exact, size_t& bytes) {
  Run r{};
  const bool tall = p.rows > p.cols;
  r.M = p.M; r.out = p.out;
  r.ld_m = p.ld_m; r.stride_m = p.stride_m; r.ld_out = p.ld_out; r.stride_out = p.stride_out;
  r.s = int(std::min(p.rows, p.cols)); r.l = int(std::max(p.rows, p.cols)); r.count = int(p.count);
  r.kind = (tall ? kTall : 0) | (p.m_dtype == MUON_F32 ? kF32 : 0) | (r.s > 64 ? kBig : 0);
  r.out_f32 = p.out_dtype == MUON_F32;
  cut(r, total_blocks, exact);
  const int64_t sp = ceil_div(r.s, 32) * 32;
  r.partials = int64_t(bytes);
  bytes += round_up(size_t(r.count) * r.chunks * tiles_of(int(ceil_div(r.s, 16))) * 2048, 256);
  r.parts = int64_t(bytes);
  bytes += round_up(size_t(r.count) * sp * sp * 8, 256);   // in fp64, or in parts of 6 bytes
  return r;
}

// Largest factor by which a step scales a singular value of at most 1: the maximum of
// |a + b x + c x x| over x in [0, 1], at least 1.
double growth(double a, double b, double c) {
  double g = std::max(std::max(1.0, std::abs(a)), std::abs(a + b + c));
  const double x = c != 0.0 ? -b / (2.0 * c) : 0.0;
  if (x > 0.0 && x < 1.0) g = std::max(g, std::abs(a + b * x + c * x * x));
  return g;
}
constexpr double kPartsGrowth = 9.0;   // log2 of what T may reach for the last product to take it in bf16 parts

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

template <typename T, typename TO, bool TALL, bool BIG>
int launch_exact(const Runs& runs, const char* ws, const Epilogue& e, hipStream_t st) {
  int64_t units = 0;
  for (int i = 0; i < runs.n; ++i) units += int64_t(runs.r[i].count) * runs.r[i].units;
  using C_ = ExactTile<T, TO, TALL, BIG>;
  static std::atomic<uint64_t> configured{0};
  if (gemm::set_lds_limit(blocks_apply_exact_kernel<T, TO, TALL, BIG>, C_::LDS_BYTES, configured) != MUON_OK) return MUON_ELAUNCH;
  launch_kernel(blocks_apply_exact_kernel<T, TO, TALL, BIG>, dim3(units), dim3(C_::THREADS), C_::LDS_BYTES, st, runs, ws, e);
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
  const double t_growth = steps == 0 ? 0.0 : steps * std::log2(growth(a, b, c));   // log2 of what T may reach
  if (t_growth > MUON_BLOCKS_MAX_GROWTH) return MUON_EINVAL;
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
  const bool exact = t_growth > kPartsGrowth;
  Run all[MUON_BLOCKS_MAX_PROBLEMS];
  int n = 0;
  size_t bytes = 0;
  for (int i = 0; i < nprobs; ++i)
    if (!empty(probs[i])) all[n++] = make_run(probs[i], total, exact, bytes);
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
                                [&](const Runs& runs) {
                                  return exact ? launch_exact<T, bf16_t, TALL, BIG>(runs, ws, e, st)
                                               : launch_apply<T, bf16_t, TALL, BIG>(runs, ws, e, st);
                                });
    if (status != MUON_OK) return status;
    return for_runs(all, n, [](const Run& r) { return r.kind == kind_of<T, TALL, BIG>() && r.out_f32; },
                    [&](const Runs& runs) {
                      return exact ? launch_exact<T, float, TALL, BIG>(runs, ws, e, st)
                                   : launch_apply<T, float, TALL, BIG>(runs, ws, e, st);
                    });
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
    return for_runs(all, n, [](const Run& r) { return (r.s + 15) / 16 == NY; }, [&](const Runs& runs) {
      int64_t blocks = 0;
      for (int i = 0; i < runs.n; ++i) blocks += runs.r[i].count;
      constexpr int LDS = 2 * SymTiles<NY>::BYTES;
      static std::atomic<uint64_t> configured{0};
      if (gemm::set_lds_limit(blocks_poly_kernel<NY>, LDS, configured) != MUON_OK) return int(MUON_ELAUNCH);
      launch_kernel(blocks_poly_kernel<NY>, dim3(blocks), dim3(64 * NY), LDS, st, runs, ws, double(a), double(b), double(c),
                    steps, int(exact));
      return launch_status();
    });
  };
  status = poly(std::integral_constant<int, 1>{});
  if (status == MUON_OK) status = poly(std::integral_constant<int, 2>{});
  if (status == MUON_OK) status = poly(std::integral_constant<int, 3>{});
  if (status == MUON_OK) status = poly(std::integral_constant<int, 4>{});
  if (status == MUON_OK) status = poly(std::integral_constant<int, 5>{});
  if (status == MUON_OK) status = poly(std::integral_constant<int, 6>{});
  if (status == MUON_OK) status = poly(std::integral_constant<int, 7>{});
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
    if (!empty(probs[i])) make_run(probs[i], total, false, bytes);
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
