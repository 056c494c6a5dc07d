// Products C = A B^T on matrix cores for the gated block (bf16) and the 8-bit integer
// products (gfx950, wave64): one tile unit for every operand layout, and a kernel for few
// rows.  What happens to a sum (scales, activation, momentum) is an `Out` of the caller.
//
// Operands.  A step of the contraction is 64 bytes of every row: 32 bf16 or 64 int8 values.
//   rows      [row][k], k contiguous.  LDS: 64-byte rows of four 16-byte chunks, chunk c of
//             row r at slot c ^ ((r / 4) % 4).
//   k-major   [k][row] (bf16 only), rows contiguous along the tile's side.  LDS: 32 k-rows of
//             2 x side bytes, chunk c of k-row k at slot c ^ (4 (k % 4)), read transposed by
//             ds_read_b64_tr_b16: lane i of 16 gets the four k-values of column i.
// Both put the k-values 8 (2 p + h) .. + 7 of a step (int8: 16 of them) into lane half h of
// matrix instruction p, so operands of different layouts go together.
//
// Unit.  BM x BN of C by (BM / WM) (BN / WN) waves.  A ring of S stages in LDS is filled by
// global -> LDS DMA, 16 bytes per lane.  Per step: wait until this wave's copies of the next
// stage have landed, s_barrier (everybody's have, and everybody is done with the stage
// before), then multiply this step's operands, and between the matrix instructions read the
// next step's from LDS and start the copy S - 1 steps ahead.
//   DUAL      the tile's columns are halves of two matrices B[0], B[1]: in every wave's WN the
//             first half are columns of B[0], the second the same columns of B[1], so that one
//             lane holds both sums of an output.
//   segments  the contraction runs over (A[0], B[0]) and then (A[1], B[1]).
//   masked    steps that the DMA cannot copy (the last one of a K that is not whole steps, and
//             every step where rows do not start at 16 bytes) go through registers, with zeros
//             past the ends.
//
// Times given as a -> b, or of one side against the other, belong to the choice that they stand
// at: both sides on one card, when it was made.  Later changes moved both.  What the products take
// now stands at mixed_kernel and direct_kernel, over several cards.
#pragma once

#include <algorithm>

#include "common.h"
#include "gemm.h"

namespace muon {
namespace tile {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

enum Kind { kBf16, kI8 };

template <int KIND> struct Math;
template <> struct Math<kBf16> {
  using acc16_t = f32x16_t;   // 32 x 32 block
  using acc4_t = f32x4_t;     // 16 x 16 block
  using sum_t = float;
  static constexpr int kBytes = 2;
  __device__ __forceinline__ static acc16_t mma32(const u32x4_t& a, const u32x4_t& b, const acc16_t& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  }
  __device__ __forceinline__ static acc4_t mma16(const u32x4_t& a, const u32x4_t& b, const acc4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  }
};
template <> struct Math<kI8> {
  using acc16_t = i32x16_t;
  using acc4_t = i32x4_t;
  using sum_t = int;
  static constexpr int kBytes = 1;
  __device__ __forceinline__ static acc16_t mma32(const u32x4_t& a, const u32x4_t& b, const acc16_t& c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
  }
  __device__ __forceinline__ static acc4_t mma16(const u32x4_t& a, const u32x4_t& b, const acc4_t& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
  }
};

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Source {
  const char* A[2];
  const char* B[2];
  int64_t lda, ldb;   // pitches in bytes
  int64_t m, n, K;    // n: columns of one B
  int segs;           // segments of the contraction (1 or 2)
};

// stages of tiles of 128 rows and more (Config::PAIRS)
constexpr int ring_of(bool a_kmajor) { return a_kmajor ? 4 : 5; }

template <int KIND_, int BM_, int BN_, int WM_, int WN_, int S_, bool AT_, bool BT_, bool DUAL_>
struct Config {
  static constexpr int KIND = KIND_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_;
  static constexpr bool AT = AT_, BT = BT_, DUAL = DUAL_;
  static constexpr int NB = DUAL ? 2 : 1, COLS = BN / NB;   // columns of C
  static constexpr int W = (BM / WM) * (BN / WN), NT = W * kWave;
  static constexpr int FM = WM / 32, FN = WN / 32;
  static constexpr int A_BYTES = BM * 64, B_BYTES = BN * 64, STAGE = A_BYTES + B_BYTES;
  static constexpr int LDW = WN + 4;                        // row pitch of the epilogue's slab, in floats
  static constexpr int LDS_BYTES = S * STAGE > W * 32 * LDW * 4 ? S * STAGE : W * 32 * LDW * 4;
  static constexpr int A_DMA = A_BYTES / 1024 / W, B_DMA = B_BYTES / 1024 / W, D = A_DMA + B_DMA;
  // Operands in rows have 64 of a cache line's 128 bytes in a stage.  With an odd number of stages
  // the two stages of a line are copied one right after the other, and the second half comes from
  // the CU's own cache: forward of 4096 x 14336 x 4096 816 -> 780 us, int8 gated 2048 x 14336 x 4096
  // 236 -> 223, 33 rows of it 32.2 -> 26.5, dx of 4096 x 14336 x 4096 (A only) 765 -> 750.  K-major rows
  // are whole lines; gathering two stages' copies of them in every other step costs 5%.
  static constexpr bool PAIRS = !AT && S % 2 == 1;
  // Tiles of few rows are bound by reading B, and all start at once: each begins at another step
  // of the contraction, or the same offsets of many rows (one memory channel, at pitches of 8 KB
  // and more) are wanted together.  33 x 14336 x 8192 bf16, both weights from memory: 125 -> 108 us.
  static constexpr bool TURNED = BM == 64;
  static constexpr int CHUNKS = STAGE / 16 / NT;            // 16-byte chunks per thread of a masked step
  static_assert(A_BYTES % (1024 * W) == 0 && B_BYTES % (1024 * W) == 0, "DMA split");
  static_assert(S >= 3 && D * (S - 2) <= 63 && LDS_BYTES <= 160 * 1024, "ring");
  static_assert((!AT || (BM >= 128 && KIND == kBf16)) && (!BT || (BN >= 128 && KIND == kBf16)), "k-major rows of 256 bytes or more");
  static_assert(!DUAL || (!BT && WN >= 64), "gate and up columns in one wave");
};

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 bytes per lane from base + off to LDS bytes [lds_addr + 16 * lane), with the wait state
// that a load to LDS needs after a scalar write of M0
__device__ __forceinline__ void dma16_at(const char* base, uint32_t off, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base),
               "s"(__builtin_amdgcn_readfirstlane(lds_addr))
               : "memory", "m0");
}
#pragma clang diagnostic pop

// a pointer that is the same in every lane, in scalar registers
__device__ __forceinline__ const char* scalar(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v)), hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
  return reinterpret_cast<const char*>((uint64_t(hi) << 32) | lo);
}

// This wave's copies but the last N have landed and all its LDS reads are done, then all
// waves meet: what lands next may overwrite the stage that was read before.
template <int N>
__device__ __forceinline__ void ring_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// all LDS accesses of the wave are done, then all waves meet; loads to registers stay under way
__device__ __forceinline__ void ring_barrier_lds() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// One tile at rows m0 and columns n0 over steps [s0, s1) of the contraction's whole steps (MASKED:
// through registers); `tail`: then the last, partial step of every segment.
template <class C_, bool MASKED, class Out>
__device__ __forceinline__ void unit(const Source& g, int64_t m0, int64_t n0, int s0, int s1, bool tail, const Out& out, char* lds) {
  using M_ = Math<C_::KIND>;
  constexpr int BM = C_::BM, BN = C_::BN, WM = C_::WM, WN = C_::WN, S = C_::S, FM = C_::FM, FN = C_::FN;
  constexpr int PER_STEP = 64 / M_::kBytes;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 31, h = lane >> 5;
  const int wm0 = (wave / (BN / WN)) * WM, wn0 = (wave % (BN / WN)) * WN;
  const int per = __builtin_amdgcn_readfirstlane(int(g.K / PER_STEP));
  // column of C of B's LDS row (or k-major column) r, and which B it is of
  auto col_of = [](int r) { return C_::DUAL ? (r / WN) * (WN / 2) + r % (WN / 2) : r; };
  auto is_up = [](int r) { return C_::DUAL && r % WN >= WN / 2; };
  // rows past the matrix read its last row; what they compute is not stored
  const int mlast = int(min(g.m - 1 - m0, int64_t(BM - 1))), nlast = int(min(g.n - 1 - n0, int64_t(C_::COLS - 1)));

  typename M_::acc16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;

  struct Frags {
    u32x4_t a[FM][2], b[FN][2];
  };
  // where a lane's operands lie in a stage
  constexpr int ROW_A = 2 * BM, ROW_B = 2 * BN;   // bytes of a k-row
  int a_at[C_::AT ? FM : 2], b_at[C_::BT ? FN : 2];
  const int tq = lane & 3, tj = (lane >> 2) & 3, ts = (lane >> 4) & 1;
  if constexpr (C_::AT) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
      a_at[i] = (8 * h + tj) * ROW_A + ((((wm0 >> 3) + 4 * i + 2 * ts + (tq >> 1)) ^ (4 * tj)) << 4) + (tq & 1) * 8;
  } else {
    a_at[0] = gemm::krow_off(wm0 + fr, h);
    a_at[1] = gemm::krow_off(wm0 + fr, 2 + h);
  }
  if constexpr (C_::BT) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
      b_at[j] = C_::A_BYTES + (8 * h + tj) * ROW_B + ((((wn0 >> 3) + 4 * j + 2 * ts + (tq >> 1)) ^ (4 * tj)) << 4) + (tq & 1) * 8;
  } else {
    b_at[0] = C_::A_BYTES + gemm::krow_off(wn0 + fr, h);
    b_at[1] = C_::A_BYTES + gemm::krow_off(wn0 + fr, 2 + h);
  }
  constexpr int READS = 2 * (FM + FN);
  auto read_one = [&](int q, const char* st, Frags& f) __attribute__((always_inline)) {
    // the operands of the first matrix instructions come first: phase 0 of B and A, then phase 1
    const int p = q / (FM + FN), k = q % (FM + FN);
    if (k < FN) {
      if constexpr (C_::BT) f.b[k][p] = gemm::read_tr_pair(st + b_at[k] + 16 * p * ROW_B, st + b_at[k] + (16 * p + 4) * ROW_B);
      else f.b[k][p] = *reinterpret_cast<const u32x4_t*>(st + b_at[p] + 2048 * k);
    } else {
      const int i = k - FN;
      if constexpr (C_::AT) f.a[i][p] = gemm::read_tr_pair(st + a_at[i] + 16 * p * ROW_A, st + a_at[i] + (16 * p + 4) * ROW_A);
      else f.a[i][p] = *reinterpret_cast<const u32x4_t*>(st + a_at[p] + 2048 * i);
    }
  };
  // one step's products; `between(n)` is what the wave issues after matrix instruction n
  constexpr int N = 2 * FM * FN;
  auto mma = [&](const Frags& f, auto&& between) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int p = n / (FM * FN), i = n % (FM * FN) / FN, j = n % FN;
      acc[i][j] = M_::mma32(f.b[j][p], f.a[i][p], acc[i][j]);
      between(n);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // How the tile leaves (below): a lane takes E columns of every RPP-th row.  What the output needs
  // from memory (a momentum's old values) is loaded a block of 32 rows ahead.
  constexpr int E = Out::E, NB = C_::NB, HALF = WN / NB, LPR = HALF / E, RPP = 64 / LPR, PASSES = 32 / RPP;
  using sum_t = typename Out::sum_t;
  const int pr = lane / LPR, pc = (lane % LPR) * E;
  const int64_t col = n0 + wn0 / NB + pc;
  const bool inside = col + E <= out.width;
  typename Out::template Pre<E> pre[2][PASSES];
  auto load_pre = [&](int i) __attribute__((always_inline)) {
    if (inside)
#pragma unroll
      for (int p = 0; p < PASSES; ++p) pre[i & 1][p] = out.template pre<E>(min(m0 + wm0 + 32 * i + pr + RPP * p, g.m - 1), col);
  };

  if constexpr (!MASKED) {
    // sources of this wave's copies
    uint32_t a_off[C_::A_DMA], b_off[C_::B_DMA];
#pragma unroll
    for (int i = 0; i < C_::A_DMA; ++i) {
      const int b = wave * C_::A_DMA + i;
      if constexpr (C_::AT) {
        constexpr int RC = BM / 8, RB = 64 / RC;
        const int r = RB * b + lane / RC, c = (lane % RC) ^ (4 * (r & 3));
        a_off[i] = uint32_t(r) * uint32_t(g.lda) + (min(c, (mlast + 1) / 8 - 1) << 4);
      } else {
        const int r = 16 * b + (lane >> 2);
        a_off[i] = uint32_t(min(r, mlast)) * uint32_t(g.lda) + (((lane & 3) ^ ((r >> 2) & 3)) << 4);
      }
    }
#pragma unroll
    for (int i = 0; i < C_::B_DMA; ++i) {
      const int b = wave * C_::B_DMA + i;
      if constexpr (C_::BT) {
        constexpr int RC = BN / 8, RB = 64 / RC;
        const int r = RB * b + lane / RC, c = (lane % RC) ^ (4 * (r & 3));
        b_off[i] = uint32_t(r) * uint32_t(g.ldb) + (min(c, (nlast + 1) / 8 - 1) << 4);
      } else {
        const int r = 16 * b + (lane >> 2);
        b_off[i] = uint32_t(min(col_of(r), nlast)) * uint32_t(g.ldb) + (((lane & 3) ^ ((r >> 2) & 3)) << 4);
      }
    }
    const int64_t a_start = C_::AT ? m0 * 2 : m0 * g.lda, b_start = C_::BT ? n0 * 2 : n0 * g.ldb;
    const int64_t a_step = C_::AT ? 32 * g.lda : 64, b_step = C_::BT ? 32 * g.ldb : 64;
    const uint32_t lds_base =
        static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)lds));
    const int nk = s1 - s0;
    const int turn = C_::TURNED && per > 0 ? int(n0 / C_::COLS * 6 % per) & ~1 : 0;   // even: pairs stay pairs
    auto issue_one = [&](int q, int kt, uint32_t off) __attribute__((always_inline)) {
      const int seg = kt >= per ? 1 : 0;
      int k = kt - seg * per;
      if constexpr (C_::TURNED) {
        k += turn;
        k = k >= per ? k - per : k;
      }
      const uint32_t st = lds_base + off;
      if (q < C_::A_DMA) {
        dma16_at(scalar((seg ? g.A[1] : g.A[0]) + a_start + k * a_step), a_off[q], st + (wave * C_::A_DMA + q) * 1024);
      } else {
        const int b = q - C_::A_DMA;
        const bool second = C_::DUAL ? is_up(16 * (wave * C_::B_DMA + b)) : seg != 0;
        dma16_at(scalar((second ? g.B[1] : g.B[0]) + b_start + k * b_step), b_off[b], st + C_::A_BYTES + (wave * C_::B_DMA + b) * 1024);
      }
    };
    auto ring_next = [](uint32_t o) {
      o += C_::STAGE;
      return o == uint32_t(S * C_::STAGE) ? 0u : o;
    };
    if (nk > 0) {
      Frags f0, f1;
      uint32_t o_cur = 0;
      int it = 0;
      constexpr int RPM = (READS + N * 3 / 4 - 1) / (N * 3 / 4);   // reads per MFMA, done after three quarters of them
      // The copies of stages kt and kt + 1 in two steps.  The first takes those of row operands for
      // both, the same rows one after the other, so that the second finds the cache lines that the
      // first has fetched, and a k-major B's for kt; the second step takes a k-major B's for kt + 1.
      constexpr int IN_FIRST = 2 * C_::A_DMA + (C_::BT ? 1 : 2) * C_::B_DMA, IN_SECOND = C_::BT ? C_::B_DMA : 0;
      auto issue_first = [&](int q, int kt, uint32_t o0, uint32_t o1) __attribute__((always_inline)) {
        if (C_::BT && q >= 2 * C_::A_DMA) issue_one(q - C_::A_DMA, kt, o0);
        else issue_one(q >> 1, kt + (q & 1), q & 1 ? o1 : o0);
      };
      auto issue_second = [&](int q, int kt, uint32_t o1) __attribute__((always_inline)) { issue_one(C_::A_DMA + q, kt + 1, o1); };
      constexpr bool PAIRS = C_::PAIRS;
      if (PAIRS && nk >= S - 1) {
#pragma unroll
        for (int s = 0; s < S - 1; s += 2) {
#pragma unroll
          for (int q = 0; q < IN_FIRST; ++q) issue_first(q, s0 + s, uint32_t(s) * C_::STAGE, uint32_t(s + 1) * C_::STAGE);
#pragma unroll
          for (int q = 0; q < IN_SECOND; ++q) issue_second(q, s0 + s, uint32_t(s + 1) * C_::STAGE);
        }
        ring_barrier<C_::D * (S - 3)>();
      } else {
#pragma unroll
        for (int s = 0; s < S - 1; ++s)
          if (s < nk)
#pragma unroll
            for (int q = 0; q < C_::D; ++q) issue_one(q, s0 + s, uint32_t(s) * C_::STAGE);
        if (!PAIRS && nk >= S - 1) ring_barrier<C_::D * (S - 2)>();
        else ring_barrier<0>();
      }
#pragma unroll
      for (int q = 0; q < READS; ++q) read_one(q, lds, f0);
      auto reads_under = [&](int n, const char* st, Frags& nxt) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < RPM; ++r)
          if (RPM * n + r < READS) read_one(RPM * n + r, st, nxt);
      };
      auto ring_before = [](uint32_t o) { return o == 0 ? uint32_t((S - 1) * C_::STAGE) : o - C_::STAGE; };
      // PAIRS: two steps, which copy the stages S - 1 and S steps ahead (to where the step before and
      // this one were read from); each finds all but the last S - 3 stages' copies landed
      auto two_steps = [&]() __attribute__((always_inline)) {
        const uint32_t o1 = ring_next(o_cur), o2 = ring_next(o1), before = ring_before(o_cur);
        ring_barrier<C_::D * (S - 3)>();
        mma(f0, [&](int n) __attribute__((always_inline)) {
          reads_under(n, lds + o1, f1);
#pragma unroll
          for (int q = 0; q < IN_FIRST; ++q)
            if (q * N / IN_FIRST == n) issue_first(q, s0 + it + S - 1, before, o_cur);
        });
        ring_barrier<C_::D * (S - 3)>();
        mma(f1, [&](int n) __attribute__((always_inline)) {
          reads_under(n, lds + o2, f0);
#pragma unroll
          for (int q = 0; q < IN_SECOND; ++q)
            if (q * N / C_::B_DMA == n) issue_second(q, s0 + it + S - 1, o_cur);
        });
        o_cur = o2;
        it += 2;
      };
      // other rings: one step, which copies the stage S - 1 steps ahead
      uint32_t o_iss = uint32_t(S - 1) * C_::STAGE;
      auto steady = [&](Frags& cur, Frags& nxt) __attribute__((always_inline)) {
        const char* st = lds + ring_next(o_cur);
        ring_barrier<C_::D * (S - 3)>();
        mma(cur, [&](int n) __attribute__((always_inline)) {
          reads_under(n, st, nxt);
#pragma unroll
          for (int q = 0; q < C_::D; ++q)
            if (q * N / C_::D == n) issue_one(q, s0 + it + S - 1, o_iss);
        });
        o_cur = ring_next(o_cur);
        o_iss = ring_next(o_iss);
        ++it;
      };
      auto drain = [&](Frags& cur, Frags& nxt) __attribute__((always_inline)) {
        if (it + 1 < nk) {
          ring_barrier<0>();
          const char* st = lds + ring_next(o_cur);
#pragma unroll
          for (int q = 0; q < READS; ++q) read_one(q, st, nxt);
        }
        mma(cur, [](int) {});
        o_cur = ring_next(o_cur);
        ++it;
      };
      if constexpr (PAIRS) {
        while (it + S < nk) two_steps();
        if (it + S - 1 < nk) {   // one more copy is due
          ring_barrier<0>();
#pragma unroll
          for (int q = 0; q < C_::D; ++q) issue_one(q, s0 + it + S - 1, ring_before(o_cur));
        }
      } else {
        while (it + S < nk) {   // two steps that both still copy a stage
          steady(f0, f1);
          steady(f1, f0);
        }
        if (it + S - 1 < nk) {   // one more copy is due
          steady(f0, f1);
          f0 = f1;
        }
      }
      while (it < nk) {
        drain(f0, f1);
        if (it < nk) drain(f1, f0);
      }
    }
  }

  if constexpr (C_::KIND == kBf16) {
    // Steps through registers.  Sixteen bytes are loaded from inside the row (rows have at least
    // eight entries), moved back where it ends, and put right before they go to LDS: no load stands
    // in a branch, where it would be waited for.
    struct Held {
      u32x4_t v[C_::CHUNKS];
      int back[C_::CHUNKS];   // entries that the start was moved back; 8: all of it lies outside
    };
    // chunk i of this thread: whether it is A's, its LDS row and chunk (NT divides both operands' chunks)
    auto place = [&](int i, bool& of_a, int& r, int& c) __attribute__((always_inline)) {
      of_a = i * C_::NT < BM * 4;
      const int x = threadIdx.x + i * C_::NT - (of_a ? 0 : BM * 4);
      const bool t = of_a ? C_::AT : C_::BT;
      const int side = of_a ? BM : BN;
      r = t ? x / (side / 8) : x >> 2;
      c = t ? x % (side / 8) : x & 3;
    };
    auto put_one = [&](int i, const Held& f, char* stage) __attribute__((always_inline)) {
      bool of_a;
      int r, c;
      place(i, of_a, r, c);
      const bool t = of_a ? C_::AT : C_::BT;
      const int at = (of_a ? 0 : C_::A_BYTES) + (t ? r * 2 * (of_a ? BM : BN) + ((c ^ (4 * (r & 3))) << 4) : gemm::krow_off(r, c));
      *reinterpret_cast<u32x4_t*>(stage + at) = f.v[i];
    };
    // entries down by `back`, zeros behind them
    auto shift = [&](Held& f) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < C_::CHUNKS; ++i) {
        const int by = f.back[i];
        u32x4_t v = f.v[i];
        if (by & 4) v = u32x4_t{v[2], v[3], 0, 0};
        if (by & 2) v = u32x4_t{v[1], v[2], v[3], 0};
        if (by & 1) v = u32x4_t{(v[0] >> 16) | (v[1] << 16), (v[1] >> 16) | (v[2] << 16), (v[2] >> 16) | (v[3] << 16), v[3] >> 16};
        if (by >= 8) v = u32x4_t{0, 0, 0, 0};
        f.v[i] = v;
      }
    };

    if constexpr (MASKED) {
      // Whole steps [s0, s1).  At step s: the operands of s are in registers, stage (s + 1) % 2 is
      // written, the loads of s + 2 and s + 3 are under way; its products go with the reads of the
      // next operands, the writes of step s + 2 and the loads of step s + 4.
      uint32_t off[C_::CHUNKS];
      Held h0, h1;
      bool ends = false;
#pragma unroll
      for (int i = 0; i < C_::CHUNKS; ++i) {
        bool of_a;
        int r, c;
        place(i, of_a, r, c);
        const int64_t len = (of_a ? g.m : g.n) - (of_a ? m0 : n0);   // of a k-row from the tile's first column
        int from = 8 * c, back = 0;
        if (of_a ? C_::AT : C_::BT) {
          from = int(min(int64_t(from), len - 8));   // may lie before the tile: rows have eight entries
          back = min(8 * c - from, 8);
          off[i] = uint32_t(r) * uint32_t(of_a ? g.lda : g.ldb) + uint32_t(from * 2 + 16);
        } else {
          off[i] = uint32_t(of_a ? min(r, mlast) : min(col_of(r), nlast)) * uint32_t(of_a ? g.lda : g.ldb) + uint32_t(from * 2 + 16);
        }
        h0.back[i] = h1.back[i] = back;
        ends |= back != 0;
      }
      ends = __any(ends);
      const int64_t a_start = C_::AT ? m0 * 2 : m0 * g.lda, b_start = C_::BT ? n0 * 2 : n0 * g.ldb;
      const int64_t a_step = C_::AT ? 32 * g.lda : 64, b_step = C_::BT ? 32 * g.ldb : 64;
      auto fetch = [&](int s, Held& f) __attribute__((always_inline)) {
        const int seg = s >= per ? 1 : 0, k = s - seg * per;
        // 16 bytes early, as off is 16 bytes late
        const char* pa = scalar((seg ? g.A[1] : g.A[0]) + a_start + k * a_step - 16);
        const char* pb0 = scalar((!C_::DUAL && seg ? g.B[1] : g.B[0]) + b_start + k * b_step - 16);
        const char* pb1 = scalar(g.B[1] + b_start + k * b_step - 16);
#pragma unroll
        for (int i = 0; i < C_::CHUNKS; ++i) {
          bool of_a;
          int r, c;
          place(i, of_a, r, c);
          const char* p = of_a ? pa : C_::DUAL && is_up(r) ? pb1 : pb0;
          const uint4 v = load16(reinterpret_cast<const bf16_t*>(p + off[i]));
          f.v[i] = u32x4_t{v.x, v.y, v.z, v.w};
        }
      };
      auto put = [&](Held& f, char* stage) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < C_::CHUNKS; ++i) put_one(i, f, stage);
      };
      char* stages[2] = {lds, lds + C_::STAGE};
      Frags f0, f1;
      if (s0 < s1) {
        fetch(s0, h0);
        if (s0 + 1 < s1) fetch(s0 + 1, h1);
        if (ends) shift(h0);
        put(h0, stages[0]);
        if (s0 + 2 < s1) fetch(s0 + 2, h0);
        if (s0 + 1 < s1) {
          if (ends) shift(h1);
          put(h1, stages[1]);
        }
        if (s0 + 3 < s1) fetch(s0 + 3, h1);
        ring_barrier_lds();
#pragma unroll
        for (int q = 0; q < READS; ++q) read_one(q, stages[0], f0);
      }
      constexpr int RPM = (READS + N * 3 / 4 - 1) / (N * 3 / 4);
      auto steady = [&](int s, const Frags& cur, Frags& nxt, Held& h, char* own, const char* other) __attribute__((always_inline)) {
        ring_barrier_lds();
        if (ends) shift(h);
        mma(cur, [&](int n) __attribute__((always_inline)) {
#pragma unroll
          for (int r = 0; r < RPM; ++r)
            if (RPM * n + r < READS) read_one(RPM * n + r, other, nxt);
#pragma unroll
          for (int i = 0; i < C_::CHUNKS; ++i)
            if (i * (N / 2) / C_::CHUNKS == n) put_one(i, h, own);
          if (n == N / 2) fetch(s + 4, h);
        });
      };
      auto drain = [&](int s, const Frags& cur, Frags& nxt, Held& h, char* own, const char* other) __attribute__((always_inline)) {
        ring_barrier_lds();
        if (s + 1 < s1)
#pragma unroll
          for (int q = 0; q < READS; ++q) read_one(q, other, nxt);
        if (s + 2 < s1) {
          if (ends) shift(h);
          put(h, own);
        }
        if (s + 4 < s1) fetch(s + 4, h);
        mma(cur, [](int) {});
      };
      int s = s0;
      for (; s + 5 < s1; s += 2) {
        steady(s, f0, f1, h0, stages[0], stages[1]);
        steady(s + 1, f1, f0, h1, stages[1], stages[0]);
      }
      for (; s < s1; s += 2) {
        drain(s, f0, f1, h0, stages[0], stages[1]);
        if (s + 1 < s1) drain(s + 1, f1, f0, h1, stages[1], stages[0]);
      }
    }

    // the partial last step of every segment
    if (tail && g.K % PER_STEP != 0)
      for (int seg = 0; seg < g.segs; ++seg) {
        const int64_t k0 = int64_t(per) * PER_STEP;
        Held f;
#pragma unroll
        for (int i = 0; i < C_::CHUNKS; ++i) {
          bool of_a;
          int r, c;
          place(i, of_a, r, c);
          const bool t = of_a ? C_::AT : C_::BT;
          const bool second = of_a || !C_::DUAL ? seg != 0 : is_up(r);
          const char* base = of_a ? (second ? g.A[1] : g.A[0]) : (second ? g.B[1] : g.B[0]);
          const int64_t ld = of_a ? g.lda : g.ldb, end = of_a ? g.m : g.n;
          // row of memory, entry in it, and how long the row is
          const int64_t row = t ? min(k0 + r, g.K - 1) : of_a ? m0 + min(r, mlast) : n0 + min(col_of(r), nlast);
          const int64_t at = t ? (of_a ? m0 : n0) + 8 * c : k0 + 8 * c, len = t ? end : g.K;
          const bool out_of = at >= len || (t && k0 + r >= g.K);
          const int64_t from = min(at, len - 8);
          const uint4 v = load16(reinterpret_cast<const bf16_t*>(base + row * ld) + from);
          f.v[i] = u32x4_t{v.x, v.y, v.z, v.w};
          f.back[i] = out_of ? 8 : int(at - from);
        }
        __syncthreads();   // everybody is done with the stage
        shift(f);
#pragma unroll
        for (int i = 0; i < C_::CHUNKS; ++i) put_one(i, f, lds);
        __syncthreads();
        Frags fr_;
#pragma unroll
        for (int q = 0; q < READS; ++q) read_one(q, lds, fr_);
        mma(fr_, [](int) {});
      }
  }

  // The tile leaves through LDS, 32 rows at a time and each wave through its own part of the
  // ring, so that rows are read and written 16 bytes per lane and whole lines at a time.
  // Accumulator v of a lane: column 8 (v / 4) + 4 h + v % 4 of B's block, row fr of A's.
  load_pre(0);
  ring_barrier_lds();
  sum_t* slab = reinterpret_cast<sum_t*>(lds) + wave * 32 * C_::LDW;
  typedef sum_t sum4_t __attribute__((ext_vector_type(4)));
  const typename Out::template Cols<E> cols = out.template cols<E>(col);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        sum4_t v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = sum_t(acc[i][j][4 * q + r]);
        *reinterpret_cast<sum4_t*>(slab + fr * C_::LDW + 32 * j + 8 * q + 4 * h) = v;
      }
    const int64_t row0 = m0 + wm0 + 32 * i + pr;
    if (i + 1 < FM) load_pre(i + 1);
    if (inside) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        sum_t v[NB][E];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int k = 0; k < E; k += 4) {
            const sum4_t x = *reinterpret_cast<const sum4_t*>(slab + (pr + RPP * p) * C_::LDW + b * HALF + pc + k);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[b][k + e] = x[e];
          }
        if (row0 + RPP * p < g.m) out.template store<E>(row0 + RPP * p, col, v, cols, pre[i & 1][p]);
      }
    } else {
      for (int p = 0; p < PASSES; ++p)
        if (row0 + RPP * p < g.m)
          for (int k = 0; k < E; ++k)
            if (col + k < out.width) {
              sum_t v[NB][1];
#pragma unroll
              for (int b = 0; b < NB; ++b) v[b][0] = slab[(pr + RPP * p) * C_::LDW + b * HALF + pc + k];
              out.template store<1>(row0 + RPP * p, col + k, v, out.template cols<1>(col + k), out.template pre<1>(row0 + RPP * p, col + k));
            }
    }
  }
}

// ---------------------------------------------------------------------------
// Parts of a split contraction
// ---------------------------------------------------------------------------
// Unjoined sums of one part: [part][batch][row][b][ldp]
template <int KIND, int NB>
struct Partial {
  using sum_t = typename Math<KIND>::sum_t;
  static constexpr int E = 4;
  sum_t* p;
  int64_t ldp, width;
  template <int N> struct Cols {};
  template <int N> struct Pre {};
  template <int N> __device__ __forceinline__ Cols<N> cols(int64_t) const { return {}; }
  template <int N> __device__ __forceinline__ Pre<N> pre(int64_t, int64_t) const { return {}; }
  template <int N>
  __device__ __forceinline__ void store(int64_t row, int64_t col, const sum_t (&v)[NB][N], const Cols<N>&, const Pre<N>&) const {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      sum_t* dst = p + (row * NB + b) * ldp + col;
      if constexpr (N == 4) {
        typedef sum_t sum4_t __attribute__((ext_vector_type(4)));
        *reinterpret_cast<sum4_t*>(dst) = sum4_t{v[b][0], v[b][1], v[b][2], v[b][3]};
      } else {
        dst[0] = v[b][0];
      }
    }
  }
};

// Tile rows walked together, column by column: 32 neighbouring tiles, one XCD's, read 4 panels of A
// and 8 of B.  Measured with 8 rows: forward of 4096 x 14336 x 4096 837 us against 821, int8 1999 x
// 4096 x 14336 135 against 128; with 16: 867 and 136; with 2 backward and weight gradients lose 2%.
constexpr int kGroupRows = 4;

// tile t of the grid of TM x TN tiles: groups of kGroupRows tile rows, column by column
__device__ __forceinline__ void tile_at(int64_t t, int64_t TM, int64_t TN, int64_t& tm, int64_t& tn) {
  const int64_t per = int64_t(kGroupRows) * TN, first = (t / per) * kGroupRows;
  const int64_t size = min(TM - first, int64_t(kGroupRows)), r = t % per;
  tm = __builtin_amdgcn_readfirstlane(int(first + r % size));
  tn = __builtin_amdgcn_readfirstlane(int(r / size));
}

struct Split {
  int parts;     // of the contraction
  int batch;     // products of the launch: A[z] with B[0] (weight gradients), 1 otherwise
  void* sums;    // [parts][batch][m][NB][ldp]
  int64_t ldp;
};

// product z of a batch
__device__ __forceinline__ Source source_at(const Source& g, int z) {
  Source s = g;
  if (z) s.A[0] = g.A[1];
  return s;
}

// All tiles of one size; with SPLIT each is sp.parts units along the contraction, whose sums
// lie one after another in sp.sums.
template <class C_, bool MASKED, bool SPLIT, class Out>
__global__ __launch_bounds__(C_::NT) void tile_kernel(Source g, Out out, Split sp) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  constexpr int PER_STEP = 64 / Math<C_::KIND>::kBytes;
  const int64_t TM = (g.m + C_::BM - 1) / C_::BM, TN = (g.n + C_::COLS - 1) / C_::COLS, tiles = TM * TN;
  const int64_t u = gemm::xcd_remap(blockIdx.x, gridDim.x);
  const int z = __builtin_amdgcn_readfirstlane(int(u / tiles % sp.batch));
  int64_t tm, tn;
  tile_at(u % tiles, TM, TN, tm, tn);
  const int steps = __builtin_amdgcn_readfirstlane(int(g.K / PER_STEP * g.segs));
  const Source s = source_at(g, z);
  if constexpr (SPLIT) {
    // a part's tiles are neighbours
    const int64_t part = u / (tiles * sp.batch);
    // (even first steps: two steps share a cache line)
    const int s0 = __builtin_amdgcn_readfirstlane(int(part * steps / sp.parts) & ~1);
    const int s1 = part == sp.parts - 1 ? steps : __builtin_amdgcn_readfirstlane(int((part + 1) * steps / sp.parts) & ~1);
    using P = Partial<C_::KIND, C_::NB>;
    const P po{static_cast<typename P::sum_t*>(sp.sums) + (part * sp.batch + z) * g.m * C_::NB * sp.ldp, sp.ldp, sp.ldp};
    unit<C_, MASKED>(s, tm * C_::BM, tn * C_::COLS, s0, s1, part == sp.parts - 1, po, lds);
  } else {
    unit<C_, MASKED>(s, tm * C_::BM, tn * C_::COLS, 0, steps, true, out.at(z), lds);
  }
}

// 256 x 256 tiles in rounds of one per CU; those of the last, partial round come in `parts`
// (2: 128 x 256, 4: 128 x 128) so that they fill the CUs.  Workgroups [0, whole) take whole tiles.
// Bound by the matrix cores at the clock that the chip holds under them (1.65 GHz, 2.0 in int8): a
// step of 32 bf16 values takes 0.67 us (0.61 in matrix instructions); prologue and epilogue of a tile
// 9 us (bf16 outputs) to 27 (fp32 momenta read and written).  Over several cards, 4096 x 14336 x 4096
// bf16: forward with g and u 768 to 791 us (1.22 to 1.25 PFLOP/s), dx 700 to 725 (1.33 to 1.37), weight
// gradients into fp32 806 to 833 (1.15 to 1.19); int8 gated 2048 x 14336 x 4096 219 to 226 us (2.1 to
// 2.2 POP/s), 1999 x 4096 x 14336 117 to 121 (1.9 to 2.0).
template <int KIND, bool AT, bool BT, bool DUAL, class Out>
__global__ __launch_bounds__(256) void mixed_kernel(Source g, Out out, int batch, int64_t whole, int parts) {
  using L = Config<KIND, 256, 256, 128, 128, ring_of(AT), AT, BT, DUAL>;
  using H = Config<KIND, 128, 256, 64, 128, ring_of(AT), AT, BT, DUAL>;
  using Q = Config<KIND, 128, 128, 64, 64, ring_of(AT), AT, BT, DUAL>;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int64_t TM = (g.m + 255) / 256, TN = (g.n + L::COLS - 1) / L::COLS, tiles = TM * TN;
  const int steps = __builtin_amdgcn_readfirstlane(int(g.K / (64 / Math<KIND>::kBytes) * g.segs));
  const int64_t b = blockIdx.x;
  int64_t t, part = 0, tm, tn;
  if (b < whole) {
    t = gemm::xcd_remap(b, whole);
  } else {
    const int64_t u = gemm::xcd_remap(b - whole, int64_t(gridDim.x) - whole);
    t = whole + u / parts;
    part = u % parts;
  }
  const int z = __builtin_amdgcn_readfirstlane(int(t / tiles));
  tile_at(t % tiles, TM, TN, tm, tn);
  const Source s = source_at(g, z);
  const Out o = out.at(z);
  if (b < whole) {
    unit<L, false>(s, tm * 256, tn * L::COLS, 0, steps, true, o, lds);
    return;
  }
  const int64_t m0 = tm * 256 + 128 * (part & 1), n0 = tn * L::COLS + Q::COLS * (part >> 1);
  if (m0 >= g.m || n0 >= g.n) return;
  if (parts == 2) unit<H, false>(s, m0, n0, 0, steps, true, o, lds);
  else unit<Q, false>(s, m0, n0, 0, steps, true, o, lds);
}

// Sums of the parts, added in their order, to the output.  Bound by reading them (777 x 768 in
// three parts: 3.9 us).
template <int KIND, int NB, class Out>
__global__ __launch_bounds__(256) void join_kernel(Out out, Split sp, int64_t m) {
  using sum_t = typename Math<KIND>::sum_t;
  typedef sum_t sum4_t __attribute__((ext_vector_type(4)));
  const int64_t per = sp.ldp / 4, t = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (t >= m * per * sp.batch) return;
  const int64_t zr = t / per, col = (t % per) * 4;   // row of the batch
  const sum_t* src = static_cast<const sum_t*>(sp.sums) + zr * NB * sp.ldp + col;
  const int64_t stride = sp.batch * m * NB * sp.ldp;
  sum_t v[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    sum4_t sum = *reinterpret_cast<const sum4_t*>(src + b * sp.ldp);
    for (int p = 1; p < sp.parts; ++p) sum += *reinterpret_cast<const sum4_t*>(src + b * sp.ldp + p * stride);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[b][e] = sum[e];
  }
  const int z = int(zr / m);
  const int64_t row = zr % m;
  const Out o = out.at(z);
  if (col + 4 <= o.width) {
    o.template store<4>(row, col, v, o.template cols<4>(col), o.template pre<4>(row, col));
  } else {
    for (int e = 0; e < 4; ++e)
      if (col + e < o.width) {
        sum_t w[NB][1];
#pragma unroll
        for (int b = 0; b < NB; ++b) w[b][0] = v[b][e];
        o.template store<1>(row, col + e, w, o.template cols<1>(col + e), o.template pre<1>(row, col + e));
      }
  }
}

// Rows of fewer than eight entries: a thread takes an output at a time, straight from the definition.
template <int NB, class Out>
__global__ __launch_bounds__(256) void plain_kernel(Source g, Out out, int batch, bool a_kmajor, bool b_kmajor) {
  for (int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x; t < g.m * g.n * batch; t += int64_t(gridDim.x) * 256) {
    const int z = int(t / (g.m * g.n));
    const int64_t row = t / g.n % g.m, col = t % g.n;
    float v[NB][1] = {};
    for (int s = 0; s < g.segs; ++s)
      for (int64_t k = 0; k < g.K; ++k) {
        const char* a = (s || z ? g.A[1] : g.A[0]) + (a_kmajor ? k * g.lda + row * 2 : row * g.lda + k * 2);
        const float av = bf16_to_f32(*reinterpret_cast<const bf16_t*>(a));
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const char* p = (s || b ? g.B[1] : g.B[0]) + (b_kmajor ? k * g.ldb + col * 2 : col * g.ldb + k * 2);
          v[b][0] = fmaf(av, bf16_to_f32(*reinterpret_cast<const bf16_t*>(p)), v[b][0]);
        }
      }
    const Out o = out.at(z);
    o.template store<1>(row, col, v, o.template cols<1>(col), o.template pre<1>(row, col));
  }
}

// ---------------------------------------------------------------------------
// Few rows
// ---------------------------------------------------------------------------
// Few rows (8 at most, see Plan; the blocks hold 16) of int8 against one B, bound by reading B: 1 x
// 4096 x 14336 12.6 us (4.6 TB/s).  Straight from memory: no tile is staged, each wave reads 16 rows
// of B and the rows of A, 128 bytes of each at a time, and multiplies them on 16 x 16 blocks.  The
// waves of a workgroup take the 128-byte groups of the contraction in turn; their sums meet in LDS.
// B is the first operand: a lane holds four consecutive columns of one row of C.
template <class Out>
__global__ __launch_bounds__(512) void direct_kernel(Source g, Out out) {
  using M_ = Math<kI8>;
  __shared__ int red[8 * 4 * 64];   // [waves][4][64]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int r = lane & 15, kq = lane >> 4;
  const int64_t n0 = int64_t(blockIdx.x) * 16;
  // 16 bytes at 16 kq and at 64 + 16 kq of the group: the same k-values for both operands
  const char* pa = g.A[0] + min(int64_t(r), g.m - 1) * g.lda + 16 * kq;
  const char* pb = g.B[0] + min(n0 + r, g.n - 1) * g.ldb + 16 * kq;
  M_::acc4_t acc = {0, 0, 0, 0};
  const int64_t groups = g.K / 128;
  auto load = [](const char* p) __attribute__((always_inline)) { return *reinterpret_cast<const u32x4_t*>(p); };
  constexpr int U = 4;   // groups whose loads are in flight together
  // each workgroup begins at another group, as TURNED tiles do
  const int64_t turn = groups > 0 ? int64_t(blockIdx.x) * 5 % groups : 0;
  for (int64_t kb0 = wave; kb0 < groups; kb0 += U * waves) {
    u32x4_t fb[U][2], fa[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int64_t at = min(kb0 + u * waves, groups - 1) + turn;   // past the end: read again, not used
      at = (at >= groups ? at - groups : at) * 128;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        fb[u][c] = load(pb + at + 64 * c);
        fa[u][c] = load(pa + at + 64 * c);
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // all loads before the first product: the compiler would take them in turn
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb0 + u * waves >= groups) break;
#pragma unroll
      for (int c = 0; c < 2; ++c) acc = M_::mma16(fb[u][c], fa[u][c], acc);
    }
  }
  if (wave == waves - 1 && g.K % 128 != 0)   // half a group is left (K is a multiple of 64)
    acc = M_::mma16(load(pb + groups * 128), load(pa + groups * 128), acc);
  if (waves > 1) {
#pragma unroll
    for (int v = 0; v < 4; ++v) red[(wave * 4 + v) * 64 + lane] = acc[v];
    __syncthreads();
    if (wave > 0) return;
  }
  int o[1][4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    o[0][v] = acc[v];
    for (int w = 1; w < waves; ++w) o[0][v] += red[(w * 4 + v) * 64 + lane];
  }
  const int64_t row = r, col = n0 + 4 * kq;
  if (row >= g.m || col >= g.n) return;
  if (col + 4 <= g.n) {
    out.template store<4>(row, col, o, out.template cols<4>(col), out.template pre<4>(row, col));
  } else {
    for (int e = 0; e < 4; ++e)
      if (col + e < g.n) {
        const int w[1][1] = {{o[0][e]}};
        out.template store<1>(row, col + e, w, out.template cols<1>(col + e), out.template pre<1>(row, col + e));
      }
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
// the tiles address the rows of a stage with 32-bit offsets (256 rows of under 2^24 bytes)
constexpr int64_t kMaxPitch = (int64_t(1) << 24) - 16;
constexpr int64_t kCus = 256;

// How a product is cut, by its sizes alone (tiles counted over all B's and the batch).
//  direct  up to 8 rows against one B in int8: straight from memory (4096 x 14336, 1 row 12.9 us
//          against 15.1 on narrow tiles, 4 rows 13.8 and 15.0, 8 rows 14.8 and 15.1, 16 rows 17.2
//          and 15.2; 14336 x 4096, 1 row 12.1 and 12.9, 4 rows 13.1 and 13.0, 8 rows 14.5 and 13.0;
//          2304 x 768 8.1 and 8.1 for all of them).  Not two B's: 1 x 14336 x 4096 24.7 and 25.0,
//          in bf16 49.2 and 44.4
//  narrow  64 rows and 64 columns (128 where an operand is k-major): up to 64 rows, and where
//          128 x 128 tiles would not be half as many as the CUs
//  small   128 x 128 tiles where 256 x 256 ones would leave more than half the CUs idle
//  large   256 x 256 tiles, the last round in halves or quarters
// Narrow and small tiles that are no more than half the CUs are cut along the contraction into
// `parts` of 20 steps or more, so that there is at most one unit per CU; a second kernel joins them.
// Two units per CU, as long, share its matrix cores and LDS and write twice the sums: backward to
// the input of 777 x 2304 x 768, 42 small tiles in 6 parts 28.6 us, in 13 34.1, 78 narrow ones in 3
// 25.5, in 6 32.0; 33 x 4096 x 14336 int8, 64 narrow tiles in 4 parts 20.5, in 8 23.1.
enum PlanKind { kDirect, kNarrow, kSmall, kLarge };
struct Plan {
  PlanKind kind;
  int parts;
};
// m, n at least 1; rows_only: both operands lie in rows, a_rows: A does; whole: the DMA can copy
// (rows start at 16 bytes).  Otherwise narrow tiles have 128 columns, and steps through registers
// wait for memory, so two units per CU are worth their sums.
inline Plan plan_product(int64_t m, int64_t n, int64_t steps, int mats, int batch, bool whole, bool rows_only, bool a_rows = true) {
  if (m <= 8 && mats == 1 && rows_only) return {kDirect, 1};
  const int64_t cols = n * mats;
  const int64_t narrow = ceil_div(m, 64) * ceil_div(cols, rows_only && whole ? 64 : 128) * batch, small = ceil_div(m, 128) * ceil_div(cols, 128) * batch;
  auto parts = [&](int64_t tiles) { return int(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(16, steps / 20), (whole ? 1 : 2) * kCus / tiles))); };
  if (a_rows && (m <= 64 || (2 * small <= kCus && narrow <= kCus))) return {kNarrow, parts(narrow)};
  if (2 * small <= kCus || 2 * ceil_div(m, 256) * ceil_div(cols, 256) * batch < kCus) return {kSmall, parts(small)};
  return {kLarge, 1};
}
// how many parts each tile of mixed_kernel's last, partial round comes in (1: there is none, or it stays whole)
inline int last_round_parts(int64_t tiles) {
  const int64_t rest = tiles % kCus;
  return rest == 0 ? 1 : rest * 4 <= kCus ? 4 : rest * 2 <= kCus ? 2 : 1;
}
// bytes of the parts' sums
inline size_t sum_bytes(const Plan& p, int64_t m, int64_t n, int mats, int batch) {
  return p.parts > 1 ? size_t(p.parts) * batch * size_t(m) * mats * size_t(ceil_div(n, 4) * 4) * 4 : 0;
}

// workgroups of 256 threads that stride over n entries; a launch has to stay under 2^32 threads
inline dim3 grid_of(int64_t n) { return dim3(unsigned(std::min<int64_t>(ceil_div(n, 256), 1 << 20))); }

template <class C_, bool MASKED, bool SPLIT, class Out>
int launch_tiles(const Source& g, const Out& out, const Split& sp, hipStream_t st) {
  auto kern = tile_kernel<C_, MASKED, SPLIT, Out>;
  const int64_t units = ceil_div(g.m, C_::BM) * ceil_div(g.n, C_::COLS) * sp.batch * sp.parts;
  if (units * C_::NT > UINT32_MAX) return MUON_EINVAL;
  static std::atomic<uint64_t> configured{0};   // devices with the LDS limit set
  if (gemm::set_lds_limit(kern, C_::LDS_BYTES, configured) != MUON_OK) return MUON_ELAUNCH;
  launch_kernel(kern, dim3(units), dim3(C_::NT), C_::LDS_BYTES, st, g, out, sp);
  const int status = launch_status();
  if (!SPLIT || status != MUON_OK) return status;
  launch_kernel(join_kernel<C_::KIND, C_::NB, Out>, dim3(ceil_div(g.m * sp.batch * (sp.ldp / 4), 256)), dim3(256), 0, st, out, sp, g.m);
  return launch_status();
}
template <int KIND, bool AT, bool BT, bool DUAL, class Out>
int launch_mixed(const Source& g, const Out& out, int batch, hipStream_t st) {
  using L = Config<KIND, 256, 256, 128, 128, ring_of(AT), AT, BT, DUAL>;
  auto kern = mixed_kernel<KIND, AT, BT, DUAL, Out>;
  const int64_t tiles = ceil_div(g.m, 256) * ceil_div(g.n, L::COLS) * batch;
  const int parts = last_round_parts(tiles);
  const int64_t whole = parts == 1 ? tiles : tiles - tiles % kCus;
  if ((whole + (tiles - whole) * parts) * L::NT > UINT32_MAX) return MUON_EINVAL;
  static std::atomic<uint64_t> configured{0};
  if (gemm::set_lds_limit(kern, L::LDS_BYTES, configured) != MUON_OK) return MUON_ELAUNCH;
  launch_kernel(kern, dim3(whole + (tiles - whole) * parts), dim3(256), L::LDS_BYTES, st, g, out, batch, whole, parts);
  return launch_status();
}
template <class C_, bool MASKED, class Out>
int launch_sized(const Source& g, const Out& out, const Split& sp, hipStream_t st) {
  return sp.parts > 1 ? launch_tiles<C_, MASKED, true>(g, out, sp, st) : launch_tiles<C_, MASKED, false>(g, out, sp, st);
}

// large tiles: outputs of whole cache lines pass the caches, others go out in whole tiles only
template <int KIND, bool AT, bool BT, bool DUAL, class Out>
int launch_large(const Source& g, const Out& out, const Split& sp, hipStream_t st) {
  using Passing = decltype(out.passing());
  if constexpr (std::is_same_v<Passing, Out>) {   // an output that never passes them (the bf16 forward's)
    return launch_mixed<KIND, AT, BT, DUAL>(g, out, sp.batch, st);
  } else {
    if (out.lines()) return launch_mixed<KIND, AT, BT, DUAL>(g, out.passing(), sp.batch, st);
    return launch_tiles<Config<KIND, 256, 256, 128, 128, ring_of(AT), AT, BT, DUAL>, false, false>(g, out, sp, st);
  }
}
template <int NB, class Out>
int launch_plain(const Source& g, const Out& out, int batch, bool a_kmajor, bool b_kmajor, hipStream_t st) {
  launch_kernel(plain_kernel<NB, Out>, grid_of(g.m * g.n * batch), dim3(256), 0, st, g, out, batch, a_kmajor, b_kmajor);
  return launch_status();
}
template <class Out>
int launch_direct(const Source& g, const Out& out, hipStream_t st) {
  const int waves = int(std::max<int64_t>(1, std::min<int64_t>(g.K / 128 / 8, 8)));   // eight groups each, up to eight waves
  launch_kernel(direct_kernel<Out>, dim3(ceil_div(g.n, 16)), dim3(64 * waves), 0, st, g, out);
  return launch_status();
}

}  // namespace tile
}  // namespace muon
