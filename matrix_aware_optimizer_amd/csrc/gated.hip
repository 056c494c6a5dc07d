// The gated feed-forward block h = act(x Wg^T) * (x Wu^T) in bf16: forward, gradients of both
// products, of the input and of the weights.
//
//   forward   g = x Wg^T, u = x Wu^T, h = a(g) u
//   backward  dg = dh u a'(g), du = dh a(g), dx = dg Wg + du Wu
//   weights   Mg <- beta Mg + alpha dg^T x, Mu <- beta Mu + alpha du^T x
//
// Sums, activations and products are fp32 and each output is rounded once.  dg and du are outputs
// in bf16, and dx and the weight gradients take them as stored: the matrix instructions read bf16,
// and a second part for what the rounding leaves would double the products (dx of 4096 x 14336 x 4096
// 1400 us for 700).  It makes dx 1.4 times its own rounding (2.3e-3 of its norm instead of 1.7e-3).
#include <algorithm>

#include "act.h"
#include "common.h"
#include "tile.h"

namespace muon {
namespace {

using tile::ceil_div;
using tile::kBf16;

// C <- beta C + alpha sum (READS) or alpha sum, one rounding to the stored type; z says which of two outputs
template <typename TC, bool READS, bool PASSING = false>
struct AxpbyOut {
  using sum_t = float;
  static constexpr int E = 16 / int(sizeof(TC));
  TC *C, *C1;
  int64_t ldc, width;
  float alpha, beta;

  template <int N> struct Cols {};
  template <int N> struct Pre { TC c[READS ? N : 1]; };
  AxpbyOut<TC, READS, true> passing() const { return {C, C1, ldc, width, alpha, beta}; }
  bool lines() const { return whole_lines(C, ldc * int64_t(sizeof(TC))) && whole_lines(C1, 0); }
  __device__ __forceinline__ AxpbyOut at(int z) const {
    AxpbyOut o = *this;
    if (z) o.C = C1;
    return o;
  }
  template <int N> __device__ __forceinline__ Cols<N> cols(int64_t) const { return {}; }
  // read once; PASSING: past the caches' order of keeping (weight gradients of 14336 x 4096 from 4096 tokens, 848 -> 833 us then)
  template <int N> __device__ __forceinline__ Pre<N> pre(int64_t row, int64_t col) const {
    Pre<N> p;
    if constexpr (READS) {
      const TC* src = C + row * ldc + col;
      if constexpr (N * sizeof(TC) == 16) {
        if constexpr (PASSING) p = __builtin_bit_cast(Pre<N>, __builtin_nontemporal_load(reinterpret_cast<const typename Unaligned<TC>::x4*>(src)));
        else p = __builtin_bit_cast(Pre<N>, load16(src));
      }
      else if constexpr (N * sizeof(TC) == 8) p = __builtin_bit_cast(Pre<N>, load8(src));
      else
#pragma unroll
        for (int k = 0; k < N; ++k) p.c[k] = src[k];
    }
    return p;
  }
  template <int N>
  __device__ __forceinline__ void store(int64_t row, int64_t col, const float (&v)[1][N], const Cols<N>&, const Pre<N>& p) const {
    float o[N];
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = alpha * v[0][k];
    if constexpr (READS)
#pragma unroll
      for (int k = 0; k < N; ++k) o[k] = fmaf(beta, to_f32(p.c[k]), o[k]);
    store_n<N, PASSING>(C + row * ldc + col, o);
  }
};

struct GradArgs {
  const bf16_t *dH, *G, *U;
  bf16_t *dG, *dU, *H;   // H may be null
  int64_t rows, cols, lddh, ldg, ldd, ldh;
};

// dg, du and h of N entries; everything is read before anything is written
template <int ACT, int N>
__device__ __forceinline__ void gradients(const GradArgs& a, int64_t row, int64_t col) {
  float dh[N], g[N], u[N], dg[N], du[N], h[N];
  load_n<N>(a.dH + row * a.lddh + col, dh);
  load_n<N>(a.G + row * a.ldg + col, g);
  load_n<N>(a.U + row * a.ldg + col, u);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float slope;
    const float act = activate<true, false>(ACT, g[k], slope);
    dg[k] = dh[k] * u[k] * slope;
    du[k] = dh[k] * act;
    h[k] = act * u[k];
  }
  store_n<N, false>(a.dG + row * a.ldd + col, dg);
  store_n<N, false>(a.dU + row * a.ldd + col, du);
  if (a.H != nullptr) store_n<N, false>(a.H + row * a.ldh + col, h);
}

// Eight columns of one row per thread.  Bound by memory: 6 bytes read and 4 (6 with h) written
// per entry; 4096 x 14336 92 us, 6.3 TB/s.
template <int ACT>
__global__ __launch_bounds__(256) void glu_gradients_kernel(GradArgs a) {
  const int64_t per = (a.cols + 7) / 8;
  for (int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x; t < a.rows * per; t += int64_t(gridDim.x) * 256) {
    const int64_t row = t / per, col = (t % per) * 8;
    if (col + 8 <= a.cols) gradients<ACT, 8>(a, row, col);
    else
      for (int64_t c = col; c < a.cols; ++c) gradients<ACT, 1>(a, row, c);
  }
}

// A product on tiles: the sizes of `plan`, through the DMA where rows start at 16 bytes (whole)
template <bool AT, bool BT, bool DUAL, class Out>
int launch_tiled(const tile::Source& g, const Out& out, const tile::Plan& plan, const tile::Split& sp, bool whole, hipStream_t st) {
  if ((AT ? g.m : g.K) < 8 || (BT ? g.n : g.K) < 8) return tile::launch_plain<DUAL ? 2 : 1>(g, out, sp.batch, AT, BT, st);
  if constexpr (!AT) {
    if (plan.kind == tile::kNarrow)
      return whole ? tile::launch_sized<tile::Config<kBf16, 64, BT ? 128 : 64, 32, 64, BT ? 8 : 9, AT, BT, DUAL>, false>(g, out, sp, st)
                   : tile::launch_sized<tile::Config<kBf16, 64, 128, 32, 64, 3, AT, BT, DUAL>, true>(g, out, sp, st);
  }
  // through registers, 256 x 256 tiles pay over 2048 and more values (14335 x 4095 weight gradients of
  // 4096 tokens 1319 us against 1501, of 300 tokens 71 against 45), and for one B only: two spill
  if (plan.kind == tile::kSmall || (!whole && (DUAL || g.K * g.segs < 2048))) {
    using Copied = tile::Config<kBf16, 128, 128, 64, 64, tile::ring_of(AT), AT, BT, DUAL>;
    using Held = tile::Config<kBf16, 128, 128, 64, 64, 3, AT, BT, DUAL>;
    if (!whole) return tile::launch_sized<Held, true>(g, out, sp, st);
    // one part for dx: where small tiles are no more than half the CUs, twice as many narrow ones are at most the CUs
    if constexpr (!AT && BT) return tile::launch_tiles<Copied, false, false>(g, out, sp, st);
    else return tile::launch_sized<Copied, false>(g, out, sp, st);
  }
  if constexpr (!DUAL)
    if (!whole) return tile::launch_tiles<tile::Config<kBf16, 256, 256, 128, 128, 3, AT, BT, DUAL>, true, false>(g, out, sp, st);
  return tile::launch_large<kBf16, AT, BT, DUAL>(g, out, sp, st);
}

bool sides_ok(int64_t tokens, int64_t out, int64_t in) {
  return tokens >= 0 && out >= 0 && in >= 0 && tokens <= MUON_GLU_MAX_SIDE && out <= MUON_GLU_MAX_SIDE && in <= MUON_GLU_MAX_SIDE;
}
// outputs that would be written over each other
bool same(const void* a, const void* b) { return a != nullptr && a == b; }
bool pitch_ok(int64_t ld, int64_t cols) { return ld >= cols && ld * 2 <= tile::kMaxPitch; }
bool run8(int64_t v) { return v % 8 == 0; }

// Plans of the three products.  The workspace queries do not see the pitches: they serve both.
tile::Plan forward_plan(int64_t tokens, int64_t out, int64_t in, bool whole) {
  return tile::plan_product(tokens, out, in / 32, 2, 1, whole, true);
}
tile::Plan input_plan(int64_t tokens, int64_t out, int64_t in, bool whole) {
  return tile::plan_product(tokens, in, 2 * (out / 32), 1, 1, whole, false);
}
tile::Plan weight_plan(int64_t tokens, int64_t out, int64_t in, bool whole) {
  return tile::plan_product(out, in, tokens / 32, 1, 2, whole, false, false);
}

// MUON_OK where the workspace serves `need` bytes
int workspace_status(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return MUON_OK;
  if (workspace == nullptr || bytes < need) return MUON_EWORKSPACE;
  return aligned16(workspace) ? MUON_OK : MUON_EALIGN;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t glu_forward_workspace_bytes(int64_t tokens, int64_t out, int64_t in) {
  if (!sides_ok(tokens, out, in) || tokens == 0 || out == 0) return 0;
  return std::max(tile::sum_bytes(forward_plan(tokens, out, in, true), tokens, out, 2, 1),
                  tile::sum_bytes(forward_plan(tokens, out, in, false), tokens, out, 2, 1));
}

int glu_forward(const void* X, int64_t ldx, const void* Wg, const void* Wu, int64_t ldw, int act, void* H, int64_t ldh, void* G,
                void* U, int64_t ldg, int64_t tokens, int64_t out, int64_t in, void* workspace, size_t ws_bytes, void* stream) {
  if (!sides_ok(tokens, out, in) || !valid_act(act)) return MUON_EINVAL;
  if (tokens == 0 || out == 0) return MUON_OK;
  if (!numel_ok(tokens * out) || same(H, G) || same(H, U) || same(G, U)) return MUON_EINVAL;
  if (H == nullptr || ldh < out || (in > 0 && (X == nullptr || Wg == nullptr || Wu == nullptr))) return MUON_EINVAL;
  if (!pitch_ok(ldx, in) || !pitch_ok(ldw, in) || (G == nullptr) != (U == nullptr) || (G != nullptr && ldg < out)) return MUON_EINVAL;
  if (!aligned16(X) || !aligned16(Wg) || !aligned16(Wu) || !aligned16(H) || !aligned16(G) || !aligned16(U)) return MUON_EALIGN;
  const bool whole = run8(ldx) && run8(ldw);
  const tile::Plan plan = forward_plan(tokens, out, in, whole);
  const int ws = workspace_status(workspace, ws_bytes, glu_forward_workspace_bytes(tokens, out, in));
  if (ws != MUON_OK) return ws;
  const char* x = static_cast<const char*>(X);
  const tile::Source g{{x, x}, {static_cast<const char*>(Wg), static_cast<const char*>(Wu)}, ldx * 2, ldw * 2, tokens, out, in, 1};
  const GluOut<bf16_t, false> o{static_cast<bf16_t*>(H), static_cast<bf16_t*>(G), static_cast<bf16_t*>(U), ldh, ldg, out, act,
                                nullptr, nullptr, nullptr};
  const tile::Split sp{plan.parts, 1, workspace, ceil_div(out, 4) * 4};
  hipStream_t hs = static_cast<hipStream_t>(stream);
  return launch_tiled<false, false, true>(g, o, plan, sp, whole, hs);
}

size_t glu_backward_workspace_bytes(int64_t tokens, int64_t out, int64_t in) {
  if (!sides_ok(tokens, out, in) || tokens == 0 || in == 0) return 0;
  return std::max(tile::sum_bytes(input_plan(tokens, out, in, true), tokens, in, 1, 1),
                  tile::sum_bytes(input_plan(tokens, out, in, false), tokens, in, 1, 1));
}

int glu_backward(const void* dH, int64_t lddh, const void* G, const void* U, int64_t ldg, int act, void* dG, void* dU, int64_t ldd,
                 void* H, int64_t ldh, const void* Wg, const void* Wu, int64_t ldw, void* dX, int64_t lddx, int64_t tokens,
                 int64_t out, int64_t in, void* workspace, size_t ws_bytes, void* stream) {
  if (!sides_ok(tokens, out, in) || !valid_act(act)) return MUON_EINVAL;
  const bool input = dX != nullptr && in > 0;
  if (tokens == 0) return MUON_OK;
  if (out > 0 && (dH == nullptr || G == nullptr || U == nullptr || dG == nullptr || dU == nullptr)) return MUON_EINVAL;
  if (!numel_ok(tokens * out) || !numel_ok(tokens * in) || (out > 0 && (same(dG, dU) || same(H, dG) || same(H, dU)))) return MUON_EINVAL;
  if (input && (same(dX, dG) || same(dX, dU) || same(dX, H) || same(dX, Wg) || same(dX, Wu))) return MUON_EINVAL;
  if (lddh < out || ldg < out || !pitch_ok(ldd, out) || (H != nullptr && ldh < out)) return MUON_EINVAL;
  // an output over an operand row by row: other pitches would write rows that are still to be read
  const auto crossed = [&](const void* o, int64_t ldo) {
    return (same(o, dH) && ldo != lddh) || ((same(o, G) || same(o, U)) && ldo != ldg);
  };
  if (tokens > 1 && out > 0 && (crossed(dG, ldd) || crossed(dU, ldd) || crossed(H, ldh))) return MUON_EINVAL;
  if (input && (lddx < in || !pitch_ok(ldw, in) || (out > 0 && (Wg == nullptr || Wu == nullptr)))) return MUON_EINVAL;
  if (!aligned16(dH) || !aligned16(G) || !aligned16(U) || !aligned16(dG) || !aligned16(dU) || !aligned16(H)) return MUON_EALIGN;
  if (input && (!aligned16(Wg) || !aligned16(Wu) || !aligned16(dX))) return MUON_EALIGN;
  if (input) {
    const int ws = workspace_status(workspace, ws_bytes, glu_backward_workspace_bytes(tokens, out, in));
    if (ws != MUON_OK) return ws;
  }
  hipStream_t hs = static_cast<hipStream_t>(stream);
  if (out > 0) {
    const GradArgs a{static_cast<const bf16_t*>(dH), static_cast<const bf16_t*>(G), static_cast<const bf16_t*>(U), static_cast<bf16_t*>(dG),
                     static_cast<bf16_t*>(dU), static_cast<bf16_t*>(H), tokens, out, lddh, ldg, ldd, ldh};
    void (*kern)(GradArgs) = act == MUON_ACT_SILU        ? glu_gradients_kernel<MUON_ACT_SILU>
                             : act == MUON_ACT_GELU      ? glu_gradients_kernel<MUON_ACT_GELU>
                             : act == MUON_ACT_GELU_TANH ? glu_gradients_kernel<MUON_ACT_GELU_TANH>
                                                         : glu_gradients_kernel<MUON_ACT_RELU>;
    launch_kernel(kern, tile::grid_of(tokens * ceil_div(out, 8)), dim3(256), 0, hs, a);
    const int status = launch_status();
    if (status != MUON_OK) return status;
  }
  if (!input) return MUON_OK;
  const bool whole = run8(ldd) && run8(ldw) && run8(in);
  const tile::Plan plan = input_plan(tokens, out, in, whole);
  const tile::Source g{{static_cast<const char*>(dG), static_cast<const char*>(dU)},
                       {static_cast<const char*>(Wg), static_cast<const char*>(Wu)}, ldd * 2, ldw * 2, tokens, in, out, 2};
  const AxpbyOut<bf16_t, false> o{static_cast<bf16_t*>(dX), nullptr, lddx, in, 1.0f, 0.0f};
  const tile::Split sp{plan.parts, 1, workspace, ceil_div(in, 4) * 4};
  return launch_tiled<false, true, false>(g, o, plan, sp, whole, hs);
}

size_t glu_weight_grad_workspace_bytes(int64_t tokens, int64_t out, int64_t in) {
  if (!sides_ok(tokens, out, in) || out == 0 || in == 0) return 0;
  return std::max(tile::sum_bytes(weight_plan(tokens, out, in, true), out, in, 1, 2),
                  tile::sum_bytes(weight_plan(tokens, out, in, false), out, in, 1, 2));
}

int glu_weight_grad(const void* dG, const void* dU, int64_t ldd, const void* X, int64_t ldx, void* Mg, void* Mu, int m_dtype, int64_t ldm,
                    int64_t tokens, int64_t out, int64_t in, float alpha, float beta, void* workspace, size_t ws_bytes, void* stream) {
  if (!sides_ok(tokens, out, in)) return MUON_EINVAL;
  if (!valid_dtype(m_dtype)) return MUON_EDTYPE;
  if (out == 0 || in == 0) return MUON_OK;
  if (!numel_ok(out * in) || same(Mg, Mu)) return MUON_EINVAL;
  if (Mg == nullptr || Mu == nullptr || ldm < in || (tokens > 0 && (dG == nullptr || dU == nullptr || X == nullptr))) return MUON_EINVAL;
  if (!pitch_ok(ldd, out) || !pitch_ok(ldx, in)) return MUON_EINVAL;
  if (!aligned16(dG) || !aligned16(dU) || !aligned16(X) || !aligned16(Mg) || !aligned16(Mu)) return MUON_EALIGN;
  const bool whole = run8(ldd) && run8(ldx) && run8(out) && run8(in);
  const tile::Plan plan = weight_plan(tokens, out, in, whole);
  const int ws = workspace_status(workspace, ws_bytes, glu_weight_grad_workspace_bytes(tokens, out, in));
  if (ws != MUON_OK) return ws;
  const char* x = static_cast<const char*>(X);
  const tile::Source g{{static_cast<const char*>(dG), static_cast<const char*>(dU)}, {x, x}, ldd * 2, ldx * 2, out, in, tokens, 1};
  const tile::Split sp{plan.parts, 2, workspace, ceil_div(in, 4) * 4};
  hipStream_t hs = static_cast<hipStream_t>(stream);
  auto go = [&](auto type, auto reads) {
    using TC = decltype(type);
    const AxpbyOut<TC, decltype(reads)::value> o{static_cast<TC*>(Mg), static_cast<TC*>(Mu), ldm, in, alpha, beta};
    return launch_tiled<true, true, false>(g, o, plan, sp, whole, hs);
  };
  if (m_dtype == MUON_F32) return beta != 0.0f ? go(float{}, std::true_type{}) : go(float{}, std::false_type{});
  return beta != 0.0f ? go(bf16_t{}, std::true_type{}) : go(bf16_t{}, std::false_type{});
}

}  // extern "C"
