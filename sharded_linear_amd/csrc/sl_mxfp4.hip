// C-ABI entry points of the MXFP4 operators: argument checks and launches.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sharded_linear.h"
#include "sl_f4.h"

namespace {

constexpr int64_t kMaxExtent = int64_t(1) << 31;
constexpr int64_t kMaxTiles = int64_t(1) << 31;        // workgroups of one launch
constexpr int64_t kMaxCastTiles = int64_t(1) << 24;    // of 256 threads: a launch has fewer than 2^32
constexpr int64_t kMaxFeatures = int64_t(1) << 23;     // rows of a tile stay within 32-bit offsets

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Extents of a product [T, out] x [out, in]: k is the contracted one, held in blocks of 32.
int check_product(int64_t T, int64_t in, int64_t out, int64_t k) {
  if (T < 0 || in < 0 || out < 0) return SL_EINVAL;
  if (T >= kMaxExtent || in >= kMaxExtent || out >= kMaxExtent) return SL_ESHAPE;
  if (in % 8 || out % 8 || k % 32 || in > kMaxFeatures || out > kMaxFeatures || k > kMaxFeatures) return SL_ESHAPE;
  return SL_OK;
}

int check_grid(int64_t M, int64_t N) { return (M + 63) / 64 * ((N + 63) / 64) < kMaxTiles ? SL_OK : SL_ESHAPE; }

int64_t ntiles(int64_t M, int64_t N, int bm, int bn) { return (M + bm - 1) / bm * ((N + bn - 1) / bn); }

// Rows up to which a product goes to the few-row kernel.  MXFP4 rows: 64 by [11008, 4096] 12.0 us there, 12.7 in
// 128x128 tiles; by [8192, 2048] 6.1 against 8.2.  bf16 rows, of which every workgroup reads all: 16 by [4096, 11008]
// 15.2 us there, 15.7 in the tiles of sl_tile_w4.hip; 32 by [11008, 4096] 14.7 against 17.5, by [4096, 5504] 13.3
// against 13.5, by [2048, 8192] 18.7 against 13.2; 48 by [11008, 4096] 20.6 against 18.1.
constexpr int64_t kFewRows = 64;
bool few_rows_bf16(int64_t T, int64_t K) { return T <= 16 || (T <= 32 && K <= 6144); }

// Splits of K over `stages` for a grid of `tiles`: up to `slots` workgroups, at least `least` stages to a split (an
// even number: the kernel starts at an even stage) and at most 16 splits.
void split_k(F4Args& g, int64_t tiles, int64_t slots, int least) {
  const int64_t stages = (g.K + kF4StageK - 1) / kF4StageK;
  int64_t s = tiles ? slots / tiles : 1;
  if (s > stages / least) s = stages / least;
  if (s > 16) s = 16;
  if (s < 1) s = 1;
  int64_t per = stages ? (stages + s - 1) / s : 2;
  per += per & 1;
  g.kt_per_split = int(per);
  g.splits = stages ? int((stages + per - 1) / per) : 1;
}

// 128x128 tiles two stages deep, of which two workgroups fit on a CU, or four stages deep, one to a CU: where there
// is about one to a CU anyway and its sum is long.  [1536, 2048] over 8192 tokens, 192 tiles of 32 stages, 29.2 us
// against 32.6; [2048, 4096] (512 tiles) 58.0 against 53.1; [1024, 1024] over 4096 (256 of 4 stages) the same.
int small_tiles(const F4Args& g, int64_t tiles) {
  const int64_t items = tiles * g.splits, stages = (g.K + kF4StageK - 1) / kF4StageK;
  return items > 128 && items <= 256 && stages >= 16 * g.splits ? 2 : 1;
}

size_t planes_bytes(const F4Args& g) { return g.splits > 1 ? size_t(g.splits) * size_t(g.M) * size_t(g.N) * 4 : 0; }

// Tiles of a bf16 result: 256x256 where they fill most of the 256 CUs, else 128x128 (2048 rows by [4096, 4096], 128
// tiles of 256x256, 33.6 us against 26.3; 4096 rows, 256 tiles, 41.9 against 45.8).  K is split where that leaves CUs
// empty and a sum is long enough to pay for the planes and their second pass: 128 rows by [4096, 11008], 43 stages,
// 34.0 us unsplit, 19.1 in 5 splits; 512 by [2048, 6144], 24 stages, 17.0 and, in 3 splits, 20.1.
F4Args product_plan(int64_t M, int64_t N, int64_t K) {
  F4Args g{};
  g.M = M; g.N = N; g.K = K;
  const int forced = block_scaled_config();
  g.cfg = forced >= 0 ? forced : ntiles(M, N, 256, 256) >= 200 ? 0 : 1;
  const int64_t tiles = g.cfg == 0 ? ntiles(M, N, 256, 256) : ntiles(M, N, 128, 128);
  split_k(g, tiles, M > kFewRows && K > 31 * kF4StageK ? 256 : 0, 8);
  if (forced < 0 && g.cfg == 1) g.cfg = small_tiles(g, tiles);
  return g;
}

// The weight gradient: 128x128 tiles up to 128 tiles of 256x256, 256x256 tiles above: [2048, 4096] over 8192 tokens
// (128 tiles of 256x256) 51.1 us against 65.2, [4096, 2816] (176) 75.2 against 70.1.
F4Args wgrad_plan(int64_t T, int64_t in, int64_t out) {
  F4Args g{};
  g.M = out; g.N = in; g.K = T;
  const int64_t t256 = ntiles(out, in, 256, 256);
  const int forced = block_scaled_config();
  g.cfg = forced >= 0 ? forced : t256 > 128 ? 0 : 1;
  const int64_t tiles = g.cfg == 0 ? t256 : ntiles(out, in, 128, 128);
  split_k(g, tiles, 256 + tiles / 2, 4);
  if (forced < 0 && g.cfg == 1) g.cfg = small_tiles(g, tiles);
  return g;
}

// bf16 rows by an MXFP4 weight: whether a bf16 copy of the weight and the bf16 product beat the tiles that expand
// the weight as they read it, T / 64 times.  They do for many rows, and in between where the tiles take more than one
// round on the chip.  Input gradient (one workgroup a CU): T 512 by [11008, 4096], 256 tiles, 76 us against 117; T 384
// by [4096, 5504], 258 tiles, 58 against 52; T 200, 172 tiles, 31 against 52.  Forward (two a CU): T 512 by
// [11008, 4096], 688 tiles, 64 against 71; T 768, 1032 tiles, 102 against 89; T 1000 by [4096, 5504], 512 tiles, 61
// against 65.  The copy is 19 us of 174 for T 2048 by [11008, 4096], 10 of 217 for T 8192 by [8192, 2048].
bool w4_by_copy(int64_t T, int64_t N, bool dgrad) {
  return T >= 1024 || (T > (dgrad ? 256 : 640) && ntiles(T, N, kW4TileT, kW4TileN) > (dgrad ? 256 : 512));
}

// Split of K of those tiles, to one workgroup a CU and at least 8 steps to a split: T 64 by [8192, 2048], input
// gradient, 16 tiles unsplit 50.5 us, in 8 splits 16.2; T 200 by [4096, 5504], forward, 128 tiles unsplit 30.8 us,
// in 2 splits 22.2, in 4 (two workgroups a CU) 25.1.
void w4_plan(F4RowsArgs& g) {
  const int64_t tiles = ntiles(g.T, g.N, kW4TileT, kW4TileN), steps = (g.K + kW4StepK - 1) / kW4StepK;
  int64_t s = tiles ? 256 / tiles : 1;
  if (s > steps / 8) s = steps / 8;
  if (s > 16) s = 16;
  if (s < 1) s = 1;
  const int64_t per = steps ? (steps + s - 1) / s : 1;
  g.steps_per_split = int(per);
  g.splits = steps ? int((steps + per - 1) / per) : 1;
}

bool few_rows(int64_t M) { return M <= kFewRows && block_scaled_config() < 0; }

size_t product_workspace(int64_t M, int64_t N, int64_t K) {
  return M == 0 || N == 0 || few_rows(M) ? 0 : planes_bytes(product_plan(M, N, K));
}

// C[M][N] = A . B^T (bf16) over K
int product(void* stream, const uint8_t* a, const uint8_t* sa, const uint8_t* b, const uint8_t* sb, void* c, int64_t M,
            int64_t N, int64_t K, void* workspace, size_t workspace_bytes) {
  if (M == 0 || N == 0) return SL_OK;
  if (!c || (K > 0 && (!a || !sa || !b || !sb))) return SL_EINVAL;
  if (!aligned16(c) || !aligned16(a) || !aligned16(b)) return SL_EALIGN;
  const int st = check_grid(M, N);
  if (st) return st;
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  if (few_rows(M)) {
    const F4RowsArgs r{a, sa, b, sb, c, M, N, K, nullptr, 1, 1};
    // an empty K may come without scales, and X without scales is bf16
    return f4_rows(hs, K ? r : F4RowsArgs{c, c, c, c, c, M, N, 0, nullptr, 1, 1}) == 0 ? SL_OK : SL_EHIP;
  }
  F4Args g = product_plan(M, N, K);
  g.a = a; g.b = b; g.sa = sa; g.sb = sb; g.c = c;
  if (g.splits == 1) return f4_gemm(hs, g) == 0 ? SL_OK : SL_EHIP;
  if (!workspace || !aligned16(workspace) || workspace_bytes < planes_bytes(g)) return SL_EWORKSPACE;
  g.ws = static_cast<float*>(workspace);
  return f4_accum(hs, g) || f4_join(hs, c, g.ws, M * N, g.splits) ? SL_EHIP : SL_OK;
}

}  // namespace

extern "C" int sl_mxfp4_quantize(void* stream, const void* x, int64_t rows, int64_t cols, uint8_t* q_rows,
                                 uint8_t* s_rows, uint8_t* q_cols, uint8_t* s_cols, int32_t rounding, uint64_t seed,
                                 const uint64_t* seed_offset) {
  if (rows < 0 || cols < 0 || (rounding != SL_ROUND_NEAREST && rounding != SL_ROUND_STOCHASTIC)) return SL_EINVAL;
  if (rows >= kMaxExtent || cols >= kMaxExtent || cols % 8) return SL_ESHAPE;
  if (!q_rows != !s_rows || !q_cols != !s_cols) return SL_EINVAL;
  if (rows == 0 || cols == 0 || (!q_rows && !q_cols)) return SL_OK;
  if (!x) return SL_EINVAL;
  if (!aligned16(x) || (q_rows && !aligned16(q_rows)) || (q_cols && !aligned16(q_cols))) return SL_EALIGN;
  if (reinterpret_cast<uintptr_t>(seed_offset) & 7u) return SL_EALIGN;
  if (ntiles(rows, cols, 128, 128) >= kMaxCastTiles) return SL_ESHAPE;
  const F4QuantArgs a{x, rows, cols, q_rows, s_rows, q_cols, s_cols, rounding == SL_ROUND_STOCHASTIC, seed, seed_offset};
  return f4_quantize(static_cast<hipStream_t>(stream), a) == 0 ? SL_OK : SL_EHIP;
}

extern "C" int sl_mxfp4_dequantize(void* stream, const uint8_t* q, const uint8_t* s, void* out, int64_t rows,
                                   int64_t cols) {
  if (rows < 0 || cols < 0) return SL_EINVAL;
  if (rows >= kMaxExtent || cols >= kMaxExtent || cols % 32) return SL_ESHAPE;
  if (rows == 0 || cols == 0) return SL_OK;
  if (!q || !s || !out) return SL_EINVAL;
  if (!aligned16(q) || !aligned16(out)) return SL_EALIGN;
  return f4_dequantize(static_cast<hipStream_t>(stream), q, s, out, rows, cols) == 0 ? SL_OK : SL_EHIP;
}

extern "C" size_t sl_mxfp4_fwd_workspace_bytes(int64_t T, int64_t in, int64_t out) {
  return check_product(T, in, out, in) ? 0 : product_workspace(T, out, in);
}

extern "C" int sl_linear_fwd_mxfp4(void* stream, const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                                   const uint8_t* Ws, void* Y, int64_t T, int64_t in, int64_t out, void* workspace,
                                   size_t workspace_bytes) {
  const int st = check_product(T, in, out, in);
  return st ? st : product(stream, Xq, Xs, Wq, Ws, Y, T, out, in, workspace, workspace_bytes);
}

extern "C" size_t sl_mxfp4_dgrad_workspace_bytes(int64_t T, int64_t in, int64_t out) {
  return check_product(T, in, out, out) ? 0 : product_workspace(T, in, out);
}

extern "C" int sl_linear_dgrad_mxfp4(void* stream, const uint8_t* dYq, const uint8_t* dYs, const uint8_t* WqT,
                                     const uint8_t* WsT, void* dX, int64_t T, int64_t in, int64_t out, void* workspace,
                                     size_t workspace_bytes) {
  const int st = check_product(T, in, out, out);
  return st ? st : product(stream, dYq, dYs, WqT, WsT, dX, T, in, out, workspace, workspace_bytes);
}

extern "C" size_t sl_mxfp4_wgrad_workspace_bytes(int64_t T, int64_t in, int64_t out) {
  if (check_product(T, in, out, T) || T == 0 || in == 0 || out == 0) return 0;
  return planes_bytes(wgrad_plan(T, in, out));
}

extern "C" int sl_linear_wgrad_accum_mxfp4(void* stream, const uint8_t* dYqT, const uint8_t* dYsT, const uint8_t* XqT,
                                           const uint8_t* XsT, float* main_grad, int64_t T, int64_t in, int64_t out,
                                           void* workspace, size_t workspace_bytes) {
  int st = check_product(T, in, out, T);
  if (st) return st;
  if (T == 0 || in == 0 || out == 0) return SL_OK;
  if (!dYqT || !dYsT || !XqT || !XsT || !main_grad) return SL_EINVAL;
  if (!aligned16(dYqT) || !aligned16(XqT) || !aligned16(main_grad)) return SL_EALIGN;
  st = check_grid(out, in);
  if (st) return st;
  F4Args g = wgrad_plan(T, in, out);
  if (g.splits > 1) {
    if (!workspace || !aligned16(workspace) || workspace_bytes < planes_bytes(g))
      return SL_EWORKSPACE;
    g.ws = static_cast<float*>(workspace);
  }
  g.a = dYqT; g.b = XqT; g.sa = dYsT; g.sb = XsT; g.c = main_grad;
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  if (f4_accum(hs, g)) return SL_EHIP;
  if (g.splits > 1 && f4_reduce(hs, main_grad, g.ws, out, in, g.splits)) return SL_EHIP;
  return SL_OK;
}

// ---- bf16 activations with MXFP4 weights ------------------------------------------------------

namespace {

// A product of T bf16 rows with an MXFP4 weight: Y[T][N] over K.
F4RowsArgs w4_args(const void* x, const void* w, const void* ws, void* y, int64_t T, int64_t N, int64_t K) {
  F4RowsArgs g{x, nullptr, w, ws, y, T, N, K, nullptr, 1, 1};
  w4_plan(g);
  return g;
}

size_t w4_workspace(int64_t T, int64_t in, int64_t out, bool dgrad) {
  if (check_product(T, in, out, in) || T == 0 || in == 0 || out == 0) return 0;
  const int64_t N = dgrad ? in : out;
  if (w4_by_copy(T, N, dgrad)) return size_t(out) * size_t(in) * 2;
  if (!dgrad && few_rows_bf16(T, in)) return 0;
  const F4RowsArgs g = w4_args(nullptr, nullptr, nullptr, nullptr, T, N, dgrad ? out : in);
  return g.splits > 1 ? size_t(g.splits) * size_t(T) * size_t(N) * 4 : 0;
}

int w4_product(void* stream, const void* x, const uint8_t* Wq, const uint8_t* Ws, void* y, int64_t T, int64_t in, int64_t out,
               bool dgrad, void* workspace, size_t workspace_bytes) {
  const int st = check_product(T, in, out, in);
  if (st) return st;
  const int64_t N = dgrad ? in : out, K = dgrad ? out : in;
  if (T == 0 || N == 0) return SL_OK;
  if (!y || (K > 0 && (!x || !Wq || !Ws))) return SL_EINVAL;
  if (!aligned16(x) || !aligned16(Wq) || !aligned16(y)) return SL_EALIGN;
  const size_t need = w4_workspace(T, in, out, dgrad);
  if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return SL_EWORKSPACE;
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  if (!w4_by_copy(T, N, dgrad)) {
    F4RowsArgs g = w4_args(x, Wq, Ws, y, T, N, K);
    g.part = static_cast<float*>(workspace);
    return (dgrad ? w4_tile_dgrad(hs, g) : few_rows_bf16(T, K) ? f4_rows(hs, g) : w4_tile_fwd(hs, g)) == 0 ? SL_OK : SL_EHIP;
  }
  if (K > 0 && f4_dequantize(hs, Wq, Ws, workspace, out, in)) return SL_EHIP;
  return (dgrad ? sl_linear_dgrad : sl_linear_fwd)(stream, x, workspace, y, T, in, out);
}

}  // namespace

extern "C" size_t sl_mxfp4w_fwd_workspace_bytes(int64_t T, int64_t in, int64_t out) { return w4_workspace(T, in, out, false); }

extern "C" size_t sl_mxfp4w_dgrad_workspace_bytes(int64_t T, int64_t in, int64_t out) { return w4_workspace(T, in, out, true); }

extern "C" int sl_linear_fwd_mxfp4w(void* stream, const void* X, const uint8_t* Wq, const uint8_t* Ws, void* Y,
                                    int64_t T, int64_t in, int64_t out, void* workspace, size_t workspace_bytes) {
  return w4_product(stream, X, Wq, Ws, Y, T, in, out, false, workspace, workspace_bytes);
}

extern "C" int sl_linear_dgrad_mxfp4w(void* stream, const void* dY, const uint8_t* Wq, const uint8_t* Ws, void* dX,
                                      int64_t T, int64_t in, int64_t out, void* workspace, size_t workspace_bytes) {
  return w4_product(stream, dY, Wq, Ws, dX, T, in, out, true, workspace, workspace_bytes);
}
