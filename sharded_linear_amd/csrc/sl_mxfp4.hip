// C-ABI entry points of the MXFP4 operators: argument checks and launches.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sharded_linear.h"
#include "sl_f4.h"

namespace {

constexpr int64_t kMaxExtent = int64_t(1) << 31;
constexpr int64_t kMaxTiles = int64_t(1) << 31;        // workgroups of one launch
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

// Tiles of a bf16 result: 256x256 where they fill most of the 256 CUs, else 128x128.
int pick_config(int64_t M, int64_t N) {
  const int forced = block_scaled_config();
  if (forced >= 0) return forced;
  return ntiles(M, N, 256, 256) >= 200 ? 0 : 1;
}

// Rows up to which a product reads the weight directly.
constexpr int64_t kFewRows = 64, kFewRowsBf16 = 32;
// Rows from which a bf16 copy of the weight pays for itself.
constexpr int64_t kManyRowsFwd = 1024, kManyRowsDgrad = 1024;

// C[M][N] = A . B^T (bf16) over K
int product(void* stream, const uint8_t* a, const uint8_t* sa, const uint8_t* b, const uint8_t* sb, void* c, int64_t M,
            int64_t N, int64_t K) {
  if (M == 0 || N == 0) return SL_OK;
  if (!c || (K > 0 && (!a || !sa || !b || !sb))) return SL_EINVAL;
  if (!aligned16(c) || !aligned16(a) || !aligned16(b)) return SL_EALIGN;
  const int st = check_grid(M, N);
  if (st) return st;
  if (M <= kFewRows && block_scaled_config() < 0) {
    const F4RowsArgs r{a, sa, b, sb, c, M, N, K};
    // an empty K may come without scales, and X without scales is bf16
    return f4_rows(static_cast<hipStream_t>(stream), K ? r : F4RowsArgs{c, c, c, c, c, M, N, 0}) == 0 ? SL_OK : SL_EHIP;
  }
  F4Args g{};
  g.a = a; g.b = b; g.sa = sa; g.sb = sb; g.c = c;
  g.M = M; g.N = N; g.K = K;
  g.splits = 1;
  g.cfg = pick_config(M, N);
  return f4_gemm(static_cast<hipStream_t>(stream), g) == 0 ? SL_OK : SL_EHIP;
}

// Tiles and split of K of the weight gradient: 256x256 tiles; where those fill about half the chip and
// 256x128 tiles fill it once, those, unsplit; otherwise K split to fill the 256 CUs, with at least 4
// stages (an even number) to a split and at most 16 splits.
F4Args wgrad_plan(int64_t T, int64_t in, int64_t out) {
  F4Args g{};
  g.M = out; g.N = in; g.K = T;
  const int64_t t256 = ntiles(out, in, 256, 256), t128 = ntiles(out, in, 256, 128), nkt = (T + kF4StageK - 1) / kF4StageK;
  const int forced = block_scaled_config();
  g.cfg = forced >= 0 ? forced : (t256 <= 144 && t128 >= 240 && t128 <= 288) ? 2 : 0;
  const int64_t tiles = g.cfg == 0 ? t256 : g.cfg == 2 ? t128 : ntiles(out, in, 128, 128);
  int64_t s = tiles < 200 ? (256 + tiles / 2) / tiles : 1;
  if (s > nkt / 4) s = nkt / 4;
  if (s > 16) s = 16;
  if (s < 1) s = 1;
  int64_t per = (nkt + s - 1) / s;
  per += per & 1;                        // the kernel starts at an even stage
  g.kt_per_split = int(per);
  g.splits = int((nkt + per - 1) / per);
  return g;
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
  if (ntiles(rows, cols, 128, 128) >= kMaxTiles) return SL_ESHAPE;
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

extern "C" int sl_linear_fwd_mxfp4(void* stream, const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                                   const uint8_t* Ws, void* Y, int64_t T, int64_t in, int64_t out) {
  const int st = check_product(T, in, out, in);
  return st ? st : product(stream, Xq, Xs, Wq, Ws, Y, T, out, in);
}

extern "C" int sl_linear_dgrad_mxfp4(void* stream, const uint8_t* dYq, const uint8_t* dYs, const uint8_t* WqT,
                                     const uint8_t* WsT, void* dX, int64_t T, int64_t in, int64_t out) {
  const int st = check_product(T, in, out, out);
  return st ? st : product(stream, dYq, dYs, WqT, WsT, dX, T, in, out);
}

extern "C" size_t sl_mxfp4_wgrad_workspace_bytes(int64_t T, int64_t in, int64_t out) {
  if (check_product(T, in, out, T) || T == 0 || in == 0 || out == 0) return 0;
  const F4Args g = wgrad_plan(T, in, out);
  return g.splits > 1 ? size_t(g.splits) * size_t(out) * size_t(in) * 4 : 0;
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
    if (!workspace || !aligned16(workspace) || workspace_bytes < sl_mxfp4_wgrad_workspace_bytes(T, in, out))
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

extern "C" size_t sl_mxfp4w_fwd_workspace_bytes(int64_t T, int64_t in, int64_t out) {
  if (check_product(T, in, out, in) || T < kManyRowsFwd || in == 0 || out == 0) return 0;
  return size_t(out) * size_t(in) * 2;
}

extern "C" size_t sl_mxfp4w_dgrad_workspace_bytes(int64_t T, int64_t in, int64_t out) {
  if (check_product(T, in, out, in) || T < kManyRowsDgrad || in == 0 || out == 0) return 0;
  return size_t(out) * size_t(in) * 2;
}

extern "C" int sl_linear_fwd_mxfp4w(void* stream, const void* X, const uint8_t* Wq, const uint8_t* Ws, void* Y,
                                    int64_t T, int64_t in, int64_t out, void* workspace, size_t workspace_bytes) {
  const int st = check_product(T, in, out, in);
  if (st) return st;
  if (T == 0 || out == 0) return SL_OK;
  if (!Y || (in > 0 && (!X || !Wq || !Ws))) return SL_EINVAL;
  if (!aligned16(X) || !aligned16(Wq) || !aligned16(Y)) return SL_EALIGN;
  if (T < kManyRowsFwd) {
    const F4RowsArgs g{X, nullptr, Wq, Ws, Y, T, out, in};
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    return (T <= kFewRowsBf16 ? f4_rows(hs, g) : w4_tile_fwd(hs, g)) == 0 ? SL_OK : SL_EHIP;
  }
  const size_t need = sl_mxfp4w_fwd_workspace_bytes(T, in, out);
  if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return SL_EWORKSPACE;
  if (in > 0 && f4_dequantize(static_cast<hipStream_t>(stream), Wq, Ws, workspace, out, in)) return SL_EHIP;
  return sl_linear_fwd(stream, X, workspace, Y, T, in, out);
}

extern "C" int sl_linear_dgrad_mxfp4w(void* stream, const void* dY, const uint8_t* Wq, const uint8_t* Ws, void* dX,
                                      int64_t T, int64_t in, int64_t out, void* workspace, size_t workspace_bytes) {
  const int st = check_product(T, in, out, in);
  if (st) return st;
  if (T == 0 || in == 0) return SL_OK;
  if (!dX || (out > 0 && (!dY || !Wq || !Ws))) return SL_EINVAL;
  if (!aligned16(dY) || !aligned16(Wq) || !aligned16(dX)) return SL_EALIGN;
  if (T < kManyRowsDgrad)
    return w4_tile_dgrad(static_cast<hipStream_t>(stream), F4RowsArgs{dY, nullptr, Wq, Ws, dX, T, in, out}) == 0 ? SL_OK : SL_EHIP;
  const size_t need = sl_mxfp4w_dgrad_workspace_bytes(T, in, out);
  if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return SL_EWORKSPACE;
  if (out > 0 && f4_dequantize(static_cast<hipStream_t>(stream), Wq, Ws, workspace, out, in)) return SL_EHIP;
  return sl_linear_dgrad(stream, dY, workspace, dX, T, in, out);
}
