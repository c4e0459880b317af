// Products of a few rows with an MXFP4 weight (gfx950): Y[T][N] = X . W^T for the tokens of a decoding
// batch, X in MXFP4 or in bf16, W[N][K] blocked along K.
//
// Such a call reads the weight once (0.53 bytes an element) and little else, so it is bound by HBM and,
// for the usual shard, by the time of one round trip.  Nothing is staged: a lane's share of a 128-wide k
// step of 16 weight rows is one 16-byte load, a whole scale block, with its scale byte.  A workgroup
// takes 16 R rows, its 8 waves split K, each keeping U k steps in flight, and their partial sums are
// added in wave order through LDS.
//   X in MXFP4: v_mfma_scale_f32_16x16x128_f8f6f4 takes both operands' codes as they are stored
//     (lane l: row l % 16, block l / 16 of the step).
//   X in bf16: the codes become bf16 in registers (exact) and four v_mfma_f32_16x16x32_bf16 take the
//     step; the j-th contracts elements 8 j .. 8 j + 7 of every lane's block, an order of k that both
//     operands share, so that X too is read in whole 64-byte pieces.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sl_device.h"
#include "sl_f4.h"
#include "sl_mx.h"

namespace sl2 {

constexpr int kRowWaves = 8;

__device__ __forceinline__ bf16x8 f4_to_bf16x8(uint32_t codes, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// XBF: X is bf16.  R: 16-row groups of W, TN: 16-row groups of X, U: k steps in flight.
template <bool XBF, int R, int TN, int U>
__global__ void __launch_bounds__(kRowWaves * 64) rows_f4(F4RowsArgs g) {
  __shared__ f32x4v part[kRowWaves][R * TN][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n0 = int64_t(blockIdx.x) * (16 * R), t0 = int64_t(blockIdx.y) * (16 * TN);
  const int r = lane & 15, q = lane >> 4;
  const int nb = int(g.K / 32), steps = (nb + 3) / 4;
  const uint4* const W = static_cast<const uint4*>(g.w);
  const uint8_t *const ws = static_cast<const uint8_t*>(g.ws), *const xs = static_cast<const uint8_t*>(g.xs);
  const uint4* const X = static_cast<const uint4*>(g.x);

  f32x4v acc[R][TN] = {};
  for (int s0 = wave * U; s0 < steps; s0 += kRowWaves * U) {
    uint4 w[U][R], x[U][TN][XBF ? 4 : 1];
    uint32_t sw[U][R], sx[U][TN];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = 4 * (s0 + u) + q;                           // this lane's block of the step
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int64_t n = n0 + 16 * i + r;
        const bool in = b < nb && n < g.N;
        w[u][i] = in ? W[n * nb + b] : make_uint4(0, 0, 0, 0);
        sw[u][i] = in ? ws[n * nb + b] : 0;
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int64_t t = t0 + 16 * j + r;
        const bool in = b < nb && t < g.T;
        if constexpr (XBF) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[u][j][e] = in ? X[(t * nb + b) * 4 + e] : make_uint4(0, 0, 0, 0);
        } else {
          x[u][j][0] = in ? X[t * nb + b] : make_uint4(0, 0, 0, 0);
          sx[u][j] = in ? xs[t * nb + b] : 0;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if constexpr (XBF) {
          const float sc = e8m0_to_f32(sw[u][i]);
          const uint32_t c[4] = {w[u][i].x, w[u][i].y, w[u][i].z, w[u][i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bf16x8 a = f4_to_bf16x8(c[e], sc);
#pragma unroll
            for (int j = 0; j < TN; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, x[u][j][e]), acc[i][j], 0, 0, 0);
          }
        } else {
          const i32x8 a = {int(w[u][i].x), int(w[u][i].y), int(w[u][i].z), int(w[u][i].w), 0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            const uint4 v = x[u][j][0];
            const i32x8 b = {int(v.x), int(v.y), int(v.z), int(v.w), 0, 0, 0, 0};
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[i][j], 4, 4, 0, int(sw[u][i]), 0, int(sx[u][j]));
          }
        }
      }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) part[wave][i * TN + j][lane] = acc[i][j];
  __syncthreads();
  // lane l of block (i, j): token 16 j + l % 16, features 16 i + 4 (l / 16) + 0..3
  for (int p = tid; p < R * TN * 64; p += kRowWaves * 64) {
    const int l = p & 63, ij = p >> 6;
    f32x4v s = part[0][ij][l];
#pragma unroll
    for (int v = 1; v < kRowWaves; ++v) s += part[v][ij][l];
    const int64_t t = t0 + 16 * (ij % TN) + (l & 15), n = n0 + 16 * (ij / TN) + 4 * (l >> 4);
    if (t < g.T && n < g.N) {
      bf16x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = static_cast<__bf16>(s[e]);
      *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(g.y) + t * g.N + n) = o;
    }
  }
}

template <bool XBF, int R, int TN, int U>
int launch_rows(hipStream_t st, const F4RowsArgs& g) {
  const dim3 grid(unsigned((g.N + 16 * R - 1) / (16 * R)), unsigned((g.T + 16 * TN - 1) / (16 * TN)));
  hipLaunchKernelGGL((rows_f4<XBF, R, TN, U>), grid, dim3(kRowWaves * 64), 0, st, g);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

template <bool XBF>
int dispatch_rows(hipStream_t st, const F4RowsArgs& g) {
  if (g.T <= 16) return g.N >= 16 * 512 ? launch_rows<XBF, 2, 1, 2>(st, g) : launch_rows<XBF, 1, 1, 4>(st, g);
  if (g.T <= 32) return launch_rows<XBF, 2, 2, 2>(st, g);
  return launch_rows<XBF, 2, 4, 1>(st, g);
}

}  // namespace sl2

int f4_rows(hipStream_t st, const F4RowsArgs& g) {
  return g.xs ? sl2::dispatch_rows<false>(st, g) : sl2::dispatch_rows<true>(st, g);
}
