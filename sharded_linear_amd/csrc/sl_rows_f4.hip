// Products of a few rows with an MXFP4 weight (gfx950): Y[T][N] = X . W^T for the tokens of a decoding
// batch, X in MXFP4 or in bf16, W[N][K] blocked along K.
//
// Such a call reads the weight once (0.53 bytes an element) and little else, so it is bound by HBM and,
// for the usual shard, by the time of one round trip.  Nothing is staged: a lane's share of a 128-wide k
// step of 16 weight rows is one 16-byte load, and a row's scales of U steps are one load too.  A
// workgroup takes 16 R rows, its 8 waves split K, each with U steps in flight, and their partial
// sums are added in wave order through LDS.
//   X in MXFP4: v_mfma_scale_f32_16x16x128_f8f6f4 takes both operands' codes as they are stored
//     (lane l: row l % 16, block l / 16 of the step).
//   X in bf16: four v_mfma_f32_16x16x32_bf16 take the step's four blocks in turn, on codes made bf16 in
//     registers (exact).  For that the four lanes of a row trade dwords, so that each holds 8 elements of
//     every block: X is then read 64 contiguous bytes to a row, as W is.  With the codes left where they
//     are loaded, X came in 16-byte pieces 64 bytes apart, four times the cache accesses.
//
// Measured: one token by [8192, 2048] 4.7 us with bf16 X, by [6144, 4096] 5.3 us with MXFP4 X (2.5 TB/s); 16 tokens
// by [11008, 4096] with bf16 X 10.6 us (2.3 TB/s).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sl_device.h"
#include "sl_f4.h"
#include "sl_mx.h"

namespace sl2 {

constexpr int kRowWaves = 8;

// The scales of blocks b .. b + 4 U - 1 (b < nb) of a row of nb, four to a word; 0 past the row's end.
// One load, whatever the address; where it would pass the end, it ends there and is shifted.
template <int U>
__device__ __forceinline__ void load_scales(const uint8_t* row, int b, int nb, uint32_t (&d)[U]) {
  if (nb >= 4 * U) {
    const int over = b + 4 * U - nb;
    __builtin_memcpy(d, row + (over > 0 ? nb - 4 * U : b), 4 * U);
    if (over > 0) {
      for (int o = over; o >= 4; o -= 4) {
#pragma unroll
        for (int u = 0; u < U; ++u) d[u] = u + 1 < U ? d[u + 1] : 0;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) d[u] = __builtin_amdgcn_alignbyte(u + 1 < U ? d[u + 1] : 0u, d[u], over & 3);
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) d[u] = 0;
    for (int e = 0; b + e < nb; ++e) {
#pragma unroll
      for (int u = 0; u < U; ++u) d[u] |= e / 4 == u ? uint32_t(row[b + e]) << (8 * (e % 4)) : 0u;
    }
  }
}

__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
}

// Word j of lane (r, q), r = lane % 16 and q = lane / 16, becomes word q of lane (r, j).
__device__ __forceinline__ void trade(uint4& v) {
  auto p = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  v.x = p[0]; v.z = p[1];
  p = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  v.y = p[0]; v.w = p[1];
  p = __builtin_amdgcn_permlane16_swap(v.x, v.y, false, false);
  v.x = p[0]; v.y = p[1];
  p = __builtin_amdgcn_permlane16_swap(v.z, v.w, false, false);
  v.z = p[0]; v.w = p[1];
}

// XBF: X is bf16.  R: 16-row groups of W, TN: 16-row groups of X, U: k steps in flight.
template <bool XBF, int R, int TN, int U>
__global__ void __launch_bounds__(kRowWaves * 64) rows_f4(F4RowsArgs g) {
  __shared__ f32x4v part[kRowWaves][R * TN][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = int64_t(blockIdx.x) * (16 * R), t0 = int64_t(blockIdx.y) * (16 * TN);
  const int r = lane & 15, q = lane >> 4;
  const int nb = int(g.K / 32), steps = (nb + 3) / 4;
  constexpr int kXBlock = XBF ? 64 : 16;                        // bytes of a block of X
  // descriptors over this workgroup's rows: rows past the end read zeros
  const int rows_n = int(g.N - n0 < 16 * R ? g.N - n0 : 16 * R), rows_t = int(g.T - t0 < 16 * TN ? g.T - t0 : 16 * TN);
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      static_cast<char*>(const_cast<void*>(g.w)) + n0 * nb * 16, 0, rows_n * nb * 16, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      static_cast<char*>(const_cast<void*>(g.x)) + t0 * nb * kXBlock, 0, rows_t * nb * kXBlock, kRsrcWord3);
  // rows of scales; those past the end repeat the last one's, whose codes are zeros
  const uint8_t* ws[R];
  const uint8_t* xs[TN];
#pragma unroll
  for (int i = 0; i < R; ++i) ws[i] = static_cast<const uint8_t*>(g.ws) + (n0 + min(16 * i + r, rows_n - 1)) * nb;
#pragma unroll
  for (int j = 0; j < TN; ++j) xs[j] = static_cast<const uint8_t*>(g.xs) + (t0 + min(16 * j + r, rows_t - 1)) * nb;

  f32x4v acc[R][TN] = {};
  for (int s0 = wave * U; s0 < steps; s0 += kRowWaves * U) {
    uint4 w[U][R], x[U][TN][XBF ? 4 : 1];
    uint32_t sw[R][U], sx[TN][U];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = 4 * (s0 + u) + q;                         // this lane's block of the step
        w[u][i] = load16(rw, b < nb ? uint32_t((16 * i + r) * nb + b) * 16 : kOOB);
      }
      load_scales(ws[i], 4 * s0, nb, sw[i]);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = 4 * (s0 + u);
        if constexpr (XBF) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[u][j][e] = load16(rx, b + e < nb ? uint32_t((16 * j + r) * nb + b + e) * 64 + q * 16 : kOOB);
        } else {
          x[u][j][0] = load16(rx, b + q < nb ? uint32_t((16 * j + r) * nb + b + q) * 16 : kOOB);
        }
      }
      if constexpr (!XBF) load_scales(xs[j], 4 * s0, nb, sx[j]);
    }
    if constexpr (XBF && U == 4) __builtin_amdgcn_sched_barrier(0);     // all on their way before the first is used
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if constexpr (XBF) {
          trade(w[u][i]);
          const uint32_t c[4] = {w[u][i].x, w[u][i].y, w[u][i].z, w[u][i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bf16x8 a = f4_to_bf16x8(c[e], e8m0_to_f32((sw[i][u] >> (8 * e)) & 0xFFu));
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
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[i][j], 4, 4, 0, int(sw[i][u] >> (8 * q)), 0,
                                                                          int(sx[j][u] >> (8 * q)));
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

// R: the 16-row groups of W that give each of the 256 CUs one workgroup.  Fewer would need a second
// round, more would leave CUs without one: 16 tokens on [11008, 4096] (688 groups) took 17.3, 15.6,
// 11.3 and 13.0 us with bf16 X and R = 1, 2, 3 and 4, on [6144, 4096] (384) 12.3, 9.1, 11.0 and 12.8.
// U: 4 steps in flight with MXFP4 X; with bf16 X, whose registers hold 4 KiB a step, 2, and 4 for
// up to 4 tokens where 2 would need a second round of loads: one token by [4096, 5504] 5.9 us with 2, 5.3 with 4, by
// [2048, 8192] 7.1 and 6.4, but 8 by [4096, 11008] 11.7 and 12.3.
template <bool XBF, int TN, int U>
int dispatch_r(hipStream_t st, const F4RowsArgs& g) {
  const int64_t groups = (g.N + 15) / 16;
  if (groups <= 256) return launch_rows<XBF, 1, TN, U>(st, g);
  if (groups <= 512) return launch_rows<XBF, 2, TN, U>(st, g);
  if (groups <= 768) return launch_rows<XBF, 3, TN, U>(st, g);
  return launch_rows<XBF, 4, TN, U>(st, g);
}

template <bool XBF>
int dispatch_rows(hipStream_t st, const F4RowsArgs& g) {
  if constexpr (XBF) {                                           // up to 32 rows
    if (g.T > 16) return dispatch_r<XBF, 2, 2>(st, g);
    return g.T <= 4 && g.K > kRowWaves * 2 * 128 ? dispatch_r<XBF, 1, 4>(st, g) : dispatch_r<XBF, 1, 2>(st, g);
  } else {
    return g.T <= 16 ? dispatch_r<XBF, 1, 4>(st, g) : g.T <= 32 ? dispatch_r<XBF, 2, 4>(st, g) : dispatch_r<XBF, 4, 4>(st, g);
  }
}

}  // namespace sl2

int f4_rows(hipStream_t st, const F4RowsArgs& g) {
  return g.xs ? sl2::dispatch_rows<false>(st, g) : sl2::dispatch_rows<true>(st, g);
}
