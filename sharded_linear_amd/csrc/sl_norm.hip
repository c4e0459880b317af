// Root-mean-square norm with the residual's addition, and its gradient (gfx950).
//
//   h = bf16(x + residual)      rstd = (mean(h^2) + eps)^-1/2      y = h * rstd * w
//   g = w * dY                  dX = dresidual + rstd * (g - h * rstd^2 * mean(g * h))
//   w_grad += sum over rows of dY * h * rstd
//
// y is rounded to bf16, or straight to MXFP8 (the OCP MX rule of the quantiser in
// sl_quant.hip), rowwise and columnwise, as the products of the all-MXFP8 step read it.  The norm is
// of the rounded h, which is what the next layer adds to and what the gradient reads again.
//
// MXFP8 has borders: where a block's largest magnitude lies within an error of a power of two, the whole block is encoded with
// another scale.  With y in plain fp32 that befell one block in some ten million, so the forward's sums end in 64 bits, rstd is
// held in two floats (to 2^-47), and h * w (exact in fp32) times rstd is rounded to odd: the code is then that of h * w by this
// rstd, which is off by the fp32 sums of a lane's few squares.  (Of results below 2^-100, fp32 cannot hold what a product leaves.)
//
// Every kernel here is bound by HBM, so each row passes through registers once: TPR threads hold a
// row, NC chunks of 8 elements a thread.  Means are fp32 sums of each of a lane's 8 columns in order, then of those; then
// of the lanes by DPP and half-wave swaps, and of the waves in order (in 64 bits in the forward).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sharded_linear.h"
#include "sl_device.h"
#include "sl_mx.h"

namespace {

using sl2::bf16x8;

typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x8 widen(uint4 v) { return __builtin_convertvector(__builtin_bit_cast(bf16x8, v), f32x8); }
__device__ __forceinline__ uint4 narrow(f32x8 v) { return __builtin_bit_cast(uint4, __builtin_convertvector(v, bf16x8)); }

template <int CTRL>
__device__ __forceinline__ float add_dpp(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double add_dpp(double x) {
  const int2 v = __builtin_bit_cast(int2, x);
  return x + __builtin_bit_cast(double, make_int2(__builtin_amdgcn_update_dpp(0, v.x, CTRL, 0xF, 0xF, false),
                                                  __builtin_amdgcn_update_dpp(0, v.y, CTRL, 0xF, 0xF, false)));
}

// Both halves' values of a swap of 16- or 32-lane halves, added.
template <int LANES>
__device__ __forceinline__ float add_halves(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  const auto r = LANES == 16 ? __builtin_amdgcn_permlane16_swap(b, b, false, false) : __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __builtin_bit_cast(float, uint32_t(r[0])) + __builtin_bit_cast(float, uint32_t(r[1]));
}
template <int LANES>
__device__ __forceinline__ double add_halves(double x) {
  const uint2 b = __builtin_bit_cast(uint2, x);
  const auto r = LANES == 16 ? __builtin_amdgcn_permlane16_swap(b.x, b.x, false, false) : __builtin_amdgcn_permlane32_swap(b.x, b.x, false, false);
  const auto s = LANES == 16 ? __builtin_amdgcn_permlane16_swap(b.y, b.y, false, false) : __builtin_amdgcn_permlane32_swap(b.y, b.y, false, false);
  return __builtin_bit_cast(double, make_uint2(r[0], s[0])) + __builtin_bit_cast(double, make_uint2(r[1], s[1]));
}

// Sum over the 64 lanes, in every lane: pairs, quads, 8 and 16 lanes by DPP, then the 16- and 32-lane halves.
template <typename S>
__device__ __forceinline__ S wave_sum(S x) {
  x = add_dpp<0xB1>(x);     // quad_perm [1,0,3,2]
  x = add_dpp<0x4E>(x);     // quad_perm [2,3,0,1]
  x = add_dpp<0x141>(x);    // row_half_mirror
  x = add_dpp<0x140>(x);    // row_mirror
  return add_halves<32>(add_halves<16>(x));
}

__device__ __forceinline__ float fold(f32x8 v) { return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7])); }

// Sum over the TPR threads of a row (a wave, or a whole workgroup).  `turn` alternates between calls, so that one
// barrier a call is enough.
template <int TPR, typename S>
__device__ __forceinline__ S row_sum(S x, S* red, int turn) {
  x = wave_sum(x);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    S* r = red + turn * W;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = x;
    __syncthreads();
    x = r[0];
#pragma unroll
    for (int w = 1; w < W; ++w) x += r[w];
  }
  return x;
}

// x^-1/2 as the nearest float and what it leaves: two terms of the series in 1 - x r^2 from the fp32 root r.
__device__ __forceinline__ float2 inverse_root(double x) {
  const float r = 1.0f / sqrtf(float(x));
  const double off = fma(-x * r, double(r), 1.0), c = r + r * off * fma(0.375, off, 0.5);
  const float hi = float(c);
  return hi - hi == 0.f ? make_float2(hi, float(c - hi)) : make_float2(r, 0.f);      // zeros, infinities and NaN as they come
}

// p times the two floats of r, rounded to odd: the last bit is set where anything was left, so that a later rounding to fewer bits
// is that of the product.  p r.x is off by up to half a unit in its last place and p r.y adds up to a whole one, so what is left is
// added before the last bit is looked at.
__device__ __forceinline__ float odd_product(float p, float2 r) {
  const float y = p * r.x, left = fmaf(p, r.y, fmaf(p, r.x, -y)), z = y + left, rest = left - (z - y);
  const uint32_t b = __float_as_uint(z), away = (__float_as_uint(rest) ^ b) >> 31 ? ~0u : 1u;
  if (left == 0.f || rest - rest != 0.f) return y;     // zeros with their sign; infinities, NaN, and what would become one
  return __uint_as_float(rest != 0.f && !(b & 1) ? b + away : b);
}

// E8M0 byte of a block whose largest magnitude has the fp32 bits `amax`: floor(log2 amax) - 8, biased; 255 (NaN) for
// a block with an infinity or a NaN.
__device__ __forceinline__ uint32_t mx8_scale(uint32_t amax) {
  const int e = int(amax >> 23) - 8;
  return amax >= 0x7F800000u ? 255u : uint32_t(e < 0 ? 0 : e);
}

// E4M3 codes of 4 elements under that scale byte, nearest-even, saturating at +-448; none in a block of zeros of
// either sign.  The conversion divides by an
// fp32 scale and gives the NaN code where a quotient rounds past 448; 2^-127 is no normal fp32 number, so blocks that
// small are moved up by 2^64 first (exactly).
__device__ __forceinline__ uint32_t mx8_codes(float a, float b, float c, float d, uint32_t s, uint32_t amax) {
  if (s == 255 || amax == 0) return 0;
  const float scale = __uint_as_float((s ? s : 64u) << 23), up = s ? 1.0f : 0x1p64f;
  sl2::s16x2 r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32((sl2::s16x2){0, 0}, a * up, b * up, scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c * up, d * up, scale, true);
  const uint32_t q = __builtin_bit_cast(uint32_t, r);
  const uint32_t nan = ((q & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return q - (nan >> 7);
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Below kBorder for a magnitude p r.x other than zero (zeros of either sign are frequent, and no border) whose odd_product may
// lie on the other side of a border, or on it: borders of E4M3's four bits, subnormal codes' among them, and powers of two have no
// bits in their last 19 places, and the product is less than two units in the last place from p r.x.  Of the unit above it, the
// last 19 bits are then 0 to 2 (3 passes the comparison too).
constexpr uint32_t kBorder = 0x7000;
__device__ __forceinline__ uint32_t border_key(uint32_t magnitude) {
  const uint32_t next = magnitude + 1;
  return (__builtin_amdgcn_alignbit(next, next, 19) ^ 0x2000) - 1;
}

enum Out { kBF16, kRows, kNothing };

struct FwdArgs {
  const uint4 *x, *res, *w;
  uint4 *y, *h;
  uint2* q;
  uint8_t* s;
  float *rstd, *left;  // left: what the rounding of rstd left, or null
  int64_t T;
  int chunks;          // H / 8
  double h_inv;        // 1 / H
  float eps;
};

// With a residual, rowwise MXFP8: [8192, 2048] 21.7 us, 118 MB, 5.4 TB/s, as a copy; one row of 4096 2.8 us, the launch.
template <int TPR, int NC, bool RES, int OUT>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_fwd(FwdArgs g) {
  constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
  __shared__ double red[TPR > 64 ? 2 * TPR / 64 : 1];
  const int lane = threadIdx.x % TPR;
  uint4 w[NC];
  if constexpr (OUT != kNothing)
#pragma unroll
    for (int j = 0; j < NC; ++j) w[j] = lane + j * TPR < g.chunks ? g.w[lane + j * TPR] : make_uint4(0, 0, 0, 0);
  int turn = 0;
  for (int64_t t = int64_t(blockIdx.x) * ROWS + threadIdx.x / TPR; t < g.T; t += int64_t(gridDim.x) * ROWS, turn ^= 1) {
    uint4 v[NC];
    const uint4* x = g.x + t * g.chunks;
#pragma unroll
    for (int j = 0; j < NC; ++j) v[j] = lane + j * TPR < g.chunks ? x[lane + j * TPR] : make_uint4(0, 0, 0, 0);
    if constexpr (RES) {
      uint4 r[NC];
      const uint4* res = g.res + t * g.chunks;
#pragma unroll
      for (int j = 0; j < NC; ++j) r[j] = lane + j * TPR < g.chunks ? res[lane + j * TPR] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        v[j] = narrow(widen(v[j]) + widen(r[j]));
        if (lane + j * TPR < g.chunks) g.h[t * g.chunks + lane + j * TPR] = v[j];
      }
    }
    f32x8 squares = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const f32x8 a = widen(v[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) squares[e] = fmaf(a[e], a[e], squares[e]);
    }
    const float2 rstd = inverse_root(row_sum<TPR>(double(fold(squares)), red, turn) * g.h_inv + g.eps);
    if (lane == 0) {
      g.rstd[t] = rstd.x;
      if (g.left) g.left[t] = rstd.y;
    }
    if constexpr (OUT != kNothing) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = lane + j * TPR;
        f32x8 y = widen(v[j]) * widen(w[j]);                     // exact
        if constexpr (OUT == kBF16) {
          if (c < g.chunks) g.y[t * g.chunks + c] = narrow(y * rstd.x);
        } else {
          const f32x8 p = y;
          y = p * rstd.x;
          uint32_t border = ~0u;
#pragma unroll
          for (int e = 0; e < 8; ++e) border = min(border, border_key(magnitude(y[e])));
          if (border < kBorder)
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = odd_product(p[e], rstd);
          // a block is the 4 chunks of a quad of lanes (chunks % 4 == 0: whole quads are in range)
          uint32_t amax = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = max(amax, magnitude(y[e]));
          amax = sl2::quad_max(amax);
          const uint32_t s = mx8_scale(amax);
          if (c < g.chunks) {
            g.q[t * g.chunks + c] = make_uint2(mx8_codes(y[0], y[1], y[2], y[3], s, amax), mx8_codes(y[4], y[5], y[6], y[7], s, amax));
            if ((lane & 3) == 0) g.s[t * (g.chunks / 4) + c / 4] = uint8_t(s);
          }
        }
      }
    }
  }
}

// ---- columnwise MXFP8 copy -----------------------------------------------------------------------
// One workgroup takes a 128 x 128 tile of h: rows of 16-byte chunks into LDS, from which each thread reads two blocks
// of 32 rows down a column by transposing reads, scales them (rstd by row, w by column) and encodes them; codes leave
// as whole 128-byte lines of the transposed copy.  The LDS layout is the quantiser's (sl_quant.hip).  [8192, 2048]: 16.5 us,
// 51 MB, 3.1 TB/s, of which the search for borders takes about 2; rstd needs whole rows before the first column, so h is read again here (from the last-level cache).
constexpr int kTile = 128, kStride = kTile + 16;

__global__ void __launch_bounds__(256) norm_cols(const uint16_t* __restrict__ h, const uint16_t* __restrict__ w, const float* __restrict__ rstd,
                                                 const float* __restrict__ left, int64_t R, int64_t C, uint8_t* __restrict__ qc, uint8_t* __restrict__ sc) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[kTile * kStride];
  __shared__ float inv[kTile], left_lds[kTile];
  uint8_t* const qbuf = reinterpret_cast<uint8_t*>(tile);
  uint8_t* const sbuf = qbuf + kTile * kTile;
  const int64_t ntc = (C + kTile - 1) / kTile;
  const int64_t r0 = int64_t(blockIdx.x) / ntc * kTile, c0 = int64_t(blockIdx.x) % ntc * kTile;
  const int t = threadIdx.x, ch = t & 15;
  uint4 raw[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t gr = r0 + (t >> 4) + 16 * k, gc = c0 + 8 * ch;
    raw[k] = (gr < R && gc < C) ? *reinterpret_cast<const uint4*>(h + gr * C + gc) : make_uint4(0, 0, 0, 0);
  }
  if (t < kTile) {
    inv[t] = r0 + t < R ? rstd[r0 + t] : 0.f;
    left_lds[t] = r0 + t < R ? left[r0 + t] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) reinterpret_cast<uint4*>(tile + ((t >> 4) + 16 * k) * kStride)[ch] = raw[k];
  __syncthreads();
  uint32_t q[2][8], s[2];
  const int64_t col = c0 + (t & (kTile - 1));
  const float wc = col < C ? __uint_as_float(uint32_t(w[col]) << 16) : 0.f;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int idx = t + 256 * b, rb = idx >> 7;
    // source lane 4j + q of a 16-lane group reads 4 columns of row j; result lane 4q + e holds 4 rows of its column
    const int s16 = t & 15, jr = s16 >> 2, qc4 = s16 & 3;
    const int col4 = ((idx & (kTile - 1)) & ~15) + 4 * qc4;
    const uint32_t a0 = sl2::lds_addr(tile + (rb * 32 + jr) * kStride + col4);
    float y[32];
    uint32_t amax = 0, border = ~0u;
#pragma unroll
    for (int r4 = 0; r4 < 8; ++r4) {
      const sl2::i16x4q v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) sl2::i16x4q*)(uintptr_t)(a0 + r4 * 4 * kStride * 2));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = __uint_as_float(uint32_t(uint16_t(v[e])) << 16);
        y[4 * r4 + e] = x * wc * inv[rb * 32 + 4 * r4 + e];
        const uint32_t m = magnitude(y[4 * r4 + e]);
        border = min(border, border_key(m));
        amax = max(amax, m);
      }
    }
    if (border < kBorder) {                   // a column's elements once more, from the tile as it stands
      amax = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float x = __uint_as_float(uint32_t(tile[(rb * 32 + i) * kStride + (idx & (kTile - 1))]) << 16);
        y[i] = odd_product(x * wc, make_float2(inv[rb * 32 + i], left_lds[rb * 32 + i]));
        amax = max(amax, magnitude(y[i]));
      }
    }
    s[b] = mx8_scale(amax);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[b][i] = mx8_codes(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3], s[b], amax);
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int idx = t + 256 * b, c = idx & (kTile - 1), rb = idx >> 7;
    uint8_t* line = qbuf + c * kTile;
    *reinterpret_cast<uint4*>(line + ((2 * rb) ^ (c & 7)) * 16) = make_uint4(q[b][0], q[b][1], q[b][2], q[b][3]);
    *reinterpret_cast<uint4*>(line + ((2 * rb + 1) ^ (c & 7)) * 16) = make_uint4(q[b][4], q[b][5], q[b][6], q[b][7]);
    sbuf[c * 4 + rb] = uint8_t(s[b]);
  }
  __syncthreads();
  const int nrb = int(R - r0 < kTile ? (R - r0) / 32 : 4);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int idx = t + 256 * p, c = idx >> 3, k = idx & 7;
    if (c0 + c < C && k < 2 * nrb)
      *reinterpret_cast<uint4*>(qc + (c0 + c) * R + r0 + k * 16) = *reinterpret_cast<const uint4*>(qbuf + c * kTile + (k ^ (c & 7)) * 16);
  }
  if (t < kTile && c0 + t < C) {
    uint8_t* d = sc + (c0 + t) * (R / 32) + r0 / 32;
    if (nrb == 4 && (reinterpret_cast<uintptr_t>(d) & 3) == 0) *reinterpret_cast<uint32_t*>(d) = *reinterpret_cast<const uint32_t*>(sbuf + t * 4);
    else for (int b = 0; b < nrb; ++b) d[b] = sbuf[t * 4 + b];
  }
}

// ---- gradient ------------------------------------------------------------------------------------

struct BwdArgs {
  const uint4 *dy, *h, *w, *dres;
  const float* rstd;
  uint4* dx;
  float* part;         // [gridDim.x][H], or null: the weight is frozen
  int64_t T;
  int chunks;
  float h_float;
};

// A workgroup walks rows with the weight gradient of its threads' columns in registers and leaves one plane of
// partial sums; the planes are added in order by norm_wgrad.  [8192, 4096] with the residual's gradient: 41.6 us, 277 MB, 6.7 TB/s
// (part of it out of the last-level cache), and 4.7 for the planes.
template <int TPR, int NC, bool RES>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_bwd(BwdArgs g) {
  constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[TPR > 64 ? 2 * TPR / 64 : 1];
  __shared__ f32x8 acc_lds[ROWS > 1 ? NC * TPR : 1];
  const int lane = threadIdx.x % TPR;
  uint4 w[NC];
  f32x8 acc[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    w[j] = lane + j * TPR < g.chunks ? g.w[lane + j * TPR] : make_uint4(0, 0, 0, 0);
    acc[j] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
  }
  int turn = 0;
  for (int64_t t = int64_t(blockIdx.x) * ROWS + threadIdx.x / TPR; t < g.T; t += int64_t(gridDim.x) * ROWS, turn ^= 1) {
    uint4 dy[NC], h[NC], dr[NC];
    const int64_t o = t * g.chunks + lane;
    const float rstd = g.rstd[t];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const bool in = lane + j * TPR < g.chunks;
      dy[j] = in ? g.dy[o + j * TPR] : make_uint4(0, 0, 0, 0);
      h[j] = in ? g.h[o + j * TPR] : make_uint4(0, 0, 0, 0);
      if constexpr (RES) dr[j] = in ? g.dres[o + j * TPR] : make_uint4(0, 0, 0, 0);
    }
    f32x8 dots = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const f32x8 a = widen(dy[j]) * widen(w[j]), b = widen(h[j]) * rstd;
#pragma unroll
      for (int e = 0; e < 8; ++e) dots[e] = fmaf(a[e], b[e], dots[e]);
    }
    const float mean = row_sum<TPR>(fold(dots), red, turn) / g.h_float;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const f32x8 d = widen(dy[j]), n = widen(h[j]) * rstd;
      f32x8 dx = (d * widen(w[j]) - n * mean) * rstd;
      if constexpr (RES) dx += widen(dr[j]);
      acc[j] += d * n;
      if (lane + j * TPR < g.chunks) g.dx[o + j * TPR] = narrow(dx);
    }
  }
  if (!g.part) return;
  if constexpr (ROWS > 1) {
    for (int r = 1; r < ROWS; ++r) {
      __syncthreads();
      if (int(threadIdx.x) / TPR == r)
#pragma unroll
        for (int j = 0; j < NC; ++j) acc_lds[j * TPR + lane] = acc[j];
      __syncthreads();
      if (threadIdx.x < TPR)
#pragma unroll
        for (int j = 0; j < NC; ++j) acc[j] += acc_lds[j * TPR + lane];
    }
    if (threadIdx.x >= TPR) return;
  }
#pragma unroll
  for (int j = 0; j < NC; ++j)
    if (lane + j * TPR < g.chunks) {
      float4* p = reinterpret_cast<float4*>(g.part + (int64_t(blockIdx.x) * g.chunks + lane + j * TPR) * 8);
      p[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
      p[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
    }
}

// w_grad[c] += the planes' sums: 32 columns by 32 parts of the planes to a workgroup, each part in order, then the parts.
__global__ void __launch_bounds__(1024) norm_wgrad(const float* __restrict__ part, float* __restrict__ grad, int planes, int64_t H) {
  __shared__ float sums[32][33];
  const int c = threadIdx.x & 31, p = threadIdx.x >> 5;
  const int64_t col = int64_t(blockIdx.x) * 32 + c;
  const int per = (planes + 31) / 32, p0 = p * per, p1 = min(p0 + per, planes);
  float sum = 0.f;
  if (col < H)
#pragma unroll 4
    for (int i = p0; i < p1; ++i) sum += part[int64_t(i) * H + col];
  sums[p][c] = sum;
  __syncthreads();
  if (p == 0 && col < H) {
    for (int i = 1; i < 32; ++i) sum += sums[i][c];
    grad[col] += sum;
  }
}

// ---- host ----------------------------------------------------------------------------------------

constexpr int64_t kMaxExtent = int64_t(1) << 31;
constexpr int64_t kMaxH = 16384;           // 1024 threads of 2 chunks of 8 elements
constexpr int64_t kMaxBlocks = int64_t(1) << 20;
constexpr int64_t kPlanes = 512;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_norm(int64_t T, int64_t H, float eps) {
  if (T < 0 || H < 0 || !(eps >= 0.f) || !(eps - eps == 0.f)) return SL_EINVAL;
  return T >= kMaxExtent || H > kMaxH || H % 8 ? SL_ESHAPE : SL_OK;
}

// Threads to a row: a wave while its lanes hold the row in 4 chunks each and there are rows enough for the chip, else
// a workgroup.  One rule serves the forward (with a residual) and the gradient; in us, forward + gradient, with 64 threads and with
// 256: [1, 2048] 4.1 + 6.7, 4.0 + 5.7; [512, 2048] 4.8 + 7.8, 4.7 + 9.1 (here the rule takes the slower); [8192, 2048] 25.0 +
// 23.3, 23.8 + 27.4; [8192, 512] 8.2 + 10.8, 11.0 + 18.3.  With 256 and with 1024: [8192, 4096] 41.8 + 37.4, 47.6 + 56.7;
// [8192, 8192] 94.1 + 80.5, 92.6 + 84.1.
int row_threads(int64_t T, int chunks) {
  if (chunks <= 256 && (T >= 1024 || chunks <= 64)) return 64;
  return chunks <= 1024 ? 256 : 1024;
}

// f(threads, chunks a thread) with both as compile-time constants
template <class F>
void with_row(int tpr, int chunks, F&& f) {
  const int nc = (chunks + tpr - 1) / tpr;
  auto by_nc = [&](auto t) {
    if (nc <= 1) f(t, sl2::ic<1>{});
    else if (nc <= 2) f(t, sl2::ic<2>{});
    else f(t, sl2::ic<4>{});
  };
  if (tpr == 64) by_nc(sl2::ic<64>{});
  else if (tpr == 256) by_nc(sl2::ic<256>{});
  else f(sl2::ic<1024>{}, sl2::ic<2>{});
}

int run_fwd(hipStream_t st, const FwdArgs& g, int out) {
  const int tpr = row_threads(g.T, g.chunks), rows = tpr < 256 ? 256 / tpr : 1;
  const int64_t blocks = (g.T + rows - 1) / rows;
  const dim3 grid(unsigned(blocks < kMaxBlocks ? blocks : kMaxBlocks)), threads(tpr < 256 ? 256 : tpr);
  with_row(tpr, g.chunks, [&](auto t, auto n) {
    constexpr int TPR = decltype(t)::value, NC = decltype(n)::value;
    auto go = [&](auto res) {
      constexpr bool RES = decltype(res)::value;
      if (out == kBF16) hipLaunchKernelGGL((norm_fwd<TPR, NC, RES, kBF16>), grid, threads, 0, st, g);
      else if (out == kRows) hipLaunchKernelGGL((norm_fwd<TPR, NC, RES, kRows>), grid, threads, 0, st, g);
      else hipLaunchKernelGGL((norm_fwd<TPR, NC, RES, kNothing>), grid, threads, 0, st, g);
    };
    g.res ? go(std::true_type{}) : go(std::false_type{});
  });
  return hipGetLastError() == hipSuccess ? SL_OK : SL_EHIP;
}

struct BwdPlan {
  int tpr, rows;
  int64_t planes;
};

BwdPlan bwd_plan(int64_t T, int chunks) {
  BwdPlan p{};
  p.tpr = row_threads(T, chunks);
  p.rows = p.tpr < 256 ? 256 / p.tpr : 1;
  p.planes = (T + p.rows - 1) / p.rows;
  if (p.planes > kPlanes) p.planes = kPlanes;
  return p;
}

}  // namespace

extern "C" int sl_rmsnorm_fwd(void* stream, const void* x, const void* residual, const void* w, float eps, void* y, void* h, float* rstd,
                              int64_t T, int64_t H) {
  const int e = check_norm(T, H, eps);
  if (e) return e;
  if (T == 0 || H == 0) return SL_OK;
  if (!x || !w || !y || !rstd || (residual && !h)) return SL_EINVAL;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(w) || !aligned16(y) || (residual && !aligned16(h)) || reinterpret_cast<uintptr_t>(rstd) & 3u)
    return SL_EALIGN;
  FwdArgs g{static_cast<const uint4*>(x), static_cast<const uint4*>(residual), static_cast<const uint4*>(w), static_cast<uint4*>(y),
            static_cast<uint4*>(h), nullptr, nullptr, rstd, nullptr, T, int(H / 8), 1.0 / double(H), eps};
  return run_fwd(static_cast<hipStream_t>(stream), g, kBF16);
}

extern "C" int sl_rmsnorm_fwd_mxfp8(void* stream, const void* x, const void* residual, const void* w, float eps, uint8_t* q_rows, uint8_t* s_rows,
                                    uint8_t* q_cols, uint8_t* s_cols, void* h, float* rstd, int64_t T, int64_t H) {
  const int e = check_norm(T, H, eps);
  if (e) return e;
  if (!q_rows != !s_rows || !q_cols != !s_cols) return SL_EINVAL;
  if ((q_rows && H % 32) || (q_cols && T % 32)) return SL_ESHAPE;
  if (T == 0 || H == 0) return SL_OK;
  if (!x || !w || !rstd || (residual && !h)) return SL_EINVAL;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(w) || (residual && !aligned16(h)) || !aligned16(q_rows) || !aligned16(q_cols) ||
      reinterpret_cast<uintptr_t>(rstd) & 3u)
    return SL_EALIGN;
  const int64_t tiles = (T + kTile - 1) / kTile * ((H + kTile - 1) / kTile);
  if (q_cols && tiles >= (int64_t(1) << 24)) return SL_ESHAPE;            // of 256 threads: a launch has fewer than 2^32
  const hipStream_t st = static_cast<hipStream_t>(stream);
  FwdArgs g{static_cast<const uint4*>(x), static_cast<const uint4*>(residual), static_cast<const uint4*>(w), nullptr, static_cast<uint4*>(h),
            reinterpret_cast<uint2*>(q_rows), s_rows, rstd, q_cols ? rstd + T : nullptr, T, int(H / 8), 1.0 / double(H), eps};
  const int f = run_fwd(st, g, q_rows ? kRows : kNothing);
  if (f || !q_cols) return f;
  hipLaunchKernelGGL(norm_cols, dim3(unsigned(tiles)), dim3(256), 0, st, static_cast<const uint16_t*>(residual ? h : x),
                     static_cast<const uint16_t*>(w), rstd, rstd + T, T, H, q_cols, s_cols);
  return hipGetLastError() == hipSuccess ? SL_OK : SL_EHIP;
}

extern "C" size_t sl_rmsnorm_bwd_workspace_bytes(int64_t T, int64_t H) {
  if (T <= 0 || H <= 0 || check_norm(T, H, 0.f)) return 0;
  return size_t(bwd_plan(T, int(H / 8)).planes) * size_t(H) * 4;
}

extern "C" int sl_rmsnorm_bwd(void* stream, const void* dY, const void* h, const void* w, const float* rstd, const void* dresidual, void* dX,
                              float* w_grad, int64_t T, int64_t H, void* workspace, size_t workspace_bytes) {
  const int e = check_norm(T, H, 0.f);
  if (e) return e;
  if (T == 0 || H == 0) return SL_OK;
  if (!dY || !h || !w || !rstd || !dX) return SL_EINVAL;
  if (!aligned16(dY) || !aligned16(h) || !aligned16(w) || !aligned16(dresidual) || !aligned16(dX) || reinterpret_cast<uintptr_t>(rstd) & 3u ||
      reinterpret_cast<uintptr_t>(w_grad) & 3u)
    return SL_EALIGN;
  if (w_grad && (!workspace || !aligned16(workspace) || workspace_bytes < sl_rmsnorm_bwd_workspace_bytes(T, H))) return SL_EWORKSPACE;
  const BwdPlan p = bwd_plan(T, int(H / 8));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  BwdArgs g{static_cast<const uint4*>(dY), static_cast<const uint4*>(h), static_cast<const uint4*>(w), static_cast<const uint4*>(dresidual), rstd,
            static_cast<uint4*>(dX), w_grad ? static_cast<float*>(workspace) : nullptr, T, int(H / 8), float(H)};
  const dim3 grid(unsigned(p.planes)), threads(p.tpr < 256 ? 256 : p.tpr);
  with_row(p.tpr, g.chunks, [&](auto t, auto n) {
    constexpr int TPR = decltype(t)::value, NC = decltype(n)::value;
    if (dresidual) hipLaunchKernelGGL((norm_bwd<TPR, NC, true>), grid, threads, 0, st, g);
    else hipLaunchKernelGGL((norm_bwd<TPR, NC, false>), grid, threads, 0, st, g);
  });
  if (hipGetLastError() != hipSuccess) return SL_EHIP;
  if (!w_grad) return SL_OK;
  hipLaunchKernelGGL(norm_wgrad, dim3(unsigned((H + 31) / 32)), dim3(1024), 0, st, g.part, w_grad, int(p.planes), H);
  return hipGetLastError() == hipSuccess ? SL_OK : SL_EHIP;
}
