// MXFP4 casts (gfx950): bf16 matrices to packed E2M1 codes with E8M0 scales per 32 elements, and back.
//
// A block is 32 elements along the axis that the consuming product contracts: rowwise along C,
// columnwise down R (stored transposed, so that the product reads its k axis contiguously).  Its
// shared exponent X and codes are
//   nearest (OCP MX v1.0):  X = clamp(floor(log2 amax) - 2, -127, 127)   (2 = E2M1's largest exponent)
//                           code = E2M1 of x / 2^X, round half to even, saturating at 6
//   stochastic:             X = the least exponent >= -127 with amax <= 6 * 2^X, so nothing saturates;
//                           with v = |x| / 2^X and s its E2M1 step (0.5 below 2, 1 below 4, else 2)
//                           |code| = s * floor((floor(v / s * 2^16) + r) / 2^16), r 16 random bits:
//                           the expectation is v up to 2^-16 s.
// The scale byte is X + 127; a block of zeros has scale 0 and codes 0; a block with an infinity or a
// NaN has the NaN scale 255 and codes 0 (E2M1 itself has neither).
//
// r comes from Philox4x32 with 7 rounds (Salmon et al., "Parallel random numbers: as easy as 1, 2,
// 3", 2011): the group of 8 elements with linear index 8 g .. 8 g + 7 of x takes the 8 half words of
// the generator at counter g and the call's 64-bit key, low half first.  An element's draw depends
// on nothing but the key and its place, so both copies round with the same draws and none is stored.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sl_f4.h"
#include "sl_mx.h"

namespace sl2 {

// 16-bit draws of the 8 elements of group g, two to a word, element 2i in the low half of word i.
__device__ __forceinline__ uint4 philox7(uint64_t g, uint64_t key) {
  uint32_t c0 = uint32_t(g), c1 = uint32_t(g >> 32), c2 = 0, c3 = 0;
  uint32_t k0 = uint32_t(key), k1 = uint32_t(key >> 32);
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t p0 = uint64_t(0xD2511F53u) * c0, p1 = uint64_t(0xCD9E8D57u) * c2;
    c0 = uint32_t(p1 >> 32) ^ c1 ^ k0;
    c1 = uint32_t(p1);
    c2 = uint32_t(p0 >> 32) ^ c3 ^ k1;
    c3 = uint32_t(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// E2M1 code of x with |x| / 2^X = |x| * mult: nearest, half to even.
__device__ __forceinline__ uint32_t e2m1_nearest(float x, float mult) {
  const float v = __builtin_fabsf(x) * mult;
  const float n = v < 2.f ? __builtin_rintf(v * 2.f) : v < 4.f ? __builtin_rintf(v) + 2.f : __builtin_rintf(v * 0.5f) + 4.f;
  return uint32_t(n < 7.f ? n : 7.f) | ((__float_as_uint(x) >> 28) & 8u);
}

// The same, stochastic with the draw r.  From 1 on, the codes order like the fp32 bits with one
// mantissa bit left, so adding the draw below that bit and cutting there is the rule above (a bf16's
// mantissa has no bits below the draw's); below 1 the step is fixed.
__device__ __forceinline__ uint32_t e2m1_stochastic(float x, float mult, uint32_t r) {
  const float v = __builtin_fabsf(x) * mult;
  const uint32_t big = ((__float_as_uint(v) + (r << 6)) >> 22) - 252u;     // bits of 1.0 are 254 << 22
  const uint32_t small = (uint32_t(v * 131072.f) + r) >> 16;
  return (v >= 1.f ? big : small) | ((__float_as_uint(x) >> 28) & 8u);
}

// Shared exponent of a block whose largest magnitude has the bf16 bits amax (finite, not zero).  A
// subnormal amax counts as 2^-127, which the clamp makes right.
template <bool SR>
__device__ __forceinline__ int mx4_exponent(uint32_t amax) {
  int X = int(amax >> 7) - 127 - 2;
  if (SR && (amax & 0x7Fu) > 0x40u) ++X;                    // amax > 1.5 * 2^(X + 2) = 6 * 2^X
  return X < -127 ? -127 : X;                               // at most 126
}

// Encodes 8 elements, two to a word, of a block with largest magnitude amax: codes of elements
// 0..7 in nibbles 0..7.  r: their draws (stochastic only).
template <bool SR>
__device__ __forceinline__ uint32_t mx4_codes(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, int X, uint4 r) {
  const uint32_t w[4] = {w0, w1, w2, w3};
  const float mult = __uint_as_float(uint32_t(127 - X) << 23);          // 2^-X, X in -127 .. 126
  uint32_t q = 0;
  if constexpr (SR) {
    const uint32_t d[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q |= e2m1_stochastic(bf16_lo(w[i]), mult, d[i] & 0xFFFFu) << (8 * i);
      q |= e2m1_stochastic(bf16_hi(w[i]), mult, d[i] >> 16) << (8 * i + 4);
    }
  } else {
    if (X > -127) {
      // one instruction for two elements; checked on every bf16 pattern against the rule
      const float scale = __uint_as_float(uint32_t(X + 127) << 23);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[0]), scale, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[1]), scale, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[2]), scale, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[3]), scale, 3);
    } else {                                                // 2^-127 is no normal fp32 scale
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q |= e2m1_nearest(bf16_lo(w[i]), mult) << (8 * i);
        q |= e2m1_nearest(bf16_hi(w[i]), mult) << (8 * i + 4);
      }
    }
  }
  return q;
}

constexpr uint32_t kNonFinite = 0x7F80u;       // bf16 magnitudes from here on are infinities and NaNs

// One thread casts one 32-element block: consecutive threads take consecutive blocks of a row, or
// (columnwise) consecutive columns of one block row.
template <bool SR, bool COL>
__global__ void __launch_bounds__(256) mx4_quant_blocks(const uint16_t* x, int64_t R, int64_t C, uint8_t* q, uint8_t* s,
                                                         uint64_t seed, const uint64_t* seed_offset) {
  const uint64_t key = seed + (SR && seed_offset ? *seed_offset : 0);
  const int64_t nb = ((COL ? R : C) + 31) / 32, lines = COL ? C : R, total = nb * lines;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    const int64_t line = COL ? i % C : i / nb, b = COL ? i / C : i % nb;
    uint32_t w[16];
    uint16_t d[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const int64_t r = COL ? b * 32 + e : line, c = COL ? line : b * 32 + e;
      const uint32_t v = r < R && c < C ? x[r * C + c] : 0;
      w[e / 2] = e & 1 ? w[e / 2] | (v << 16) : v;
      if constexpr (SR) {
        const int64_t at = r * C + c;
        const uint4 p = philox7(uint64_t(at) / 8, key);
        const uint32_t word = (at & 4) ? ((at & 2) ? p.w : p.z) : ((at & 2) ? p.y : p.x);
        d[e] = uint16_t(at & 1 ? word >> 16 : word);
      }
    }
    const uint32_t amax = mag_max(w);
    uint32_t out[4] = {0, 0, 0, 0}, scale = 0;
    if (amax >= kNonFinite) {
      scale = 255;
    } else if (amax) {
      const int X = mx4_exponent<SR>(amax);
      scale = uint32_t(X + 127);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 r = make_uint4(0, 0, 0, 0);
        if constexpr (SR)
          r = make_uint4(d[8 * j] | (d[8 * j + 1] << 16), d[8 * j + 2] | (d[8 * j + 3] << 16),
                         d[8 * j + 4] | (d[8 * j + 5] << 16), d[8 * j + 6] | (d[8 * j + 7] << 16));
        out[j] = mx4_codes<SR>(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3], X, r);
      }
    }
    reinterpret_cast<uint4*>(q)[line * nb + b] = make_uint4(out[0], out[1], out[2], out[3]);
    s[line * nb + b] = uint8_t(scale);
  }
}

// bf16 values of codes: rows hold whole blocks, so chunk i is 8 elements, one code dword and scale
// byte i / 4, with no row arithmetic.  The product is exact (an E2M1 value has two significant bits;
// the smallest, 2^-128, is a bf16 subnormal), up to scales of 2^126 and more, whose 4 and 6 or 3
// pass bf16's range and become infinite.
__global__ void __launch_bounds__(256) mx4_dequant_bf16(const uint32_t* q, const uint8_t* s, uint4* out, int64_t n8) {
  constexpr int U = 4;
  const int64_t stride = int64_t(gridDim.x) * blockDim.x;
  for (int64_t base = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; base < n8; base += U * stride) {
    uint32_t c[U];
    float sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = base + u * stride;
      if (i < n8) {
        c[u] = q[i];
        sc[u] = e8m0_to_f32(s[i >> 2]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = base + u * stride;
      if (i < n8) {
        uint32_t o[4];
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], sc[u], 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], sc[u], 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], sc[u], 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u], sc[u], 3));
        out[i] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

template <bool SR, bool COL>
int launch_quant(hipStream_t st, const F4QuantArgs& a, uint8_t* q, uint8_t* s) {
  const int64_t total = ((COL ? a.R : a.C) + 31) / 32 * (COL ? a.C : a.R);
  int64_t blocks = (total + 255) / 256;
  if (blocks > 65536) blocks = 65536;
  hipLaunchKernelGGL((mx4_quant_blocks<SR, COL>), dim3(unsigned(blocks)), dim3(256), 0, st,
                     static_cast<const uint16_t*>(a.x), a.R, a.C, q, s, a.seed, a.seed_offset);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace sl2

int f4_quantize(hipStream_t st, const F4QuantArgs& a) {
  if (a.R == 0 || a.C == 0) return 0;
  if (a.qr) {
    const int r = a.stochastic ? sl2::launch_quant<true, false>(st, a, a.qr, a.sr) : sl2::launch_quant<false, false>(st, a, a.qr, a.sr);
    if (r) return r;
  }
  if (a.qc) return a.stochastic ? sl2::launch_quant<true, true>(st, a, a.qc, a.sc) : sl2::launch_quant<false, true>(st, a, a.qc, a.sc);
  return 0;
}

int f4_dequantize(hipStream_t st, const uint8_t* q, const uint8_t* s, void* out, int64_t rows, int64_t cols) {
  const int64_t n8 = rows * (cols / 8);
  if (n8 == 0) return 0;
  int64_t blocks = (n8 + 1023) / 1024;          // 256 threads x 4 chunks each
  if (blocks > 16384) blocks = 16384;
  hipLaunchKernelGGL(sl2::mx4_dequant_bf16, dim3(unsigned(blocks)), dim3(256), 0, st, reinterpret_cast<const uint32_t*>(q),
                     s, static_cast<uint4*>(out), n8);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}
