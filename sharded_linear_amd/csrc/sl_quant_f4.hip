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

#include "sl_device.h"
#include "sl_f4.h"
#include "sl_mx.h"

namespace sl2 {

__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) { return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96); }

// 16-bit draws of the 8 elements of group g, two to a word, element 2i in the low half of word i.
__device__ __forceinline__ uint4 philox7(uint64_t g, uint64_t key) {
  uint32_t c0 = uint32_t(g), c1 = uint32_t(g >> 32), c2 = 0, c3 = 0;
  uint32_t k0 = uint32_t(key), k1 = uint32_t(key >> 32);
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t p0 = uint64_t(0xD2511F53u) * c0, p1 = uint64_t(0xCD9E8D57u) * c2;
    c0 = xor3(uint32_t(p1 >> 32), c1, k0);
    c1 = uint32_t(p1);
    c2 = xor3(uint32_t(p0 >> 32), c3, k1);
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

// The sign bits of 8 elements, two to a word, at bit 3 of nibbles 0..7.
__device__ __forceinline__ uint32_t signs8(const uint32_t (&w)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x07030501u);      // high bytes: elements 0, 2, 1, 3
  const uint32_t b = __builtin_amdgcn_perm(w[3], w[2], 0x07030501u);
  const uint32_t even = __builtin_amdgcn_perm(b, a, 0x05040100u) & 0x80808080u;
  const uint32_t odd = __builtin_amdgcn_perm(b, a, 0x07060302u) & 0x80808080u;
  return (even >> 4) | odd;
}

// The magnitude's code of x with |x| / 2^X = v, stochastic.  E2M1's magnitudes in order are the
// fp32 numbers 0, 2^-127, 2^-126 and 1.5, 2, 3, 4, 6 times 2^-126, which have one mantissa bit and, below
// 2^-126, the fixed step of a subnormal as E2M1 has below 1: the bits from 22 up are the code.  So the draw is added
// below that bit of 2^-126 v, which is cut off at 2^-149 (the kernel rounds toward zero), far below the draw's last bit.
// draws: two of them, HI the upper one's, taken as it is by a 16-bit multiply-add.  e: -126 - X.
template <bool HI>
__device__ __forceinline__ uint32_t e2m1_stochastic(float x, int e, uint32_t draws) {
  const uint32_t v = __float_as_uint(__builtin_ldexpf(__builtin_fabsf(x), e));
  uint32_t s;
  if constexpr (HI) asm("v_mad_u32_u16 %0, %1, 64, %2 op_sel:[1,0,0,0]" : "=v"(s) : "v"(draws), "v"(v));
  else asm("v_mad_u32_u16 %0, %1, 64, %2" : "=v"(s) : "v"(draws), "v"(v));
  return s >> 22;
}
// Sets the wave's fp32 rounding toward zero (MODE bits 0..1) and returns -126, on which every float operation
// that needs it has to depend: the compiler moves float operations past a change of the mode, but not past
// their operands.  before1, before2: wave-uniform values whose computation needs the mode that was.
__device__ __forceinline__ int round_toward_zero(uint32_t before1, uint32_t before2) {
  int e;
  asm volatile("s_setreg_imm32_b32 hwreg(HW_REG_MODE, 0, 2), 3\n\ts_movk_i32 %0, 0xff82" : "=s"(e) : "s"(before1), "s"(before2));
  return e;
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
// 0..7 in nibbles 0..7.  r: their draws, unit: -126 from round_toward_zero (stochastic only).
template <bool SR>
__device__ __forceinline__ uint32_t mx4_codes(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, int X, uint4 r, int unit) {
  const uint32_t w[4] = {w0, w1, w2, w3};
  uint32_t q = 0;
  if constexpr (SR) {
    const uint32_t d[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {                             // each code enters at the top
      q = __builtin_amdgcn_alignbit(e2m1_stochastic<false>(bf16_lo(w[i]), unit - X, d[i]), q, 4);
      q = __builtin_amdgcn_alignbit(e2m1_stochastic<true>(bf16_hi(w[i]), unit - X, d[i]), q, 4);
    }
    q |= signs8(w);
  } else {
    if (X > -127) {
      // one instruction for two elements; checked on every bf16 pattern against the rule
      const float scale = __uint_as_float(uint32_t(X + 127) << 23);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[0]), scale, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[1]), scale, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[2]), scale, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[3]), scale, 3);
    } else {                                                // 2^-127 is no normal fp32 scale
      const float mult = __uint_as_float(0x7F000000u);        // 2^127
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

// Scale byte of a block, and its exponent (unused where the block has no codes: zeros, or not finite).
template <bool SR>
__device__ __forceinline__ uint32_t mx4_scale(uint32_t amax, int& X) {
  X = mx4_exponent<SR>(amax);
  if (!SR && amax == 0) X = 0;                              // padding need not take the way of the smallest blocks
  return amax >= kNonFinite ? 255u : amax ? uint32_t(X + 127) : 0u;
}

// One workgroup casts 64 H x 128 elements.  Each thread loads four 16-byte chunks of every 64 rows, 16
// adjacent lanes to a tile row, so that a quad of lanes holds a row block: it shares the block's amax
// through two DPP permutes and each lane stores its chunk's 8 codes.  For the columnwise copy the elements,
// and with stochastic rounding their draws, are staged in LDS, 64 rows at a time, and read back transposed
// (ds_read_b64_tr_b16), a 32-row block of one column to a thread; the codes go back through LDS and leave
// 32 H bytes a column.  Nearest is bound by HBM ([8192, 4096] both copies 20.0 us, 5130 GB/s; [8192, 11008]
// 62 us, 4410 GB/s), stochastic by its vector instructions ([8192, 11008] 70 us): 1531 for 64 elements a lane in both
// copies, 112 of them the generator's 64-bit multiplications, which count four times: 7.7 thousand issue cycles a
// wave, 21.5 waves a SIMD, 69 us at 2.4 GHz.  The generator is 29 % of that, the encoding about 40 %, the rest
// maxima, places and packing.
//
// H = 1 up to this many tiles of 128 rows, 4 to a CU, so that more CUs work at a time: [1536, 2048] both
// copies 5.2 us against 5.9, [8192, 2048] (1024 tiles) 12.5 against 13.0;
// [8192, 4096] 21.0 against 20.0, and [8192, 11008], whose columns then leave in half lines, 83 against 62.
constexpr int64_t kSmallTiles = 1024;
constexpr int kQC = 128, kQH = 64;       // tile columns, rows of half a tile
constexpr int kQS = kQC + 16;            // LDS row stride in elements: 4 rows x 4 column quads of a transposing read in distinct banks

template <bool SR, bool ROWS, bool COLS, int H>
__global__ void __launch_bounds__(256) mx4_quant_tile(F4QuantArgs a) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[COLS ? kQH * kQS : 8];
  __shared__ __attribute__((aligned(16))) uint16_t dtile[COLS && SR ? kQH * kQS : 8];
  // kDown tiles down, then across, on one XCD: their pieces of the columnwise copy are whole 128-byte lines
  // (across alone: [8192, 11008] stochastic 74 us against 70)
  constexpr uint32_t kDown = COLS ? 4 / H : 1;
  const uint32_t ntc = uint32_t((a.C + kQC - 1) / kQC), ntr = uint32_t((a.R + H * kQH - 1) / (H * kQH));
  const uint32_t b = uint32_t(xcd_remap(int(blockIdx.x), int(gridDim.x))), g = b / (kDown * ntc), p = b % (kDown * ntc);
  const uint32_t down = min(kDown, ntr - g * kDown);
  const uint32_t tr = g * kDown + p % down, tc = p / down;
  const int64_t r0 = int64_t(tr) * (H * kQH), c0 = int64_t(tc) * kQC;
  const int t = threadIdx.x, ch = t & 15;
  const uint64_t key = a.seed + (SR && a.seed_offset ? *a.seed_offset : 0);
  const int64_t nbr = (a.C + 31) / 32, nbc = (a.R + 31) / 32;   // blocks of a row, of a column
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  // chunk k of this thread: row r0 + t / 16 + 16 k, columns gc .. gc + 7
  const int64_t gr0 = r0 + (t >> 4), gc = c0 + 8 * ch, at0 = gr0 * (a.C / 8) + gc / 8, qat0 = gr0 * nbr + gc / 32;
  const int left = int(a.R - gr0 < H * kQH ? a.R - gr0 : H * kQH);      // rows from the first on
  uint4 raw[4 * H];
#pragma unroll
  for (int k = 0; k < 4 * H; ++k)                                   // C % 8 == 0: a chunk is inside or outside
    raw[k] = 16 * k < left && gc < a.C ? reinterpret_cast<const uint4*>(x)[at0 + k * (2 * a.C)] : make_uint4(0, 0, 0, 0);
  int unit = 0;
  if constexpr (SR) unit = round_toward_zero(tr, tc);           // the tile's place by a division, which uses fp32 itself
  uint32_t q[H][4], s[H];                                       // columnwise codes and scales, a block from each half
#pragma unroll
  for (int h = 0; h < H; ++h) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = (t >> 4) + 16 * k;
      const int n = 4 * h + k;
      const uint4 v = raw[4 * h + k];
      uint4 d = make_uint4(0, 0, 0, 0);
      if constexpr (SR) d = philox7(uint64_t(at0 + n * (2 * a.C)), key);
      if constexpr (COLS) {
        reinterpret_cast<uint4*>(tile + row * kQS)[ch] = v;
        if constexpr (SR) reinterpret_cast<uint4*>(dtile + row * kQS)[ch] = d;
      }
      if constexpr (ROWS) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const uint32_t amax = quad_max(mag_max(w));              // every lane takes part
        int X;
        const uint32_t sc = mx4_scale<SR>(amax, X);
        uint32_t c = mx4_codes<SR>(w[0], w[1], w[2], w[3], X, d, unit);
        if (amax == 0 || amax >= kNonFinite) c = 0;
        if (16 * n < left && gc < nbr * 32) {
          const int64_t at = qat0 + n * (16 * nbr);
          reinterpret_cast<uint32_t*>(a.qr)[at * 4 + (ch & 3)] = c;
          if ((ch & 3) == 0) a.sr[at] = uint8_t(sc);
        }
      }
    }
    if constexpr (COLS) {
      __syncthreads();
      // Thread t: column t % 128, rows 32 (t / 128) .. of this half.  Lane 4 j + i of a 16-lane group
      // addresses 4 adjacent columns (quad i of the group's 16) of row j and receives 4 rows of its own column.
      const int s16 = t & 15, jr = s16 >> 2, qc4 = s16 & 3;
      const int at = ((t >> 7) * 32 + jr) * kQS + ((t & (kQC - 1)) & ~15) + 4 * qc4;
      uint32_t v[16], d[16];
#pragma unroll
      for (int r4 = 0; r4 < 8; ++r4) {
        const uint2 p = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) i16x4q*)(uintptr_t)lds_addr(tile + at + r4 * 4 * kQS)));
        v[2 * r4] = p.x;
        v[2 * r4 + 1] = p.y;
        if constexpr (SR) {
          const uint2 e = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) i16x4q*)(uintptr_t)lds_addr(dtile + at + r4 * 4 * kQS)));
          d[2 * r4] = e.x;
          d[2 * r4 + 1] = e.y;
        }
      }
      const uint32_t amax = mag_max(v);
      int X;
      s[h] = mx4_scale<SR>(amax, X);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint4 r = make_uint4(0, 0, 0, 0);
        if constexpr (SR) r = make_uint4(d[4 * e], d[4 * e + 1], d[4 * e + 2], d[4 * e + 3]);
        q[h][e] = mx4_codes<SR>(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3], X, r, unit);
        if (amax == 0 || amax >= kNonFinite) q[h][e] = 0;
      }
      __syncthreads();
    }
  }
  if constexpr (COLS) {
    // 16-byte chunk rb of a column's 64-byte line sits in slot rb ^ (col / 2): 8 adjacent columns in distinct banks
    uint8_t* const qbuf = reinterpret_cast<uint8_t*>(tile);
    uint8_t* const sbuf = qbuf + kQC * 64;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int col = t & (kQC - 1), rb = 2 * h + (t >> 7);
      *reinterpret_cast<uint4*>(qbuf + col * 64 + ((rb ^ (col >> 1)) & 3) * 16) = make_uint4(q[h][0], q[h][1], q[h][2], q[h][3]);
      sbuf[col * 4 + rb] = uint8_t(s[h]);
    }
    __syncthreads();
    const int nrb = int(nbc - r0 / 32 < 2 * H ? nbc - r0 / 32 : 2 * H);   // row blocks of this tile
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int idx = t + 256 * h, col = idx >> 2, c = idx & 3;
      const int64_t gc = c0 + col;
      if (gc < a.C && c < nrb)
        *reinterpret_cast<uint4*>(a.qc + (gc * nbc + r0 / 32 + c) * 16) =
            *reinterpret_cast<const uint4*>(qbuf + col * 64 + ((c ^ (col >> 1)) & 3) * 16);
    }
    if (t < kQC && c0 + t < a.C) {
      uint8_t* const dst = a.sc + (c0 + t) * nbc + r0 / 32;
      if (nrb == 4 && (reinterpret_cast<uintptr_t>(dst) & 3) == 0) *reinterpret_cast<uint32_t*>(dst) = reinterpret_cast<const uint32_t*>(sbuf)[t];
      else for (int e = 0; e < nrb; ++e) dst[e] = sbuf[t * 4 + e];
    }
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

template <bool SR, bool ROWS, bool COLS, int H>
int launch_tiles(hipStream_t st, const F4QuantArgs& a) {
  const int64_t tiles = (a.C + kQC - 1) / kQC * ((a.R + H * kQH - 1) / (H * kQH));
  hipLaunchKernelGGL((mx4_quant_tile<SR, ROWS, COLS, H>), dim3(unsigned(tiles)), dim3(256), 0, st, a);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

template <bool SR, bool ROWS, bool COLS>
int launch_quant(hipStream_t st, const F4QuantArgs& a) {
  const int64_t tiles = (a.C + kQC - 1) / kQC * ((a.R + 2 * kQH - 1) / (2 * kQH));
  return tiles <= kSmallTiles ? launch_tiles<SR, ROWS, COLS, 1>(st, a) : launch_tiles<SR, ROWS, COLS, 2>(st, a);
}

template <bool SR>
int dispatch_quant(hipStream_t st, const F4QuantArgs& a) {
  if (a.qr && a.qc) return launch_quant<SR, true, true>(st, a);
  if (a.qr) return launch_quant<SR, true, false>(st, a);
  return launch_quant<SR, false, true>(st, a);
}

}  // namespace sl2

int f4_quantize(hipStream_t st, const F4QuantArgs& a) {
  if (a.R == 0 || a.C == 0 || (!a.qr && !a.qc)) return 0;
  return a.stochastic ? sl2::dispatch_quant<true>(st, a) : sl2::dispatch_quant<false>(st, a);
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
