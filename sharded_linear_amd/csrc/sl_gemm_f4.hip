// Products of two MXFP4 operands (gfx950): C = A . B^T with A[M][K], B[N][K] blocked along K.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes E2M1 codes with an E8M0 scale per 32 elements as they are
// stored.  Its operand layout for 4-bit data (checked on the hardware): lane l of a 32-row fragment
// holds row l % 32, elements [32 g, 32 g + 32) of the 64-wide k step for g = l / 32, which are one
// 16-byte chunk and exactly one scale block, whose scale byte the same lane supplies.
//
// One wave computes a 32 x 32 block straight from memory.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sl_device.h"
#include "sl_f4.h"

namespace sl2 {

constexpr int kF4Fmt = 4;                       // cbsz / blgp of E2M1 operands

// Fragment of row r at k block kb: zeros (and scale 1) past the last block.
__device__ __forceinline__ i32x8 f4_frag(const uint4* codes, int64_t r, int64_t kb, int64_t nb) {
  const uint4 v = kb < nb ? codes[r * nb + kb] : make_uint4(0, 0, 0, 0);
  return i32x8{int(v.x), int(v.y), int(v.z), int(v.w), 0, 0, 0, 0};
}

template <bool ACC>
__global__ void __launch_bounds__(256) gemm_f4_simple(F4Args g) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t tn = (g.N + 63) / 64;
  const int64_t m0 = int64_t(blockIdx.x) / tn * 64 + (wave >> 1) * 32, n0 = int64_t(blockIdx.x) % tn * 64 + (wave & 1) * 32;
  const int64_t nb = g.K / 32, r = lane & 31, h = lane >> 5;
  // rows past the edge repeat the last row; their results are not stored
  const int64_t ma = m0 + r < g.M ? m0 + r : g.M - 1, na = n0 + r < g.N ? n0 + r : g.N - 1;
  const uint4 *A = static_cast<const uint4*>(g.a), *B = static_cast<const uint4*>(g.b);
  const uint8_t *sa = static_cast<const uint8_t*>(g.sa), *sb = static_cast<const uint8_t*>(g.sb);
  f32x16 acc = {};
  for (int64_t kb = 0; kb < nb; kb += 2) {
    const int64_t b = kb + h;
    const int xa = b < nb ? sa[ma * nb + b] : 127, xb = b < nb ? sb[na * nb + b] : 127;
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f4_frag(B, na, b, nb), f4_frag(A, ma, b, nb), acc, kF4Fmt,
                                                          kF4Fmt, 0, xb, 0, xa);
  }
  // B first: lane l has row m0 + l % 32 and in registers 4q .. 4q + 3 columns n0 + 8 q + 4 (l / 32) + 0..3
  const int64_t m = m0 + r;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t n = n0 + 8 * q + 4 * h;
    if (m >= g.M || n >= g.N) continue;
    if constexpr (ACC) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(g.c) + m * g.N + n);
      float4 o = *p;
      o.x += acc[4 * q]; o.y += acc[4 * q + 1]; o.z += acc[4 * q + 2]; o.w += acc[4 * q + 3];
      *p = o;
    } else {
      bf16x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = static_cast<__bf16>(acc[4 * q + e]);
      *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(g.c) + m * g.N + n) = v;
    }
  }
}

template <bool ACC>
int launch_f4(hipStream_t st, const F4Args& g) {
  const int64_t tiles = (g.M + 63) / 64 * ((g.N + 63) / 64);
  hipLaunchKernelGGL(gemm_f4_simple<ACC>, dim3(unsigned(tiles)), dim3(256), 0, st, g);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace sl2

int f4_gemm(hipStream_t st, const F4Args& g) { return sl2::launch_f4<false>(st, g); }

int f4_accum(hipStream_t st, const F4Args& g) { return sl2::launch_f4<true>(st, g); }
