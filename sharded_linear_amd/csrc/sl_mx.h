// Device helpers of the microscaled formats (MXFP8, MXFP4), internal.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace sl2 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef short i16x4q __attribute__((ext_vector_type(4)));

// Largest magnitude field of N words of two bf16 elements: |bf16| orders like its 15-bit magnitude.
// Both halves are compared at once (packed 16-bit max).
template <int N>
__device__ __forceinline__ uint32_t mag_max(const uint32_t (&w)[N]) {
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < N; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu));
  return m[0] > m[1] ? m[0] : m[1];
}

// Largest value of m over the four lanes of a quad (DPP quad permutes [1,0,3,2] and [2,3,0,1]).
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0xB1, 0xF, 0xF, false));
  m = o > m ? o : m;
  o = uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x4E, 0xF, 0xF, false));
  return o > m ? o : m;
}

// An E8M0 scale byte as fp32: 2^(s - 127), s = 0 as the subnormal 2^-127, s = 255 as NaN; the two set the
// top mantissa bit.
__device__ __forceinline__ float e8m0_to_f32(uint32_t s) {
  return __builtin_bit_cast(float, (s << 23) | (((s + 1) & 0xFEu) == 0 ? 0x00400000u : 0u));
}

// 8 E2M1 codes (nibbles 0..7 of a word) times a scale, exact.
typedef __bf16 bf16x8_mx __attribute__((ext_vector_type(8)));
__device__ __forceinline__ bf16x8_mx f4_to_bf16x8(uint32_t codes, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8_mx{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

}  // namespace sl2
