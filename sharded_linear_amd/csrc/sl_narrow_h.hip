// Newton-Schulz steps of matrices with up to 256 rows (gfx950): a step in two launches.
//
// For few rows the products are small and a step's time is that of its launches, one behind the other.  The polynomial
// is applied from the right side of the parenthesis,
//   y = a x + b u + A (c u),   u = A x,
// so that a workgroup computes 32 columns of y from the same columns of x and the whole of A, with nothing to wait for in
// between; the columns of y are then in LDS, and their share of the next Gram matrix, y y^T, is one more product there,
// kept in accumulators over all columns that the workgroup takes.  The second launch adds the workgroups' shares in order.
// A's rows stay in registers for both products with it: of 256 rows wave w holds the blocks of 16 rows w and 15 - w, which
// together have 17 blocks on and below the diagonal whatever w, and only those of the Gram matrix are computed and kept
// (all 32 of a wave took 128 registers and twice the stores: a step of [256, 512] 13.2 us against 10.8).  Of 128 rows wave w
// holds block w and of the Gram matrix 5 blocks (all 8: 16 of [128, 2048] 126 us against 119).
//
// Rounded to fp16 are y, A and w = c u (at a quarter of the others' scale: its elements may be larger); u stays in fp32.
// With l what the rounding of x left, y has a l, and w takes (b + c) l in before its rounding: near singular values of 1, where
// the sum of the three coefficients is small, a l alone would add a multiple of l that the polynomial has not.  w is the
// largest of the errors: of up to 128 rows it is held in two fp16 numbers, 22 bits, for a second pass of the second product.
// Against 64 bits, with the 1.7e-3 of the result's rounding to bf16: [33, 18] 2.0e-3, [64, 1997] 2.1e-3; with y = a x +
// A (b x + c u), the parenthesis rounded as one, 2.5e-3 and 2.3e-3, and single matrices of 256 rows 3 to 6 % faster.
//
// Five steps and what surrounds them: [64, 64] 47 us, [128, 1024] 57, [512, 256] 80, [256, 8192] 155, 16 of [128, 2048] 119.  A
// launch for a step takes 4.5 (128 rows) to 11 us (256), its join 2.5 to 4: a chain of two products, three barriers and the loads
// of A and x behind each other in a workgroup, most of it latency, so that the matrix units are busy for less than a tenth.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sl_device.h"
#include "sl_narrow_h.h"

namespace sl2 {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kCols = 32, kRow = kCols + 8;    // a slice's columns, and its row in LDS: 80 bytes against bank conflicts

template <int M>
struct Narrow {
  static constexpr int TI = M / 128, KS = M / 32, TJ = M / 16;
  // Blocks of 16 rows of wave w; and the blocks of the Gram matrix that it keeps.  256 rows: of its rows, those on and below the
  // diagonal.  128: of its row the diagonal and the next four, counted round the edge; the last of these is also that of wave
  // w + 4, transposed.
  __device__ __host__ static constexpr int row(int w, int i) { return i == 0 ? w : TJ - 1 - w; }
  static constexpr int kBlocks = TI == 1 ? 5 : TJ + 1;
  __device__ __host__ static constexpr int half(int w, int t) { return TI == 1 || t <= w ? 0 : 1; }
  __device__ __host__ static constexpr int col(int w, int t) { return TI == 1 ? (w + t) % TJ : t <= w ? t : t - w - 1; }
  __device__ __host__ static constexpr bool mirrored(int w, int t) { return TI == 1 ? t % 4 != 0 : col(w, t) != row(w, half(w, t)); }
  static constexpr int kHalves = TI == 1 ? 2 : 1;              // fp16 numbers that hold w
  static constexpr int kChunks = M * kCols / 8 / 512;          // 16-byte chunks of a slice for each thread
};

__device__ __forceinline__ f32x4v mfma_h(f16x8 b, f16x8 a, f32x4v c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(b, a, c, 0, 0, 0); }

// B operand of 32 rows from k0 and 16 columns from c0 of an LDS slice: result lane 4q + e of a 16-lane group gets 4 rows
// of column 4q + e through each transposing read.
__device__ __forceinline__ f16x8 columns(const _Float16* s, int k0, int c0, int lane) {
  const int g = lane >> 4, j = (lane & 15) >> 2, q = lane & 3;
  const _Float16* p = s + (k0 + 8 * g + j) * kRow + c0 + 4 * q;
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)p);
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(p + 4 * kRow));
  const short __attribute__((ext_vector_type(8))) v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(f16x8, v);
}

template <int M, bool STEP, bool GRAM>
__global__ void __launch_bounds__(512) narrow_kernel(NarrowArgs g) {
  using P = Narrow<M>;
  constexpr int TI = P::TI, KS = P::KS;
  __shared__ __attribute__((aligned(16))) _Float16 xs[M * kRow];
  __shared__ __attribute__((aligned(16))) _Float16 ws[STEP ? P::kHalves : 1][STEP ? M * kRow : 8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int batch = blockIdx.x / g.groups, group = blockIdx.x % g.groups;
  const int rl = lane & 15, gl = lane >> 4;
  int rows[TI];                                // this lane's row in each of its wave's blocks
#pragma unroll
  for (int i = 0; i < TI; ++i) rows[i] = 16 * P::row(wave, i) + rl;
  const _Float16* x = static_cast<const _Float16*>(g.x) + int64_t(batch) * M * g.N;
  const int slices = g.N / kCols, per = (slices + g.groups - 1) / g.groups;
  const int s0 = group * per, s1 = min(s0 + per, slices);

  // this thread's chunks of the next slice, row p / 4, chunk p % 4, and l of its part of the results (loads return in order:
  // behind the stores of a slice they would wait for those)
  u32x4 next[P::kChunks];
  int next_l[STEP ? TI : 1][2];
  const uint8_t* const lo = STEP && g.lo ? static_cast<const uint8_t*>(g.lo) + int64_t(batch) * M * g.N : nullptr;
  auto fetch = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < P::kChunks; ++k) {
      const int p = k * 512 + threadIdx.x;
      next[k] = *reinterpret_cast<const u32x4*>(x + int64_t(p >> 2) * g.N + s * kCols + 8 * (p & 3));
    }
    if constexpr (STEP)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          next_l[i][j] = lo ? *reinterpret_cast<const int*>(lo + int64_t(rows[i]) * g.N + s * kCols + 16 * j + 4 * gl) : 0;
  };
  if (s0 < s1) fetch(s0);
  f16x8 a[STEP ? TI : 1][STEP ? KS : 1];
  if constexpr (STEP) {
    const _Float16* A = static_cast<const _Float16*>(g.A) + int64_t(batch) * M * M;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int k = 0; k < KS; ++k) a[i][k] = *reinterpret_cast<const f16x8*>(A + rows[i] * M + 32 * k + 8 * gl);
  }
  f32x4v gram[GRAM ? P::kBlocks : 1];
  if constexpr (GRAM)
#pragma unroll
    for (int t = 0; t < P::kBlocks; ++t) gram[t] = f32x4v{0.f, 0.f, 0.f, 0.f};

  for (int s = s0; s < s1; ++s) {
#pragma unroll
    for (int k = 0; k < P::kChunks; ++k) {
      const int p = k * 512 + threadIdx.x;
      *reinterpret_cast<u32x4*>(xs + (p >> 2) * kRow + 8 * (p & 3)) = next[k];
    }
    int left[STEP ? TI : 1][2];
    if constexpr (STEP)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) left[i][j] = next_l[i][j];
    __syncthreads();
    if (s + 1 < s1) fetch(s + 1);
    if constexpr (STEP) {
      const int64_t at0 = int64_t(batch) * M * g.N + s * kCols + 4 * gl;
      // u = A x; a lane holds row 16 i + l % 16 and columns 16 j + 4 (l / 16) + 0..3 of its wave's rows
      f32x4v acc[TI][2], sum[TI][2];
      auto product = [&](f32x4v (&to)[TI][2], const _Float16* from) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const f16x8 b = columns(from, 32 * k, 16 * j, lane);
#pragma unroll
            for (int i = 0; i < TI; ++i) to[i][j] = mfma_h(b, a[i][k], to[i][j]);
          }
      };
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = sum[i][j] = f32x4v{0.f, 0.f, 0.f, 0.f};
      product(acc, xs);
      auto kept = [&](int i, int j) {          // l
        const auto a = __builtin_amdgcn_cvt_pk_f32_bf8(left[i][j], false), b = __builtin_amdgcn_cvt_pk_f32_bf8(left[i][j], true);
        return f32x4v{a[0], a[1], b[0], b[1]};
      };
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int at = rows[i] * kRow + 16 * j + 4 * gl;
          const f32x4v w = acc[i][j] * (0.25f * g.c * g.unit) + kept(i, j) * ((g.b + g.c) * 0x1p-13f);
          const f16x4 hi = __builtin_convertvector(w, f16x4);
          *reinterpret_cast<f16x4*>(ws[0] + at) = hi;
          if constexpr (P::kHalves == 2) *reinterpret_cast<f16x4*>(ws[1] + at) = __builtin_convertvector(w - __builtin_convertvector(hi, f32x4v), f16x4);
        }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < P::kHalves; ++h) product(sum, ws[h]);
      // y, in place of x in LDS (of which every wave has read the others' rows before the last barrier)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int at = rows[i] * kRow + 16 * j + 4 * gl;
          const f32x4v own = __builtin_convertvector(*reinterpret_cast<const f16x4*>(xs + at), f32x4v);
          const f32x4v v = (own + kept(i, j) * 0x1p-11f) * g.a + acc[i][j] * (g.b * g.unit) + sum[i][j] * (4.f * g.unit);
          const f16x4 hi = __builtin_convertvector(v, f16x4);
          *reinterpret_cast<f16x4*>(xs + at) = hi;
          if (g.ylo) {
            const f32x4v r = (v - __builtin_convertvector(hi, f32x4v)) * 0x1p11f;
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(g.ylo) + at0 + int64_t(rows[i]) * g.N + 16 * j) =
                uint32_t(__builtin_amdgcn_cvt_pk_bf8_f32(r[2], r[3], __builtin_amdgcn_cvt_pk_bf8_f32(r[0], r[1], 0, false), true));
          }
        }
      __syncthreads();
      _Float16* y = static_cast<_Float16*>(g.y) + int64_t(batch) * M * g.N;
#pragma unroll
      for (int k = 0; k < P::kChunks; ++k) {
        const int p = k * 512 + threadIdx.x;
        *reinterpret_cast<u32x4*>(y + int64_t(p >> 2) * g.N + s * kCols + 8 * (p & 3)) = *reinterpret_cast<const u32x4*>(xs + (p >> 2) * kRow + 8 * (p & 3));
      }
    }
    if constexpr (GRAM) {
      f16x8 r[TI];
#pragma unroll
      for (int i = 0; i < TI; ++i) r[i] = *reinterpret_cast<const f16x8*>(xs + rows[i] * kRow + 8 * gl);
#pragma unroll
      for (int t = 0; t < P::kBlocks; ++t) {
        const f16x8 b = *reinterpret_cast<const f16x8*>(xs + (16 * P::col(wave, t) + rl) * kRow + 8 * gl);
        gram[t] = mfma_h(b, P::half(wave, t) == 0 ? r[0] : r[TI - 1], gram[t]);
      }
    }
    __syncthreads();
  }
  if constexpr (GRAM) {
    // in the accumulators' order: [wave][block][lane], whole lines a store
    f32x4v* to = reinterpret_cast<f32x4v*>(g.planes) + (int64_t(blockIdx.x) * 8 + wave) * (P::kBlocks * 64) + lane;
#pragma unroll
    for (int t = 0; t < P::kBlocks; ++t) to[t * 64] = gram[t];
  }
}

// A wave adds a block's 4 elements a lane over a part of the planes, 4 blocks of a matrix in 4 parts to a workgroup.
template <int M>
__global__ void __launch_bounds__(1024) narrow_join_kernel(const f32x4v* __restrict__ planes, _Float16* __restrict__ A, int groups, float unit) {
  using P = Narrow<M>;
  __shared__ f32x4v sums[3][256];
  constexpr int kAll = 8 * P::kBlocks;
  static_assert(kAll % 4 == 0, "whole workgroups");
  const int batch = blockIdx.x / (kAll / 4), lane = threadIdx.x & 63, place = threadIdx.x & 255;
  const int block = __builtin_amdgcn_readfirstlane(blockIdx.x % (kAll / 4) * 4 + place / 64), part = threadIdx.x >> 8;
  const int per = (groups + 3) / 4, g0 = part * per, g1 = min(g0 + per, groups);
  f32x4v sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int g = g0; g < g1; ++g) sum += planes[(int64_t(batch) * groups + g) * (kAll * 64) + block * 64 + lane];
  if (part) sums[part - 1][place] = sum;
  __syncthreads();
  if (part) return;
  sum = ((sum + sums[0][place]) + sums[1][place]) + sums[2][place];
  const int wave = block / P::kBlocks, t = block % P::kBlocks;
  const int row = 16 * P::row(wave, P::half(wave, t)) + (lane & 15), col = 16 * P::col(wave, t) + 4 * (lane >> 4);
  const f16x4 v = __builtin_convertvector(sum * unit, f16x4);
  _Float16* const a = A + int64_t(batch) * M * M;
  *reinterpret_cast<f16x4*>(a + row * M + col) = v;
  if (P::mirrored(wave, t))
#pragma unroll
    for (int e = 0; e < 4; ++e) a[(col + e) * M + row] = v[e];
}

template <bool STEP, bool GRAM>
int launch_narrow(hipStream_t st, const NarrowArgs& g) {
  const dim3 grid(unsigned(g.batches * g.groups)), block(512);
  if (g.M == 128) hipLaunchKernelGGL((narrow_kernel<128, STEP, GRAM>), grid, block, 0, st, g);
  else hipLaunchKernelGGL((narrow_kernel<256, STEP, GRAM>), grid, block, 0, st, g);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace sl2

size_t narrow_plane_bytes(int M) { return size_t(8 * (M == 128 ? sl2::Narrow<128>::kBlocks : sl2::Narrow<256>::kBlocks)) * 1024; }

int narrow_groups(int M, int N, int64_t batches) {
  const int64_t slices = N / sl2::kCols;
  int64_t most = 512 / batches;                // two workgroups a CU
  if (most > (M == 128 ? 128 : 64)) most = M == 128 ? 128 : 64;
  if (most < 1) most = 1;
  if (most > slices) most = slices;
  const int64_t per = (slices + most - 1) / most;
  return int((slices + per - 1) / per);
}

int narrow_gram(hipStream_t st, const NarrowArgs& g) { return sl2::launch_narrow<false, true>(st, g); }

int narrow_step(hipStream_t st, const NarrowArgs& g) { return g.planes ? sl2::launch_narrow<true, true>(st, g) : sl2::launch_narrow<true, false>(st, g); }

int narrow_join(hipStream_t st, const float* planes, void* A, int M, int groups, int64_t batches, float unit) {
  const dim3 grid(unsigned(batches * (M == 128 ? sl2::Narrow<128>::kBlocks : sl2::Narrow<256>::kBlocks) * 2)), block(1024);
  const sl2::f32x4v* p = reinterpret_cast<const sl2::f32x4v*>(planes);
  if (M == 128) hipLaunchKernelGGL(sl2::narrow_join_kernel<128>, grid, block, 0, st, p, static_cast<_Float16*>(A), groups, unit);
  else hipLaunchKernelGGL(sl2::narrow_join_kernel<256>, grid, block, 0, st, p, static_cast<_Float16*>(A), groups, unit);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}
