// Newton-Schulz steps of matrices with up to 256 rows (gfx950): a step in two launches.
//
// For few rows the products are small and a step's time is that of its launches, one behind the other.  The polynomial
// is applied from the right side of the parenthesis,
//   y = a x + A (b x + c (A x)),
// so that a workgroup computes 32 columns of y from the same columns of x and the whole of A, with nothing to wait for in
// between; the columns of y are then in LDS, and their share of the next Gram matrix, y y^T, is one more product there,
// kept in accumulators over all columns that the workgroup takes.  The second launch adds the workgroups' shares in order.
// A's rows stay in registers for both products with it: of 256 rows wave w holds the blocks of 16 rows w and 15 - w, which
// together have 17 blocks on and below the diagonal whatever w, and only those of the Gram matrix are computed and kept
// (all 32 of a wave took 128 registers and twice the stores: a step of [256, 512] 13.2 us against 10.8).  Of 128 rows wave w
// holds block w, and all of the Gram matrix is computed.
//
// Each of b x + c A x, y and A is rounded to fp16 once, the first at a quarter of the others' scale (its elements may be larger).
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
  static constexpr int kBlocks = TI == 1 ? TJ : TJ + 1;        // blocks of the Gram matrix that a wave keeps
  // Block t of wave w: row block and column block.
  __device__ __host__ static constexpr int row(int w, int i) { return i == 0 ? w : TJ - 1 - w; }
  __device__ __host__ static constexpr int half(int w, int t) { return TI == 1 || t <= w ? 0 : 1; }
  __device__ __host__ static constexpr int col(int w, int t) { return TI == 1 || t <= w ? t : t - w - 1; }
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
  constexpr int TI = P::TI, KS = P::KS, TJ = P::TJ;
  __shared__ __attribute__((aligned(16))) _Float16 xs[M * kRow];
  __shared__ __attribute__((aligned(16))) _Float16 zs[STEP ? M * kRow : 8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int batch = blockIdx.x / g.groups, group = blockIdx.x % g.groups;
  const int rl = lane & 15, gl = lane >> 4;
  int rows[TI];                                // this lane's row in each of its wave's blocks
#pragma unroll
  for (int i = 0; i < TI; ++i) rows[i] = 16 * P::row(wave, i) + rl;
  const _Float16* x = static_cast<const _Float16*>(g.x) + int64_t(batch) * M * g.N;
  const int slices = g.N / kCols, per = (slices + g.groups - 1) / g.groups;
  const int s0 = group * per, s1 = min(s0 + per, slices);

  // this thread's chunks of a slice: row p / 4, chunk p % 4
  u32x4 next[P::kChunks];
  auto fetch = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < P::kChunks; ++k) {
      const int p = k * 512 + threadIdx.x;
      next[k] = *reinterpret_cast<const u32x4*>(x + int64_t(p >> 2) * g.N + s * kCols + 8 * (p & 3));
    }
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
    __syncthreads();
    if (s + 1 < s1) fetch(s + 1);
    if constexpr (STEP) {
      const int64_t at0 = int64_t(batch) * M * g.N + s * kCols + 4 * gl;
      // z = b x + c A x; a lane holds row 16 i + l % 16 and columns 16 j + 4 (l / 16) + 0..3 of its wave's rows
      f32x4v acc[TI][2];
#pragma unroll
      for (int i = 0; i < TI; ++i) acc[i][0] = acc[i][1] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const f16x8 b0 = columns(xs, 32 * k, 0, lane), b1 = columns(xs, 32 * k, 16, lane);
#pragma unroll
        for (int i = 0; i < TI; ++i) {
          acc[i][0] = mfma_h(b0, a[i][k], acc[i][0]);
          acc[i][1] = mfma_h(b1, a[i][k], acc[i][1]);
        }
      }
      auto own = [&](int at) { return __builtin_convertvector(*reinterpret_cast<const f16x4*>(xs + at), f32x4v); };
      const uint8_t* const lo = g.lo ? static_cast<const uint8_t*>(g.lo) + at0 : nullptr;
      uint32_t left[TI][2];
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int at = rows[i] * kRow + 16 * j + 4 * gl;
          const f32x4v z = (own(at) * g.b + acc[i][j] * (g.c / g.scale)) * 0.25f;
          *reinterpret_cast<f16x4*>(zs + at) = __builtin_convertvector(z, f16x4);
          acc[i][j] = f32x4v{0.f, 0.f, 0.f, 0.f};
          left[i][j] = lo ? *reinterpret_cast<const uint32_t*>(lo + int64_t(rows[i]) * g.N + 16 * j) : 0u;
        }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const f16x8 b0 = columns(zs, 32 * k, 0, lane), b1 = columns(zs, 32 * k, 16, lane);
#pragma unroll
        for (int i = 0; i < TI; ++i) {
          acc[i][0] = mfma_h(b0, a[i][k], acc[i][0]);
          acc[i][1] = mfma_h(b1, a[i][k], acc[i][1]);
        }
      }
      // y, in place of x in LDS (of which every wave has read the others' rows before the last barrier)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int at = rows[i] * kRow + 16 * j + 4 * gl;
          const auto l0 = __builtin_amdgcn_cvt_pk_f32_bf8(int(left[i][j]), false), l1 = __builtin_amdgcn_cvt_pk_f32_bf8(int(left[i][j]), true);
          const f32x4v v = (own(at) + f32x4v{l0[0], l0[1], l1[0], l1[1]} * 0x1p-11f) * g.a + acc[i][j] * (4.f / g.scale);
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
__global__ void __launch_bounds__(1024) narrow_join_kernel(const f32x4v* __restrict__ planes, _Float16* __restrict__ A, int groups, float scale) {
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
  const f16x4 v = __builtin_convertvector(sum * (1.f / scale), f16x4);
  _Float16* const a = A + int64_t(batch) * M * M;
  *reinterpret_cast<f16x4*>(a + row * M + col) = v;
  if (P::TI > 1 && row / 16 != col / 16)
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

int narrow_join(hipStream_t st, const float* planes, void* A, int M, int groups, int64_t batches, float scale) {
  const dim3 grid(unsigned(batches * (M == 128 ? sl2::Narrow<128>::kBlocks : sl2::Narrow<256>::kBlocks) * 2)), block(1024);
  const sl2::f32x4v* p = reinterpret_cast<const sl2::f32x4v*>(planes);
  if (M == 128) hipLaunchKernelGGL(sl2::narrow_join_kernel<128>, grid, block, 0, st, p, static_cast<_Float16*>(A), groups, scale);
  else hipLaunchKernelGGL(sl2::narrow_join_kernel<256>, grid, block, 0, st, p, static_cast<_Float16*>(A), groups, scale);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}
