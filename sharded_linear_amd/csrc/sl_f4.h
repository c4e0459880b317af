// Internal interface of the MXFP4 kernels (not part of the C ABI).
//
// An MXFP4 matrix [R][K] (K a multiple of 32) is packed E2M1 codes [R][K/2], element 2j of a row in
// the low nibble of byte j, and E8M0 scales [R][K/32]: element (r, k) stands for
// E2M1(code) * 2^(scale[r][k/32] - 127).  E2M1 = sign, 2 exponent bits (bias 1), 1 mantissa bit
// (0, 0.5, 1, 1.5, 2, 3, 4, 6).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

// Status of the launchers below: 0, or -5 where the HIP runtime reported an error at launch.

// Quantises x[R][C] (bf16, row-major, 16-byte aligned, C % 8 == 0): rowwise codes qr[R][Cp/2] and
// scales sr[R][Cp/32], and columnwise ones, stored transposed, qc[C][Rp/2] and sc[C][Rp/32], Cp and
// Rp the extents rounded up to 32 (the last block padded with zeros).  A null pair is skipped.
// Rounds to nearest, or stochastically with the key seed + (seed_offset ? *seed_offset : 0).
struct F4QuantArgs {
  const void* x;
  int64_t R, C;
  uint8_t *qr, *sr, *qc, *sc;
  bool stochastic;
  uint64_t seed;
  const uint64_t* seed_offset;
};
int f4_quantize(hipStream_t st, const F4QuantArgs& a);

// bf16 out[rows][cols] of codes q and scales s; cols % 32 == 0.
int f4_dequantize(hipStream_t st, const uint8_t* q, const uint8_t* s, void* out, int64_t rows, int64_t cols);

// C[M][N] = A . B^T of two MXFP4 operands A[M][K], B[N][K]: bf16 C, or fp32 C += (f4_accum), unsplit or
// with the partial sums of each split of K in its plane of ws[splits][M][N].  N % 8 == 0.
struct F4Args {
  const void *a, *b;    // codes
  const void *sa, *sb;  // scales
  void* c;
  int64_t M, N, K;
  float* ws;
  int splits;           // splits of K, of kt_per_split stages each (accumulating product only)
  int kt_per_split;
  int cfg;              // tile configuration: 0 256x256, 1 128x128, 2 128x128 staged four deep
};
constexpr int kF4StageK = 256;                  // k elements of one stage
int f4_gemm(hipStream_t st, const F4Args& g);
int f4_accum(hipStream_t st, const F4Args& g);

// Y[T][N] = X . W^T for few rows T: X bf16 (xs null) or MXFP4, W MXFP4, both blocked along K; up to 32 rows of bf16.
struct F4RowsArgs {
  const void *x, *xs, *w, *ws;
  void* y;
  int64_t T, N, K;
  // w4_tile_*: K in `splits` ranges of steps_per_split steps of kW4StepK, none empty; with more than one, their
  // f32 sums in part[splits][T][N]
  float* part;
  int splits, steps_per_split;
};
int f4_rows(hipStream_t st, const F4RowsArgs& g);
// The same with bf16 X for any T (w4_tile_fwd), and Y[T][N] = X[T][K] . W[K][N] with W blocked along N
// (w4_tile_dgrad), in tiles of kW4TileT rows by kW4TileN columns.
constexpr int kW4TileT = 64, kW4TileN = 128, kW4StepK = 128;
int w4_tile_fwd(hipStream_t st, const F4RowsArgs& g);
int w4_tile_dgrad(hipStream_t st, const F4RowsArgs& g);

// bf16 y[n] = the sum of the planes part[splits][n] in order, rounded once; n % 4 == 0 (sl_gemm_f4.hip).
int f4_join(hipStream_t st, void* y, const float* part, int64_t n, int splits);

// The SL_TUNE_F8_CONFIG knob: a forced tile configuration of the block-scaled products, or -1 (sl_gemm.hip).
int block_scaled_config();
// main_grad[M][N] += the planes of ws in split order (sl_gemm.hip).
int f4_reduce(hipStream_t st, float* c, const float* ws, int64_t M, int64_t N, int splits);
