// Internal interface of the fp16 products of the orthogonalised update (not part of the C ABI).
#pragma once
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

// C[M][N] = alpha * A . B + beta * D (+ diag * I) for each of `batches` matrices, summed in fp32 and rounded to fp16 once.
//   half_gemm_sym: A [M][K] by the transpose of B [N][K], known to be symmetric; D is fp16, like C, or null (then there is no
//                  diagonal either)
//   half_gemm_nn:  A [M][K] by B [K][N]; D is bytes [M][N] in E5M2, or null; with D and clo, what the rounding of C left,
//                  times 2^11, goes there in E5M2 (clo may be D)
// M, N and K are multiples of 128; matrices are dense and follow each other without gaps.
struct HalfArgs {
  const void *a, *b;           // the first matrix of each
  const void* d;
  void *c, *clo;               // C is no operand and not D
  int M, N, K;
  int64_t batches;
  float alpha, beta, diag;
  float* ws;                   // half_gemm_workspace_bytes() for split sums
  // set by the launchers
  int tiles_m, tiles_n, full, rest, splits, kt_per_split, quarters, first;
};
constexpr int kHalfPad = 128;

// The symmetric product (M == N) computes the tiles on and below the diagonal and writes those below it a second time,
// transposed.
int half_gemm_sym(hipStream_t st, HalfArgs g);
int half_gemm_nn(hipStream_t st, HalfArgs g);
// Workspace of either with these extents (nn: M, N, K; sym: M == N).
size_t half_gemm_workspace_bytes(int M, int N, int K, int64_t batches, bool sym);
// What either takes its result apart into: tiles of 256x256, tiles of 128x128 for the rest or for all of it, how many of
// these have their sums split, and in how many parts.
struct HalfTiles { int64_t big, small, split, parts; };
HalfTiles half_gemm_tiles(int M, int N, int K, int64_t batches, bool sym);
