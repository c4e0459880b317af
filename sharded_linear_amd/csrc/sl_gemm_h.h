// Internal interface of the fp16 products of the orthogonalised update (not part of the C ABI).
#pragma once
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

// C[M][N] = alpha * A . B + beta * D + diag * I for each of `batches` matrices, summed in fp32 and rounded to fp16 once;
// with clo, what that rounding left, times 2^11, goes there (fp16).  A is [M][K] and B [N][K] (half_gemm_sym) or [K][N]
// (half_gemm_nn).  M, N and K are multiples of 128; matrices are dense and follow each other without gaps.
struct HalfArgs {
  const void *a, *b;           // the first matrix of each
  const void* d;               // like C, or null
  void *c, *clo;               // C is no operand and not D; clo null, or like C, D itself if need be
  int M, N, K;
  int64_t batches;
  float alpha, beta, diag;
  float* ws;                   // half_gemm_workspace_bytes() for split sums
  // set by the launchers
  int tiles_m, tiles_n, full, rest, splits, kt_per_split;
};
constexpr int kHalfPad = 128;

// A . B^T of a product known to be symmetric (M == N): tiles on and below the diagonal are computed and those below it
// written a second time, transposed.
int half_gemm_sym(hipStream_t st, HalfArgs g);
int half_gemm_nn(hipStream_t st, HalfArgs g);
// Workspace of either with these extents (nn: M, N, K; sym: M == N).
size_t half_gemm_workspace_bytes(int M, int N, int K, int64_t batches, bool sym);
