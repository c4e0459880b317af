// Internal interface of the fp16 products of the orthogonalised update (not part of the C ABI).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

// C[M][N] = alpha * A . B + beta * (D + Dlo / 2^11) for each of `batches` matrices, sums in fp32, results rounded to
// fp16 once; with clo, what the rounding left, times 2^11, goes there (fp16).  A is [M][K]; B is [N][K] (half_gemm_nt) or
// [K][N] (half_gemm_nn).  M, N and K are multiples of 128; matrices are dense and follow each other without gaps.
struct HalfArgs {
  const void *a, *b;           // the first matrix of each
  const void *d, *dlo;         // like C; may be null, dlo alone too
  void *c, *clo;               // c is no operand and not d; clo null, or another matrix or dlo itself
  int M, N, K;
  int64_t batches;
  float alpha, beta;
  // set by the launchers, and by the kernels to the matrix of the workgroup
  int64_t lda, ldb;
  uint32_t a_bytes, b_bytes;
  int tiles_m, tiles_n;
};
constexpr int kHalfPad = 128;

// A and B K-major.  Where the result is known to be symmetric (`sym`, M == N), tiles on and below the diagonal are
// computed and those below written a second time, transposed.
int half_gemm_nt(hipStream_t st, HalfArgs g, bool sym);
int half_gemm_nn(hipStream_t st, HalfArgs g);
