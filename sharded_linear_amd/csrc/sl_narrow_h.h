// Internal interface of the Newton-Schulz steps of matrices with few rows (not part of the C ABI).
#pragma once
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

constexpr int kNarrowRows = 256;               // the most rows (128 or 256 after padding)

struct NarrowArgs {
  const void* A;               // [batches][M][M] fp16: the Gram matrices of x, times 1 / unit
  const void* x;               // [batches][M][N] fp16, times 1 / unit
  void* y;                     // the step's result, like x
  const void* lo;              // what the rounding of x left, times 2^11 / unit, in E5M2, or null
  void* ylo;                   // the same of y, or null; may be lo
  float* planes;               // [batches][groups] partial Gram matrices of the result, or null
  int M, N, groups;
  int64_t batches;
  float a, b, c, unit;
};

// Workgroups (and so planes) of one matrix, and the bytes of one plane.
size_t narrow_plane_bytes(int M);
int narrow_groups(int M, int N, int64_t batches);
// planes = the Gram matrices of x in parts.
int narrow_gram(hipStream_t st, const NarrowArgs& g);
// A = the sum of the planes.
int narrow_join(hipStream_t st, const float* planes, void* A, int M, int groups, int64_t batches, float unit);
// y = a x + A (b x + c A x), and the planes of y.  |c A x| may reach 60.
int narrow_step(hipStream_t st, const NarrowArgs& g);
