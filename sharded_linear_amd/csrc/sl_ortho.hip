// The orthogonalised update (gfx950): Newton-Schulz iterations on a gradient, and the optimiser step around them.
//
//   X = U / |U|_F, as [m, n] with m <= n;   each step:  A = X X^T,  P = a I + b A + c A^2,  X <- P X
//   step of a weight:  M <- mu M + G,  U = G + mu M (Nesterov) or M,  W <- (1 - lr wd) W - lr s X
//
// The polynomial a + b z^3 + c z^5 moves every singular value towards 1; all of the work is products of [m, m] and
// [m, n] matrices.  They run in fp16: singular values stay below 3 (checked on the host for the coefficients given), so
// every element of X, A and P lies within fp16's range at one fixed scale, 2^12, where fp16 keeps 11 bits and
// bf16 would keep 8.  Against 64 bits, on [512, 2048] of normal values, the result is 2.2e-3 off in fp16, 1.7e-3 of it its own
// rounding to bf16, and 1.2e-2 in bf16 (relative, in the 2-norm).  A rounding of X in a direction whose singular value is
// small is multiplied by up to a each step, so the first kLoSteps steps add a times what the rounding of X left (kept in
// E5M2 beside it: the whole is then held to 2^-14) to P X: with singular values falling over four decades the error is 2.4e-3
// with it and 9e-3 without.  (P has a on its diagonal rather than the epilogue adding a X: P's rounding scales X and so leaves
// small singular values their place, P is nearer to 1 than P - a I in the last steps, and X is not read a second time.)
//
// Around the products: one pass for the momentum and the norm (sums of squares in 64 bits: any finite gradient has a
// norm), one that scales, transposes a tall matrix and pads to multiples of 128 with zeros, and one that writes the
// result or the weight.  The three are bound by HBM: for 2 x [4096, 5504] 91 us (541 MB, 6.0 TB/s), 101 (496 MB, 4.9) and 46
// (271 MB, 5.9) of 3250.  G and M are read twice, for the norm has to be known before the first element of X, and U in fp32
// would be as many bytes.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "sharded_linear.h"
#include "sl_device.h"
#include "sl_gemm_h.h"
#include "sl_narrow_h.h"

namespace {

constexpr int kMats = 32;                  // matrices of one launch: their pointers travel in the kernel's arguments
constexpr int kNormBlocks = 512;           // partial sums of squares of a matrix
constexpr int kLoSteps = 3;
constexpr float kScale = 4096.f;

struct Mats {
  const void* g[kMats];                    // gradients, fp32 or bf16
  float* m[kMats];                         // momenta
  void* w[kMats];                          // results or weights, bf16
  float* master[kMats];                    // fp32 weights
};

struct PassArgs {
  int64_t rows, cols;
  int mp, np;                              // padded extents of X
  float mu;
  bool nesterov, has_m, g_bf16, tall, vec; // vec: rows begin at multiples of 4 elements
  double* part;                            // [matrices][kNormBlocks]
  int blocks;
  _Float16* x;
  uint32_t* lo;                            // four E5M2 bytes a word
  float keep, step;                        // W <- keep W - step X
  bool update, has_master;
};

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// Four elements from `at` of an fp32 or bf16 array; n of them are there.
__device__ __forceinline__ f32x4 load4(const void* p, bool is_bf16, int64_t at, int n, bool vec) {
  if (is_bf16) {
    const __bf16* b = static_cast<const __bf16*>(p) + at;
    if (vec && n == 4) return __builtin_convertvector(*reinterpret_cast<const bf16x4*>(b), f32x4);
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) v[e] = float(b[e]);
    return v;
  }
  const float* f = static_cast<const float*>(p) + at;
  if (vec && n == 4) return *reinterpret_cast<const f32x4*>(f);
  f32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) v[e] = f[e];
  return v;
}

template <typename T4, typename T>
__device__ __forceinline__ void store4(T* p, f32x4 v, int n, bool vec) {
  if (vec && n == 4) {
    *reinterpret_cast<T4*>(p) = __builtin_convertvector(v, T4);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) p[e] = static_cast<T>(v[e]);
  }
}

__device__ __forceinline__ double block_sum(double x, double* red) {
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = red[0];
  for (int w = 1; w < int(blockDim.x >> 6); ++w) s += red[w];
  return s;
}

// Momentum, and the sum of squares of U over this workgroup's part of matrix blockIdx.y.
__global__ void __launch_bounds__(512) ortho_norm(Mats mats, PassArgs a) {
  __shared__ double red[8];
  const int l = blockIdx.y;
  const int64_t n = a.rows * a.cols, groups = (n + 3) / 4;
  float* const m = a.has_m ? mats.m[l] : nullptr;
  double sum = 0;
  for (int64_t i = int64_t(blockIdx.x) * 512 + threadIdx.x; i < groups; i += int64_t(gridDim.x) * 512) {
    const int64_t at = 4 * i;
    const int k = n - at < 4 ? int(n - at) : 4;
    f32x4 u = load4(mats.g[l], a.g_bf16, at, k, a.vec);
    if (m) {
      const f32x4 g = u;
      u = load4(m, false, at, k, a.vec) * a.mu + g;
      store4<f32x4>(m + at, u, k, a.vec);
      if (a.nesterov) u = g + u * a.mu;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum += double(u[e]) * double(u[e]);
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) a.part[l * kNormBlocks + blockIdx.x] = sum;
}

constexpr int kEdge = 64;                  // tiles of the passes below

// X = U / |U| * 2^12 in fp16, and what the rounding left times 2^11 in E5M2, padded with zeros; one tile of U to a workgroup.
__global__ void __launch_bounds__(256) ortho_scale(Mats mats, PassArgs a) {
  __shared__ double red[4];
  __shared__ float tile[kEdge][kEdge + 1];
  const int l = blockIdx.y;
  double sum = 0;
  for (int i = threadIdx.x; i < a.blocks; i += 256) sum += a.part[l * kNormBlocks + i];
  sum = block_sum(sum, red);
  const double inv = sum > 0 ? double(kScale) / sqrt(sum) : sum == 0 ? 0.0 : sum;      // NaN stays NaN
  const int across = (a.tall ? a.mp : a.np) / kEdge;
  const int64_t r0 = int64_t(blockIdx.x / across) * kEdge, c0 = int64_t(blockIdx.x % across) * kEdge;
  const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4;
  const float* const m = a.has_m ? mats.m[l] : nullptr;
  f32x4 x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = r0 + tr + 16 * k, c = c0 + 4 * tc;
    const int n = r < a.rows && c < a.cols ? (a.cols - c < 4 ? int(a.cols - c) : 4) : 0;
    x[k] = f32x4{0, 0, 0, 0};
    if (n > 0) {
      f32x4 u = load4(mats.g[l], a.g_bf16, r * a.cols + c, n, a.vec);
      if (m) {
        const f32x4 v = load4(m, false, r * a.cols + c, n, a.vec);
        u = a.nesterov ? u + v * a.mu : v;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x[k][e] = float(double(u[e]) * inv);
    }
  }
  if (a.tall) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) tile[4 * tc + e][tr + 16 * k] = x[k][e];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[k][e] = tile[tr + 16 * k][4 * tc + e];
  }
  const int64_t xr = a.tall ? c0 : r0, xc = a.tall ? r0 : c0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t at = (int64_t(l) * a.mp + xr + tr + 16 * k) * a.np + xc + 4 * tc;
    const f16x4 hi = __builtin_convertvector(x[k], f16x4);
    *reinterpret_cast<f16x4*>(a.x + at) = hi;
    const f32x4 left = (x[k] - __builtin_convertvector(hi, f32x4)) * 0x1p11f;
    a.lo[at / 4] = uint32_t(__builtin_amdgcn_cvt_pk_bf8_f32(left[2], left[3], __builtin_amdgcn_cvt_pk_bf8_f32(left[0], left[1], 0, false), true));
  }
}

// The result, or the weights' update, from X; one tile of the result to a workgroup.
__global__ void __launch_bounds__(256) ortho_write(Mats mats, PassArgs a) {
  __shared__ float tile[kEdge][kEdge + 1];
  const int l = blockIdx.y;
  const int across = int((a.cols + kEdge - 1) / kEdge);
  const int64_t r0 = int64_t(blockIdx.x / across) * kEdge, c0 = int64_t(blockIdx.x % across) * kEdge;
  const int64_t xr = a.tall ? c0 : r0, xc = a.tall ? r0 : c0;
  const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4;
  f32x4 x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    x[k] = __builtin_convertvector(*reinterpret_cast<const f16x4*>(a.x + (int64_t(l) * a.mp + xr + tr + 16 * k) * a.np + xc + 4 * tc), f32x4) * (1.f / kScale);
  if (a.tall) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) tile[4 * tc + e][tr + 16 * k] = x[k][e];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[k][e] = tile[tr + 16 * k][4 * tc + e];
  }
  __bf16* const w = static_cast<__bf16*>(mats.w[l]);
  float* const master = a.has_master ? mats.master[l] : nullptr;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = r0 + tr + 16 * k, c = c0 + 4 * tc, at = r * a.cols + c;
    const int n = r < a.rows && c < a.cols ? (a.cols - c < 4 ? int(a.cols - c) : 4) : 0;
    if (n == 0) continue;
    f32x4 v = x[k];
    if (a.update) {
      v = load4(master ? static_cast<const void*>(master) : w, !master, at, n, a.vec) * a.keep - v * a.step;
      if (master) store4<f32x4>(master + at, v, n, a.vec);
    }
    store4<bf16x4>(w + at, v, n, a.vec);
  }
}

// ---- host ----------------------------------------------------------------------------------------

constexpr int64_t kMaxExtent = int64_t(1) << 31;
constexpr int64_t kMaxBytes = 0x7FFFFFF0LL - 16;         // of one fp16 matrix: the products' 32-bit offsets
constexpr int kMaxSteps = 64;

bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & uintptr_t(bytes - 1)) == 0; }

// What a slice of a 16-byte aligned batch has: four elements are loaded at once where rows begin at multiples of four (bf16 slices
// then begin at multiples of 8 bytes), others element by element.
bool aligned_matrix(const void* p, int64_t rows, int64_t cols, int bytes) {
  return aligned(p, cols % 4 ? bytes : rows % 2 * (cols % 8) * bytes % 16 ? 8 : 16);
}

struct OrthoPlan {
  int64_t mp, np;
  bool tall, narrow;
  int64_t x_bytes, a_bytes, part_bytes, bytes;           // one [L, mp, np] and one [L, mp, mp] fp16 array; the norms' sums
};

// Whether the steps go to the kernels of sl_narrow_h.hip (left), or to the tiles (right): [128, 1024] 57 and 119 us, 16 of
// [128, 8192] 231 and 278; [256, 512] 80 and 127, [256, 8192] 155 and 210, 16 of [256, 512] 134 and 131, 16 of [256, 8192]
// 597 and 473.
bool few_rows(int64_t mp, int64_t np, int64_t L) { return mp <= kNarrowRows / 2 || (mp <= kNarrowRows && L * np <= 8192); }

int ortho_plan(int64_t L, int64_t rows, int64_t cols, OrthoPlan& p) {
  if (L < 0 || rows < 0 || cols < 0) return SL_EINVAL;
  if (L >= kMaxExtent || rows >= kMaxExtent || cols >= kMaxExtent) return SL_ESHAPE;
  p.tall = rows > cols;
  auto pad = [](int64_t x) { return (x + kHalfPad - 1) / kHalfPad * kHalfPad; };
  p.mp = pad(p.tall ? cols : rows);
  p.np = pad(p.tall ? rows : cols);
  if (p.mp > kMaxBytes / 2 / (p.np ? p.np : 1)) return SL_ESHAPE;
  // of a launch's tiles: fewer than 2^24 of 256 threads
  if (L * (p.np / 64) * (p.mp / 64) >= (int64_t(1) << 24) || L > 65535) return SL_ESHAPE;
  p.x_bytes = L * p.mp * p.np * 2;
  p.a_bytes = L * p.mp * p.mp * 2;
  p.part_bytes = L * kNormBlocks * 8;
  p.bytes = 2 * p.x_bytes + p.x_bytes / 2 + 2 * p.a_bytes + p.part_bytes;
  if (L == 0 || p.mp == 0 || p.np == 0) return SL_OK;
  p.narrow = few_rows(p.mp, p.np, L);
  size_t planes = 0;                                     // of the products' split sums, or of the Gram matrices' shares
  if (p.narrow) planes = size_t(L) * size_t(narrow_groups(int(p.mp), int(p.np), L)) * narrow_plane_bytes(int(p.mp));
  else for (size_t b : {half_gemm_workspace_bytes(int(p.mp), int(p.mp), int(p.np), L, true), half_gemm_workspace_bytes(int(p.mp), int(p.mp), int(p.mp), L, true),
                   half_gemm_workspace_bytes(int(p.mp), int(p.np), int(p.mp), L, false)})
    planes = b > planes ? b : planes;
  p.bytes += int64_t(planes);
  return SL_OK;
}

// The largest |a s + b s^3 + c s^5| over 0 <= s <= top, and the largest |a + b z + c z^2| over 0 <= z <= top^2.
void step_bounds(const float* k, double top, double& x, double& inner) {
  const double a = k[0], b = k[1], c = k[2];
  auto p = [&](double s) { return std::fabs(s * (a + s * s * (b + c * s * s))); };
  auto q = [&](double z) { return std::fabs(a + z * (b + c * z)); };
  x = p(top);
  inner = std::fmax(q(0), q(top * top));
  if (c != 0) {
    const double z = -b / (2 * c), d = 9 * b * b - 20 * a * c;
    if (z > 0 && z < top * top) inner = std::fmax(inner, q(z));
    if (d >= 0)
      for (double sign : {-1.0, 1.0}) {
        const double u = (-3 * b + sign * std::sqrt(d)) / (10 * c);
        if (u > 0 && u < top * top) x = std::fmax(x, p(std::sqrt(u)));
      }
  } else if (b != 0 && -a / (3 * b) > 0 && -a / (3 * b) < top * top) {
    x = std::fmax(x, p(std::sqrt(-a / (3 * b))));
  }
}

// Whether X, A and a I + b A + c A^2 stay in range at kScale: |X| <= 3 (12288), |A| <= 9 (36864), the third <= 15 (61440);
// and c A X at a quarter of it: <= 60.
int check_steps(int32_t steps, const float* coeffs) {
  if (steps < 0 || steps > kMaxSteps || (steps && !coeffs)) return SL_EINVAL;
  double top = 1;
  for (int i = 0; i < steps; ++i) {
    double x, inner;
    step_bounds(coeffs + 3 * i, top, x, inner);
    if (!(x <= 3) || !(inner <= 15) || !(std::fabs(coeffs[3 * i + 2]) * top * top * top <= 60)) return SL_EINVAL;
    top = x * 1.01;                                      // roundings
  }
  return SL_OK;
}

// Sums of squares, X, and the products; afterwards X is in `*result`.
int iterate(hipStream_t st, const Mats& mats, PassArgs a, const OrthoPlan& p, int64_t L, int32_t steps, const float* coeffs, char* ws,
            int64_t first, _Float16** result) {
  char* at = ws;
  _Float16* x[2];
  x[0] = reinterpret_cast<_Float16*>(at); at += p.x_bytes;
  x[1] = reinterpret_cast<_Float16*>(at); at += p.x_bytes;
  uint32_t* lo = reinterpret_cast<uint32_t*>(at); at += p.x_bytes / 2;
  _Float16* A = reinterpret_cast<_Float16*>(at); at += p.a_bytes;
  _Float16* P = reinterpret_cast<_Float16*>(at); at += p.a_bytes;
  a.part = reinterpret_cast<double*>(at) + first * kNormBlocks; at += p.part_bytes;
  a.x = x[0] + first * p.mp * p.np;
  a.lo = lo + first * p.mp * p.np / 4;
  const int64_t groups = (a.rows * a.cols + 3) / 4;
  a.blocks = int((groups + 2047) / 2048 < kNormBlocks ? (groups + 2047) / 2048 : kNormBlocks);
  const int64_t left = L - first < kMats ? L - first : kMats;
  hipLaunchKernelGGL(ortho_norm, dim3(a.blocks, unsigned(left)), dim3(512), 0, st, mats, a);
  if (hipGetLastError() != hipSuccess) return SL_EHIP;
  hipLaunchKernelGGL(ortho_scale, dim3(unsigned(p.mp / kEdge * (p.np / kEdge)), unsigned(left)), dim3(256), 0, st, mats, a);
  if (hipGetLastError() != hipSuccess) return SL_EHIP;
  *result = x[steps & 1];
  if (first + left < L) return SL_OK;                    // the products take all matrices at once
  if (p.narrow) {
    NarrowArgs g{};
    g.A = A; g.lo = lo;
    g.M = int(p.mp); g.N = int(p.np); g.batches = L;
    g.groups = narrow_groups(g.M, g.N, L);
    g.unit = 1.f / kScale;
    float* const planes = reinterpret_cast<float*>(at);
    for (int k = 0; k < steps; ++k) {
      const int kept = steps < kLoSteps ? steps : kLoSteps;
      g.x = x[k & 1]; g.y = x[~k & 1];
      g.planes = planes;
      if (k == 0 && narrow_gram(st, g)) return SL_EHIP;
      if (narrow_join(st, planes, A, g.M, g.groups, L, 1.f / kScale)) return SL_EHIP;
      g.planes = k + 1 < steps ? planes : nullptr;
      g.lo = k < kept ? lo : nullptr;
      g.ylo = k + 1 < kept ? lo : nullptr;
      g.a = coeffs[3 * k]; g.b = coeffs[3 * k + 1]; g.c = coeffs[3 * k + 2];
      if (narrow_step(st, g)) return SL_EHIP;
    }
    return SL_OK;
  }
  for (int k = 0; k < steps; ++k) {
    const float ca = coeffs[3 * k], cb = coeffs[3 * k + 1], cc = coeffs[3 * k + 2];
    const int kept = steps < kLoSteps ? steps : kLoSteps;
    HalfArgs g{};
    g.batches = L;
    g.ws = reinterpret_cast<float*>(at);
    g.a = g.b = x[k & 1]; g.c = A;
    g.M = g.N = int(p.mp); g.K = int(p.np);
    g.alpha = 1.f / kScale;
    if (half_gemm_sym(st, g)) return SL_EHIP;
    g.a = g.b = g.d = A; g.c = P;
    g.K = int(p.mp);
    g.alpha = cc / kScale; g.beta = cb; g.diag = ca * kScale;
    if (half_gemm_sym(st, g)) return SL_EHIP;
    g.a = P; g.b = x[k & 1]; g.c = x[~k & 1];
    g.N = int(p.np);
    g.d = k < kept ? lo : nullptr;
    g.clo = k + 1 < kept ? lo : nullptr;
    g.alpha = 1.f / kScale; g.beta = ca * 0x1p-11f; g.diag = 0.f;
    if (half_gemm_nn(st, g)) return SL_EHIP;
  }
  return SL_OK;
}

int write_out(hipStream_t st, const Mats& mats, const PassArgs& a, int64_t count) {
  const int64_t tiles = (a.rows + kEdge - 1) / kEdge * ((a.cols + kEdge - 1) / kEdge);
  hipLaunchKernelGGL(ortho_write, dim3(unsigned(tiles), unsigned(count)), dim3(256), 0, st, mats, a);
  return hipGetLastError() == hipSuccess ? SL_OK : SL_EHIP;
}

}  // namespace

extern "C" size_t sl_orthogonalize_workspace_bytes(int64_t L, int64_t rows, int64_t cols) {
  OrthoPlan p{};
  if (ortho_plan(L, rows, cols, p) || L == 0 || rows == 0 || cols == 0) return 0;
  return size_t(p.bytes);
}

extern "C" int sl_orthogonalize_tiles(int64_t L, int64_t rows, int64_t cols, int64_t* tiles) {
  OrthoPlan p{};
  if (!tiles) return SL_EINVAL;
  const int e = ortho_plan(L, rows, cols, p);
  if (e) return e;
  for (int i = 0; i < 12; ++i) tiles[i] = 0;
  if (L == 0 || rows == 0 || cols == 0 || p.narrow) return SL_OK;
  const int m = int(p.mp), n = int(p.np);
  const HalfTiles t[3] = {half_gemm_tiles(m, m, n, L, true), half_gemm_tiles(m, m, m, L, true), half_gemm_tiles(m, n, m, L, false)};
  for (int i = 0; i < 3; ++i) {
    const int64_t v[4] = {t[i].big, t[i].small, t[i].split, t[i].parts};
    for (int k = 0; k < 4; ++k) tiles[4 * i + k] = v[k];
  }
  return SL_OK;
}

extern "C" int sl_orthogonalize(void* stream, const void* G, int32_t g_bytes, void* O, int64_t L, int64_t rows, int64_t cols, int32_t steps,
                                const float* coeffs, void* workspace, size_t workspace_bytes) {
  OrthoPlan p{};
  int e = ortho_plan(L, rows, cols, p);
  if (e) return e;
  if (g_bytes != 2 && g_bytes != 4) return SL_EINVAL;
  if ((e = check_steps(steps, coeffs))) return e;
  if (L == 0 || rows == 0 || cols == 0) return SL_OK;
  if (!G || !O) return SL_EINVAL;
  if (!aligned_matrix(G, rows, cols, g_bytes) || !aligned_matrix(O, rows, cols, 2)) return SL_EALIGN;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < size_t(p.bytes)) return SL_EWORKSPACE;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  PassArgs a{};
  a.rows = rows; a.cols = cols; a.mp = int(p.mp); a.np = int(p.np);
  a.g_bf16 = g_bytes == 2; a.tall = p.tall; a.vec = cols % 4 == 0;
  Mats mats{};
  auto fill = [&](int64_t first) {
    const int64_t n = L - first < kMats ? L - first : kMats;
    for (int64_t i = 0; i < n; ++i) {
      mats.g[i] = static_cast<const char*>(G) + (first + i) * rows * cols * g_bytes;
      mats.w[i] = static_cast<char*>(O) + (first + i) * rows * cols * 2;
    }
    return n;
  };
  _Float16* x = nullptr;
  for (int64_t first = 0; first < L; first += kMats) {
    fill(first);
    if ((e = iterate(st, mats, a, p, L, steps, coeffs, static_cast<char*>(workspace), first, &x))) return e;
  }
  for (int64_t first = 0; first < L; first += kMats) {
    const int64_t n = fill(first);
    a.x = x + first * p.mp * p.np;
    if ((e = write_out(st, mats, a, n))) return e;
  }
  return SL_OK;
}

extern "C" int sl_muon_step(void* stream, void* const* W, float* const* master, const float* const* G, float* const* M, int64_t L, int64_t rows,
                            int64_t cols, float lr, float momentum, int32_t nesterov, float weight_decay, float scale, int32_t steps,
                            const float* coeffs, void* workspace, size_t workspace_bytes) {
  OrthoPlan p{};
  int e = ortho_plan(L, rows, cols, p);
  if (e) return e;
  if ((e = check_steps(steps, coeffs))) return e;
  if (!std::isfinite(lr) || !std::isfinite(momentum) || !std::isfinite(weight_decay) || !std::isfinite(scale)) return SL_EINVAL;
  if (L == 0 || rows == 0 || cols == 0) return SL_OK;
  if (!W || !G || !M) return SL_EINVAL;
  for (int64_t i = 0; i < L; ++i) {
    if (!W[i] || !G[i] || !M[i] || (master && !master[i])) return SL_EINVAL;
    if (!aligned_matrix(W[i], rows, cols, 2) || !aligned_matrix(G[i], rows, cols, 4) || !aligned_matrix(M[i], rows, cols, 4) ||
        (master && !aligned_matrix(master[i], rows, cols, 4)))
      return SL_EALIGN;
  }
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < size_t(p.bytes)) return SL_EWORKSPACE;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  PassArgs a{};
  a.rows = rows; a.cols = cols; a.mp = int(p.mp); a.np = int(p.np);
  a.mu = momentum; a.nesterov = nesterov != 0; a.has_m = true;
  a.tall = p.tall; a.vec = cols % 4 == 0;
  a.keep = 1.0f - lr * weight_decay; a.step = lr * scale;
  a.update = true; a.has_master = master != nullptr;
  Mats mats{};
  auto fill = [&](int64_t first) {
    const int64_t n = L - first < kMats ? L - first : kMats;
    for (int64_t i = 0; i < n; ++i) {
      mats.g[i] = G[first + i];
      mats.m[i] = M[first + i];
      mats.w[i] = W[first + i];
      if (master) mats.master[i] = master[first + i];
    }
    return n;
  };
  _Float16* x = nullptr;
  for (int64_t first = 0; first < L; first += kMats) {
    fill(first);
    if ((e = iterate(st, mats, a, p, L, steps, coeffs, static_cast<char*>(workspace), first, &x))) return e;
  }
  for (int64_t first = 0; first < L; first += kMats) {
    const int64_t n = fill(first);
    a.x = x + first * p.mp * p.np;
    if ((e = write_out(st, mats, a, n))) return e;
  }
  return SL_OK;
}
