// fp16 products of the orthogonalised update (gfx950): the fixed-order main loop of the bf16 kernels (sl_gemm4.h) on
// v_mfma_f32_16x16x32_f16, with batches of matrices, symmetric results, and an epilogue that adds a multiple of a third
// matrix in fp32 before the one rounding.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>

#include "sl_gemm4.h"
#include "sl_gemm_h.h"

namespace sl2 {

// Lower triangle of a grid of tiles, row by row: tile t is row i, column j <= i.
__device__ __forceinline__ void triangle(int t, int& i, int& j) {
  i = int((sqrtf(8.f * float(t) + 1.f) - 1.f) * 0.5f);
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  while (i * (i + 1) / 2 > t) --i;
  j = t - i * (i + 1) / 2;
}

template <int WM, int WN>
__device__ __forceinline__ void store_rows(char* ep, _Float16* C, int64_t ldc, int M, int N, int mw, int nw, int lane) {
  using E = Epi<WN, WM, false>;
  const int rr = lane / E::kCPR, cr = lane % E::kCPR, n = nw + cr * 8;
#pragma unroll
  for (int t = 0; t < WM / E::kRPI; ++t) {
    const int r = t * E::kRPI + rr, m = mw + r;
    const uint4 v = *reinterpret_cast<const uint4*>(ep + E::off(r, cr));
    if (m < M && n < N) *reinterpret_cast<uint4*>(C + int64_t(m) * ldc + n) = v;
  }
}

// The same wave tile, transposed: a group of 16 lanes reads 4 x 16 blocks through transposing reads (source lane 4j + q:
// row j, columns 4q .. 4q + 3; result lane s: column s, 4 rows), twice for 8 rows of its column, and the four groups take
// 32 rows, so that a row of the result gets 64 bytes a store.
template <int WM, int WN>
__device__ __forceinline__ void store_transposed(char* ep, _Float16* C, int64_t ldc, int M, int N, int mw, int nw, int lane) {
  using E = Epi<WN, WM, false>;
  const int g = lane >> 4, s = lane & 15, j = s >> 2, q = s & 3;
#pragma unroll
  for (int cb = 0; cb < WN / 16; ++cb) {
    const int col = 16 * cb + 4 * q;
#pragma unroll
    for (int mb = 0; mb < WM / 32; ++mb) {
      const int row = 32 * mb + 8 * g;
      const char* p0 = ep + E::off(row + j, col / 8) + 2 * (col % 8);
      const char* p1 = ep + E::off(row + 4 + j, col / 8) + 2 * (col % 8);
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)p0);
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)p1);
      const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
      const int n = nw + 16 * cb + s, m = mw + row;
      if (n < N && m < M) *reinterpret_cast<uint4*>(C + int64_t(n) * ldc + m) = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
}

template <class P, bool SYM, int OCC>
__global__ void __launch_bounds__(P::WAVES * 64, OCC) half_gemm(HalfArgs g) {
  constexpr int WM = P::WM, WN = P::WN, TM = P::TM, TN = P::TN;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = SYM ? g.tiles_m * (g.tiles_m + 1) / 2 : g.tiles_m * g.tiles_n;
  const int t = xcd_remap(blockIdx.x, gridDim.x), batch = t / per, tile = t % per;
  int tm, tn;
  if constexpr (SYM) {
    triangle(tile, tm, tn);
  } else {
    constexpr int GR = 4;
    const int first = tile / (GR * g.tiles_n) * GR, rows = min(g.tiles_m - first, GR), in = tile % (GR * g.tiles_n);
    tm = first + in % rows;
    tn = in / rows;
  }
  const int m0 = tm * P::BM, n0 = tn * P::BN;
  g.a = static_cast<const _Float16*>(g.a) + int64_t(batch) * g.M * g.K;
  g.b = static_cast<const _Float16*>(g.b) + int64_t(batch) * g.N * g.K;

  f32x4v acc[TM][TN];
  gemm4_core<P>(g, smem, lane, wave, m0, n0, 0, (g.K + P::BK - 1) / P::BK, acc);
  asm_wait_vm<0>();
  __syncthreads();          // every wave is past its last operand read: the ring becomes epilogue space

  // Lane l holds row 16 i + l % 16 and columns 16 j + 4 (l / 16) + 0..3 of its wave tile.  Each wave stages its own
  // part of LDS, and reads D where its accumulators lie.
  const int64_t base = int64_t(batch) * g.M * g.N, ldc = g.N;
  const int mw = m0 + wave / P::WGN * WM, nw = n0 + wave % P::WGN * WN;
  const int rl = lane & 15, gl = lane >> 4;
  char* ep = smem + wave * Epi<WN, WM, false>::kBytes;
  const _Float16* D = static_cast<const _Float16*>(g.d);
  const _Float16* Dlo = static_cast<const _Float16*>(g.dlo);
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      acc[i][j] *= g.alpha;
      const int m = mw + 16 * i + rl, n = nw + 16 * j + 4 * gl;
      if (D && m < g.M && n < g.N) {
        const int64_t at = base + int64_t(m) * ldc + n;
        f32x4v d = __builtin_convertvector(*reinterpret_cast<const f16x4*>(D + at), f32x4v);
        if (Dlo) d += __builtin_convertvector(*reinterpret_cast<const f16x4*>(Dlo + at), f32x4v) * 0x1p-11f;
        acc[i][j] += d * g.beta;
      }
    }
  auto stage = [&](auto part) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        *reinterpret_cast<f16x4*>(ep + Epi<WN, WM, false>::off(i * 16 + rl, 2 * j + (gl >> 1)) + 8 * (gl & 1)) = part(acc[i][j]);
    asm volatile("" ::: "memory");       // the wave's lanes read each other's pieces, in order behind these writes
  };
  auto high = [](f32x4v v) { return __builtin_convertvector(v, f16x4); };
  stage(high);
  _Float16* C = static_cast<_Float16*>(g.c) + base;
  store_rows<WM, WN>(ep, C, ldc, g.M, g.N, mw, nw, lane);
  if constexpr (SYM) {
    if (tm != tn) store_transposed<WM, WN>(ep, C, ldc, g.M, g.N, mw, nw, lane);
  } else {
    if (g.clo) {
      asm volatile("" ::: "memory");
      stage([&](f32x4v v) { return __builtin_convertvector((v - __builtin_convertvector(high(v), f32x4v)) * 0x1p11f, f16x4); });
      store_rows<WM, WN>(ep, static_cast<_Float16*>(g.clo) + base, ldc, g.M, g.N, mw, nw, lane);
    }
  }
}

template <class P, bool SYM, int OCC>
int launch_half(hipStream_t st, HalfArgs g) {
  auto kfn = half_gemm<P, SYM, OCC>;
  static std::atomic<uint64_t> attr{0};
  if (smem_attr_once(reinterpret_cast<const void*>(kfn), P::kLds, attr)) return -5;
  g.tiles_m = (g.M + P::BM - 1) / P::BM;
  g.tiles_n = (g.N + P::BN - 1) / P::BN;
  const int64_t tiles = SYM ? int64_t(g.tiles_m) * (g.tiles_m + 1) / 2 : int64_t(g.tiles_m) * g.tiles_n;
  hipLaunchKernelGGL(kfn, dim3(unsigned(tiles * g.batches)), dim3(P::WAVES * 64), P::kLds, st, g);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

// 256x256 tiles of 8 waves, one workgroup a CU, and 128x128 tiles of 4 waves, two a CU; both two stages of 64 k.
template <bool B_KM> using Big = G4<true, B_KM, false, 2, 2, 4, 64, 256, 16, 256, true>;
template <bool B_KM> using Small = G4<true, B_KM, false, 2, 2, 2, 64, 128, 16, 128, true>;

// Whether 256x256 tiles fill the chip: their rounds over 256 CUs cost less than those of 128x128 tiles over 512 places,
// whose workgroups reach about 0.7 of their rate.
bool big_tiles(const HalfArgs& g, bool sym) {
  auto tiles = [&](int64_t e) {
    const int64_t m = (g.M + e - 1) / e, n = (g.N + e - 1) / e;
    return g.batches * (sym ? m * (m + 1) / 2 : m * n);
  };
  const double big = double((tiles(256) + 255) / 256), small = double((tiles(128) + 511) / 512) * 0.5 / 0.7;
  return big <= small;
}

template <bool B_KM, bool SYM>
int run_half(hipStream_t st, HalfArgs g) {
  g.lda = g.K;
  g.ldb = B_KM ? g.K : g.N;
  g.a_bytes = uint32_t(int64_t(g.M) * g.K * 2);
  g.b_bytes = uint32_t(int64_t(g.N) * g.K * 2);
  return big_tiles(g, SYM) ? launch_half<Big<B_KM>, SYM, 1>(st, g) : launch_half<Small<B_KM>, SYM, 2>(st, g);
}

}  // namespace sl2

int half_gemm_nt(hipStream_t st, HalfArgs g, bool sym) {
  return sym ? sl2::run_half<true, true>(st, g) : sl2::run_half<true, false>(st, g);
}

int half_gemm_nn(hipStream_t st, HalfArgs g) { return sl2::run_half<false, false>(st, g); }
