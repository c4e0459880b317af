// fp16 products of the orthogonalised update (gfx950) on v_mfma_f32_16x16x32_f16: batches of matrices, symmetric
// results, and an epilogue that adds a multiple of a third matrix and of the unit matrix in fp32 before the one rounding.
//
// A workgroup walks a list of items (a tile, or a part of a tile's sum) and the stages of one item follow those of the
// item before without a gap: operands go HBM -> LDS directly, 64 k to a stage, two stages deep, in the fixed issue order
// of the bf16 kernels (sl_gemm4.h holds the operand layouts).  The loads of stage s + 2 go out behind the barrier that ends the
// reads of stage s, whichever item it belongs to, so an item starts with its first two stages in LDS or under way, and
// only its results' stores stand between its products and the next item's.  Results leave straight from the
// accumulators: the 16-lane groups of a wave trade pieces, so that a lane has 8 columns of a row.
//
// What bounds it: a 64 k stage of 256 x 256 takes 1.45 us on all CUs, 1.48 PFLOP/s, which is what the power limit leaves a large
// product here (the library's reaches 1.47 to 1.51).  On top of it come 15 us a round: 3.4 from the start to the first data, the
// results' loads and stores, and the drain at the end; two accumulator tiles, which would let the results leave under the next
// tile's products, do not fit into the registers.  P X of 2 x [4096, 5504]: 279 to 291 us without what roundings left (1.27 to
// 1.32 PFLOP/s, matrix units 0.66 busy), 307 to 318 with it read and written; of 16 x [1536, 2048] 137 to 140 and 162 to 165 in
// three rounds.
//
// The kernels that add D and the diagonal (b A + c A^2 + a I) do not fit their registers: 62 and 50 scalar ones are spilled, with 24
// bytes of scratch a lane that every piece of the epilogue reads back, and their join takes 126 registers where the others take 61
// to 64.  The kernels that keep what roundings left spill 12 and 5 scalar ones; the rest spill none or 2.
//
// Tiles of 256 x 256 are dealt out in whole rounds of the chip; what remains, or the whole of a small product, goes to
// tiles of 128 x 128 in a launch of its own, and where its last round would leave places idle, sums are split into fp32
// planes (kept in the accumulators' own order, whole lines a store) which another kernel adds in order and finishes through
// the same epilogue.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>

#include "sl_gemm4.h"
#include "sl_gemm_h.h"

namespace sl2 {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---- items ---------------------------------------------------------------------------------------

// plane < 0: the whole sum; mirror: the transposed tile too; all wave-uniform
struct HalfItem { int batch, m0, n0, kt0, kt1, plane; bool mirror; };

// Row and column of tile `t` of a lower triangle of n x n tiles in groups of 4 rows, column by column, so that tiles near each other in the
// order share rows and columns: group q holds (4 q + 1) columns of all its rows, then the corner at the diagonal.
__device__ __forceinline__ int2 triangle(int t, int n) {
  int q = int((sqrtf(4.f + 32.f * float(t)) - 2.f) * (1.f / 16.f));
  while ((8 * (q + 1) + 2) * (q + 1) <= t) ++q;
  while ((8 * q + 2) * q > t) --q;
  const int rows = min(n - 4 * q, 4), whole = (4 * q + 1) * rows, u = t - (8 * q + 2) * q;
  if (u < whole) return make_int2(4 * q + u % rows, u / rows);
  // the corner's columns of rows - 1, rows - 2, .. tiles
  const int v = u - whole, d = v < rows - 1 ? 1 : v < 2 * rows - 3 ? 2 : 3;
  const int j = 4 * q + d;
  return make_int2(j + v - (d == 1 ? 0 : d == 2 ? rows - 1 : 2 * rows - 3), j);
}

template <class P, bool SYM>
__device__ __forceinline__ HalfItem half_item(const HalfArgs& g, int x) {
  const int stages = g.K / P::BK;
  const bool part = x >= g.full;               // the parts of a tile are neighbours in the order
  const int plane = part ? x - g.full : -1, tile = part ? g.full + plane / g.splits : x;
  const int kt0 = part ? plane % g.splits * g.kt_per_split : 0, kt1 = part ? min(stages, kt0 + g.kt_per_split) : stages;
  // quarters of the tiles from g.first on of a grid of twice the edge, where g.quarters
  const int q = g.quarters ? 1 : 0, all = g.quarters ? g.first + tile / 4 : tile;
  const int rows = (g.tiles_m + q) >> q, cols = (g.tiles_n + q) >> q;
  const int per = SYM ? rows * (rows + 1) / 2 : rows * cols, batch = all / per, t = all % per;
  int tm, tn;
  if constexpr (SYM) {
    const int2 at = triangle(t, rows);
    tm = at.x;
    tn = at.y;
  } else {
    constexpr int GR = 4;
    const int first = t / (GR * cols) * GR, high = min(rows - first, GR), in = t % (GR * cols);
    tm = first + in % high;
    tn = in / high;
  }
  const bool mirror = SYM && tm != tn;
  if (g.quarters) {                            // those past the matrix's edge load zeros and store nothing
    tm = 2 * tm + (tile >> 1 & 1);
    tn = 2 * tn + (tile & 1);
  }
  return HalfItem{batch, __builtin_amdgcn_readfirstlane(tm * P::BM), __builtin_amdgcn_readfirstlane(tn * P::BN), kt0, kt1, plane, mirror};
}

// ---- epilogue ------------------------------------------------------------------------------------
// A wave finishes 32 rows by 64 columns at a time: lane l holds row 16 i + l % 16 and columns 16 j + 4 (l / 16) + 0..3 of
// blocks [2][4].  M and N are multiples of 128, so such a piece lies wholly inside the matrix or outside.

// Blocks j and j + 1 as fp16 words: afterwards lane group g holds columns 8 (g / 2) .. + 7 of block j + g % 2 (its own
// inverse).
__device__ __forceinline__ u32x4 trade(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v[0], v[2], false, false), b = __builtin_amdgcn_permlane16_swap(v[1], v[3], false, false);
  return u32x4{a[0], b[0], a[1], b[1]};
}

// Words of the four blocks of a row of blocks, transposed between them and the lane groups: afterwards group g holds all 4
// words of block g (its own inverse).
__device__ __forceinline__ u32x4 gather(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v[0], v[1], false, false), b = __builtin_amdgcn_permlane16_swap(v[2], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false), d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  return u32x4{c[0], d[0], c[1], d[1]};
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t half_rows(const void* p, int64_t first, int64_t bytes, bool in) {
  return __builtin_amdgcn_make_buffer_rsrc(static_cast<char*>(const_cast<void*>(p)) + first, 0, in ? int(bytes) : 0, kRsrcWord3);
}

constexpr int kStageBytes = 32 * 64 * 2;       // a wave's piece in LDS, for its transposed copy

// What a kernel's epilogue adds: nothing; D in fp16 and the diagonal; what roundings left (E5M2); that, and keeping it anew.
enum HalfEpi { kPlain, kAdd, kLeft, kLeftKeep };

// D's part of a piece, in the order in which results are stored: rows of 64 fp16 elements, two loads of half a row's columns, or
// rows of 64 bytes.
template <int EPI>
__device__ __forceinline__ void half_fetch(const HalfArgs& g, u32x4 (&d)[2][2], int batch, int m, int n, int lane) {
  constexpr int E = EPI == kAdd ? 2 : 1;
  const int rl = lane & 15, gl = lane >> 4;
  const uint32_t off = uint32_t(rl) * uint32_t(g.N) * E + uint32_t(n + 16 * (E == 2 ? gl & 1 : gl) + (E == 2 ? 8 * (gl >> 1) : 0)) * E;
  const auto rd = half_rows(g.d, (int64_t(batch) * g.M + m) * g.N * E, int64_t(32) * g.N * E, m < g.M && n < g.N);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int p = 0; p < E; ++p)
      d[i][p] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rd, off + 64 * p + i * uint32_t(g.N) * 16 * E, 0, 0));
}

// `lds`: kStageBytes of the wave's own, used where `mirror` asks for the transposed copy too.
template <int EPI>
__device__ __forceinline__ void half_finish(const HalfArgs& g, f32x4v (&acc)[2][4], const u32x4 (&d)[2][2], int batch, int m, int n, bool mirror,
                                            uint32_t lds, int lane) {
  const bool in = m < g.M && n < g.N;
  const int64_t first = (int64_t(batch) * g.M + m) * g.N * 2, bytes = int64_t(32) * g.N * 2;
  const int rl = lane & 15, gl = lane >> 4;
  const uint32_t off = uint32_t(rl) * uint32_t(g.N) * 2 + uint32_t(n + 16 * (gl & 1) + 8 * (gl >> 1)) * 2;
  const uint32_t down = uint32_t(g.N) * 32;    // 16 rows
  auto wide = [](uint32_t a, uint32_t b) { return __builtin_convertvector(__builtin_bit_cast(f16x4, make_uint2(a, b)), f32x4v); };
  auto words = [](f32x4v v) { return __builtin_bit_cast(uint2, __builtin_convertvector(v, f16x4)); };
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] *= g.alpha;
  if constexpr (EPI == kAdd) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const u32x4 w = trade(d[i][p]);
        acc[i][2 * p] += wide(w[0], w[1]) * g.beta;
        acc[i][2 * p + 1] += wide(w[2], w[3]) * g.beta;
      }
  }
  if constexpr (EPI >= kLeft) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4 w = gather(d[i][0]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_bf8(int(w[j]), false), hi = __builtin_amdgcn_cvt_pk_f32_bf8(int(w[j]), true);
        acc[i][j] += f32x4v{lo[0], lo[1], hi[0], hi[1]} * g.beta;
      }
    }
  }
  if (EPI == kAdd && m < n + 64 && n < m + 32) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (m + 16 * i + rl == n + 16 * j + 4 * gl + e) acc[i][j][e] += g.diag;
  }
  const auto rc = half_rows(g.c, first, bytes, in);
  u32x4 hi[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint2 a = words(acc[i][2 * p]), b = words(acc[i][2 * p + 1]);
      hi[i][p] = trade(u32x4{a.x, a.y, b.x, b.y});
      __builtin_amdgcn_raw_buffer_store_b128(hi[i][p], rc, off + 64 * p + i * down, 0, 0);
    }
  if constexpr (EPI == kLeftKeep) {
    const auto rk = half_rows(g.clo, first / 2, bytes / 2, in);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u32x4 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4v v = acc[i][j], left = (v - __builtin_convertvector(__builtin_convertvector(v, f16x4), f32x4v)) * 0x1p11f;
        w[j] = uint32_t(__builtin_amdgcn_cvt_pk_bf8_f32(left[2], left[3], __builtin_amdgcn_cvt_pk_bf8_f32(left[0], left[1], 0, false), true));
      }
      __builtin_amdgcn_raw_buffer_store_b128(gather(w), rk, uint32_t(rl) * uint32_t(g.N) + uint32_t(n + 16 * gl) + i * uint32_t(g.N) * 16, 0, 0);
    }
  }
  if (!mirror) return;
  // Rows of 8 chunks in LDS, chunks XOR-swizzled by row; a group of 16 lanes then reads 4 x 16 blocks through transposing
  // reads (source lane 4j + q: row j, columns 4q .. 4q + 3; result lane s: column s, 4 rows), twice for 8 rows of its
  // column, and the four groups take the 32 rows, so that a row of the copy gets 64 bytes a store.
  typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  auto at = [&](int r, int c) { return lds + uint32_t(r * 128 + ((c ^ (r & 7)) << 4)); };
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int p = 0; p < 2; ++p) *(lds_u32x4*)(uintptr_t)at(16 * i + rl, 4 * p + 2 * (gl & 1) + (gl >> 1)) = hi[i][p];
  asm volatile("" ::: "memory");
  const auto rt = half_rows(g.c, (int64_t(batch) * g.M + n) * g.N * 2, int64_t(64) * g.N * 2, in);
  const int jr = rl >> 2, q = rl & 3;
#pragma unroll
  for (int cb = 0; cb < 4; ++cb) {
    const int col = 16 * cb + 4 * q, row = 8 * gl + jr;
    const i16x4 lo4 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(uintptr_t)(at(row, col / 8) + 2 * (col % 8)));
    const i16x4 hi4 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(uintptr_t)(at(row + 4, col / 8) + 2 * (col % 8)));
    const uint2 a = __builtin_bit_cast(uint2, lo4), b = __builtin_bit_cast(uint2, hi4);
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{a.x, a.y, b.x, b.y}, rt, uint32_t(16 * cb + rl) * uint32_t(g.N) * 2 + uint32_t(m + 8 * gl) * 2, 0, 0);
  }
  asm volatile("" ::: "memory");
}

// ---- the kernel ----------------------------------------------------------------------------------

template <class P, bool SYM, int EPI, int OCC>
__global__ void __launch_bounds__(P::WAVES * 64, OCC) half_gemm(HalfArgs g) {
  constexpr int BK = P::BK, WAVES = P::WAVES, WM = P::WM, WN = P::WN, TM = P::TM, TN = P::TN, KS = P::KS;
  constexpr int LA = P::LA, LB = P::LB, LPS = LA + LB, kStage = P::kStage, NR = TM + TN;
  constexpr bool B_KM = P::B_KM;
  using OA = typename P::OA;
  using OB = typename P::OB;
  static_assert(P::S == 2 && BK == 2 * KS && TN == 4 && WN == 64 && TM % 2 == 0, "two steps a stage, pieces of 32 x 64");
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / P::WGN, wn = wave % P::WGN;
  const uint32_t lds0 = lds_addr(smem);

  // Each XCD takes a contiguous range of the whole tiles and one of the parts, its workgroups side by side in them.
  const int xcd = blockIdx.x % kXCD, slot0 = blockIdx.x / kXCD, stride = (int(gridDim.x) - xcd + kXCD - 1) / kXCD;
  auto range = [&](int n, int& lo, int& hi) {
    const int per = n / kXCD, rem = n % kXCD;
    lo = xcd * per + min(xcd, rem);
    hi = lo + per + (xcd < rem);
  };
  int f0, f1, p0, p1;
  range(g.full, f0, f1);
  range(g.rest * g.splits, p0, p1);
  const int nf = f1 - f0 > slot0 ? (f1 - f0 - slot0 + stride - 1) / stride : 0;
  const int np = p1 - p0 > slot0 ? (p1 - p0 - slot0 + stride - 1) / stride : 0;
  const int count = nf + np;
  if (count == 0) return;
  auto nth = [&](int q) { return half_item<P, SYM>(g, q < nf ? f0 + slot0 + q * stride : g.full + p0 + slot0 + (q - nf) * stride); };

  // Lane offsets of the loads and fragment reads, the same for every tile: descriptors begin at the tile.  A wave's loads
  // of an operand differ by whole multiples of 16 rows, over which the swizzles repeat, so one lane offset and a scalar
  // serve them all; a K-major fragment's second step is the other half of each 128-byte row.
  uint32_t va[1], vb[1], ofb[B_KM ? 1 : TN];
  const int64_t ldb = B_KM ? g.K : g.N;
  OA::template prep<WAVES>(va, lane, wave, 0, P::BM, g.K);
  OB::template prep<WAVES>(vb, lane, wave, 0, P::BN, ldb);
  const uint32_t ofa = kmaj_frag_off16<OA>(wm * WM, 0, lane);
  if constexpr (B_KM) ofb[0] = OA::kBytes + kmaj_frag_off16<OB>(wn * WN, 0, lane);
  else
#pragma unroll
    for (int j = 0; j < TN; ++j) ofb[j] = OA::kBytes + mnmaj_frag_off16<OB>(wn * WN + 16 * j, lane);
  constexpr int kRowsA = WAVES * 64 / OA::kCPR, kRowsB = WAVES * 64 / OB::kCPR;        // rows of one load of all waves
  static_assert(kRowsA % 16 == 0 && kRowsB % 16 == 0, "the swizzles' period");
  const uint32_t a_rows = uint32_t(kRowsA) * uint32_t(g.K) * 2, b_rows = uint32_t(kRowsB) * uint32_t(ldb) * 2;
  const uint32_t ka_step = BK * 2, kb_step = B_KM ? BK * 2 : uint32_t(BK) * uint32_t(g.N) * 2;

  // The item being loaded: operands as descriptors from the tile's first element to the matrix's end.  A tile's second
  // half of rows may lie past the end as a whole (extents are multiples of 128): its descriptor then has no bytes, and the
  // loads write zeros.  Columns past a K x N operand's edge read the next row's first ones (zeros behind the last row), and no
  // result of theirs is stored.
  i32x4 ra, rb;
  int a_high, b_high;                          // bytes of the second halves' descriptors
  uint32_t ka, kb;
  int lq = 0, left;
  auto open = [&](const HalfItem it) {
    ra = rsrc_uniform(static_cast<const _Float16*>(g.a) + (int64_t(it.batch) * g.M + it.m0) * g.K, uint32_t(int64_t(g.M - it.m0) * g.K * 2));
    a_high = it.m0 + P::BM / 2 < g.M ? ra[2] : 0;
    if constexpr (B_KM)
      rb = rsrc_uniform(static_cast<const _Float16*>(g.b) + (int64_t(it.batch) * g.N + it.n0) * g.K, uint32_t(int64_t(g.N - it.n0) * g.K * 2));
    else
      rb = rsrc_uniform(static_cast<const _Float16*>(g.b) + int64_t(it.batch) * g.K * g.N + it.n0, uint32_t((int64_t(g.K) * g.N - it.n0) * 2));
    b_high = !B_KM || it.n0 + P::BN / 2 < g.N ? rb[2] : 0;
    ka = uint32_t(it.kt0) * ka_step;
    kb = uint32_t(it.kt0) * kb_step;
    left = it.kt1 - it.kt0;
  };
  auto advance = [&]() {                       // to the next stage of the list; past its end, descriptors of no bytes
    ka += ka_step;
    kb += kb_step;
    if (--left == 0) {
      if (++lq < count) open(nth(lq));
      else ra[2] = rb[2] = a_high = b_high = 0;
    }
  };
  auto load_one = [&](auto ic_l, uint32_t base) {
    constexpr int l = decltype(ic_l)::value;
    i32x4 r = l < LA ? ra : rb;
    if constexpr (l >= LA / 2 && l < LA) r[2] = a_high;
    if constexpr (l >= LA + LB / 2) r[2] = b_high;
    if constexpr (l < LA) lds_dma16s(r, base + (l * WAVES + wave) * 1024, va[0], ka + l * a_rows);
    else lds_dma16s(r, base + OA::kBytes + ((l - LA) * WAVES + wave) * 1024, vb[0], kb + (l - LA) * b_rows);
  };

  f32x4v acc[TM][TN];
  f16x8 fa[2][TM], fb[2][TN];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x4v{0.f, 0.f, 0.f, 0.f};
  };
  auto half8 = [](bf16x8 v) __attribute__((always_inline)) { return __builtin_bit_cast(f16x8, v); };    // 16 bits either way
  auto read_one = [&](auto ic_m, auto ic_to, auto ic_ks, uint32_t base) {
    constexpr int m = decltype(ic_m)::value, to = decltype(ic_to)::value, ks = decltype(ic_ks)::value;
    if constexpr (m < TM) fa[to][m] = half8(lds_rd128<m * 16 * OA::kRowBytes>((base + ofa) ^ (64 * ks)));
    else if constexpr (B_KM) fb[to][m - TM] = half8(lds_rd128<(m - TM) * 16 * OB::kRowBytes>((base + ofb[0]) ^ (64 * ks)));
    else fb[to][m - TM] = half8(lds_rd_tr<ks * KS * OB::kRowBytes, (ks * KS + 4) * OB::kRowBytes>(base + ofb[m - TM]));
  };
  // One step: the products on buffer CUR, with the next step's fragment reads over the first three quarters of them and,
  // in a stage's second step, the loads spread over all.
  auto step = [&](auto ic_cur, uint32_t rbase, uint32_t lbase) {
    constexpr int cur = decltype(ic_cur)::value, NL = cur ? LPS : 0, NQ = TM * TN, RQ = NQ * 3 / 4;
    static_for<NQ>([&](auto qc) {
      constexpr int q = decltype(qc)::value, i = q / TN, j = (i & 1) ? TN - 1 - q % TN : q % TN;
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[cur][j], fa[cur][i], acc[i][j], 0, 0, 0);
      constexpr int rlo = q < RQ ? q * NR / RQ : NR, rhi = q < RQ ? (q + 1) * NR / RQ : NR;
      static_for<rhi - rlo>([&](auto mc) { read_one(ic<rlo + decltype(mc)::value>{}, ic<cur ^ 1>{}, ic<cur ^ 1>{}, rbase); });
      constexpr int llo = (2 * q * NL + NQ) / (2 * NQ), lhi = (2 * (q + 1) * NL + NQ) / (2 * NQ);
      static_for<lhi - llo>([&](auto mc) { load_one(ic<llo + decltype(mc)::value>{}, lbase); });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  HalfItem it = nth(0);
  open(it);
  static_for<LPS>([&](auto lc) { load_one(lc, lds0); });
  advance();
  static_for<LPS>([&](auto lc) { load_one(lc, lds0 + kStage); });
  advance();
  asm_wait_vm<LPS>();
  bare_barrier();
  static_for<NR>([&](auto mc) { read_one(mc, ic<0>{}, ic<0>{}, lds0); });
  __builtin_amdgcn_sched_barrier(0);
  clear();

  uint32_t cur = lds0, nxt = lds0 + kStage;
  bool stores = false;                         // the results of an item went out since the last wait
  for (int q = 0;;) {
    for (int k = it.kt0; k < it.kt1; ++k) {
      step(ic<0>{}, cur, 0);
      // The next stage has landed: memory operations return in order, and each item's results are at least 2 TM stores of
      // every wave, all younger than that stage's loads.
      if (stores) asm_wait_vm<2 * TM>();
      else asm_wait_vm<0>();
      stores = false;
      lds_barrier();
      step(ic<1>{}, nxt, cur);
      advance();
      const uint32_t t = cur;
      cur = nxt;
      nxt = t;
    }
    const int m = it.m0 + wm * WM, n = it.n0 + wn * WN;
    if (it.plane < 0) {
      int l = lane;                            // from here on: what follows from it is not kept in registers over the stages
      asm volatile("" : "+v"(l));
      u32x4 d[2][2][2];                        // two pieces ahead
      if constexpr (EPI != kPlain) {
        half_fetch<EPI>(g, d[0], it.batch, m, n, l);
        half_fetch<EPI>(g, d[1], it.batch, m + 32, n, l);
      }
#pragma unroll
      for (int i = 0; i < TM / 2; ++i) {
        f32x4v piece[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) piece[h][j] = acc[2 * i + h][j];
        half_finish<EPI>(g, piece, d[i % 2], it.batch, m + 32 * i, n, SYM && it.mirror, lds0 + 2 * kStage + wave * kStageBytes, l);
        if (EPI != kPlain && i + 2 < TM / 2) half_fetch<EPI>(g, d[i % 2], it.batch, m + 32 * (i + 2), n, l);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      f32x4v* to = reinterpret_cast<f32x4v*>(g.ws) + (int64_t(it.plane) * WAVES + wave) * (TM * TN * 64) + lane;
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) to[(i * TN + j) * 64] = acc[i][j];
    }
    asm volatile("" ::: "memory");
    if (++q == count) break;
    stores = true;
    // the next item's first fragments once more: kept over the results, they would push what the results need out of registers
    static_for<NR>([&](auto mc) { read_one(mc, ic<0>{}, ic<0>{}, cur); });
    __builtin_amdgcn_sched_barrier(0);
    clear();
    it = nth(q);
  }
  asm_wait_vm<0>();
}

// Adds the planes of the tiles from g.full on, in order, and finishes them: a wave to 32 rows by 64 columns.
template <class P, bool SYM, int EPI>
__global__ void __launch_bounds__(64) half_join(HalfArgs g) {
  __shared__ __attribute__((aligned(16))) char stage[kStageBytes];
  constexpr int PIECES = P::TM / 2;
  const int lane = threadIdx.x, piece = blockIdx.x % PIECES, wave = blockIdx.x / PIECES % P::WAVES, tile = blockIdx.x / (PIECES * P::WAVES);
  const HalfItem it = half_item<P, SYM>(g, g.full + tile * g.splits);
  const int m = it.m0 + wave / P::WGN * P::WM + 32 * piece, n = it.n0 + wave % P::WGN * P::WN;
  u32x4 d[2][2];
  if constexpr (EPI != kPlain) half_fetch<EPI>(g, d, it.batch, m, n, lane);
  f32x4v acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int s = 0; s < g.splits; ++s) {
    const f32x4v* from = reinterpret_cast<const f32x4v*>(g.ws) + (int64_t(tile * g.splits + s) * P::WAVES + wave) * (P::TM * P::TN * 64) + lane;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += from[((2 * piece + i) * P::TN + j) * 64];
  }
  half_finish<EPI>(g, acc, d, it.batch, m, n, SYM && it.mirror, lds_addr(stage), lane);
}

// ---- host ----------------------------------------------------------------------------------------

// 256x256 tiles of 8 waves, one workgroup a CU, and 128x128 tiles of 4 waves, two a CU.
template <bool B_KM> using Big = G4<true, B_KM, false, 2, 2, 4, 64, 256, 16, 256>;
template <bool B_KM> using Small = G4<true, B_KM, false, 2, 2, 2, 64, 128, 16, 128>;

// A product: `big` tiles of 256x256, from the first on, and `small` tiles of 128x128 for the rest, or for all of it (big ==
// 0); of these `rest` are split in `splits` parts.
struct HalfPlan {
  int64_t big, small, rest;
  int splits, kt_per_split;
  double us;
};

// Times in us, fitted to measured products with every split count (36 to 504 items of 5 to 128 stages: [1024, 1024] over 4096
// unsplit 41 us, in 2, 4, 6, 8 and 14 parts 28, 19, 19, 21 and 23; [2048, 2048] over 8192 in 1, 2 and 3 parts 88, 68 and 57).
// 128x128 tiles: a 64 k stage by the workgroups under way on 256 CUs; what an item costs beside its stages; a launch; and a
// split, by the planes that go out and come back.
void plan_small(HalfPlan& p, int stages) {
  constexpr int64_t places = 512;
  auto stage = [](int64_t items) { return items <= 256 ? 0.57 : 0.92; };
  constexpr double full_stage = 1.05, fixed = 3.0, launch = 4.0, join = 3.0, plane = 0.018;
  p.rest = p.small % places;
  p.splits = 1;
  p.kt_per_split = stages;
  double last = p.rest ? fixed + stages * stage(p.rest) : 0;
  for (int s = 2; p.rest && s <= places / p.rest && s <= stages / 4; ++s) {
    const int per = (stages + s - 1) / s, parts = (stages + per - 1) / per;
    const int64_t items = p.rest * parts;
    const double t = fixed + per * stage(items) + join + double(items) * plane;
    if (t < last) {
      last = t;
      p.splits = parts;
      p.kt_per_split = per;
    }
  }
  if (p.splits == 1) p.rest = 0;
  p.us += launch + double(p.small / places) * (fixed + stages * full_stage) + last;
}

// 256x256 tiles: rounds of the chip, each with its stores behind it.  16 x [1536, 2048]: the Gram products (336 tiles) 107 us in
// two rounds, 108 as one round and quarters, 104 in 128x128 tiles; the squares 93, 91 and 83; P X (768 tiles) 140 in three
// rounds, 173 in 128x128 tiles.  2 x [4096, 5504], Gram products (272 tiles): 240, 179 and 199.
HalfPlan half_plan(int M, int N, int K, int64_t batches, bool sym) {
  const int stages = K / 64;
  auto tiles = [&](int edge) {
    const int64_t m = (M + edge - 1) / edge, n = (N + edge - 1) / edge;
    return batches * (sym ? m * (m + 1) / 2 : m * n);
  };
  constexpr double stage = 1.38, fixed = 15.0, launch = 6.0, quarters = 3.0;
  HalfPlan best{};
  const int64_t all = tiles(256);
  for (int64_t big : {int64_t(0), all / 256 * 256, all}) {
    HalfPlan p{};
    p.big = big;
    p.small = big == 0 ? tiles(128) : 4 * (all - big);
    if (big) p.us = launch + double((big + 255) / 256) * (fixed + stages * stage) + (p.small ? quarters : 0);
    if (p.small) plan_small(p, stages);
    if (best.us == 0 || p.us < best.us) best = p;
  }
  return best;
}

template <class P, bool SYM, int EPI, int OCC>
int launch_half(hipStream_t st, const HalfArgs& g) {
  auto kfn = half_gemm<P, SYM, EPI, OCC>;
  constexpr int kLds = 2 * P::kStage + (SYM ? P::WAVES * kStageBytes : 0);
  static_assert(OCC * kLds <= 160 * 1024, "LDS");
  static std::atomic<uint64_t> attr{0};
  if (smem_attr_once(reinterpret_cast<const void*>(kfn), kLds, attr)) return -5;
  const int64_t items = g.full + int64_t(g.rest) * g.splits, places = OCC * 256;
  hipLaunchKernelGGL(kfn, dim3(unsigned(items < places ? items : places)), dim3(P::WAVES * 64), kLds, st, g);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

template <bool SYM, int EPI>
int run_half(hipStream_t st, HalfArgs g) {
  const HalfPlan p = half_plan(g.M, g.N, g.K, g.batches, SYM);
  if (p.big) {
    g.tiles_m = (g.M + 255) / 256;
    g.tiles_n = (g.N + 255) / 256;
    g.full = int(p.big);
    g.rest = 0;
    g.splits = 1;
    g.quarters = 0;
    if (launch_half<Big<SYM>, SYM, EPI, 1>(st, g)) return -5;
  }
  if (!p.small) return 0;
  using P = Small<SYM>;
  g.tiles_m = g.M / 128;
  g.tiles_n = g.N / 128;
  g.full = int(p.small - p.rest);
  g.rest = int(p.rest);
  g.splits = p.splits;
  g.kt_per_split = p.kt_per_split;
  g.quarters = p.big != 0;
  g.first = int(p.big);
  if (launch_half<P, SYM, EPI, 2>(st, g)) return -5;
  if (!p.rest) return 0;
  hipLaunchKernelGGL((half_join<P, SYM, EPI>), dim3(unsigned(p.rest * P::WAVES * P::TM / 2)), dim3(64), 0, st, g);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace sl2

int half_gemm_sym(hipStream_t st, HalfArgs g) { return g.d ? sl2::run_half<true, sl2::kAdd>(st, g) : sl2::run_half<true, sl2::kPlain>(st, g); }

int half_gemm_nn(hipStream_t st, HalfArgs g) {
  return !g.d ? sl2::run_half<false, sl2::kPlain>(st, g) : g.clo ? sl2::run_half<false, sl2::kLeftKeep>(st, g) : sl2::run_half<false, sl2::kLeft>(st, g);
}

HalfTiles half_gemm_tiles(int M, int N, int K, int64_t batches, bool sym) {
  const sl2::HalfPlan p = sl2::half_plan(M, N, K, batches, sym);
  return HalfTiles{p.big, p.small, p.rest, p.rest ? p.splits : 1};
}

size_t half_gemm_workspace_bytes(int M, int N, int K, int64_t batches, bool sym) {
  const HalfTiles t = half_gemm_tiles(M, N, K, batches, sym);
  return size_t(t.split) * size_t(t.parts) * (128 * 128 * 4);
}
