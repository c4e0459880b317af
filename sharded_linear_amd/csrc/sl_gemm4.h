// Operand tiles and the fixed-order main loop of the 16-bit GEMM kernels with direct HBM->LDS staging (gfx950), shared by
// the bf16 kernels of the linear step (sl_gemm2.hip) and the fp16 kernels of the orthogonalised update (sl_gemm_h.hip).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "sl_device.h"
#include "sl_epi.h"

namespace sl2 {

// ---- K-major operand: LDS [R rows][BK] bf16 -----------------------------------------------
template <int R, int BK, int SW = 0>
struct KMaj {
  static constexpr int kRowBytes = BK * 2;
  static constexpr int kCPR = BK / 8;                  // 16-byte chunks per row
  static constexpr int kBytes = R * kRowBytes;
  static constexpr int kLoads = kBytes / 1024;         // wave-loads of 1 KiB per stage
  static_assert(BK == 32 || BK == 64, "row swizzles are defined for BK 32 and 64");
  // XOR swizzle of 16-byte chunks by row, chosen by measurement: a wave's ds_read_b128 of one
  // fragment (32 rows, two chunks) runs at the rate of linear addresses -- full LDS rate with 8
  // waves per CU -- with these, while the 64-byte-row alternative ((r >> 1) ^ (r >> 3)) & 3,
  // conflict-free on paper for 8 and 16 consecutive lanes, ran 1.7x slower.
  // SW 1 serves the 16x16x32 fragment read (16 rows, four chunks) at BK 64: a ds_read_b128 pairs
  // lanes 0-7 with 16-23 (rows r with chunks c, c+1), so the four same-parity rows of an 8-row
  // block need distinct swizzles in bits {1,2} and in bits {0,2}, and rows r, r+8 distinct ones;
  // {0,3,5,6} by bits 1-2 of r, complemented for rows 8-15, meets all three and measured at the
  // linear rate.
  __device__ static __forceinline__ int swz(int r) {
    if constexpr (SW == 1) {
      static_assert(BK == 64, "16x16 swizzle is defined for BK 64");
      return ((0x6530 >> (4 * ((r >> 1) & 3))) & 7) ^ (((r >> 3) & 1) * 7);
    } else if constexpr (BK == 64) {
      return (r & 7) ^ ((r >> 3) & 1);
    } else {
      return (r ^ (r >> 2)) & 3;
    }
  }

  // Wave `w` issues loads wl = w, w + waves, ...; lane i fills LDS bytes [1024 wl + 16 i, +16).
  template <int WAVES, int LO = 0, int HI = kLoads / WAVES>
  __device__ static __forceinline__ void load(i32x4 rs, char* lds, int lane, int wave,
                                              int row0, int rows, int k0, int K, int64_t ld) {
#pragma unroll
    for (int it = LO; it < HI; ++it) {
      const int wl = it * WAVES + wave;
      const int p = wl * 64 + lane;                      // 16-byte slot
      const int r = p / kCPR, c = (p % kCPR) ^ swz(p / kCPR);
      const int gr = row0 + r, k = k0 + c * 8;
      const uint32_t off = (gr < rows && k < K) ? uint32_t((int64_t(gr) * ld + k) * 2) : kOOB;
      lds_dma16(rs, lds_addr(lds + wl * 1024), off);
    }
  }
  // Byte offsets of this thread's loads relative to the stage's first k (rows outside the matrix
  // -> kOOB).  A stage wholly inside K then loads with these and a scalar offset of 2 k0.
  template <int WAVES, int N = kLoads / WAVES>
  __device__ static __forceinline__ void prep(uint32_t (&voff)[N], int lane, int wave, int row0, int rows,
                                              int64_t ld) {
#pragma unroll
    for (int it = 0; it < N; ++it) {
      const int p = (it * WAVES + wave) * 64 + lane;
      const int r = p / kCPR, c = (p % kCPR) ^ swz(p / kCPR);
      voff[it] = row0 + r < rows ? uint32_t((int64_t(row0 + r) * ld + c * 8) * 2) : kOOB;
    }
  }
  // fragment of 32 rows starting at r0, k16 step ks: lane l gets row r0 + l%32, k 8(l/32)..+7
  // (the compiler-scheduled kernels; the fixed-order ones compute offsets once, see kmaj_frag_off)
  __device__ static __forceinline__ bf16x8 frag(const char* lds, int r0, int ks, int lane) {
    const int r = r0 + (lane & 31);
    const int c = ks * 2 + (lane >> 5);
    const uint4 v = *reinterpret_cast<const uint4*>(lds + r * kRowBytes + ((c ^ swz(r)) << 4));
    return __builtin_bit_cast(bf16x8, v);
  }
};

// ---- MN-major operand: LDS [BK rows (k)][R] bf16 -------------------------------------------
template <int R, int BK, int SW = 0>
struct MNMaj {
  static constexpr int kRowBytes = R * 2;
  static constexpr int kCPR = R / 8;
  static constexpr int kBytes = BK * kRowBytes;
  static constexpr int kLoads = kBytes / 1024;
  static_assert(kRowBytes % 128 == 0, "rows must span whole bank windows");
  // XOR swizzle of 16-byte chunks by k row: for the 4 rows x 16 free indices read by each
  // 16-lane group of ds_read_b64_tr_b16 (and the 4 x 32 read by 32 lanes), the 32-byte chunk
  // pairs are pair ^ {0, 5, 2, 7}, distinct within 128- and 256-byte bank windows.
  // SW 1 serves the 16x16x32 fragment read, whose 32 lanes read k rows kb..kb+3 and kb+8..kb+11
  // of the same 16 free indices: those rows also flip the low pair bit ({1, 4, 3, 6}), so the
  // eight 32-byte pieces fill a 256-byte window.  Bit 3 of k is constant over a fragment's rows,
  // so its k32 steps and second read stay immediates.
  __device__ static __forceinline__ int swz(int k) {
    if constexpr (SW == 1) return (((k & 3) ^ ((k & 1) << 2)) ^ ((k >> 3) & 1)) << 1;
    else return ((k & 3) ^ ((k & 1) << 2)) << 1;
  }

  template <int WAVES, int LO = 0, int HI = kLoads / WAVES>
  __device__ static __forceinline__ void load(i32x4 rs, char* lds, int lane, int wave,
                                              int col0, int cols, int k0, int K, int64_t ld) {
#pragma unroll
    for (int it = LO; it < HI; ++it) {
      const int wl = it * WAVES + wave;
      const int p = wl * 64 + lane;
      const int k = p / kCPR, c = (p % kCPR) ^ swz(p / kCPR);
      const int gk = k0 + k, gc = col0 + c * 8;
      const uint32_t off = (gk < K && gc < cols) ? uint32_t((int64_t(gk) * ld + gc) * 2) : kOOB;
      lds_dma16(rs, lds_addr(lds + wl * 1024), off);
    }
  }
  // Byte offsets relative to the stage's first k row (columns outside the matrix -> kOOB); a
  // stage wholly inside K loads with these and a scalar offset of 2 k0 ld.
  template <int WAVES, int N = kLoads / WAVES>
  __device__ static __forceinline__ void prep(uint32_t (&voff)[N], int lane, int wave, int col0, int cols,
                                              int64_t ld) {
#pragma unroll
    for (int it = 0; it < N; ++it) {
      const int p = (it * WAVES + wave) * 64 + lane;
      const int k = p / kCPR, c = (p % kCPR) ^ swz(p / kCPR);
      const int gc = col0 + c * 8;
      voff[it] = gc < cols ? uint32_t((int64_t(k) * ld + gc) * 2) : kOOB;
    }
  }
  // fragment of 32 free indices from f0, k16 step ks, via two transposing reads
  __device__ static __forceinline__ bf16x8 frag(const char* lds, int f0, int ks, int lane) {
    const int g = lane >> 4, s = lane & 15, j = s >> 2, q = s & 3;
    const int f = f0 + 16 * (g & 1) + 4 * q;
    const int k = ks * 16 + 8 * (g >> 1) + j;
    const int cb = f >> 3, eb = (f & 7) << 1;
    const char* p0 = lds + k * kRowBytes + ((cb ^ swz(k)) << 4) + eb;
    const char* p1 = lds + (k + 4) * kRowBytes + ((cb ^ swz(k + 4)) << 4) + eb;
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)p0);
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)p1);
    const short __attribute__((ext_vector_type(8))) v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, v);
  }
};

template <bool KM, int R, int BK, int SW = 0>
struct OpSel { using T = KMaj<R, BK, SW>; };
template <int R, int BK, int SW>
struct OpSel<false, R, BK, SW> { using T = MNMaj<R, BK, SW>; };

// Loads [LO, HI) of one stage of an operand with precomputed offsets (wave `w` issues wave-loads
// it * WAVES + w, each 1 KiB of LDS).
// `koff` is the stage's byte offset along k, applied through the instruction's scalar offset.
template <int WAVES, int LO, int HI, int N>
__device__ __forceinline__ void load_pre(i32x4 rs, char* lds, int wave, const uint32_t (&voff)[N], uint32_t koff) {
#pragma unroll
  for (int it = LO; it < HI; ++it) lds_dma16s(rs, lds_addr(lds + (it * WAVES + wave) * 1024), voff[it], koff);
}

// ---- kernels with a fixed issue order ------------------------------------------------------------
// WGM x WGN waves (4 or 8), each computing a WM x WN part of a BM x BN tile with TM x TN
// accumulator blocks, so an MFMA step (k16 for 32x32 blocks, k32 for 16x16) is TM*TN MFMAs against
// TM + TN fragment reads.  The LDS ring holds S stages of BK k; the loads of stage s + S go out
// right after the barrier that ends the reads of stage s, so every load has S - 1 stages of MFMA
// work to land.  Each step interleaves its MFMAs with the fragment reads of the next step and,
// where due, the HBM->LDS loads; sched_barrier fences keep exactly that order.  The stage barrier
// sits before a stage's last step: that step's fragments are already in registers, so its MFMAs
// cover the first reads of the next stage issued just after the barrier, and no wave starts a
// stage waiting on LDS.
//
// Barrier B(s+1), before the last step of stage s, certifies (i) every wave's loads of stage s + 1
// have landed (each wave waits for its own with vmcnt first) and (ii) every wave has read all of
// stage s (its last-step fragments were waited for), so its slot can take stage s + S.
//
// MF selects the matrix instruction: 32 for v_mfma_f32_32x32x16_bf16 (k16 steps, 32x32 blocks),
// 16 for v_mfma_f32_16x16x32_bf16 (k32 steps, 16x16 blocks).  Both run at the same rate per clock,
// but the 16x16 form draws less power, so the part holds a higher clock under it.
template <bool A_KM_, bool B_KM_, bool ACC, int S_, int WGM, int WGN_, int BK_, int BN_ = 256, int MF_ = 32, int BM_ = 256>
struct G4 {
  static constexpr bool A_KM = A_KM_, B_KM = B_KM_;
  static constexpr int S = S_, WGN = WGN_, MF = MF_;
  static constexpr int BM = BM_, BN = BN_, BK = BK_, WAVES = WGM * WGN, WM = BM / WGM, WN = BN / WGN;
  static constexpr int TM = WM / MF, TN = WN / MF;
  static constexpr int KS = 512 / MF;                   // k per MFMA step
  using OA = typename OpSel<A_KM, BM, BK, MF == 16 ? 1 : 0>::T;
  using OB = typename OpSel<B_KM, BN, BK, MF == 16 ? 1 : 0>::T;
  using AccT = std::conditional_t<MF == 32, f32x16, f32x4v>;
  static constexpr int kStage = OA::kBytes + OB::kBytes;
  static constexpr int LA = OA::kLoads / WAVES, LB = OB::kLoads / WAVES, LPS = LA + LB;
  static constexpr int kRing = S * kStage;
  static constexpr int kEpi = WAVES * EpiOf<WM, WN, ACC>::kBytes;
  static constexpr int kLds = kRing > kEpi ? kRing : kEpi;
  static_assert(OA::kLoads % WAVES == 0 && OB::kLoads % WAVES == 0, "loads per wave");
  static_assert(S >= 2 && kLds <= 160 * 1024, "ring");
};

// Per-lane LDS byte offset of the first fragment (32 rows from r0) of a K-major operand for k16
// step ks, relative to the operand's base in a stage.  The row swizzle repeats every 32 rows, so
// the other fragments add immediates; steps change the swizzled chunk and need their own offset.
template <class O>
__device__ __forceinline__ uint32_t kmaj_frag_off(int r0, int ks, int lane) {
  const int r = r0 + (lane & 31), c = ks * 2 + (lane >> 5);
  return uint32_t(r * O::kRowBytes + ((c ^ O::swz(r)) << 4));
}
// Same for an MN-major operand's first transposing read (k rows kb..kb+3 of step 0).  The chunk
// swizzle of these rows depends on k % 4 only, so steps (16 rows) and the second read (4 rows
// further) are immediates; fragments differ in their swizzled chunk and need their own offsets.
template <class O>
__device__ __forceinline__ uint32_t mnmaj_frag_off(int f0, int lane) {
  const int g = lane >> 4, s = lane & 15, j = s >> 2, q = s & 3;
  const int f = f0 + 16 * (g & 1) + 4 * q;
  const int k = 8 * (g >> 1) + j;
  return uint32_t(k * O::kRowBytes + (((f >> 3) ^ O::swz(k)) << 4) + ((f & 7) << 1));
}

// The 16x16x32 forms: a fragment is 16 rows (or free indices) x 32 k, lane l holding row l%16
// and k 8(l/16) .. 8(l/16)+7.  K-major: the swizzle repeats every 16 rows, so fragments add
// immediates and each k32 step has its own offset.  MN-major: the four 16-lane groups read k
// rows 8g .. 8g+3 (and 8g+4 .. 8g+7 in the second read) of the same 16 free indices.
template <class O>
__device__ __forceinline__ uint32_t kmaj_frag_off16(int r0, int ks, int lane) {
  const int r = r0 + (lane & 15), c = ks * 4 + (lane >> 4);
  return uint32_t(r * O::kRowBytes + ((c ^ O::swz(r)) << 4));
}
template <class O>
__device__ __forceinline__ uint32_t mnmaj_frag_off16(int f0, int lane) {
  const int g = lane >> 4, s = lane & 15, j = s >> 2, q = s & 3;
  const int f = f0 + 4 * q;
  const int k = 8 * g + j;
  return uint32_t(k * O::kRowBytes + (((f >> 3) ^ O::swz(k)) << 4) + ((f & 7) << 1));
}

template <int OFF>
__device__ __forceinline__ bf16x8 lds_rd128(uint32_t addr) {
  const auto* p = reinterpret_cast<const __attribute__((address_space(3))) uint4*>(addr + OFF);
  return __builtin_bit_cast(bf16x8, *p);
}
template <int OFF0, int OFF1>
__device__ __forceinline__ bf16x8 lds_rd_tr(uint32_t addr) {
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(uintptr_t)(addr + OFF0));
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(uintptr_t)(addr + OFF1));
  const short __attribute__((ext_vector_type(8))) v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8, v);
}

template <int N>
__device__ __forceinline__ void asm_wait_vm() { asm volatile("s_waitcnt vmcnt(%0)" : : "i"(N) : "memory"); }

// acc = the product of rows m0 .. of A and n0 .. of B over the k tiles kt0 .. kt0 + nk - 1 (at least S of them).
// G provides a, b, a_bytes, b_bytes, lda, ldb, M, N and K.  On return loads may be in flight and other waves may
// still read the ring.
template <class P, class G>
__device__ __forceinline__ void gemm4_core(const G& g, char* smem, int lane, int wave, int m0, int n0, int kt0, int nk,
                                           typename P::AccT (&acc)[P::TM][P::TN]) {
  constexpr bool A_KM = P::A_KM, B_KM = P::B_KM;
  constexpr int S = P::S, MF = P::MF, KS = P::KS, NACC = MF == 32 ? 16 : 4;
  using OA = typename P::OA;
  using OB = typename P::OB;
  constexpr int BK = P::BK, WAVES = P::WAVES, WM = P::WM, WN = P::WN, TM = P::TM, TN = P::TN;
  constexpr int LA = P::LA, LB = P::LB, LPS = P::LPS, kStage = P::kStage;
  const int wm = wave / P::WGN, wn = wave % P::WGN, nkt = (g.K + BK - 1) / BK;
  // The k tiles are walked from a starting point that depends on the XCD (blocks are dealt to
  // the XCDs round-robin): stage j of this split (0 <= j < nk) is k tile kmap(j), a rotation by
  // (3x mod 8) eighths of the split on XCD x (measured 1 % ahead of x eighths).  Without it every
  // workgroup of the chip loads the same k column of its rows at the same time; with rows a power
  // of two apart in HBM (K = 2048 or 8192 bf16), those loads pile onto the same memory channels.
  // The workgroups of one XCD keep one phase, so the operand panels they share in that XCD's L2
  // are still loaded once.  Each tile keeps one fixed k order, so results stay deterministic.
  const int rot = ((((int(blockIdx.x) % kXCD) * 3) % kXCD) * nk) / kXCD;
  auto kmap = [&](int j) { const int x = j + rot; return kt0 + (x >= nk ? x - nk : x); };

  const i32x4 ra = rsrc(g.a, g.a_bytes), rb = rsrc(g.b, g.b_bytes);
  // load offsets relative to a stage's first k; the ragged last stage (K % 32 != 0) uses a copy
  // with the lanes past K sent out of range
  uint32_t voa[LA], vob[LB], vra[LA], vrb[LB];
  OA::template prep<WAVES>(voa, lane, wave, m0, g.M, g.lda);
  OB::template prep<WAVES>(vob, lane, wave, n0, g.N, g.ldb);
  {
    const int kr = g.K - (nkt - 1) * BK;          // k extent of the last stage
#pragma unroll
    for (int it = 0; it < LA; ++it) {
      const int p = (it * WAVES + wave) * 64 + lane;
      const int kk = A_KM ? ((p % OA::kCPR) ^ OA::swz(p / OA::kCPR)) * 8 : p / OA::kCPR;
      vra[it] = kk < kr ? voa[it] : kOOB;
    }
#pragma unroll
    for (int it = 0; it < LB; ++it) {
      const int p = (it * WAVES + wave) * 64 + lane;
      const int kk = B_KM ? ((p % OB::kCPR) ^ OB::swz(p / OB::kCPR)) * 8 : p / OB::kCPR;
      vrb[it] = kk < kr ? vob[it] : kOOB;
    }
  }
  const uint32_t ka_step = A_KM ? BK * 2 : uint32_t(BK * g.lda * 2);
  const uint32_t kb_step = B_KM ? BK * 2 : uint32_t(BK * g.ldb * 2);
  const uint32_t lds0 = lds_addr(smem);

  // fragment read offsets (per lane), K-major: one per MFMA step; MN-major: one per fragment
  constexpr int NPS = BK / KS;
  uint32_t ofa[A_KM ? NPS : TM], ofb[B_KM ? NPS : TN];
  auto kfo_a = [&](int ks) { return MF == 32 ? kmaj_frag_off<OA>(wm * WM, ks, lane) : kmaj_frag_off16<OA>(wm * WM, ks, lane); };
  auto kfo_b = [&](int ks) { return MF == 32 ? kmaj_frag_off<OB>(wn * WN, ks, lane) : kmaj_frag_off16<OB>(wn * WN, ks, lane); };
  auto mfo_a = [&](int f0) { return MF == 32 ? mnmaj_frag_off<OA>(f0, lane) : mnmaj_frag_off16<OA>(f0, lane); };
  auto mfo_b = [&](int f0) { return MF == 32 ? mnmaj_frag_off<OB>(f0, lane) : mnmaj_frag_off16<OB>(f0, lane); };
  if constexpr (A_KM)
#pragma unroll
    for (int ks = 0; ks < NPS; ++ks) ofa[ks] = kfo_a(ks);
  else
#pragma unroll
    for (int i = 0; i < TM; ++i) ofa[i] = mfo_a(wm * WM + MF * i);
  if constexpr (B_KM)
#pragma unroll
    for (int ks = 0; ks < NPS; ++ks) ofb[ks] = OA::kBytes + kfo_b(ks);
  else
#pragma unroll
    for (int j = 0; j < TN; ++j) ofb[j] = OA::kBytes + mfo_b(wn * WN + MF * j);

#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < NACC; ++r) acc[i][j][r] = 0.f;
  bf16x8 fa[2][TM], fb[2][TN];

  // fragment i (A) or j (B) of MFMA step ks from the stage at LDS byte `base`
  auto read_a = [&](bf16x8& d, uint32_t base, auto ic_i, auto ic_ks) {
    constexpr int i = decltype(ic_i)::value, ks = decltype(ic_ks)::value;
    if constexpr (A_KM) d = lds_rd128<i * MF * OA::kRowBytes>(base + ofa[ks]);
    else d = lds_rd_tr<ks * KS * OA::kRowBytes, (ks * KS + 4) * OA::kRowBytes>(base + ofa[i]);
  };
  auto read_b = [&](bf16x8& d, uint32_t base, auto ic_j, auto ic_ks) {
    constexpr int j = decltype(ic_j)::value, ks = decltype(ic_ks)::value;
    if constexpr (B_KM) d = lds_rd128<j * MF * OB::kRowBytes>(base + ofb[ks]);
    else d = lds_rd_tr<ks * KS * OB::kRowBytes, (ks * KS + 4) * OB::kRowBytes>(base + ofb[j]);
  };
  // wave-load `l` (A: l < LA, then B) of the stage at k tile kt into LDS slot `slot`
  auto load_one = [&](auto ic_l, int kt, int slot, bool ragged) {
    constexpr int l = decltype(ic_l)::value;
    const uint32_t base = lds0 + slot * kStage;
    if constexpr (l < LA) {
      lds_dma16s(ra, base + (l * WAVES + wave) * 1024, ragged ? vra[l] : voa[l], uint32_t(kt) * ka_step);
    } else {
      constexpr int lb = l - LA;
      lds_dma16s(rb, base + OA::kBytes + (lb * WAVES + wave) * 1024, ragged ? vrb[lb] : vob[lb], uint32_t(kt) * kb_step);
    }
  };
  // Memory operation m of a step: m < NR reads fragment piece m into buffer NX; after that the
  // loads [L0, L0 + LPS/2) (or all LPS when ONE) of stage kt into slot `slot` (when `loads`).
  // ONE (the 16x16 kernels): a stage's loads all go out in the step right after the barrier that
  // frees its slot.  Under the 16x16 instruction the part clocks higher, a stage takes less time,
  // and loads issued a step later than that no longer land before the barrier that waits for them.
  constexpr bool ONE = MF == 16;
  constexpr int NR = TM + TN, LH = LPS / 2;
  static_assert(ONE || LPS % 2 == 0, "loads split over two steps");
  auto memop = [&](auto ic_m, auto ic_nx, auto ic_ks, auto ic_l0, uint32_t rbase, bool loads, int kt, int slot,
                   bool ragged) {
    constexpr int m = decltype(ic_m)::value, nx = decltype(ic_nx)::value, l0 = decltype(ic_l0)::value;
    if constexpr (m < NR) {
      if constexpr (m < TM) read_a(fa[nx][m], rbase, ic<m>{}, ic_ks);
      else read_b(fb[nx][m - TM], rbase, ic<m - TM>{}, ic_ks);
    } else {
      if (loads) load_one(ic<l0 + m - NR>{}, kt, slot, ragged);
    }
  };
  // One MFMA step: TM x TN MFMAs on buffer CUR with NM memory operations among them.  The
  // fragment reads go out over the first three quarters of the MFMAs, so they have landed when
  // the step ends (the stage barrier waits for them); the loads are spread evenly over the whole
  // step, one every NQ/NL MFMAs, which keeps the texture-address queue from filling.
  auto step = [&](auto ic_cur, auto ic_nm, auto&& mem) {
    constexpr int cur = decltype(ic_cur)::value, NM = decltype(ic_nm)::value;
    // MFMAs row by row over the A fragments, the B fragments in serpentine order (odd rows run j
    // backwards), so that every MFMA shares an operand with the one before it: the part is held
    // at its power limit, and fewer operand changes measured 0.3-0.6 % faster per launch on every
    // product.
    static_for<TM * TN>([&](auto qc) {
      constexpr int q = decltype(qc)::value, i = q / TN, j = (i & 1) ? TN - 1 - q % TN : q % TN;
      if constexpr (MF == 32)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[cur][j], fa[cur][i], acc[i][j], 0, 0, 0);
      else
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[cur][j], fa[cur][i], acc[i][j], 0, 0, 0);
      constexpr int NQ = TM * TN, NRD = NR < NM ? NR : NM, NL = NM - NRD;
      constexpr int RQ = NQ * 3 / 4 > 0 ? NQ * 3 / 4 : 1;
      constexpr int rlo = q < RQ ? q * NRD / RQ : NRD, rhi = q < RQ ? (q + 1) * NRD / RQ : NRD;
      static_for<rhi - rlo>([&](auto mc) { mem(ic<rlo + decltype(mc)::value>{}); });
      constexpr int llo = NL ? (2 * q * NL + NQ) / (2 * NQ) : 0, lhi = NL ? (2 * (q + 1) * NL + NQ) / (2 * NQ) : 0;
      static_for<lhi - llo>([&](auto mc) { mem(ic<NRD + llo + decltype(mc)::value>{}); });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  {
    // Prologue: stages 0..S-2 and the first half of stage S-1, or all S stages when ONE (the host
    // launches this kernel only when every split has at least S stages).  From then on the loads of
    // stage x are issued in the last step of stage x - S (just after the barrier that frees its
    // slot): all of them when ONE, else the first half there and the second in the first step of
    // stage x - S + 1.  Either way, at barrier B(s+1) the loads issued after stage s + 1's are the
    // S - 2 whole stages s + 2 .. s + S - 1.
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const bool rag = kmap(s) == nkt - 1;
      if (ONE || s < S - 1) static_for<LPS>([&](auto lc) { load_one(lc, kmap(s), s, rag); });
      else static_for<LH>([&](auto lc) { load_one(lc, kmap(s), s, rag); });
    }
    // stage 0 is complete once at most the later prologue stages' loads (S - 1 of them, the last
    // one only half issued unless ONE) are outstanding
    asm_wait_vm<ONE ? LPS * (S - 1) : LPS * (S - 2) + LH>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    static_for<TM>([&](auto ic_i) { read_a(fa[0][decltype(ic_i)::value], lds0, ic_i, ic<0>{}); });
    static_for<TN>([&](auto ic_j) { read_b(fb[0][decltype(ic_j)::value], lds0, ic_j, ic<0>{}); });
    __builtin_amdgcn_sched_barrier(0);

    // Stage s: steps 0 .. NPS-2, each on buffer t % 2 and reading step t + 1 into the other (the
    // first also issues the second half of stage s + S - 1); barrier; the last step on buffer 1
    // (NPS is even), reading the next stage's step 0 into buffer 0 and issuing the first half of
    // stage s + S into s's slot.  At the barrier the loads issued after the last one of stage
    // s + 1 are the S - 2 whole stages s + 2 .. s + S - 1.
    constexpr int NPS_ = BK / KS;
    static_assert(NPS_ % 2 == 0, "steps per stage");
    auto stage = [&](int s, auto ic_vm, auto ic_la, auto ic_lb, auto ic_last) {
      constexpr int VM = decltype(ic_vm)::value;
      constexpr bool LDA = decltype(ic_la)::value, LDB = decltype(ic_lb)::value, LAST = decltype(ic_last)::value;
      const int slot = s % S;
      const uint32_t cur = lds0 + slot * kStage;
      static_for<NPS_ - 1>([&](auto tc) {
        constexpr int t = decltype(tc)::value;
        constexpr bool ld = !ONE && LDA && t == 0;
        const int kt = kmap(s + S - 1), lslot = (s + S - 1) % S;
        const bool rag = kt == nkt - 1;
        step(ic<t % 2>{}, ic<ld ? NR + LH : NR>{},
             [&](auto ic_m) { memop(ic_m, ic<(t + 1) % 2>{}, ic<t + 1>{}, ic<LH>{}, cur, ld, kt, lslot, rag); });
      });
      if constexpr (!LAST) {
        asm_wait_vm<VM>();
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        const uint32_t nxt = lds0 + ((s + 1) % S) * kStage;
        const int kt = kmap(s + S);
        const bool rag = kt == nkt - 1;
        step(ic<1>{}, ic<LDB ? NR + (ONE ? LPS : LH) : NR>{},
             [&](auto ic_m) { memop(ic_m, ic<0>{}, ic<0>{}, ic<0>{}, nxt, LDB, kt, slot, rag); });
      } else {
        step(ic<1>{}, ic<0>{}, [&](auto) {});
      }
    };
    using T_ = std::true_type;
    using F_ = std::false_type;
    for (int s = 0; s < nk - S; ++s) stage(s, ic<LPS * (S - 2)>{}, T_{}, T_{}, F_{});
    // The last S stages issue no new stages (the first still completes stage nk - 1); stage
    // nk-S+j waits for stage nk-S+j+1, after which S-2-j whole stages remain outstanding.
    static_for<S>([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      if constexpr (j == S - 1) stage(nk - S + j, ic<0>{}, std::bool_constant<j == 0>{}, F_{}, T_{});
      else stage(nk - S + j, ic<(S - 2 - j) * LPS>{}, std::bool_constant<j == 0>{}, F_{}, F_{});
    });
  }
}

}  // namespace sl2
