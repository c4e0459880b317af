// Operand tiles in LDS, their loads and their fragment reads, of the 16-bit GEMM kernels with direct HBM->LDS staging (gfx950):
// shared by the bf16 kernels of the linear step (sl_gemm2.hip) and the fp16 kernels of the orthogonalised update
// (sl_gemm_h.hip), whose main loops are their own.
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
template <bool A_KM, bool B_KM_, bool ACC, int S_, int WGM, int WGN_, int BK_, int BN_ = 256, int MF = 32, int BM_ = 256>
struct G4 {
  static constexpr bool B_KM = B_KM_;
  static constexpr int S = S_, WGN = WGN_;
  static constexpr int BM = BM_, BN = BN_, BK = BK_, WAVES = WGM * WGN, WM = BM / WGM, WN = BN / WGN;
  static constexpr int TM = WM / MF, TN = WN / MF;
  static constexpr int KS = 512 / MF;                   // k per MFMA step
  using OA = typename OpSel<A_KM, BM, BK, MF == 16 ? 1 : 0>::T;
  using OB = typename OpSel<B_KM, BN, BK, MF == 16 ? 1 : 0>::T;
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

}  // namespace sl2
