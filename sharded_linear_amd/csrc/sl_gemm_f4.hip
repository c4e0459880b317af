// Products of two MXFP4 operands (gfx950): C = A . B^T with A[M][K], B[N][K] blocked along K.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes E2M1 codes with an E8M0 scale per 32 elements as they are
// stored.  Its operand layout for 4-bit data (checked on the hardware): lane l of a 32-row fragment
// holds row l % 32, elements [32 g, 32 g + 32) of the 64-wide k step for g = l / 32, which are one
// 16-byte chunk and exactly one scale block, whose scale byte the same lane supplies (any byte of a
// register, chosen by the instruction).
//
// Both operands go HBM -> LDS directly, 256 k elements (128 bytes of a row) to a stage, two stages
// deep, with 16-byte chunks XOR-swizzled by row.  At the fp4 rate a 256 x 256 tile's k step of 64
// takes 512 cycles of its four matrix units; with four waves of 128 x 128 it reads 32 KiB of
// fragments in that time and writes 16 KiB, 75 % of the LDS's 128 bytes a cycle, where eight waves of
// 128 x 64 would read 48 KiB and be bound by it.  So one wave runs on each SIMD, with 256
// accumulator registers, and has to hide its own latencies: while one k step's MFMAs run, one LDS
// read after each MFMA fetches the next step's fragments into a second set of registers.  The
// fragments of a stage's last step are in registers before its MFMAs start, so the barrier that
// hands the stage's slot over stands there, and the first fragments of the next stage and the loads of the
// stage after it are issued between that last step's MFMAs.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sl_device.h"
#include "sl_epi.h"
#include "sl_f4.h"

namespace sl2 {

constexpr int kF4Fmt = 4;                       // cbsz / blgp of E2M1 operands
constexpr int kF4Row = kF4StageK / 2;           // bytes of a row's stage
constexpr int kF4Blocks = kF4StageK / 32;       // scale blocks (and 16-byte chunks) of a row's stage

__device__ __forceinline__ int f4_swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

typedef int i32x2 __attribute__((ext_vector_type(2)));

// LDS reads by byte address
template <class T>
__device__ __forceinline__ T lds_read(uint32_t a) {
  return *reinterpret_cast<const __attribute__((address_space(3))) T*>(uintptr_t(a));
}
// A barrier alone: no counter is waited for, and no memory access moves across it.
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ i32x8 f4_operand(i32x4 v) {           // the 4-bit forms read the lower four registers
  return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}

// Block scales, two ways.  SC: where every row of scales starts 16-byte aligned (K % 512 == 0), the
// scales of two stages come at once, 16 bytes a row, into a double-buffered cache behind the
// operand slots.  Otherwise each stage brings, into its slot, the three aligned dwords that hold a row's 8 bytes,
// wherever they start, and the reader shifts them into place.
// One operand of a workgroup's tile: rows row0 .. row0 + R - 1 of a matrix of `rows` rows.
template <int R, int WAVES, bool SC>
struct F4Side {
  static constexpr int kLoads = R * kF4Row / 1024 / WAVES;       // code loads of a wave in a stage
  // scale loads of a wave, for a group of two stages or for one stage, and their LDS bytes: whole
  // rounds of the waves' loads, the surplus reading zeros
  static constexpr int kScaleLoads = (R * (SC ? 1 : 3) / 64 + WAVES - 1) / WAVES;
  static constexpr int kScaleBytes = kScaleLoads * WAVES * 64 * (SC ? 16 : 4);
  static_assert(R * kF4Row % (1024 * WAVES) == 0 && WAVES % 2 == 0, "loads per wave");
  i32x4 rc, rs;
  uint32_t voff, step, nb, rows, sbase;
  int chunk;

  __device__ __forceinline__ void init(const void* codes, const void* scales, int64_t row0, int64_t all, int64_t K,
                                       int lane, int wave) {
    nb = uint32_t(K / 32);
    rows = uint32_t(all - row0 < R ? all - row0 : R);
    // descriptors over this tile's rows: offsets fit 32 bits whatever the matrix's size, and rows
    // past the end read zeros
    rc = rsrc(static_cast<const char*>(codes) + row0 * (K / 2), rows * uint32_t(K / 2));
    const uintptr_t s = reinterpret_cast<uintptr_t>(scales) + uintptr_t(row0 * nb);
    sbase = uint32_t(s & 3);
    rs = rsrc(reinterpret_cast<const void*>(s & ~uintptr_t(3)), (sbase + rows * nb + 3) & ~3u);
    // wave-load wl = it * WAVES + wave covers rows 8 wl .. 8 wl + 7, 8 lanes a row; its swizzle depends
    // on the wave alone, since WAVES is even
    chunk = (lane & 7) ^ f4_swz(8 * wave + (lane >> 3));
    voff = uint32_t(8 * wave + (lane >> 3)) * uint32_t(K / 2) + uint32_t(chunk) * 16;
    step = uint32_t(8 * WAVES) * uint32_t(K / 2);
  }
  // lane offset of stage kt's code loads; chunks past the end of a row read zeros
  __device__ __forceinline__ uint32_t at(int kt) const {
    return uint32_t(kt) * kF4Blocks + uint32_t(chunk) < nb ? voff + uint32_t(kt) * kF4Row : kOOB;
  }
  __device__ __forceinline__ void load(uint32_t lds, uint32_t off, int it, int wave) const {
    lds_dma16(rc, lds + uint32_t(it * WAVES + wave) * 1024, off + uint32_t(it) * step);
  }
  // SC: wave-load q of scale group G: 16 bytes of rows 64 q .. 64 q + 63
  __device__ __forceinline__ void load_group(uint32_t lds, int q, int G, int lane) const {
    const uint32_t r = uint32_t(q * 64 + lane);
    lds_dma16(rs, lds + uint32_t(q) * 1024, r < rows && uint32_t(G) * 16 < nb ? r * nb + uint32_t(G) * 16 : kOOB);
  }
  // not SC: wave-load q of the stage's scale dwords [3][R]; dword d of row r holds bytes 4 d .. of the
  // aligned words that start at or below the row's first byte of this stage
  __device__ __forceinline__ void load_scales(uint32_t lds, int q, int kt, int lane) const {
    const uint32_t i = uint32_t(q * 64 + lane), d = i / R, r = i % R;
    const uint32_t a = ((sbase + r * nb + uint32_t(kt) * kF4Blocks) & ~3u) + d * 4;
    lds_dma4(rs, lds + uint32_t(q) * 256, d < 3 && r < rows && uint32_t(kt) * kF4Blocks < nb ? a : kOOB);
  }
};

template <int BM, int BN, int WGM, int WGN, bool ACC, bool SC>
struct F4Layout {
  static constexpr int WAVES = WGM * WGN;
  static constexpr int kCodes = (BM + BN) * kF4Row;
  using SA = F4Side<BM, WAVES, SC>;
  using SB = F4Side<BN, WAVES, SC>;
  static constexpr int kScaleB = kCodes + SA::kScaleBytes;       // not SC: B's scales in the slot, A's at kCodes
  static constexpr int kSlot = kCodes + (SC ? 0 : SA::kScaleBytes + SB::kScaleBytes);
  static constexpr int kCache = 2 * kSlot;
  static constexpr int kGroup = SA::kScaleBytes + SB::kScaleBytes;
  static constexpr int kRing = kCache + (SC ? 2 * kGroup : 0);
  static constexpr int kEpi = WAVES * EpiOf<BM / WGM, BN / WGN, ACC>::kBytes;
  static constexpr int kLds = kRing > kEpi ? kRing : kEpi;
  static_assert(kLds <= 160 * 1024, "LDS");
};

// The four scale bytes that lane group h needs of 8 consecutive ones, 2 ks + h in byte ks.
__device__ __forceinline__ int f4_pick(uint32_t lo, uint32_t hi, uint32_t sel) {
  return int(__builtin_amdgcn_perm(hi, lo, sel));
}

template <int BM, int BN, int WGM, int WGN, bool ACC, bool SC>
__global__ void __launch_bounds__(WGM * WGN * 64) gemm_f4(F4Args g) {
  using L = F4Layout<BM, BN, WGM, WGN, ACC, SC>;
  constexpr int WAVES = WGM * WGN, WM = BM / WGM, WN = BN / WGN, TM = WM / 32, TN = WN / 32;
  using SA = F4Side<BM, WAVES, SC>;
  using SB = F4Side<BN, WAVES, SC>;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const uint32_t lds = lds_addr(smem);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WGN, wn = wave % WGN;

  const int tiles_m = int((g.M + BM - 1) / BM), tiles_n = int((g.N + BN - 1) / BN);
  const int t = xcd_remap(blockIdx.x, tiles_m * tiles_n);
  const int group = t / (8 * tiles_n), first_m = group * 8, gsz = min(tiles_m - first_m, 8);
  const int tm = first_m + (t % (8 * tiles_n)) % gsz, tn = (t % (8 * tiles_n)) / gsz;
  const int m0 = tm * BM, n0 = tn * BN;
  const int split = blockIdx.z;
  const int nkt = int((g.K + kF4StageK - 1) / kF4StageK);
  const int kt0 = ACC ? split * g.kt_per_split : 0;
  const int kt1 = ACC ? min(nkt, kt0 + g.kt_per_split) : nkt;

  SA a;
  SB b;
  a.init(g.a, g.sa, m0, g.M, g.K, lane, wave);
  b.init(g.b, g.sb, n0, g.N, g.K, lane, wave);

  // fragment addresses: row r's chunk 2 ks + h sits in slot (2 ks + h) ^ swz(r) of the row's eight
  const int fr = lane & 31, h = lane >> 5;
  const uint32_t fa0 = lds + uint32_t(wm * WM + fr) * kF4Row + uint32_t((h ^ f4_swz(fr)) << 4);
  const uint32_t fb0 = lds + BM * kF4Row + uint32_t(wn * WN + fr) * kF4Row + uint32_t((h ^ f4_swz(fr)) << 4);
  const uint32_t sel = h ? 0x07050301u : 0x06040200u;

  auto load_group = [&](int G) {                                 // SC
    const uint32_t c = lds + L::kCache + uint32_t(G & 1) * L::kGroup;
#pragma unroll
    for (int it = 0; it < SA::kScaleLoads; ++it) a.load_group(c, it * WAVES + wave, G, lane);
#pragma unroll
    for (int it = 0; it < SB::kScaleLoads; ++it) b.load_group(c + SA::kScaleBytes, it * WAVES + wave, G, lane);
  };
  auto load_scales = [&](int kt, uint32_t slot) {                // not SC
#pragma unroll
    for (int it = 0; it < SA::kScaleLoads; ++it) a.load_scales(slot + L::kCodes, it * WAVES + wave, kt, lane);
#pragma unroll
    for (int it = 0; it < SB::kScaleLoads; ++it) b.load_scales(slot + L::kScaleB, it * WAVES + wave, kt, lane);
  };
  // the LDS words with the scales of row r, A's or B's, of a stage in half `par` of its group and in
  // slot `par`; and the register of scale bytes made of them
  struct Raw { uint32_t d[SC ? 2 : 3]; };
  auto read_scales = [&](auto is_a, int r, int kt, auto par) {
    constexpr bool A = decltype(is_a)::value != 0;
    Raw w;
    if constexpr (SC) {
      const i32x2 v = lds_read<i32x2>(lds + L::kCache + uint32_t((kt >> 1) & 1) * L::kGroup + (A ? 0 : SA::kScaleBytes) +
                                      uint32_t(r) * 16 + par.value * 8);
      w.d[0] = v[0];
      w.d[1] = v[1];
    } else {
      const uint32_t at = lds + par.value * L::kSlot + (A ? L::kCodes : L::kScaleB) + uint32_t(r) * 4;
#pragma unroll
      for (int d = 0; d < 3; ++d) w.d[d] = lds_read<uint32_t>(at + d * (A ? BM : BN) * 4);
    }
    return w;
  };
  auto make_scales = [&](auto is_a, const Raw& w, int r, int kt) -> int {
    if constexpr (SC) {
      return f4_pick(w.d[0], w.d[1], sel);
    } else {
      const uint32_t nb = a.nb, base = decltype(is_a)::value ? a.sbase : b.sbase;
      const uint32_t sh = (base + uint32_t(r) * nb) & 3;
      const int v = f4_pick(__builtin_amdgcn_alignbyte(w.d[1], w.d[0], sh), __builtin_amdgcn_alignbyte(w.d[2], w.d[1], sh), sel);
      // what follows a row's last block is another row's scale, perhaps a NaN: the zero codes there get 2^-127
      const int left = int(nb) - kt * kF4Blocks - h;
      return v & (left > 6 ? -1 : left > 4 ? 0xFFFFFF : left > 2 ? 0xFFFF : left > 0 ? 0xFF : 0);
    }
  };
  const int ar = wm * WM + fr, br = wn * WN + fr;                // this lane's first fragment rows

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // One stage, in slot P = (kt - kt0) % 2.  No branch stands inside (the loads past the last stage
  // read out of range, the reads past it are not used): the fixed order below holds within a basic block.
  constexpr int kReads = TM + TN, kMfma = TM * TN, kLoads = SA::kLoads + SB::kLoads;
  i32x4 fa[2][TM], fb[2][TN];
  int sca[TM], scb[TN];
  auto stage = [&](int kt, auto par) {
    constexpr int P = decltype(par)::value;
    const uint32_t cur = P * L::kSlot, nxt = L::kSlot - cur;
    Raw na[TM], nb[TN];
    static_for<4>([&](auto kc) {
      constexpr int ks = decltype(kc)::value, p = ks & 1;
      uint32_t oa = kOOB, ob = kOOB;
      if constexpr (ks == 3) {
        // this wave has read all of its slot, and its loads of the next stage have landed
        wait_lgkm0();
        wait_vmcnt<0>();
        bare_barrier();
        oa = kt + 2 < kt1 ? a.at(kt + 2) : kOOB;
        ob = kt + 2 < kt1 ? b.at(kt + 2) : kOOB;
        if constexpr (!SC) load_scales(kt + 2, lds + cur);
        else if constexpr (P == 0) load_group((kt + 2) >> 1);
      }
      const uint32_t ra = (ks == 3 ? fa0 + nxt : (fa0 ^ uint32_t((ks + 1) << 5)) + cur);
      const uint32_t rb = (ks == 3 ? fb0 + nxt : (fb0 ^ uint32_t((ks + 1) << 5)) + cur);
      // side operations of this step: fragment reads of the next one; in the last step also the next
      // stage's scales and the loads of the stage after it
      auto read = [&](auto nc) {
        constexpr int n = decltype(nc)::value;
        if constexpr (n < TN) fb[p ^ 1][n] = lds_read<i32x4>(rb + n * 32 * kF4Row);
        else if constexpr (n < kReads) fa[p ^ 1][n - TN] = lds_read<i32x4>(ra + (n - TN) * 32 * kF4Row);
        else if constexpr (ks == 3 && n < kReads + TN) nb[n - kReads] = read_scales(ic<0>{}, br + (n - kReads) * 32, kt + 1, ic<1 - P>{});
        else if constexpr (ks == 3 && n < 2 * kReads) na[n - kReads - TN] = read_scales(ic<1>{}, ar + (n - kReads - TN) * 32, kt + 1, ic<1 - P>{});
      };
      auto load = [&](auto nc) {
        constexpr int n = decltype(nc)::value;
        if constexpr (ks == 3 && n < SA::kLoads) a.load(lds + cur, oa, n, wave);
        else if constexpr (ks == 3 && n < kLoads) b.load(lds + cur + BM * kF4Row, ob, n - SA::kLoads, wave);
      };
      constexpr int kReadsPer = ks == 3 ? (4 * kReads + kMfma - 1) / kMfma : (kReads + kMfma - 1) / kMfma;
      constexpr int kLoadsPer = (kLoads + kMfma - 1) / kMfma;
      static_for<kMfma>([&](auto mc) {
        // odd rows run j backwards, so every MFMA shares an operand with the one before it
        constexpr int n = decltype(mc)::value, i = n / TN, j = (i & 1) ? TN - 1 - n % TN : n % TN;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f4_operand(fb[p][j]), f4_operand(fa[p][i]), acc[i][j],
                                                                    kF4Fmt, kF4Fmt, ks, scb[j], ks, sca[i]);
        static_for<kReadsPer>([&](auto rc) { read(ic<n * kReadsPer + decltype(rc)::value>{}); });
        static_for<kLoadsPer>([&](auto rc) { load(ic<n * kLoadsPer + decltype(rc)::value>{}); });
        __builtin_amdgcn_sched_barrier(0);
      });
    });
#pragma unroll
    for (int j = 0; j < TN; ++j) scb[j] = make_scales(ic<0>{}, nb[j], br + j * 32, kt + 1);
#pragma unroll
    for (int i = 0; i < TM; ++i) sca[i] = make_scales(ic<1>{}, na[i], ar + i * 32, kt + 1);
  };

  if (kt0 < kt1) {
    // stages kt0 (even) and kt0 + 1
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int kt = kt0 + s;
      const uint32_t slot = lds + s * L::kSlot, oa = kt < kt1 ? a.at(kt) : kOOB, ob = kt < kt1 ? b.at(kt) : kOOB;
      if constexpr (!SC) load_scales(kt, slot);
      else if (s == 0) load_group(kt >> 1);
#pragma unroll
      for (int it = 0; it < SA::kLoads; ++it) a.load(slot, oa, it, wave);
#pragma unroll
      for (int it = 0; it < SB::kLoads; ++it) b.load(slot + BM * kF4Row, ob, it, wave);
    }
    wait_vmcnt<kLoads>();
    bare_barrier();
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[0][j] = lds_read<i32x4>(fb0 + j * 32 * kF4Row);
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[0][i] = lds_read<i32x4>(fa0 + i * 32 * kF4Row);
#pragma unroll
    for (int j = 0; j < TN; ++j) scb[j] = make_scales(ic<0>{}, read_scales(ic<0>{}, br + j * 32, kt0, ic<0>{}), br + j * 32, kt0);
#pragma unroll
    for (int i = 0; i < TM; ++i) sca[i] = make_scales(ic<1>{}, read_scales(ic<1>{}, ar + i * 32, kt0, ic<0>{}), ar + i * 32, kt0);

    // an odd last stage is followed by one of zeros: with one exit the accumulators stay in place
    for (int kt = kt0; kt < kt1; kt += 2) {
      stage(kt, ic<0>{});
      stage(kt + 1, ic<1>{});
    }
  }
  wait_vmcnt<0>();
  __syncthreads();    // every wave is past its last operand read: the slots become epilogue space
  store_tile<WM, WN, TM, TN, ACC>(g, acc, smem, m0 + wm * WM, n0 + wn * WN, split, lane, wave);
}

template <int BM, int BN, int WGM, int WGN, bool ACC, bool SC>
int launch_f4_sc(hipStream_t st, const F4Args& g) {
  constexpr int lds = F4Layout<BM, BN, WGM, WGN, ACC, SC>::kLds;
  auto kfn = gemm_f4<BM, BN, WGM, WGN, ACC, SC>;
  static std::atomic<uint64_t> attr{0};
  if (smem_attr_once(reinterpret_cast<const void*>(kfn), lds, attr)) return -5;
  const int64_t tiles = (g.M + BM - 1) / BM * ((g.N + BN - 1) / BN);
  hipLaunchKernelGGL(kfn, dim3(unsigned(tiles), 1, ACC ? g.splits : 1), dim3(WGM * WGN * 64), lds, st, g);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

template <int BM, int BN, int WGM, int WGN, bool ACC>
int launch_f4(hipStream_t st, const F4Args& g) {
  const bool sc = g.K % 512 == 0 && ((reinterpret_cast<uintptr_t>(g.sa) | reinterpret_cast<uintptr_t>(g.sb)) & 15u) == 0;
  return sc ? launch_f4_sc<BM, BN, WGM, WGN, ACC, true>(st, g) : launch_f4_sc<BM, BN, WGM, WGN, ACC, false>(st, g);
}

template <bool ACC>
int dispatch_f4(hipStream_t st, const F4Args& g) {
  switch (g.cfg) {
    case 0: return launch_f4<256, 256, 2, 2, ACC>(st, g);
    case 1: return launch_f4<128, 128, 2, 2, ACC>(st, g);
    case 2: return launch_f4<256, 128, 2, 2, ACC>(st, g);
    default: return -1;
  }
}

}  // namespace sl2

int f4_gemm(hipStream_t st, const F4Args& g) { return sl2::dispatch_f4<false>(st, g); }

int f4_accum(hipStream_t st, const F4Args& g) { return sl2::dispatch_f4<true>(st, g); }
