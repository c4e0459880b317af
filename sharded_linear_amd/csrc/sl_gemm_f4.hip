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

// Block scales are 8 bytes a row and stage, far less than the 128-byte lines they lie in: direct loads
// to LDS of 16 bytes a row and two stages moved a line for every 16 bytes and cost 335 of a stage's 3150
// cycles, and where rows of scales start at odd addresses (4-byte pieces) 2100 of 5300.  So each thread
// loads its rows' scales of 8 stages (64 bytes a row) into registers ahead of time, and they go to
// LDS together when the 8 stages before them are done.  On the way a row's bytes are shifted into place
// and cut at the row's end, so any K and any address takes the same path.
template <int BM, int BN, int WGM, int WGN, bool ACC>
struct F4Layout {
  static constexpr int WAVES = WGM * WGN;
  static constexpr int kSlot = (BM + BN) * kF4Row;
  static constexpr int kRows = (BM + BN + WAVES * 64 - 1) / (WAVES * 64);   // rows of scales of a thread
  static constexpr int kCache = 2 * kSlot;
  static constexpr int kRing = kCache + kRows * WAVES * 64 * 8 * kF4Blocks;
  static constexpr int kEpi = WAVES * EpiOf<BM / WGM, BN / WGN, ACC>::kBytes;
  static constexpr int kLds = kRing > kEpi ? kRing : kEpi;
  static_assert(kLds <= 160 * 1024, "LDS");
};

// One operand of a workgroup's tile: rows row0 .. row0 + R - 1 of a matrix of `rows` rows.
template <int R, int WAVES>
struct F4Side {
  static constexpr int kLoads = R * kF4Row / 1024 / WAVES;       // code loads of a wave in a stage
  static_assert(R * kF4Row % (1024 * WAVES) == 0 && WAVES % 2 == 0, "loads per wave");
  i32x4 rc;
  uint32_t voff, step, nb;
  int chunk;

  __device__ __forceinline__ void init(const void* codes, int64_t row0, int64_t all, int64_t K, int lane, int wave) {
    nb = uint32_t(K / 32);
    // a descriptor over this tile's rows: offsets fit 32 bits whatever the matrix's size, and rows
    // past the end read zeros
    const uint32_t rows = uint32_t(all - row0 < R ? all - row0 : R);
    rc = rsrc(static_cast<const char*>(codes) + row0 * (K / 2), rows * uint32_t(K / 2));
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
};

// LDS place of the 8 scale bytes of stage u (0 .. 7 of its group) of row r: every 32 consecutive rows
// of a stage lie in distinct banks.
__device__ __forceinline__ uint32_t f4_scale_at(int r, int u) {
  return uint32_t(r) * (8 * kF4Blocks) + (uint32_t(u ^ ((r >> 2) & 7)) << 3);
}

// A row's scales of a group of 8 stages, as the 17 aligned dwords that hold their 64 bytes.
struct F4Scales {
  __amdgpu_buffer_rsrc_t rs;
  uint32_t first, nb;        // byte offset of the row's first scale in rs, and its scales
  uint32_t w[17];

  // row r of the tile at row0 (r < rows) of a matrix of scales; other rows hold zeros
  __device__ __forceinline__ void init(const void* scales, int64_t row0, uint32_t rows, uint32_t r, int64_t K) {
    nb = uint32_t(K / 32);
    const uintptr_t s = reinterpret_cast<uintptr_t>(scales) + uintptr_t(row0 * nb);
    const uint32_t low = uint32_t(s & 3);
    // the first and last word may hold up to 3 bytes beside the tile's scales; of a load that passes the
    // extent, the words inside arrive
    rs = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(s & ~uintptr_t(3)), 0, int((low + rows * nb + 3) & ~3u),
                                           kRsrcWord3);
    first = low + r * nb;
    if (r >= rows) nb = 0;
  }
  // stages kt .. kt + 7
  __device__ __forceinline__ void load(int kt) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const uint32_t off = uint32_t(kt) * kF4Blocks < nb ? (first + uint32_t(kt) * kF4Blocks) & ~3u : kOOB;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off + q * 16, 0, 0));
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * q + e] = v[e];
    }
    w[16] = __builtin_amdgcn_raw_buffer_load_b32(rs, off + 64, 0, 0);
  }
  // to row r of the cache at lds; CUT: the group that starts at stage kt passes the row's end
  template <bool CUT>
  __device__ __forceinline__ void store(uint32_t lds, int r, int kt) const {
    const uint32_t sh = first & 3;
    // what follows a row's last block is another row's scale, perhaps a NaN: the zero codes there get 2^-127
    const int left = int(nb) - kt * kF4Blocks;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      i32x2 d;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t v = __builtin_amdgcn_alignbyte(w[2 * u + e + 1], w[2 * u + e], sh);
        const int n = left - 4 * (2 * u + e);                    // bytes of this dword within the row
        d[e] = int(!CUT || n >= 4 ? v : n <= 0 ? 0u : v & (0xFFFFFFFFu >> (32 - 8 * n)));
      }
      *reinterpret_cast<__attribute__((address_space(3))) i32x2*>(uintptr_t(lds + f4_scale_at(r, u))) = d;
    }
  }
};

// The four scale bytes that lane group h needs of 8 consecutive ones, 2 ks + h in byte ks.
__device__ __forceinline__ int f4_pick(uint32_t lo, uint32_t hi, uint32_t sel) {
  return int(__builtin_amdgcn_perm(hi, lo, sel));
}

template <int BM, int BN, int WGM, int WGN, bool ACC>
__global__ void __launch_bounds__(WGM * WGN * 64) gemm_f4(F4Args g) {
  using L = F4Layout<BM, BN, WGM, WGN, ACC>;
  constexpr int WAVES = WGM * WGN, WM = BM / WGM, WN = BN / WGN, TM = WM / 32, TN = WN / 32;
  using SA = F4Side<BM, WAVES>;
  using SB = F4Side<BN, WAVES>;
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
  a.init(g.a, m0, g.M, g.K, lane, wave);
  b.init(g.b, n0, g.N, g.K, lane, wave);
  // row q of A's then B's rows belongs to thread q % threads; every wave's rows are of one operand
  F4Scales sc[L::kRows];
  const uint32_t rows_a = uint32_t(min(g.M - m0, int64_t(BM))), rows_b = uint32_t(min(g.N - n0, int64_t(BN)));
#pragma unroll
  for (int n = 0; n < L::kRows; ++n) {
    const int q0 = n * WAVES * 64 + wave * 64;
    if (q0 < BM) sc[n].init(g.sa, m0, rows_a, q0 + lane, g.K);
    else sc[n].init(g.sb, n0, rows_b, q0 - BM + lane, g.K);
  }

  // fragment addresses: row r's chunk 2 ks + h sits in slot (2 ks + h) ^ swz(r) of the row's eight
  const int fr = lane & 31, h = lane >> 5;
  const uint32_t fa0 = lds + uint32_t(wm * WM + fr) * kF4Row + uint32_t((h ^ f4_swz(fr)) << 4);
  const uint32_t fb0 = lds + BM * kF4Row + uint32_t(wn * WN + fr) * kF4Row + uint32_t((h ^ f4_swz(fr)) << 4);
  const uint32_t sel = h ? 0x07050301u : 0x06040200u;

  auto load_scales = [&](int kt) {
#pragma unroll
    for (int n = 0; n < L::kRows; ++n) sc[n].load(kt);
  };
  auto store_scales = [&](int kt) {
#pragma unroll
    for (int n = 0; n < L::kRows; ++n) {
      const uint32_t c = lds + L::kCache;
      if (kt * kF4Blocks + 8 * kF4Blocks <= int(g.K / 32)) sc[n].template store<false>(c, n * WAVES * 64 + tid, kt);
      else sc[n].template store<true>(c, n * WAVES * 64 + tid, kt);
    }
  };
  auto read_scales = [&](int r, int kt) { return lds_read<i32x2>(lds + L::kCache + f4_scale_at(r, (kt - kt0) & 7)); };
  auto make_scales = [&](i32x2 w) -> int { return f4_pick(w[0], w[1], sel); };
  const int ar = wm * WM + fr, br = BM + wn * WN + fr;          // this lane's first fragment rows, A's and B's

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
    i32x2 na[TM], nb[TN];
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
      }
      const uint32_t ra = (ks == 3 ? fa0 + nxt : (fa0 ^ uint32_t((ks + 1) << 5)) + cur);
      const uint32_t rb = (ks == 3 ? fb0 + nxt : (fb0 ^ uint32_t((ks + 1) << 5)) + cur);
      // side operations of this step: fragment reads of the next one; in the last step also the next
      // stage's scales and the loads of the stage after it
      auto read = [&](auto nc) {
        constexpr int n = decltype(nc)::value;
        if constexpr (n < TN) fb[p ^ 1][n] = lds_read<i32x4>(rb + n * 32 * kF4Row);
        else if constexpr (n < kReads) fa[p ^ 1][n - TN] = lds_read<i32x4>(ra + (n - TN) * 32 * kF4Row);
        else if constexpr (ks == 3 && n < kReads + TN) nb[n - kReads] = read_scales(br + (n - kReads) * 32, kt + 1);
        else if constexpr (ks == 3 && n < 2 * kReads) na[n - kReads - TN] = read_scales(ar + (n - kReads - TN) * 32, kt + 1);
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
    for (int j = 0; j < TN; ++j) scb[j] = make_scales(nb[j]);
#pragma unroll
    for (int i = 0; i < TM; ++i) sca[i] = make_scales(na[i]);
  };

  if (kt0 < kt1) {
    auto load_stage = [&](int kt, uint32_t slot) {
      const uint32_t oa = kt < kt1 ? a.at(kt) : kOOB, ob = kt < kt1 ? b.at(kt) : kOOB;
#pragma unroll
      for (int it = 0; it < SA::kLoads; ++it) a.load(slot, oa, it, wave);
#pragma unroll
      for (int it = 0; it < SB::kLoads; ++it) b.load(slot + BM * kF4Row, ob, it, wave);
    };
    load_scales(kt0);
    load_stage(kt0, lds);
    wait_vmcnt<0>();
    load_stage(kt0 + 1, lds + L::kSlot);
    store_scales(kt0);
    wait_lgkm0();
    bare_barrier();
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[0][j] = lds_read<i32x4>(fb0 + j * 32 * kF4Row);
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[0][i] = lds_read<i32x4>(fa0 + i * 32 * kF4Row);
#pragma unroll
    for (int j = 0; j < TN; ++j) scb[j] = make_scales(read_scales(br + j * 32, kt0));
#pragma unroll
    for (int i = 0; i < TM; ++i) sca[i] = make_scales(read_scales(ar + i * 32, kt0));

    // an odd last stage is followed by one of zeros: with one exit the accumulators stay in place
    for (int kt = kt0; kt < kt1; kt += 2) {
      const int u = (kt - kt0) & 7;
      if (u == 0) load_scales(kt + 8);
      stage(kt, ic<0>{});
      if (u == 6) {
        // the group's last scales are in registers once every wave is here; the next group's landed long
        // ago and is read after the coming stage's barrier
        wait_lgkm0();
        bare_barrier();
        store_scales(kt + 2);
      }
      stage(kt + 1, ic<1>{});
    }
  }
  wait_vmcnt<0>();
  __syncthreads();    // every wave is past its last operand read: the slots become epilogue space
  store_tile<WM, WN, TM, TN, ACC>(g, acc, smem, m0 + wm * WM, n0 + wn * WN, split, lane, wave);
}

template <int BM, int BN, int WGM, int WGN, bool ACC>
int launch_f4(hipStream_t st, const F4Args& g) {
  constexpr int lds = F4Layout<BM, BN, WGM, WGN, ACC>::kLds;
  auto kfn = gemm_f4<BM, BN, WGM, WGN, ACC>;
  static std::atomic<uint64_t> attr{0};
  if (smem_attr_once(reinterpret_cast<const void*>(kfn), lds, attr)) return -5;
  const int64_t tiles = (g.M + BM - 1) / BM * ((g.N + BN - 1) / BN);
  hipLaunchKernelGGL(kfn, dim3(unsigned(tiles), 1, ACC ? g.splits : 1), dim3(WGM * WGN * 64), lds, st, g);
  return hipGetLastError() == hipSuccess ? 0 : -5;
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
