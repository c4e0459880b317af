// Products of two MXFP4 operands (gfx950): C = A . B^T with A[M][K], B[N][K] blocked along K.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes E2M1 codes with an E8M0 scale per 32 elements as they are
// stored.  Its operand layout for 4-bit data (checked on the hardware): lane l of a 32-row fragment
// holds row l % 32, elements [32 g, 32 g + 32) of the 64-wide k step for g = l / 32, which are one
// 16-byte chunk and exactly one scale block, whose scale byte the same lane supplies (any byte of a
// register, chosen by the instruction).
//
// Both operands go HBM -> LDS directly, 256 k elements (128 bytes of a row) to a stage, S stages
// deep, with 16-byte chunks XOR-swizzled by row.  At the fp4 rate a 256 x 256 tile's k step of 64
// takes 512 cycles of its four matrix units; with four waves of 128 x 128 it reads 32 KiB of
// fragments in that time and writes 16 KiB, 75 % of the LDS's 128 bytes a cycle, where eight waves of
// 128 x 64 would read 48 KiB and be bound by it.  So one wave runs on each SIMD, with 256
// accumulator registers, and has to hide its own latencies: while one k step's MFMAs run, one LDS
// read after each MFMA fetches the next step's fragments into a second set of registers.  The
// fragments of a stage's last step are in registers before its MFMAs start, so the barrier that
// hands the stage's slot over stands there, and the first fragments of the next stage and the loads of the
// stage after it are issued between that last step's MFMAs.
//
// Measured: [8192, 4096] over 11008 184 us, 4.0 PFLOP/s; [8192, 8192] over 2048 85 us, 3.2 PFLOP/s, of which the
// results' 134 MB take 26; accumulating [11008, 4096] over 8192 237 us.  A loop of these MFMAs alone holds 6.4
// PFLOP/s (1.5-1.6 GHz, the power limit), this one without its loads 4.2-4.5.  In the first of these products the
// matrix units are busy 51 % of the cycles, at about 1.9 GHz: neither the power limit nor the LDS's bytes (75 % of
// that 51 %) hold it, but the waits of one wave a SIMD in its fixed order of reads, loads and products.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sl_device.h"
#include "sl_f4.h"
#include "sl_mx.h"

namespace sl2 {

constexpr int kF4Fmt = 4;                       // cbsz / blgp of E2M1 operands
constexpr int kF4Row = kF4StageK / 2;           // bytes of a row's stage
constexpr int kF4Blocks = kF4StageK / 32;       // scale blocks (and 16-byte chunks) of a row's stage

__device__ __forceinline__ int f4_swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// LDS reads by byte address
template <class T>
__device__ __forceinline__ T lds_read(uint32_t a) {
  return *reinterpret_cast<const __attribute__((address_space(3))) T*>(uintptr_t(a));
}
// Block scales are 8 bytes a row and stage, far less than the 128-byte lines they lie in: direct loads
// to LDS of 16 bytes a row and two stages moved a line for every 16 bytes and cost 335 of a stage's 3150
// cycles, and where rows of scales start at odd addresses (4-byte pieces) 2100 of 5300.  So each thread
// loads its rows' scales of 8 stages (64 bytes a row) into registers ahead of time, and they go to
// LDS together when the 8 stages before them are done.  On the way a row's bytes are shifted into place
// and cut at the row's end, so any K and any address takes the same path.
template <int BM, int BN, int WGM, int WGN, int S>
struct F4Layout {
  static constexpr int WAVES = WGM * WGN;
  static constexpr int kSlot = (BM + BN) * kF4Row;
  static constexpr int kRows = (BM + BN + WAVES * 64 - 1) / (WAVES * 64);   // rows of scales of a thread
  static constexpr int kCache = S * kSlot;
  static constexpr int kLds = kCache + kRows * WAVES * 64 * 8 * kF4Blocks;
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

  // a descriptor over the tile's rows: offsets fit 32 bits whatever the matrix's size, and rows past the
  // end read zeros
  __device__ __forceinline__ void set_rows(const void* codes, int row0, int all, int64_t K) {
    rc = rsrc_uniform(static_cast<const char*>(codes) + int64_t(row0) * (K / 2), uint32_t(min(all - row0, R)) * uint32_t(K / 2));
  }
  __device__ __forceinline__ void init(int64_t K, int lane, int wave) {
    nb = uint32_t(K / 32);
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
  uint32_t w[17];
  uint32_t sh;               // bytes before the group's first in w[0]
  int left;                  // the row's bytes from the group's first on, none for rows past the edge

  // stages kt .. kt + 7 of row r of the tile at row0, of a matrix of `all` rows; rows past the end hold zeros
  template <int R>
  __device__ __forceinline__ void load(const void* scales, int row0, int all, uint32_t r, int64_t K, int kt) {
    const uint32_t nb = uint32_t(K / 32), rows = uint32_t(min(all - row0, R));
    const uintptr_t s = reinterpret_cast<uintptr_t>(scales) + uintptr_t(int64_t(row0) * nb);
    const uint32_t low = uint32_t(s & 3);
    // the first and last word may hold up to 3 bytes beside the tile's scales; of a load that passes the
    // extent, the words inside arrive
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(s & ~uintptr_t(3)), 0,
                                                                        int((low + rows * nb + 3) & ~3u), kRsrcWord3);
    const uint32_t at = low + r * nb + uint32_t(kt) * kF4Blocks;
    sh = at & 3;
    left = r < rows ? int(nb) - kt * kF4Blocks : 0;
    const uint32_t off = left > 0 ? at & ~3u : kOOB;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off + q * 16, 0, 0));
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * q + e] = v[e];
    }
    w[16] = __builtin_amdgcn_raw_buffer_load_b32(rs, off + 64, 0, 0);
  }
  // to row r of the cache at lds; CUT: the group passes the row's end
  template <bool CUT>
  __device__ __forceinline__ void store(uint32_t lds, int r) const {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      i32x2 d;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t v = __builtin_amdgcn_alignbyte(w[2 * u + e + 1], w[2 * u + e], sh);
        // what follows a row's last block is another row's scale, perhaps a NaN: the zero codes there get 2^-127
        const int n = left - 4 * (2 * u + e);                    // bytes of this dword within the row
        d[e] = int(!CUT || n >= 4 ? v : n <= 0 ? 0u : v & (0xFFFFFFFFu >> (32 - 8 * n)));
      }
      *reinterpret_cast<__attribute__((address_space(3))) i32x2*>(uintptr_t(lds + f4_scale_at(r, u))) = d;
    }
  }
};

// v, as a value that the compiler computes with where it stands: what follows from it is not kept in
// registers through the loops around.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The four scale bytes that lane group h needs of 8 consecutive ones, 2 ks + h in byte ks.
__device__ __forceinline__ int f4_pick(uint32_t lo, uint32_t hi, uint32_t sel) {
  return int(__builtin_amdgcn_perm(hi, lo, sel));
}

// Stores a wave's blocks straight from the accumulators.  The MFMAs take the B fragment first, so lane l
// of block (i, j) has row 32 i + l % 32 and in registers 4q .. 4q + 3 the columns
// 32 j + 8 q + 4 (l / 32) + 0..3: 16 bytes of fp32 as they are; for bf16 the halves of the wave trade
// pieces, so that each lane has 8 columns.  No LDS is used: the next tile's stages land there meanwhile.
// Rows and columns past the edges go to offsets that the descriptors refuse, so that no branch stands
// between the blocks and few accumulators are read ahead.

// Keeps a block in its accumulator registers up to here: otherwise all of them are copied out together.
__device__ __forceinline__ void f4_pin(f32x16& v) { asm volatile("" : "+a"(v)); }

// Rows m .. m + 31 of a matrix of M rows of N elements of E bytes.
template <int E>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t f4_rows(const void* c, int64_t m, int64_t M, int64_t N) {
  const int rows = __builtin_amdgcn_readfirstlane(int(M - m < 0 ? 0 : M - m < 32 ? M - m : 32));
  return __builtin_amdgcn_make_buffer_rsrc(static_cast<char*>(const_cast<void*>(c)) + m * N * E, 0, rows * int(N) * E, kRsrcWord3);
}

template <int TM, int TN>
__device__ __forceinline__ void f4_store_bf16(const F4Args& g, f32x16 (&acc)[TM][TN], int m0, int n0, int lane) {
  const int h = lane / 32, n = n0 + 8 * h;
  const uint32_t off = uint32_t(lane % 32) * uint32_t(g.N) * 2 + uint32_t(n) * 2;
  static_for<TM>([&](auto ic_) {
    constexpr int i = decltype(ic_)::value;
    const __amdgpu_buffer_rsrc_t rs = f4_rows<2>(g.c, m0 + 32 * i, g.M, g.N);
    static_for<TN * 2>([&](auto jc) {
      constexpr int j = decltype(jc)::value / 2, q = decltype(jc)::value % 2 * 2;
      if constexpr (q == 0) f4_pin(acc[i][j]);
      uint32_t w[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          bf16x2 v;
          v[0] = static_cast<__bf16>(acc[i][j][4 * (q + e) + 2 * d]);
          v[1] = static_cast<__bf16>(acc[i][j][4 * (q + e) + 2 * d + 1]);
          w[e][d] = __builtin_bit_cast(uint32_t, v);
        }
      const auto s0 = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
      const auto s1 = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
      const u32x4 o = {s0[0], s1[0], s0[1], s1[1]};
      constexpr int c = j * 32 + 8 * q;
      __builtin_amdgcn_raw_buffer_store_b128(o, rs, n + c < g.N ? off + c * 2 : kOOB, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    });
  });
}

// fp32: added to C, or, with K split, stored to the split's plane, which the reduce kernel launched next
// on the stream adds up in split order.  Old values are loaded two blocks ahead.
template <bool ADD, int TM, int TN>
__device__ __forceinline__ void f4_store_f32(const F4Args& g, float* c, f32x16 (&acc)[TM][TN], int m0, int n0, int lane) {
  const int n = n0 + 4 * (lane / 32);
  const uint32_t off = uint32_t(lane % 32) * uint32_t(g.N) * 4 + uint32_t(n) * 4;
  constexpr int TB = TN / 2;                                     // batches of two blocks in a row of blocks
  u32x4 old[2][2][4];
  auto at = [&](int j, int q) { return n + j * 32 + 8 * q < g.N ? off + (j * 32 + 8 * q) * 4 : kOOB; };
  auto load = [&](int b, u32x4 (&o)[2][4]) {
    const __amdgpu_buffer_rsrc_t rs = f4_rows<4>(c, m0 + 32 * (b / TB), g.M, g.N);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[j][q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, at(b % TB * 2 + j, q), 0, 0));
  };
  if constexpr (ADD) load(0, old[0]);
  __builtin_amdgcn_sched_barrier(0);
  static_for<TM * TB>([&](auto bc) {
    constexpr int b = decltype(bc)::value, i = b / TB;
    if constexpr (ADD && b + 1 < TM * TB) load(b + 1, old[(b + 1) & 1]);
    __builtin_amdgcn_sched_barrier(0);
    const __amdgpu_buffer_rsrc_t rs = f4_rows<4>(c, m0 + 32 * i, g.M, g.N);
    static_for<8>([&](auto jc) {
      constexpr int jj = decltype(jc)::value / 4, j = b % TB * 2 + jj, q = decltype(jc)::value % 4;
      if constexpr (q == 0) f4_pin(acc[i][j]);
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = acc[i][j][4 * q + e];
        if constexpr (ADD) x += __uint_as_float(old[b & 1][jj][q][e]);
        v[e] = __float_as_uint(x);
      }
      __builtin_amdgcn_raw_buffer_store_b128(v, rs, at(j, q), 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    });
  });
}

// What a workgroup computes at a time: a tile over the stages [kt0, kt1).
struct F4Item { int m0, n0, kt0, kt1, split; };

// A workgroup takes several items, and the stages of one follow those of the item before without a
// gap: during an item's last S stages the loads are the next one's, so only the results' stores
// stand between the matrix instructions of two items.
template <int BM, int BN, int WGM, int WGN, int S, bool ACC>
__global__ void __launch_bounds__(WGM * WGN * 64) gemm_f4(F4Args g) {
  using L = F4Layout<BM, BN, WGM, WGN, S>;
  constexpr int WAVES = WGM * WGN, WM = BM / WGM, WN = BN / WGN, TM = WM / 32, TN = WN / 32;
  using SA = F4Side<BM, WAVES>;
  using SB = F4Side<BN, WAVES>;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const uint32_t lds = lds_addr(smem);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WGN, wn = wave % WGN;

  // Consecutive workgroups go to the 8 XCDs in turn.  Each XCD takes a contiguous range of the items,
  // its workgroups side by side in it, so that what runs there at a time shares rows in its L2: 6 tiles
  // down, then across (over 8 down, 2-3 % shorter with bf16 results and 5-11 % in accumulating 8192 x 8192;
  // 4 and 16 down are no better).
  constexpr int kDown = 6;
  const int tiles_m = int((g.M + BM - 1) / BM), tiles_n = int((g.N + BN - 1) / BN), tiles = tiles_m * tiles_n;
  const int nkt = int((g.K + kF4StageK - 1) / kF4StageK);
  auto item = [&](int x) {
    F4Item it;
    it.split = ACC ? x / tiles : 0;
    const int t = ACC ? x % tiles : x;
    const int group = t / (kDown * tiles_n), first_m = group * kDown, gsz = min(tiles_m - first_m, kDown);
    it.m0 = (first_m + (t % (kDown * tiles_n)) % gsz) * BM;
    it.n0 = (t % (kDown * tiles_n)) / gsz * BN;
    it.kt0 = ACC ? it.split * g.kt_per_split : 0;
    it.kt1 = ACC ? min(nkt, it.kt0 + g.kt_per_split) : nkt;
    it.m0 = __builtin_amdgcn_readfirstlane(it.m0);
    it.n0 = __builtin_amdgcn_readfirstlane(it.n0);
    return it;
  };
  const int items = tiles * (ACC ? g.splits : 1), xcd = blockIdx.x % kXCD;
  const int per = items / kXCD, rem = items % kXCD;
  const int end = (xcd + 1) * per + min(xcd + 1, rem), stride = (int(gridDim.x) - xcd + kXCD - 1) / kXCD;
  int x = xcd * per + min(xcd, rem) + int(blockIdx.x) / kXCD;
  if (x >= end) return;

  // fragment addresses: row r's chunk 2 ks + h sits in slot (2 ks + h) ^ swz(r) of the row's eight
  const int fr = lane & 31, h = lane >> 5;
  const uint32_t fa0 = lds + uint32_t(wm * WM + fr) * kF4Row + uint32_t((h ^ f4_swz(fr)) << 4);
  const uint32_t fb0 = lds + BM * kF4Row + uint32_t(wn * WN + fr) * kF4Row + uint32_t((h ^ f4_swz(fr)) << 4);
  const uint32_t sel = h ? 0x07050301u : 0x06040200u;

  // row q of A's then B's rows belongs to thread q % threads; every wave's rows are of one operand
  F4Scales sc[L::kRows];
  bool cut = false;                                              // the group held passes the rows' end
  auto load_scales = [&](const F4Item& it, int kt) {
    const int l = here(lane);
#pragma unroll
    for (int n = 0; n < L::kRows; ++n) {
      const int q0 = n * WAVES * 64 + wave * 64;
      if (q0 < BM) sc[n].template load<BM>(g.sa, it.m0, int(g.M), q0 + l, g.K, kt);
      else sc[n].template load<BN>(g.sb, it.n0, int(g.N), q0 - BM + l, g.K, kt);
    }
    cut = (kt + 8) * kF4Blocks > int(g.K / 32);
  };
  auto store_scales = [&]() {
    const int t = here(tid);
#pragma unroll
    for (int n = 0; n < L::kRows; ++n) {
      if (cut) sc[n].template store<true>(lds + L::kCache, n * WAVES * 64 + t);
      else sc[n].template store<false>(lds + L::kCache, n * WAVES * 64 + t);
    }
  };
  auto read_scales = [&](int r, int u) { return lds_read<i32x2>(lds + L::kCache + f4_scale_at(r, u)); };
  auto make_scales = [&](i32x2 w) -> int { return f4_pick(w[0], w[1], sel); };
  const int ar = wm * WM + fr, br = BM + wn * WN + fr;          // this lane's first fragment rows, A's and B's

  f32x16 acc[TM][TN];

  // the operands of the item being loaded, its next stage and its end
  SA a;
  SB b;
  a.init(g.K, lane, wave);
  b.init(g.K, lane, wave);
  int lkt = 0, lend = 0;
  auto load_from = [&](const F4Item& it) {
    a.set_rows(g.a, it.m0, int(g.M), g.K);
    b.set_rows(g.b, it.n0, int(g.N), g.K);
    lkt = it.kt0;
    lend = it.kt1;
  };

  // One stage, in slot P of two, or in the slot at `slot`.  u: the next stage's place in its scale group.  No branch stands inside (loads
  // past the last stage read out of range, reads past it are not used): the fixed order below holds
  // within a basic block.
  constexpr int kReads = TM + TN, kMfma = TM * TN, kLoads = SA::kLoads + SB::kLoads;
  i32x4 fa[2][TM], fb[2][TN];
  int sca[TM], scb[TN];
  uint32_t slot = 0;
  auto stage = [&](int u, auto par) __attribute__((always_inline)) {
    constexpr int P = decltype(par)::value;
    const uint32_t cur = S == 2 ? uint32_t(P * L::kSlot) : slot;
    const uint32_t nxt = S == 2 ? L::kSlot - cur : cur == (S - 1) * L::kSlot ? 0 : cur + L::kSlot;
    slot = nxt;
    i32x2 na[TM], nb[TN];
    static_for<4>([&](auto kc) {
      constexpr int ks = decltype(kc)::value, p = ks & 1;
      uint32_t oa = kOOB, ob = kOOB;
      if constexpr (ks == 3) {
        // this wave has read all of its slot, and its loads of the next stage have landed
        wait_lgkm0();
        wait_vmcnt<(S - 2) * kLoads>();
        bare_barrier();
        oa = lkt < lend ? a.at(lkt) : kOOB;
        ob = lkt < lend ? b.at(lkt) : kOOB;
        ++lkt;
      }
      const uint32_t ra = (ks == 3 ? fa0 + nxt : (fa0 ^ uint32_t((ks + 1) << 5)) + cur);
      const uint32_t rb = (ks == 3 ? fb0 + nxt : (fb0 ^ uint32_t((ks + 1) << 5)) + cur);
      // side operations of this step: fragment reads of the next one; in the last step also the next
      // stage's scales and the loads of the stage after that
      auto read = [&](auto nc) {
        constexpr int n = decltype(nc)::value;
        if constexpr (n < TN) fb[p ^ 1][n] = lds_read<i32x4>(rb + n * 32 * kF4Row);
        else if constexpr (n < kReads) fa[p ^ 1][n - TN] = lds_read<i32x4>(ra + (n - TN) * 32 * kF4Row);
        else if constexpr (ks == 3 && n < kReads + TN) nb[n - kReads] = read_scales(br + (n - kReads) * 32, u);
        else if constexpr (ks == 3 && n < 2 * kReads) na[n - kReads - TN] = read_scales(ar + (n - kReads - TN) * 32, u);
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
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f4_operand(fb[p][j]), f4_operand(fa[p][i]),
                                                                    acc[i][j], kF4Fmt, kF4Fmt, ks, scb[j], ks, sca[i]);
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

  F4Item cur = item(x);
  auto load_stage = [&](uint32_t to) {
    const uint32_t oa = lkt < lend ? a.at(lkt) : kOOB, ob = lkt < lend ? b.at(lkt) : kOOB;
    ++lkt;
#pragma unroll
    for (int it = 0; it < SA::kLoads; ++it) a.load(to, oa, it, wave);
#pragma unroll
    for (int it = 0; it < SB::kLoads; ++it) b.load(to + BM * kF4Row, ob, it, wave);
  };
  load_scales(cur, cur.kt0);
  load_from(cur);
  load_stage(lds);
  wait_vmcnt<0>();
#pragma unroll
  for (int i = 1; i < S; ++i) load_stage(lds + i * L::kSlot);
  store_scales();
  wait_lgkm0();
  bare_barrier();
#pragma unroll
  for (int j = 0; j < TN; ++j) fb[0][j] = lds_read<i32x4>(fb0 + j * 32 * kF4Row);
#pragma unroll
  for (int i = 0; i < TM; ++i) fa[0][i] = lds_read<i32x4>(fa0 + i * 32 * kF4Row);
#pragma unroll
  for (int j = 0; j < TN; ++j) scb[j] = make_scales(read_scales(br + j * 32, 0));
#pragma unroll
  for (int i = 0; i < TM; ++i) sca[i] = make_scales(read_scales(ar + i * 32, 0));

  for (;;) {
    x += stride;
    const bool more = x < end;
    const F4Item nx = item(more ? x : x - stride);
    // Stages in pairs: an odd last one is followed by one of zeros (an empty K is a pair of zeros), so
    // that the accumulators stay in place.
    const int nk = max(S, (cur.kt1 - cur.kt0 + 1) & ~1);
    // a zero that is made here: a constant one is kept in registers of its own and copied
    const float zero = __int_as_float(here(0));
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = zero;
    for (int k = 0; k < nk; k += 2) {
      const bool last = k + 2 == nk;
      if ((k & 7) == 0) {
        if (k + 8 < nk) load_scales(cur, cur.kt0 + k + 8);
        else load_scales(nx, nx.kt0);
      }
      if (k + S == nk) {                                         // from this stage on the loads are the next item's
        load_from(nx);
        if (!more) lend = lkt;
      }
      stage((k + 1) & 7, ic<0>{});
      if (last || (k & 7) == 6) {
        // the group's last scales are in registers once every wave is here; those of the next landed
        // before the stage's barrier, and are read after the coming stage's
        wait_lgkm0();
        bare_barrier();
        store_scales();
      }
      stage(last ? 0 : (k + 2) & 7, ic<1>{});
    }
    const int l = here(lane);
    const int m = cur.m0 + wm * WM, n = cur.n0 + wn * WN;
    if constexpr (!ACC) f4_store_bf16<TM, TN>(g, acc, m, n, l);
    else if (g.splits == 1) f4_store_f32<true, TM, TN>(g, static_cast<float*>(g.c), acc, m, n, l);
    else f4_store_f32<false, TM, TN>(g, g.ws + int64_t(cur.split) * g.M * g.N, acc, m, n, l);
    if (!more) break;
    cur = nx;
  }
  wait_vmcnt<0>();   // loads past the end still write zeros to LDS
}

template <int BM, int BN, int WGM, int WGN, int S, bool ACC>
int launch_f4(hipStream_t st, const F4Args& g) {
  constexpr int lds = F4Layout<BM, BN, WGM, WGN, S>::kLds;
  constexpr int kResident = 256 * (160 * 1024 / lds);            // workgroups on the 256 CUs at a time
  auto kfn = gemm_f4<BM, BN, WGM, WGN, S, ACC>;
  static std::atomic<uint64_t> attr{0};
  if (smem_attr_once(reinterpret_cast<const void*>(kfn), lds, attr)) return -5;
  const int64_t items = (g.M + BM - 1) / BM * ((g.N + BN - 1) / BN) * (ACC ? g.splits : 1);
  hipLaunchKernelGGL(kfn, dim3(unsigned(items < kResident ? items : kResident)), dim3(WGM * WGN * 64), lds, st, g);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

template <bool ACC>
int dispatch_f4(hipStream_t st, const F4Args& g) {
  switch (g.cfg) {
    case 0: return launch_f4<256, 256, 2, 2, 2, ACC>(st, g);
    case 1: return launch_f4<128, 128, 2, 2, 2, ACC>(st, g);
    default: return launch_f4<128, 128, 2, 2, 4, ACC>(st, g);
  }
}

// y = the splits' sums in order, rounded once
__global__ void __launch_bounds__(256) join_f4(const float* part, __bf16* y, int64_t n4, int splits) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n4) return;
  f32x4v v = reinterpret_cast<const f32x4v*>(part)[i];
  for (int s = 1; s < splits; ++s) v += reinterpret_cast<const f32x4v*>(part)[s * n4 + i];
  bf16x4 o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = static_cast<__bf16>(v[e]);
  reinterpret_cast<bf16x4*>(y)[i] = o;
}

}  // namespace sl2

int f4_join(hipStream_t st, void* y, const float* part, int64_t n, int splits) {
  hipLaunchKernelGGL(sl2::join_f4, dim3(unsigned((n / 4 + 255) / 256)), dim3(256), 0, st, part, static_cast<__bf16*>(y), n / 4, splits);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

int f4_gemm(hipStream_t st, const F4Args& g) { return sl2::dispatch_f4<false>(st, g); }

int f4_accum(hipStream_t st, const F4Args& g) { return sl2::dispatch_f4<true>(st, g); }
