// Products of bf16 activations with an MXFP4 weight W[out][in] blocked along in (gfx950), for more rows
// than sl_rows_f4.hip takes and fewer than pay for a bf16 copy of the weight:
//   forward  Y[T][out] = X[T][in] . W^T        input gradient  dX[T][in] = dY[T][out] . W
//
// A workgroup of 8 waves computes 64 tokens x 128 features over steps of 128 contracted elements; the waves
// share a step out along the contraction too and add their sums through LDS at the end.  Forward: four waves
// of 64 x 32 for each half of a step (101 registers, so that two workgroups fit on a CU; four waves of whole
// steps wait for their own LDS reads, 1.1 us a step against 0.75, and waves of 32 x 64 expand every block
// twice: 200 tokens by [4096, 5504] 33.8 us against 30.8).  Gradient: two waves of 64 x 64 for each quarter,
// which read a third less from LDS (58.6 -> 54.4 us for 200 tokens by [8192, 2048] unsplit; LDS is busy half
// of the time, the matrix unit a quarter).  Reading a step's fragments while the step before is multiplied
// (170 registers) gained nothing.  Activations, codes and scales go HBM -> LDS directly, three steps deep.
// Small grids split the contraction: f32 planes, added in order by a second launch.  The gradient takes these tiles
// for any number of tokens: one token through [8192, 2048] 12.1 us and 3.5 for the join.
//   forward: a lane's share of 16 weight rows is one 16-byte chunk, a whole scale block, made bf16 in
//     registers (exact); the j-th of the step's four v_mfma_f32_16x16x32_bf16 contracts elements
//     8 j .. 8 j + 7 of every lane's block, and the activations are read from LDS in that order.
//   gradient: the contraction runs down the weight's rows, so each thread expands one 32-element block to
//     bf16 in LDS, a step ahead of the products, and the fragments are read transposed
//     (ds_read_b64_tr_b16); 64-byte pieces of rows 8 .. 15 of 16 are swapped, so that the four groups of 8
//     rows that one read takes lie in distinct banks by pairs.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sl_device.h"
#include "sl_f4.h"
#include "sl_mx.h"

namespace sl2 {

constexpr int kTM = kW4TileT, kTN = kW4TileN, kTK = kW4StepK, kTSlots = 3, kTWaves = 8;
constexpr int kTX = kTM * kTK * 2;                               // bytes of a step's activations
constexpr int kTCodes = 128 * 64;                                // of its codes, and behind them
constexpr int kTW = kTCodes + kTWaves * 256;                     // the aligned dwords [2][128 rows] around its scales (half unused)
constexpr int kTRow = kTN * 2 + 32;                              // row of expanded weights: 4 rows x 4 column quads in distinct banks
constexpr int kTXLoads = kTX / 1024 / kTWaves, kTLoads = kTXLoads + kTCodes / 1024 / kTWaves + 1;   // loads of a wave in a step

template <bool DG>
__global__ void __launch_bounds__(kTWaves * 64) tile_w4(F4RowsArgs g) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];  // activations [3], codes and scales [3], expanded weights [2]
  char* const wslots = smem + kTSlots * kTX;
  char* const wtiles = wslots + kTSlots * kTW;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // a wave: kNI * 16 features over kKS * 32 elements of a step
  constexpr int kNI = DG ? 4 : 2, kKS = DG ? 1 : 2, kWN = kTN / (kNI * 16);
  const int kp = wave / kWN, wn = wave % kWN;
  const int tiles_m = int((g.T + kTM - 1) / kTM);
  const int x = xcd_remap(blockIdx.x, gridDim.x);               // workgroups of one weight tile side by side on an XCD
  const int tiles_n = int((g.N + kTN - 1) / kTN);
  const int t0 = x % tiles_m * kTM, n0 = x / tiles_m % tiles_n * kTN;
  const int split = x / tiles_m / tiles_n;
  const int K = int(g.K), nb = int((DG ? g.N : g.K) / 32);      // contracted extent; scale blocks of a weight row
  const int k0 = split * g.steps_per_split;                     // first step
  const int left = (K + kTK - 1) / kTK - k0, steps = left < g.steps_per_split ? left : g.steps_per_split;

  const int rows_t = int(g.T) - t0 < kTM ? int(g.T) - t0 : kTM;
  const i32x4 rx = rsrc(static_cast<const char*>(g.x) + int64_t(t0) * K * 2, uint32_t(rows_t) * uint32_t(K) * 2);
  // The weight's rows of a step: forward the tile's features, columns on; gradient the step's 128 contracted
  // rows, the tile's columns.  wp, sp: the first row's codes and scales of the next load; rows: those left.
  const int row0 = DG ? k0 * kTK : n0;
  const char* wp = static_cast<const char*>(g.w) + int64_t(row0) * nb * 16;
  uintptr_t sp = reinterpret_cast<uintptr_t>(g.ws) + uintptr_t(int64_t(row0) * nb);
  int rows = __builtin_amdgcn_readfirstlane((DG ? K : int(g.N)) - row0);
  const uint32_t sbase = uint32_t(sp);

  // this lane's places in the loads
  const int xr = wave * 4 + lane / 16, xc = (lane % 16) ^ (xr & 15);      // + 32 rows in the second activation load
  uint32_t xoff = uint32_t(xr) * uint32_t(K) * 2 + uint32_t(xc) * 16 + uint32_t(k0) * (kTK * 2);
  const uint32_t xstep = 32u * uint32_t(K) * 2;
  int xleft = K - xc * 8 - k0 * kTK;                                       // elements from this lane's chunk to the row's end
  const int wr = wave * 16 + lane / 4, wc = (lane % 4) ^ ((wr >> 1) & 3);
  const int c0 = DG ? n0 / 32 : 4 * k0;                         // first block column
  uint32_t woff = uint32_t(wr * nb + wc + c0) * 16;
  int wleft = nb - wc - c0;                     // blocks from this lane's to the row's end
  const int sr = wave < 4 ? (wave & 1) * 64 + lane : 1 << 24;   // waves 4 .. 7 load nothing
  uint32_t soff = ((sbase & 3) + uint32_t(sr & 127) * uint32_t(nb) + uint32_t(c0) & ~3u) + 4 * (uint32_t(wave) >> 1 & 1);

  auto load_x = [&](uint32_t slot) {
    const uint32_t lds = lds_addr(smem) + slot * kTX;
    const uint32_t o = xleft > 0 ? xoff : kOOB;                  // past the last step too
    lds_dma16(rx, lds + uint32_t(wave) * 1024, o);
    lds_dma16(rx, lds + uint32_t(8 + wave) * 1024, o + xstep);
    xoff += kTK * 2;
    xleft -= kTK;
  };
  auto load_w = [&](uint32_t slot) {
    const uint32_t lds = lds_addr(wslots) + slot * kTW;
    const int n = rows < 0 ? 0 : rows < 128 ? rows : 128;
    lds_dma16(rsrc_uniform(wp, uint32_t(n * nb) * 16), lds + uint32_t(wave) * 1024, wleft > 0 ? woff : kOOB);
    const uint32_t low = uint32_t(sp & 3);
    lds_dma4(rsrc_uniform(reinterpret_cast<const void*>(sp & ~uintptr_t(3)), (low + uint32_t(n * nb) + 3) & ~3u),
             lds + kTCodes + uint32_t(wave) * 256, sr < n && (DG || wleft + wc > 0) ? soff : kOOB);
    if constexpr (DG) {
      wp += int64_t(128) * nb * 16;
      sp += uintptr_t(int64_t(128) * nb);
      rows -= 128;
    } else {
      woff += 64;
      soff += 4;
      wleft -= 4;
    }
  };
  // The four scale bytes of weight row r of the step in a slot.  128 rows and 4 blocks are multiples of 4 bytes, so
  // their place in the words does not depend on the step.
  auto scales = [&](const char* slot, int r) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(slot + kTCodes);
    return __builtin_amdgcn_alignbyte(p[128 + r], p[r], (sbase + uint32_t(r) * uint32_t(nb)) & 3);
  };
  auto next = [](uint32_t slot) { return slot == kTSlots - 1 ? 0 : slot + 1; };

  const int q = lane >> 4, l16 = lane & 15;
  f32x4v acc[kNI][4] = {};
  // gradient: this thread's block of a step, row tid / 4, block tid % 4, to an expanded tile; 16-byte pieces
  // are swapped by the block, so that the writes lie in distinct banks
  auto expand = [&](const char* slot, char* wt) {
    const int r = tid >> 2, b = tid & 3;
    const uint4 v = *reinterpret_cast<const uint4*>(slot + r * 64 + ((b ^ ((r >> 1) & 3)) << 4));
    const float sc = e8m0_to_f32((scales(slot, r) >> (8 * b)) & 0xFFu);
    const uint32_t c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<bf16x8*>(wt + r * kTRow + (b ^ (r >> 2 & 2)) * 64 + ((e ^ b) << 4)) = f4_to_bf16x8(c[e], sc);
  };
  if constexpr (DG) load_w(2);                                  // step 0, expanded before the loop
  load_x(0);
  load_w(0);
  if constexpr (DG) {
    wait_vmcnt<kTLoads>();
    lds_barrier();
    expand(wslots + 2 * kTW, wtiles);
  }
  load_x(1);
  load_w(1);
  uint32_t cur = 0;                                             // slots: activations of step s; gradient: codes of step s + 1
  for (int s = 0; s < steps; ++s) {
    // these have landed, the next step's may be on their way; the reads and expansions of the step before are done
    wait_vmcnt<kTLoads>();
    lds_barrier();
    const uint32_t free = next(next(cur));
    load_x(free);
    load_w(free);
    const char *slot = smem + cur * kTX, *wslot = wslots + cur * kTW;
    cur = next(cur);
    auto act = [&](int j, int c) {                               // 8 elements of token 16 j + l16, chunk c of the step
      const int r = j * 16 + l16;
      return *reinterpret_cast<const bf16x8*>(slot + r * (kTK * 2) + ((c ^ (r & 15)) << 4));
    };
    if constexpr (!DG) {
      uint32_t code[kNI][2];
      float sc[kNI];
#pragma unroll
      for (int i = 0; i < kNI; ++i) {
        const int r = (wn * kNI + i) * 16 + l16;
        const uint2 v = *reinterpret_cast<const uint2*>(wslot + r * 64 + ((q ^ ((r >> 1) & 3)) << 4) + 8 * kp);
        code[i][0] = v.x; code[i][1] = v.y;
        // past the row's end the codes are zeros and the scale another row's, perhaps a NaN
        const uint32_t b = (scales(wslot, r) >> (8 * q)) & 0xFFu;
        sc[i] = e8m0_to_f32(4 * (k0 + s) + q < nb ? b : 0u);
      }
      // every read before the first product: a wave's own LDS latency is met once a step
      bf16x8 xf[kKS][4];
#pragma unroll
      for (int j = 0; j < kKS; ++j)
#pragma unroll
        for (int m = 0; m < 4; ++m) xf[j][m] = act(m, 4 * q + kKS * kp + j);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < kKS; ++j)
#pragma unroll
        for (int i = 0; i < kNI; ++i) {
          const bf16x8 w = f4_to_bf16x8(code[i][j], sc[i]);
#pragma unroll
          for (int m = 0; m < 4; ++m) acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, xf[j][m], acc[i][m], 0, 0, 0);
        }
    } else {
      const uint32_t wt = lds_addr(wtiles) + uint32_t(s & 1) * (128 * kTRow);
      bf16x8 xf[4], wf[kNI];
#pragma unroll
      for (int m = 0; m < 4; ++m) xf[m] = act(m, 4 * kp + q);
#pragma unroll
      for (int i = 0; i < kNI; ++i) {
        // rows 8 q .. 8 q + 7 of this quarter, column 16 i + l16: two reads of 4 rows
        const int b = wn * 2 + (i >> 1), piece = (i & 1) * 2 + (l16 >> 1 & 1), r = 32 * kp + 8 * q + (l16 >> 2);
        const uint32_t a = wt + uint32_t(r) * kTRow + uint32_t((b ^ (2 * q & 2)) * 64 + ((piece ^ b) << 4) + 8 * (l16 & 1));
        const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4q*)(uintptr_t)a));
        const uint2 hi = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4q*)(uintptr_t)(a + 4 * kTRow)));
        wf[i] = __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
      }
      __builtin_amdgcn_sched_barrier(0);
      expand(wslot, wtiles + ((s + 1) & 1) * (128 * kTRow));     // the next step's
#pragma unroll
      for (int i = 0; i < kNI; ++i)
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[i], xf[m], acc[i][m], 0, 0, 0);
    }
  }
  // the sums of a step's parts through LDS: the upper half of the waves to the lower, then, of quarters, the second's
  wait_vmcnt<0>();
  f32x4v* const part = reinterpret_cast<f32x4v*>(smem) + (wave & 3) * kNI * 4 * 64 + lane;
  auto put = [&]() {
#pragma unroll
    for (int i = 0; i < kNI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) part[(i * 4 + j) * 64] = acc[i][j];
  };
  auto add = [&](const f32x4v* p) {
#pragma unroll
    for (int i = 0; i < kNI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += p[(i * 4 + j) * 64];
  };
  lds_barrier();
  if (wave >= 4) put();
  lds_barrier();
  if (wave < 4) add(part);
  if constexpr (kWN == 2) {
    if (kp == 1) put();
    lds_barrier();
    if (kp == 0) add(part + 2 * kNI * 4 * 64);
  }
  if (kp > 0) return;
  // lane l of block (i, j): token 16 j + l % 16, features 16 i + 4 (l / 16) + 0..3
#pragma unroll
  for (int i = 0; i < kNI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + j * 16 + l16, n = n0 + (wn * kNI + i) * 16 + 4 * q;
      const f32x4v v = acc[i][j];
      if (t < g.T && n < g.N) {
        if (g.splits > 1) {
          *reinterpret_cast<f32x4v*>(g.part + (int64_t(split) * g.T + t) * g.N + n) = v;
        } else {
          bf16x4 o;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = static_cast<__bf16>(v[e]);
          *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(g.y) + t * g.N + n) = o;
        }
      }
    }
}

template <bool DG>
int launch_tile_w4(hipStream_t st, const F4RowsArgs& g) {
  constexpr int lds = kTSlots * (kTX + kTW) + (DG ? 2 * 128 * kTRow : 0);
  static_assert(lds <= 160 * 1024, "LDS");
  static std::atomic<uint64_t> attr{0};
  if (smem_attr_once(reinterpret_cast<const void*>(tile_w4<DG>), lds, attr)) return -5;
  const int64_t tiles = (g.T + kTM - 1) / kTM * ((g.N + kTN - 1) / kTN);
  hipLaunchKernelGGL(tile_w4<DG>, dim3(unsigned(tiles * g.splits)), dim3(kTWaves * 64), lds, st, g);
  if (g.splits > 1) {
    if (hipGetLastError() != hipSuccess) return -5;
    return f4_join(st, g.y, g.part, g.T * g.N, g.splits);
  }
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace sl2

int w4_tile_fwd(hipStream_t st, const F4RowsArgs& g) { return sl2::launch_tile_w4<false>(st, g); }

int w4_tile_dgrad(hipStream_t st, const F4RowsArgs& g) { return sl2::launch_tile_w4<true>(st, g); }
