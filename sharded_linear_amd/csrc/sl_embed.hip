// Vocabulary-parallel embedding (gfx950): lookup in a shard of the table, and its gradient into the
// fp32 buffer.
//
//   Y[t]          = bf16(scale * W[ids[t] - start])              zeros where the id is another rank's
//   main_grad[v] += scale * sum of dY[t] over ids[t] - start = v
//
// The lookup moves 4 H bytes a token and nothing else.  The gradient reads the rank's rows of dY once,
// and reads and writes once each row of main_grad that a token names; what stands between is to bring
// equal ids together, in an order that the same call always takes, without atomics on sums:
//
//  * Sort.  Ids fall into buckets by their low bits (frequent ids are neighbours in many vocabularies,
//    so ranges of ids would fill unevenly).  One workgroup per bucket walks all ids, which stay in L2:
//    it counts its own by (id, wave) in LDS, counts the ids of the buckets before it, which gives its
//    place in the sorted list without a word from any other workgroup, and walks again to write its
//    places.  A wave takes a fixed part of the list and ranks equal ids by lane, so the order is fixed.
//  * Sums.  The sorted list is cut into chunks of kChunk places.  A workgroup adds up its chunk's rows
//    in fp32 registers and writes each finished run of equal ids to main_grad; a run that crosses a
//    chunk's border goes to one of the chunk's two planes of partial sums.
//  * Join.  The chunks in which a crossing run begins are listed as the sums find them (the list's order is not fixed, and
//    no result depends on it); a workgroup adds the planes of such a run, 4 waves a contiguous part each, in order.
// 8192 tokens, half of them here, rows of 2048: sort 8.3 us, sums 13.6 (53 MB, 3.9 TB/s), join 5.0; the first and the last are
// chains of short loads behind each other, not bytes.
// Up to kFewTokens tokens one kernel does it all: a workgroup for each place whose id no earlier place has (1013 tokens, rows of
// 1032: 6.1 us, of which the walk over the ids is most).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "sharded_linear.h"
#include "sl_device.h"

namespace {

using sl2::bf16x8;

typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x8 widen(uint4 v) {
  const bf16x8 b = __builtin_bit_cast(bf16x8, v);
  return __builtin_convertvector(b, f32x8);
}

__device__ __forceinline__ uint4 narrow(f32x8 v) { return __builtin_bit_cast(uint4, __builtin_convertvector(v, bf16x8)); }

// Row of the shard that token t names, or -1.
template <typename I>
__device__ __forceinline__ int64_t local_row(const I* ids, int64_t t, int64_t start, int64_t V) {
  const int64_t id = int64_t(ids[t]);
  return id >= start && id - start < V ? id - start : -1;
}

// ---- lookup --------------------------------------------------------------------------------------
// LPR lanes to a row, so that a lane has four chunks of it where the row is long enough; they are all loaded before the first is
// stored.  8192 tokens, half of them here, in us with 8, 16, 32 and 64 lanes: rows of 2048 elements 11.6, 11.2, 10.2, 10.0; of 512
// 5.4, 5.2, 5.3, 5.8; of 256 4.4, 4.7, 4.7, 5.0.  Bound by HBM (33.5 MB written, up to as many read) for wide rows, by the launch
// for narrow ones.
template <int LPR, typename I>
__global__ void __launch_bounds__(256) embed_lookup(const I* __restrict__ ids, const uint4* __restrict__ W, uint4* __restrict__ Y,
                                                    int64_t T, int64_t V, int chunks, int64_t start, float scale) {
  for (int64_t t = int64_t(blockIdx.x) * (256 / LPR) + threadIdx.x / LPR; t < T; t += int64_t(gridDim.x) * (256 / LPR)) {
    const int64_t row = local_row(ids, t, start, V);
    const uint4* src = W + (row < 0 ? 0 : row) * chunks;       // loads stand behind no condition: each would be waited for
    uint4* dst = Y + t * chunks;
    for (int c0 = threadIdx.x % LPR; c0 < chunks; c0 += 4 * LPR) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = src[min(c0 + u * LPR, chunks - 1)];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = c0 + u * LPR;
        if (row < 0) v[u] = make_uint4(0, 0, 0, 0);
        if (c < chunks) dst[c] = scale == 1.0f || row < 0 ? v[u] : narrow(widen(v[u]) * scale);
      }
    }
  }
}

// ---- gradient: sort ------------------------------------------------------------------------------

constexpr int kSortWaves = 16;
constexpr int kSortBins = 1000;           // most ids of one bucket, kSortWaves counters each in LDS
// Sorted places to a workgroup of the sums, its rows all in flight: 4 took 29.5 us, 16 58.8 where 8 took 28.7 (8192 tokens, rows
// of 2048).
constexpr int kChunk = 8;
// Tokens up to which one kernel does it all.  In us, one kernel against three: 1024 tokens of a uniform vocabulary 8.1 and 13.8,
// 2048 12.7 and 16.3; but a frequent token's rows are one workgroup's there, and of skewed ids 1024 take 8.3 and 11.6, 1500
// 17.4 and 13.3.
constexpr int kFewTokens = 1024;

struct EmbedPlan {
  int bits;               // log2 of the number of buckets
  int64_t chunks;         // chunks of the longest sorted list
  int64_t cross_off, key_off, part_off, bytes;
};

// Buckets: 256, one workgroup a CU (a call of 8192 tokens, rows of 2048: 24.8 us; 128 buckets 27.1, 512 25.8), or as many as
// leave kSortBins ids to each.
EmbedPlan embed_plan(int64_t T, int64_t V, int64_t H) {
  EmbedPlan p{};
  if (T <= kFewTokens) return p;
  p.bits = 8;
  while ((V + (int64_t(1) << p.bits) - 1) >> p.bits > kSortBins) ++p.bits;
  p.chunks = (T + kChunk - 1) / kChunk;
  const int64_t list = (T * 4 + 255) / 256 * 256;
  p.key_off = 256 + list;                 // 256 bytes of header: the lengths of the sorted list and of the list of crossing runs
  p.cross_off = p.key_off + list;
  p.part_off = p.cross_off + (p.chunks * 4 + 255) / 256 * 256;
  p.bytes = p.part_off + p.chunks * 2 * H * 4;
  return p;
}

constexpr int kHeld = 8;                  // ids of a lane in flight, and held from the first walk to the second

template <typename I>
__global__ void __launch_bounds__(kSortWaves * 64) embed_sort(const I* __restrict__ ids, int64_t T, int64_t V, int64_t start,
                                                              int bits, int* __restrict__ head, int* __restrict__ order,
                                                              int* __restrict__ key) {
  extern __shared__ int count[];          // [bins][kSortWaves]
  __shared__ int wave_before[kSortWaves], wave_sum[kSortWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t bucket = blockIdx.x, mask = (int64_t(1) << bits) - 1;
  const int bins = int((V + mask) >> bits);
  for (int i = threadIdx.x; i < bins * kSortWaves; i += kSortWaves * 64) count[i] = 0;
  __syncthreads();
  // wave w walks places [t0, t1), 64 at a time
  const int64_t per = ((T + kSortWaves * 64 - 1) / (kSortWaves * 64)) * 64;
  const int64_t t0 = wave * per, t1 = t0 + per < T ? t0 + per : T;
  const uint32_t rows32 = start < (int64_t(1) << 31) ? uint32_t(V) : 0;      // rows that an id of 32 bits reaches
  int before = 0;                         // the rank's ids of smaller buckets in this lane's places
  int held[kHeld];                        // this lane's rows of the last kHeld groups walked
  auto load = [&](int64_t tb) {
    I id[kHeld];
    const I* from = ids + tb + lane;
    if (t1 - tb >= 64 * kHeld) {
#pragma unroll
      for (int u = 0; u < kHeld; ++u) id[u] = from[64 * u];
    } else {                              // behind a condition of its own each load would be waited for by itself
      const int last = int(t1 - tb) - 1;
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const int i = 64 * u + lane;
        id[u] = ids[tb + min(i, last)];
        if (i > last) id[u] = -1;
      }
    }
    // V is at most 2^24: below it, the difference has no wrap that a nonnegative id could bring about
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      if constexpr (sizeof(I) == 4) {
        const uint32_t r = uint32_t(id[u]) - uint32_t(start);
        held[u] = id[u] >= 0 && r < rows32 ? int(r) : -1;
      } else {
        const uint64_t r = uint64_t(id[u]) - uint64_t(start);
        held[u] = id[u] >= 0 && r < uint64_t(V) ? int(r) : -1;
      }
    }
  };
  for (int64_t tb = t0; tb < t1; tb += 64 * kHeld) {
    load(tb);
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int b = held[u] & int(mask);
      before += held[u] >= 0 && b < int(bucket);
      if (held[u] >= 0 && b == int(bucket)) atomicAdd(&count[(held[u] >> bits) * kSortWaves + wave], 1);
    }
  }
  for (int d = 1; d < 64; d <<= 1) before += __shfl_xor(before, d);
  if (lane == 0) wave_before[wave] = before;
  __syncthreads();
  // exclusive sums of the counters, (id, wave) in order: each thread a contiguous run of them
  const int total = bins * kSortWaves, each = (total + kSortWaves * 64 - 1) / (kSortWaves * 64);
  const int i0 = min(int(threadIdx.x) * each, total), i1 = min(i0 + each, total);
  int sum = 0;
  for (int i = i0; i < i1; ++i) sum += count[i];
  int incl = sum;
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  int base = 0, mine = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    base += wave_before[w];
    if (w < wave) base += wave_sum[w];
    mine += wave_sum[w];
  }
  if (threadIdx.x == 0 && bucket == mask) {
    int all = mine;
    for (int w = 0; w < kSortWaves; ++w) all += wave_before[w];
    head[0] = all;
    head[1] = 0;                          // runs that cross chunks, counted by the sums
  }
  int at = base + incl - sum;
  for (int i = i0; i < i1; ++i) {
    const int c = count[i];
    count[i] = at;
    at += c;
  }
  __syncthreads();
  if (mine == 0) return;
  // places: lanes with the same id take consecutive ones; only this wave moves its counters
  for (int64_t tb = t0; tb < t1; tb += 64 * kHeld) {
    if (per > 64 * kHeld) load(tb);
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      bool open = held[u] >= 0 && (held[u] & int(mask)) == int(bucket);
      const int bin = held[u] >> bits;
      uint64_t left = __ballot(open);
      while (left) {
        const int first = __builtin_ctzll(left);
        const int b = __builtin_amdgcn_readlane(bin, first);
        const bool same = open && bin == b;
        const uint64_t peers = __ballot(same);
        int* const counter = &count[b * kSortWaves + wave];
        const int at0 = __hip_atomic_load(counter, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        if (same) {
          const int place = at0 + __popcll(peers & ((uint64_t(1) << lane) - 1));
          order[place] = int(tb + 64 * u + lane);
          key[place] = held[u];
          open = false;
        }
        if (lane == first) __hip_atomic_store(counter, at0 + __popcll(peers), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        left &= ~peers;
      }
    }
  }
}

// ---- gradient: sums ------------------------------------------------------------------------------

__device__ __forceinline__ void add_row(float* g, f32x8 v) {
  float4* p = reinterpret_cast<float4*>(g);
  float4 a = p[0], b = p[1];
  p[0] = make_float4(a.x + v[0], a.y + v[1], a.z + v[2], a.w + v[3]);
  p[1] = make_float4(b.x + v[4], b.y + v[5], b.z + v[6], b.w + v[7]);
}

__device__ __forceinline__ void put_row(float* g, f32x8 v) {
  float4* p = reinterpret_cast<float4*>(g);
  p[0] = make_float4(v[0], v[1], v[2], v[3]);
  p[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A workgroup takes one chunk of the sorted list and blockDim.x * 8 columns; a thread owns 8 columns.
__global__ void __launch_bounds__(256) embed_sums(const uint4* __restrict__ dY, float* __restrict__ grad, int* __restrict__ head,
                                                  int* __restrict__ cross, const int* __restrict__ order, const int* __restrict__ key,
                                                  float* __restrict__ part, int64_t H, int slices, float scale) {
  const int64_t chunk = blockIdx.x / slices;
  const int n = head[0];
  const int64_t p0 = chunk * kChunk;
  if (p0 >= n) return;
  const int len = n - p0 < kChunk ? int(n - p0) : kChunk;
  if (threadIdx.x == 0 && blockIdx.x % slices == 0 && p0 + len < n && key[p0 + len] == key[p0 + len - 1] &&
      !(p0 > 0 && key[p0 - 1] == key[p0 + len]))
    cross[atomicAdd(&head[1], 1)] = int(chunk);          // a run begins in this chunk and goes on
  const int64_t col = (int64_t(blockIdx.x % slices) * blockDim.x + threadIdx.x) * 8;
  if (col >= H) return;
  const int64_t row_chunks = H / 8;
  uint4 v[kChunk];
#pragma unroll
  for (int i = 0; i < kChunk; ++i) v[i] = dY[int64_t(order[p0 + min(i, len - 1)]) * row_chunks + col / 8];
  bool open = p0 > 0 && key[p0 - 1] == key[p0];       // the current run began in an earlier chunk
  // the rows that this chunk finishes are read ahead, so that no store waits for a load
  float4 old[kChunk][2];
  bool ends[kChunk], whole[kChunk];
  int k[kChunk];
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    k[i] = key[p0 + min(i, len - 1)];
    ends[i] = i < len && (p0 + i + 1 >= n || key[p0 + i + 1] != k[i]);
    whole[i] = ends[i] && !open;
    if (ends[i]) open = false;
    const float4* p = reinterpret_cast<const float4*>(grad + int64_t(k[i]) * H + col);
    old[i][0] = p[0];
    old[i][1] = p[1];
  }
  f32x8 acc = {0, 0, 0, 0, 0, 0, 0, 0};
  bool first = p0 > 0 && key[p0 - 1] == key[p0];
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    if (i >= len) break;
    acc += widen(v[i]);
    if (whole[i]) {
      acc *= scale;
      const float4 a = old[i][0], b = old[i][1];
      put_row(grad + int64_t(k[i]) * H + col, f32x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w} + acc);
    } else if (ends[i] || i + 1 == len) {
      put_row(part + (chunk * 2 + (first ? 0 : 1)) * H + col, acc);
    }
    if (ends[i]) {
      acc = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
      first = false;
    }
  }
}

constexpr int kJoinWaves = 4;              // most runs have one or two planes: few waves to each, and many at once
constexpr int64_t kJoinBlocks = 2048;      // 8 a CU

// The runs that cross chunks: planes 2c + 1 (begins in chunk c) and 2k (goes on in chunk k > c).  Workgroups walk the
// list of (run, 512 columns).
__global__ void __launch_bounds__(kJoinWaves * 64) embed_join(float* __restrict__ grad, const int* __restrict__ head, const int* __restrict__ cross,
                                                              const int* __restrict__ key, const float* __restrict__ part,
                                                              int64_t H, int slices, float scale) {
  __shared__ f32x8 sums[kJoinWaves][64];
  const int64_t n = head[0], chunks = (n + kChunk - 1) / kChunk, items = int64_t(head[1]) * slices;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t x = blockIdx.x; x < items; x += gridDim.x) {
    const int64_t c = cross[x / slices];
    const int k = key[(c + 1) * kChunk];
    // Chunks c + 1 .. from hold the rest.  The chunks that begin with k follow each other, so 64 are asked at a time, in steps
    // that grow until one does not and shrink again.
    int64_t from = c + 1;
    for (int64_t step = 1; step > 0;) {
      const int64_t y = from + (lane + 1) * step;
      const uint64_t past = __ballot(y >= chunks || key[y * kChunk] != k);
      from += step * (past ? __builtin_ctzll(past) : 64);
      step = past ? step / 64 : step * 64;
    }
    const int64_t col = (x % slices * 64 + lane) * 8;
    const int64_t per = (from - c + kJoinWaves - 1) / kJoinWaves;
    const int64_t a0 = c + 1 + wave * per, a1 = a0 + per < from + 1 ? a0 + per : from + 1;
    auto plane = [&](int64_t i) {
      const float4* p = reinterpret_cast<const float4*>(part + i * H + col);
      const float4 a = p[0], b = p[1];
      return f32x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    };
    f32x8 acc = {0, 0, 0, 0, 0, 0, 0, 0};
    if (col < H) {
#pragma unroll 4
      for (int64_t y = a0; y < a1; ++y) acc += plane(2 * y);
      if (wave == 0) acc = plane(2 * c + 1) + acc;
    }
    sums[wave][lane] = acc;
    __syncthreads();
    if (wave == 0 && col < H) {
      for (int w = 1; w < kJoinWaves; ++w) acc += sums[w][lane];
      add_row(grad + int64_t(k) * H + col, acc * scale);
    }
    __syncthreads();
  }
}

// ---- gradient of few tokens ----------------------------------------------------------------------
// One launch.  The workgroup of place t leaves where an earlier place has its id; else it lists the places of that id in
// order and adds up their rows, its groups of `width` threads (8 columns each) every G-th row, eight in flight.
constexpr int kFewThreads = 512;

template <typename I>
__global__ void __launch_bounds__(kFewThreads) embed_few(const I* __restrict__ ids, const uint4* __restrict__ dY, float* __restrict__ grad, int T,
                                                         int64_t V, int64_t H, int64_t start, int width, int slices, float scale) {
  constexpr int kEach = kFewTokens / kFewThreads;
  __shared__ int places[kFewTokens], counts[kEach][kFewThreads / 64];
  __shared__ f32x8 sums[kFewThreads];
  const int t = blockIdx.x / slices, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = local_row(ids, t, start, V);
  if (row < 0) return;
  const I mine = ids[t];
  bool same[kEach], earlier = false;
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int p = u * kFewThreads + threadIdx.x;
    same[u] = p < T && ids[p] == mine;
    earlier |= same[u] && p < t;
  }
  if (__syncthreads_or(earlier)) return;
  uint64_t ballot[kEach];
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    ballot[u] = __ballot(same[u]);
    if (lane == 0) counts[u][wave] = __popcll(ballot[u]);
  }
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int u = 0; u < kEach; ++u)
#pragma unroll
    for (int w = 0; w < kFewThreads / 64; ++w) {
      if (w == wave && same[u]) places[n + __popcll(ballot[u] & ((uint64_t(1) << lane) - 1))] = u * kFewThreads + threadIdx.x;
      n += counts[u][w];
    }
  __syncthreads();
  const int groups = kFewThreads / width, group = threadIdx.x / width, at = threadIdx.x % width;
  const int64_t col = (int64_t(blockIdx.x % slices) * width + at) * 8;
  f32x8 acc = {0, 0, 0, 0, 0, 0, 0, 0};
  if (group < groups && col < H)
    for (int i = group; i < n; i += 8 * groups) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = dY[int64_t(places[min(i + u * groups, n - 1)]) * (H / 8) + col / 8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i + u * groups < n) acc += widen(v[u]);
    }
  if (n > 1) {
    sums[threadIdx.x] = acc;
    __syncthreads();
    if (group == 0)
      for (int g = 1; g < groups && g < n; ++g) acc += sums[g * width + at];
  }
  if (group == 0 && col < H) add_row(grad + row * H + col, acc * scale);
}

constexpr int64_t kMaxExtent = int64_t(1) << 31;
constexpr int64_t kMaxThreads = int64_t(1) << 32;
constexpr int64_t kMaxSorted = int64_t(1) << 26;         // tokens of one gradient call
constexpr int64_t kMaxRows = int64_t(1) << 24;           // of a shard: buckets x ids walked stay in proportion

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_embed(const void* ids, int32_t ids_bytes, int64_t T, int64_t V, int64_t H, int64_t start, float scale) {
  if (T < 0 || V < 0 || H < 0 || start < 0 || (ids_bytes != 4 && ids_bytes != 8) || !(scale - scale == 0.0f)) return SL_EINVAL;
  if (T >= kMaxExtent || V > kMaxRows || H >= kMaxExtent || H % 8) return SL_ESHAPE;
  if (T > 0 && H > 0 && !ids) return SL_EINVAL;
  return reinterpret_cast<uintptr_t>(ids) % uintptr_t(ids_bytes) ? SL_EALIGN : SL_OK;
}

template <int LPR>
void launch_lookup(hipStream_t st, const void* ids, int32_t ids_bytes, const void* W, void* Y, int64_t T, int64_t V, int chunks,
                   int64_t start, float scale) {
  int64_t blocks = (T + 256 / LPR - 1) / (256 / LPR);
  if (blocks > (1 << 20)) blocks = 1 << 20;
  const dim3 grid{unsigned(blocks)};
  const uint4* w = static_cast<const uint4*>(V > 0 ? W : Y);      // read, and not used, for a shard without rows
  uint4* y = static_cast<uint4*>(Y);
  if (ids_bytes == 4)
    hipLaunchKernelGGL((embed_lookup<LPR, int32_t>), grid, dim3(256), 0, st, static_cast<const int32_t*>(ids), w, y, T, V, chunks, start, scale);
  else
    hipLaunchKernelGGL((embed_lookup<LPR, int64_t>), grid, dim3(256), 0, st, static_cast<const int64_t*>(ids), w, y, T, V, chunks, start, scale);
}

}  // namespace

extern "C" int sl_embedding_fwd(void* stream, const void* ids, int32_t ids_bytes, const void* W, void* Y, int64_t T, int64_t V,
                                int64_t H, int64_t vocab_start, float scale) {
  const int e = check_embed(ids, ids_bytes, T, V, H, vocab_start, scale);
  if (e) return e;
  if (T == 0 || H == 0) return SL_OK;
  if (!Y || (V > 0 && !W)) return SL_EINVAL;
  if (!aligned16(W) || !aligned16(Y)) return SL_EALIGN;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int chunks = int(H / 8);
  (chunks > 128 ? launch_lookup<64> : chunks > 64 ? launch_lookup<32> : chunks > 32 ? launch_lookup<16> : launch_lookup<8>)(
      st, ids, ids_bytes, W, Y, T, V, chunks, vocab_start, scale);
  return hipGetLastError() == hipSuccess ? SL_OK : SL_EHIP;
}

extern "C" size_t sl_embedding_wgrad_workspace_bytes(int64_t T, int64_t V, int64_t H) {
  if (T <= 0 || V <= 0 || H <= 0 || T > kMaxSorted || V > kMaxRows || H >= kMaxExtent || H % 8) return 0;
  return size_t(embed_plan(T, V, H).bytes);
}

extern "C" int sl_embedding_wgrad_accum(void* stream, const void* ids, int32_t ids_bytes, const void* dY, float* main_grad, int64_t T,
                                        int64_t V, int64_t H, int64_t vocab_start, float scale, void* workspace,
                                        size_t workspace_bytes) {
  const int e = check_embed(ids, ids_bytes, T, V, H, vocab_start, scale);
  if (e) return e;
  if (T == 0 || H == 0 || V == 0) return SL_OK;
  if (!dY || !main_grad) return SL_EINVAL;
  if (!aligned16(dY) || !aligned16(main_grad)) return SL_EALIGN;
  if (T > kMaxSorted) return SL_ESHAPE;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int threads = H >= 2048 ? 256 : int((H / 8 + 63) / 64 * 64);
  const int64_t slices = (H + threads * 8 - 1) / (threads * 8);
  const uint4* dy = static_cast<const uint4*>(dY);
  if (T <= kFewTokens) {
    if (T * slices * kFewThreads >= kMaxThreads) return SL_ESHAPE;
    const dim3 grid(unsigned(T * slices)), block(kFewThreads);
    if (ids_bytes == 4)
      hipLaunchKernelGGL(embed_few<int32_t>, grid, block, 0, st, static_cast<const int32_t*>(ids), dy, main_grad, int(T), V, H, vocab_start, threads, int(slices), scale);
    else
      hipLaunchKernelGGL(embed_few<int64_t>, grid, block, 0, st, static_cast<const int64_t*>(ids), dy, main_grad, int(T), V, H, vocab_start, threads, int(slices), scale);
    return hipGetLastError() == hipSuccess ? SL_OK : SL_EHIP;
  }
  const EmbedPlan p = embed_plan(T, V, H);
  if (!workspace || !aligned16(workspace) || workspace_bytes < size_t(p.bytes)) return SL_EWORKSPACE;
  const int64_t join_slices = (H + 511) / 512;
  if (p.chunks * slices * threads >= kMaxThreads) return SL_ESHAPE;
  char* ws = static_cast<char*>(workspace);
  int* head = reinterpret_cast<int*>(ws);
  int* order = reinterpret_cast<int*>(ws + 256);
  int* key = reinterpret_cast<int*>(ws + p.key_off);
  int* cross = reinterpret_cast<int*>(ws + p.cross_off);
  float* part = reinterpret_cast<float*>(ws + p.part_off);
  const int bins = int((V + (int64_t(1) << p.bits) - 1) >> p.bits);
  const dim3 buckets(1u << p.bits), sort_threads(kSortWaves * 64);
  const size_t lds = size_t(bins) * kSortWaves * 4;
  if (ids_bytes == 4)
    hipLaunchKernelGGL(embed_sort<int32_t>, buckets, sort_threads, lds, st, static_cast<const int32_t*>(ids), T, V, vocab_start, p.bits, head, order, key);
  else
    hipLaunchKernelGGL(embed_sort<int64_t>, buckets, sort_threads, lds, st, static_cast<const int64_t*>(ids), T, V, vocab_start, p.bits, head, order, key);
  if (hipGetLastError() != hipSuccess) return SL_EHIP;
  hipLaunchKernelGGL(embed_sums, dim3(unsigned(p.chunks * slices)), dim3(threads), 0, st, dy, main_grad, head, cross, order, key, part, H,
                     int(slices), scale);
  if (hipGetLastError() != hipSuccess) return SL_EHIP;
  const int64_t most = (p.chunks - 1) * join_slices;     // crossing runs, at most
  hipLaunchKernelGGL(embed_join, dim3(unsigned(most < kJoinBlocks ? most : kJoinBlocks)), dim3(kJoinWaves * 64), 0, st, main_grad, head, cross, key,
                     part, H, int(join_slices), scale);
  return hipGetLastError() == hipSuccess ? SL_OK : SL_EHIP;
}
