// Tokens into expert order and back: a stable counting sort of the (token, rank) slots by
// expert, the copy of every token's row to its slots' places (moe_permute), the weighted sum
// of the slots' rows back into tokens (moe_unpermute), and both gradients. All of it is bound
// by memory: nothing is computed on a row but one multiply-add per element, so each kernel
// touches every row once with 16-byte accesses and keeps its sums in fp32 registers.
//
// Rows are addressed with the strides the caller gives. gfx950 reads and writes 16 bytes at
// element alignment, so odd widths and strides take the same instructions as aligned ones;
// only the last, partial vector of a row goes element by element.
#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "group_count.h"
#include "hmoe_internal.h"

namespace hmoe {

// ---------------------------------------------------------------------------
// counting sort of n ids over G groups
// ---------------------------------------------------------------------------

// threads of a sort block: every wave keeps a counter per group in LDS, so 16 waves up to
// kSortWideGroups groups (41 KB of counters), 4 waves beyond. 4 waves also for up to
// kSortFewIds ids, whose barriers cost less: the adapters' backward pass (2048 -> 1536, rank 8)
// takes 15.3 us so and 17.6 with 16 waves at 64 rows of 8, 25.8 and 24.5 at 1500 of 2
constexpr int kSortWide = 1024, kSortNarrow = 256, kSortWideGroups = 640, kSortFewIds = 1024;
// up to this many ids one block counts and places; more ids are counted and placed by
// several blocks of kSortChunk ids in two launches
constexpr int kSortOneBlock = 8192, kSortChunk = 2048;

struct SortArgs {
  const int32_t* ids;
  int n, G;
  int groups;           // G, or G + 1 when ids outside [0, G) form a group of their own
  int chunk;            // ids per block
  int nb;               // blocks
  int32_t* counts;      // [nb, groups] (nb > 1)
  int32_t* sorted;
  int32_t* slot_row;    // may be null
  int32_t* off;         // [groups + 1]
  int tile_rows;        // rows per tile of the tile table (0: no table)
  int max_tiles;
  SortTile* tile;
  int32_t* tile_first;  // [groups + 1]
  SortTranspose turn;
};

// inclusive sum over the block of one value per thread; *total: the block's sum
template <int THREADS>
__device__ __forceinline__ int block_scan(int v, int* s_part, int* total) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == kWave - 1) s_part[wave] = v;
  __syncthreads();
  int p = lane < THREADS / kWave ? s_part[lane] : 0;
#pragma unroll
  for (int o = 1; o < THREADS / kWave; o <<= 1) {
    const int u = __shfl_up(p, o);
    if (lane >= o) p += u;
  }
  *total = __shfl(p, THREADS / kWave - 1);
  const int add = wave ? __shfl(p, wave - 1) : 0;
  return v + add;
}

// per-block group counts of a sort over several blocks
__global__ __launch_bounds__(kSortWide) void sort_count_kernel(SortArgs a) {
  __shared__ int32_t s_cnt[kMaxGroups + 1];
  for (int e = threadIdx.x; e < a.groups; e += kSortWide) s_cnt[e] = 0;
  __syncthreads();
  const int c0 = min((long)blockIdx.x * a.chunk, (long)a.n), c1 = min(c0 + (long)a.chunk, (long)a.n);
  const int bits = group_bits(a.groups);
  for (int s0 = c0; s0 < c1; s0 += kSortWide) {
    const int s = s0 + (int)threadIdx.x;
    count_groups(s < c1 ? sort_key(a.ids[s], a.G, a.groups) : -1, bits, s_cnt);
  }
  __syncthreads();
  int32_t* out = a.counts + (size_t)blockIdx.x * a.groups;
  for (int e = threadIdx.x; e < a.groups; e += kSortWide) out[e] = s_cnt[e];
}

// 16 bytes at element alignment
struct __attribute__((packed, aligned(2))) Raw16 {
  uint32_t w[4];
};

// Eight columns of eight ranks a thread, turned in registers: 16-byte reads and writes. Threads
// run over the ranks first, so that eight of them share a row's 128 bytes (rank 64) on the way
// in and eight on the way out: 48 adapters of 4096 x 64 (50 MB moved) in 16 us with the sort, 32
// with the columns first.
__device__ __forceinline__ void transpose_block(const SortTranspose& t, long i) {
  const int nb = t.N / 8, rb = t.r / 8;
  if (i >= (long)t.G * rb * nb) return;
  const int k = (int)(i % rb);
  const long gb = i / rb, g = gb / nb;
  const int b = (int)(gb % nb);
  Raw16 v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = *reinterpret_cast<const Raw16*>(t.in + (g * t.N + b * 8 + j) * t.r + k * 8);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    Raw16 o;
#pragma unroll
    for (int p = 0; p < 4; ++p)
      o.w[p] = __builtin_amdgcn_perm(v[2 * p + 1].w[j >> 1], v[2 * p].w[j >> 1],
                                     (j & 1) ? 0x07060302u : 0x05040100u);
    *reinterpret_cast<Raw16*>(t.out + (g * t.r + k * 8 + j) * t.N + b * 8) = o;
  }
}

// Places one block's chunk: every wave owns a contiguous part of it, so the order is that
// of a serial counting sort whatever the timing. With one block the counts are its own;
// else each block sums the count table of all blocks (read from L2, eight loads in flight).
// Bound by latency: 7.5 us for 4096 ids of 9 groups with their tile table, 4.9 (the counts) and
// 6.9 us for 32768 ids of 256 experts.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void sort_place_kernel(SortArgs a) {
  constexpr int kWaves = THREADS / kWave;
  constexpr int kGroups = THREADS == kSortWide ? kSortWideGroups : kMaxGroups + 1;
  constexpr int kBatch = 4, kTable = 8;
  __shared__ int32_t s_w[kWaves][kGroups];  // per-wave counts, then positions
  __shared__ int32_t s_base[kGroups];       // first row of each group
  __shared__ int32_t s_tile[kGroups + 1];   // first tile of each group
  __shared__ int32_t s_part[kWaves];
  if ((int)blockIdx.x >= a.nb) {  // blocks beside the sort: four waves each, over more CUs
    if (threadIdx.x < kSortNarrow)
      transpose_block(a.turn, (long)(blockIdx.x - a.nb) * kSortNarrow + threadIdx.x);
    return;
  }
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
  const int c0 = min((long)blockIdx.x * a.chunk, (long)a.n), c1 = min(c0 + (long)a.chunk, (long)a.n);
  const int part = ((c1 - c0 + THREADS - 1) / THREADS) * kWave;  // ids per wave
  const int w0 = min(c0 + wave * part, c1), w1 = min(w0 + part, c1);
  for (int e = tid; e < a.groups; e += THREADS)
    for (int w = 0; w < kWaves; ++w) s_w[w][e] = 0;
  __syncthreads();
  const int bits = group_bits(a.groups);
  int id[kBatch];
  auto load_ids = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int s = s0 + i * kWave + lane;
      id[i] = a.ids[min(s, w1 - 1)];   // no branch: the loads leave together
      id[i] = s < w1 ? sort_key(id[i], a.G, a.groups) : -1;
    }
  };
  for (int s0 = w0; s0 < w1; s0 += kBatch * kWave) {
    load_ids(s0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (s0 + i * kWave < w1) count_groups(id[i], bits, s_w[wave]);
  }
  __syncthreads();
  int placed = 0, tiles = 0;
  for (int e0 = 0; e0 < a.groups; e0 += THREADS) {
    const int e = e0 + tid;
    int tot = 0, before = 0;
    if (e < a.groups) {
      if (a.nb == 1) {
        for (int w = 0; w < kWaves; ++w) tot += s_w[w][e];
      } else {
        for (int b0 = 0; b0 < a.nb; b0 += kTable) {
          int c[kTable];
#pragma unroll
          for (int i = 0; i < kTable; ++i)
            c[i] = b0 + i < a.nb ? a.counts[(size_t)(b0 + i) * a.groups + e] : 0;
#pragma unroll
          for (int i = 0; i < kTable; ++i) {
            tot += c[i];
            if (b0 + i < (int)blockIdx.x) before += c[i];
          }
        }
      }
    }
    int sum;
    const int excl = placed + block_scan<THREADS>(tot, s_part, &sum) - tot;
    placed += sum;
    if (e < a.groups) {
      int run = excl + before;
      for (int w = 0; w < kWaves; ++w) {
        const int c = s_w[w][e];
        s_w[w][e] = run;
        run += c;
      }
      if (blockIdx.x == 0) a.off[e] = excl;
    }
    if (a.tile_rows) {
      const int nt = (tot + a.tile_rows - 1) / a.tile_rows;
      const int tx = tiles + block_scan<THREADS>(nt, s_part, &sum) - nt;
      tiles += sum;
      if (e < a.groups) {
        s_tile[e] = tx;
        s_base[e] = excl;
        if (blockIdx.x == 0) a.tile_first[e] = tx;
      }
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.off[a.groups] = placed;
    if (a.tile_rows) a.tile_first[a.groups] = tiles;
  }
  __syncthreads();
  const int gid = blockIdx.x * THREADS + tid, gsz = a.nb * THREADS;
  for (int i = placed + gid; i < a.n; i += gsz) a.sorted[i] = -1;
  if (a.tile_rows) {
    // Entry i is what block i of a launch takes. Blocks go to the 8 XCDs in turn, so the
    // tiles are dealt out in 8 runs: neighbouring tiles, which read the same adapter, share
    // an L2. Tile t belongs to the last group whose first tile is at or before t.
    const int run = (tiles + 7) / 8;
    for (int i = gid; i < a.max_tiles; i += gsz) {
      const int t = (i >> 3) < run ? (i & 7) * run + (i >> 3) : tiles;
      int lo = 0, hi = a.groups - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_tile[mid] <= t) lo = mid; else hi = mid - 1;
      }
      SortTile d{-1, 0, 0, 0};
      if (t < tiles) {
        const int end = lo + 1 < a.groups ? s_base[lo + 1] : placed;
        d.group = lo;
        d.start = s_base[lo] + (t - s_tile[lo]) * a.tile_rows;
        d.rows = min(a.tile_rows, end - d.start);
        d.index = t;
      }
      a.tile[i] = d;
    }
  }
  for (int s0 = w0; s0 < w1; s0 += kBatch * kWave) {
    if (w1 - w0 > kBatch * kWave) load_ids(s0);   // else they are still here
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (s0 + i * kWave >= w1) break;
      const int s = s0 + i * kWave + lane;
      const int e = max(id[i], 0);
      const uint64_t m = same_group(id[i], bits);
      const int rank = __popcll(m & ((1ull << lane) - 1ull));
      const int cnt = __popcll(m);
      int pos = -1;
      if (id[i] >= 0) pos = s_w[wave][e] + rank;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (id[i] >= 0) {
        a.sorted[pos] = s;
        if (rank == cnt - 1) s_w[wave][e] += cnt;
      }
      if (a.slot_row && s < w1) a.slot_row[s] = pos;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// Blocks of a sort: fewer and larger ones where the count table that every block reads
// (blocks * groups entries) would grow past 64 K entries.
static int sort_blocks(int n, int groups) {
  if (n <= kSortOneBlock) return 1;
  return std::min({(n + kSortChunk - 1) / kSortChunk, std::max(1, (1 << 16) / groups), 256});
}

size_t sort_count_words(int n, int groups) {
  const int nb = sort_blocks(n, groups);
  return nb > 1 ? (size_t)nb * groups : 0;
}

hipError_t launch_sort(const GroupSort& g, hipStream_t s) {
  SortArgs a{};
  a.ids = g.ids;
  a.n = g.n;
  a.G = g.G;
  a.groups = g.groups;
  a.nb = sort_blocks(g.n, g.groups);
  a.chunk = ((g.n + a.nb - 1) / a.nb + kSortWide - 1) / kSortWide * kSortWide;
  a.counts = g.counts;
  a.sorted = g.sorted;
  a.slot_row = g.slot_row;
  a.off = g.off;
  a.tile_rows = g.tile_rows;
  a.max_tiles = g.max_tiles;
  a.tile = g.tile;
  a.tile_first = g.tile_first;
  if (a.nb > 1) hipLaunchKernelGGL(sort_count_kernel, dim3(a.nb), dim3(kSortWide), 0, s, a);
  a.turn = g.turn;
  const long turns = g.turn.in ? (long)g.turn.G * (g.turn.N / 8) * (g.turn.r / 8) : 0;
  const dim3 blocks((unsigned)(a.nb + (turns + kSortNarrow - 1) / kSortNarrow));
  if (g.groups <= kSortWideGroups && g.n > kSortFewIds)
    hipLaunchKernelGGL(sort_place_kernel<kSortWide>, blocks, dim3(kSortWide), 0, s, a);
  else
    hipLaunchKernelGGL(sort_place_kernel<kSortNarrow>, blocks, dim3(kSortNarrow), 0, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------

constexpr int kRowThreads = 256;

// element types of the rows: conversion of one 16-byte vector and of one element
struct Bf16 {
  static constexpr int kSize = 2, kVec = 8;
  static __device__ __forceinline__ void unpack(const Raw16& v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(v.w[i]);
      f[2 * i + 1] = bf16_hi(v.w[i]);
    }
  }
  static __device__ __forceinline__ Raw16 pack(const float* f) {
    Raw16 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    return v;
  }
  static __device__ __forceinline__ float load(const char* p) {
    return bf16_lo(*reinterpret_cast<const uint16_t*>(p));
  }
  static __device__ __forceinline__ void store(char* p, float f) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)pack_bf16(f, 0.f);
  }
};

struct Fp16 {
  static constexpr int kSize = 2, kVec = 8;
  static __device__ __forceinline__ void unpack(const Raw16& v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2 h = __builtin_bit_cast(f16x2, v.w[i]);
      f[2 * i] = (float)h[0];
      f[2 * i + 1] = (float)h[1];
    }
  }
  static __device__ __forceinline__ Raw16 pack(const float* f) {
    Raw16 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.w[i] = pack_f16(f[2 * i], f[2 * i + 1]);
    return v;
  }
  static __device__ __forceinline__ float load(const char* p) {
    return fp16_to_f32(*reinterpret_cast<const uint16_t*>(p));
  }
  static __device__ __forceinline__ void store(char* p, float f) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)pack_f16(f, 0.f);
  }
};

struct Fp32 {
  static constexpr int kSize = 4, kVec = 4;
  static __device__ __forceinline__ void unpack(const Raw16& v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v.w[i]);
  }
  static __device__ __forceinline__ Raw16 pack(const float* f) {
    Raw16 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.w[i] = __float_as_uint(f[i]);
    return v;
  }
  static __device__ __forceinline__ float load(const char* p) { return *reinterpret_cast<const float*>(p); }
  static __device__ __forceinline__ void store(char* p, float f) { *reinterpret_cast<float*>(p) = f; }
};

// Blocks of a row kernel: `chunks` blocks of 256 threads a token, 16 bytes a thread, on one
// grid axis (block b: token b / chunks, bytes from (b % chunks) * 4096)
struct RowPlace {
  int t;
  long at;
};
__device__ __forceinline__ RowPlace row_place(int chunks) {
  const int t = blockIdx.x / (unsigned)chunks;
  return {t, ((long)(blockIdx.x - t * chunks) * kRowThreads + threadIdx.x) * 16};
}

// Rows that no cache will hold until they are used again are read and written past the caches'
// replacement order (STREAM). On MI355X, bf16 rows of 6144, 8 slots a token, three sets of rows
// in turn: the weighted sum at 2000 tokens (197 MB of rows) takes 38 us so and 47 otherwise, at
// 700 (69 MB) 17.1 and 15.3; its gradient 83 and 87, 29 and 32 us, and at 300 (29 MB) 16.8 and
// 13.7; the copy 49 and 54, and the same below 70 MB.
constexpr long kStreamBytes = 64L << 20;

typedef uint32_t Vec16 __attribute__((ext_vector_type(4), aligned(2)));

// the bytes [at, at + 16) of a row of `bytes` bytes; a row's last, partial vector is read
// and written two bytes at a time (rows are whole elements of 2 or 4 bytes)
template <bool STREAM>
__device__ __forceinline__ Raw16 load_raw(const char* row, long at, long bytes) {
  Raw16 v{};
  if (at + 16 <= bytes) {
    if constexpr (STREAM) {
      const Vec16 q = __builtin_nontemporal_load(reinterpret_cast<const Vec16*>(row + at));
#pragma unroll
      for (int i = 0; i < 4; ++i) v.w[i] = q[i];
    } else {
      v = *reinterpret_cast<const Raw16*>(row + at);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at + 2 * i < bytes)
        v.w[i >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(row + at + 2 * i) << (16 * (i & 1));
  }
  return v;
}

template <bool STREAM>
__device__ __forceinline__ void store_raw(char* row, long at, long bytes, const Raw16& v) {
  if (at + 16 <= bytes) {
    if constexpr (STREAM)
      __builtin_nontemporal_store(Vec16{v.w[0], v.w[1], v.w[2], v.w[3]}, reinterpret_cast<Vec16*>(row + at));
    else
      *reinterpret_cast<Raw16*>(row + at) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at + 2 * i < bytes)
        *reinterpret_cast<uint16_t*>(row + at + 2 * i) = (uint16_t)(v.w[i >> 1] >> (16 * (i & 1)));
  }
}

// Copies each token's row to its slots' places: x is read once, every row written once. Bound
// by HBM: 4096 tokens of 8 slots, bf16 rows of 6144 (453 MB) in 82 us, 5.5 TB/s; a large copy
// reaches 5.05. Taking 16 KiB of a row a block was no faster (85 us).
template <bool STREAM>
__global__ __launch_bounds__(kRowThreads) void permute_copy_kernel(
    const char* __restrict__ x, long xs, const int32_t* __restrict__ slot_row, int k, int chunks,
    long bytes, char* __restrict__ rows, long rs) {
  const auto [tok, at] = row_place(chunks);
  const long t = tok;
  if (at >= bytes) return;
  const Raw16 v = load_raw<false>(x + t * xs, at, bytes);
  for (int j = 0; j < k; ++j) {
    const int r = slot_row[t * k + j];
    if (r >= 0) store_raw<STREAM>(rows + (long)r * rs, at, bytes, v);
  }
}

struct PermuteSmallArgs {
  const char* x;
  long xs;
  const int32_t* ids;
  int M, k, E, chunks;
  long bytes;
  char* rows;
  long rs;
  int32_t* sorted;
  int32_t* slot_row;
  int32_t* off;
};

// The whole permutation in one launch, for few ids: every block ranks its own token's slots
// against all ids (how many lie before it in the sorted order, 16 to 64 lanes a slot) while
// its part of the token's row is on the way. One more block writes the offsets. Bound by
// latency: 8 slots, rows of 2048: 3.0 us.
__global__ __launch_bounds__(kRowThreads) void permute_small_kernel(PermuteSmallArgs a) {
  __shared__ __align__(16) int32_t s_id[kPermuteSmall];
  __shared__ int32_t s_cnt[kMaxExperts];
  __shared__ int32_t s_row[kMaxTopK];
  __shared__ int32_t s_part[kRowThreads / kWave];
  const int tid = threadIdx.x, n = a.M * a.k;
  const auto [t, at] = row_place(a.chunks);
  const bool first = at < kRowThreads * 16;  // the token's first block
  if (t == a.M) {  // offsets and the end of sorted_slots
    for (int e = tid; e < a.E; e += kRowThreads) s_cnt[e] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kRowThreads) {
      const int e = a.ids[i];
      if ((unsigned)e < (unsigned)a.E) atomicAdd(&s_cnt[e], 1);
    }
    __syncthreads();
    int placed = 0;
    for (int e0 = 0; e0 < a.E; e0 += kRowThreads) {
      const int e = e0 + tid;
      const int c = e < a.E ? s_cnt[e] : 0;
      int sum;
      const int incl = placed + block_scan<kRowThreads>(c, s_part, &sum);
      placed += sum;
      if (e < a.E) a.off[e] = incl - c;
    }
    if (tid == 0) a.off[a.E] = placed;
    for (int i = placed + tid; i < n; i += kRowThreads) a.sorted[i] = -1;
    return;
  }
  Raw16 v{};
  if (at < a.bytes) v = load_raw<false>(a.x + t * a.xs, at, a.bytes);
  // ids past the last and dropped ones sort behind every expert
  const int quads = (n + 3) / 4;
  for (int i = tid; i < quads * 4; i += kRowThreads) {
    const int e = a.ids[min(i, n - 1)];
    s_id[i] = i < n && (unsigned)e < (unsigned)a.E ? e : INT_MAX;
  }
  __syncthreads();
  // 16, 32 or 64 lanes a slot
  const int lanes = a.k <= 4 ? 64 : a.k <= 8 ? 32 : 16, j = tid / lanes;
  if (j < a.k) {
    const int s = t * a.k + j, e = s_id[s];
    int before = 0;
    for (int i = tid & (lanes - 1); i < quads; i += lanes) {
      const int4 v = *reinterpret_cast<const int4*>(&s_id[i * 4]);
      const int o = s - i * 4;  // equal ids of earlier slots come before
      before += (v.x < e || (v.x == e && 0 < o)) + (v.y < e || (v.y == e && 1 < o)) +
                (v.z < e || (v.z == e && 2 < o)) + (v.w < e || (v.w == e && 3 < o));
    }
    for (int o = lanes / 2; o > 0; o >>= 1) before += __shfl_xor(before, o);
    if ((tid & (lanes - 1)) == 0) {
      const int r = e != INT_MAX ? before : -1;
      s_row[j] = r;
      if (first) {
        a.slot_row[s] = r;
        if (r >= 0) a.sorted[r] = s;
      }
    }
  }
  __syncthreads();
  if (at < a.bytes)
    for (int q = 0; q < a.k; ++q) {
      const int r = s_row[q];
      if (r >= 0) store_raw<false>(a.rows + (long)r * a.rs, at, a.bytes, v);
    }
}

struct CombineArgs {
  const char* rows;
  long rs;
  const int32_t* slot_row;
  const float* w;   // null: plain sums (the gradient of the permutation)
  int k, n, chunks;
  long bytes;
  char* y;
  long ys;
};

// y[t] = sum_j w[t, j] * rows[slot_row[t, j]] in fp32, j ascending, rounded once. A thread
// owns one 16-byte column of one token; the loads of up to eight rows are issued together
// before the first is used, which is what keeps enough bytes in flight. Bound by HBM: 4096
// tokens of 8 slots, bf16 rows of 6144 (453 MB) in 76 us, 6.0 TB/s; fp32 rows of 2049, 1021
// tokens of 6 slots (59 MB, in the caches in part) in 12.6 us.
template <typename T, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(CombineArgs a) {
  constexpr int kBatch = 8;
  const auto [tok, at] = row_place(a.chunks);
  const long t = tok;
  if (at >= a.bytes) return;
  float acc[T::kVec] = {};
  for (int j0 = 0; j0 < a.k; j0 += kBatch) {
    Raw16 v[kBatch];
    int r[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      r[i] = j0 + i < a.k ? a.slot_row[t * a.k + j0 + i] : -1;
      if ((unsigned)r[i] < (unsigned)a.n) v[i] = load_raw<STREAM>(a.rows + (long)r[i] * a.rs, at, a.bytes);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if ((unsigned)r[i] < (unsigned)a.n) {
        const float w = a.w ? a.w[t * a.k + j0 + i] : 1.f;
        float f[T::kVec];
        T::unpack(v[i], f);
#pragma unroll
        for (int q = 0; q < T::kVec; ++q) acc[q] = fmaf(w, f[q], acc[q]);
      }
  }
  store_raw<STREAM>(a.y + t * a.ys, at, a.bytes, T::pack(acc));
}

struct UnpermuteBwdArgs {
  const char* dy;
  long dys;
  const char* rows;
  long rs;
  const int32_t* slot_row;
  const float* w;
  int k, n;
  long bytes;
  char* drows;
  long drs;
  float* dw;
};

// drows[slot_row[t, j]] = w[t, j] * dy[t] and dw[t, j] = <dy[t], rows[slot_row[t, j]]>: one
// block a token, so dy is read once and the dot products of all its slots stay in registers
// until the row's end. Bound by HBM: 4096 tokens, 8 slots of which a quarter are here, fp16 rows
// of 6144 (252 MB) in 52 us, 4.8 TB/s.
template <typename T, int KM, bool STREAM>
__global__ __launch_bounds__(kRowThreads) void unpermute_bwd_kernel(UnpermuteBwdArgs a) {
  __shared__ float s_dot[kRowThreads / kWave][KM];
  const long t = blockIdx.x;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  int r[KM];
  float w[KM], dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    const int v = j < a.k ? a.slot_row[t * a.k + j] : -1;
    r[j] = (unsigned)v < (unsigned)a.n ? v : -1;
    w[j] = j < a.k ? a.w[t * a.k + j] : 0.f;
    dot[j] = 0.f;
  }
  for (long at = threadIdx.x * 16; at < a.bytes; at += (long)blockDim.x * 16) {
    Raw16 v[KM];
    const Raw16 dv = load_raw<STREAM>(a.dy + t * a.dys, at, a.bytes);
#pragma unroll
    for (int j = 0; j < KM; ++j)
      if (r[j] >= 0) v[j] = load_raw<STREAM>(a.rows + (long)r[j] * a.rs, at, a.bytes);
    float d[T::kVec];
    T::unpack(dv, d);
#pragma unroll
    for (int j = 0; j < KM; ++j)
      if (r[j] >= 0) {
        float f[T::kVec], g[T::kVec];
        T::unpack(v[j], f);
#pragma unroll
        for (int q = 0; q < T::kVec; ++q) {
          dot[j] = fmaf(d[q], f[q], dot[j]);
          g[q] = w[j] * d[q];
        }
        store_raw<STREAM>(a.drows + (long)r[j] * a.drs, at, a.bytes, T::pack(g));
      }
  }
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    const float s = group_sum<64>(dot[j]);
    if (lane == 0) s_dot[wave][j] = s;
  }
  __syncthreads();
  if ((int)threadIdx.x < a.k) {
    float s = 0.f;
    for (int i = 0; i < (int)blockDim.x / kWave; ++i) s += s_dot[i][threadIdx.x];
    a.dw[t * a.k + threadIdx.x] = s;
  }
}

// f(row type, whether the rows are streamed)
template <typename F>
static hipError_t by_type(int dtype, long row_bytes, F f) {
  auto with = [&](auto t) { row_bytes > kStreamBytes ? f(t, std::true_type{}) : f(t, std::false_type{}); };
  switch (dtype) {
    case HMOE_DTYPE_BF16: with(Bf16{}); break;
    case HMOE_DTYPE_FP16: with(Fp16{}); break;
    default: with(Fp32{}); break;
  }
  return hipGetLastError();
}

static int row_chunks(long bytes) { return (int)((bytes + kRowThreads * 16 - 1) / (kRowThreads * 16)); }

bool row_grid_fits(long M, long bytes) {
  return (M + 1) * ((bytes + kRowThreads * 16 - 1) / (kRowThreads * 16)) < (1L << 24);
}

hipError_t launch_permute(const PermuteRows& p, const int32_t* ids, int E, int32_t* sorted,
                          int32_t* off, int32_t* counts, hipStream_t s) {
  const long n = (long)p.M * p.k, bytes = (long)p.H * p.esize;
  const int chunks = row_chunks(bytes);
  if (n <= kPermuteSmall) {
    PermuteSmallArgs a{(const char*)p.src, p.src_stride * p.esize, ids, p.M, p.k, E, chunks, bytes,
                       (char*)p.dst, p.dst_stride * p.esize, sorted, const_cast<int32_t*>(p.slot_row), off};
    hipLaunchKernelGGL(permute_small_kernel, dim3(p.M * chunks + 1), dim3(kRowThreads), 0, s, a);
    return hipGetLastError();
  }
  GroupSort g{};
  g.ids = ids;
  g.n = (int)n;
  g.G = g.groups = E;
  g.counts = counts;
  g.sorted = sorted;
  g.slot_row = const_cast<int32_t*>(p.slot_row);
  g.off = off;
  hipError_t err = launch_sort(g, s);
  if (err != hipSuccess) return err;
  const auto copy = n * bytes > kStreamBytes ? permute_copy_kernel<true> : permute_copy_kernel<false>;
  hipLaunchKernelGGL(copy, dim3(p.M * chunks), dim3(kRowThreads), 0, s,
                     (const char*)p.src, p.src_stride * p.esize, p.slot_row, p.k, chunks, bytes, (char*)p.dst,
                     p.dst_stride * p.esize);
  return hipGetLastError();
}

hipError_t launch_combine(const PermuteRows& p, const float* w, hipStream_t s) {
  const long bytes = (long)p.H * p.esize;
  const int chunks = row_chunks(bytes);
  CombineArgs a{(const char*)p.src, p.src_stride * p.esize, p.slot_row, w, p.k, p.M * p.k, chunks,
                bytes, (char*)p.dst, p.dst_stride * p.esize};
  return by_type(p.dtype, (long)p.M * p.k * bytes, [&](auto t, auto stream) {
    hipLaunchKernelGGL((combine_kernel<decltype(t), stream.value>), dim3(p.M * chunks), dim3(kRowThreads), 0, s, a);
  });
}

hipError_t launch_unpermute_bwd(const PermuteRows& p, const void* rows, long rows_stride,
                                const float* w, float* dw, hipStream_t s) {
  const long bytes = (long)p.H * p.esize;
  UnpermuteBwdArgs a{(const char*)p.src, p.src_stride * p.esize, (const char*)rows,
                     rows_stride * p.esize, p.slot_row, w, p.k, p.M * p.k, bytes, (char*)p.dst,
                     p.dst_stride * p.esize, dw};
  // threads: one 16-byte vector each up to 256
  const int threads = bytes > 2048 ? 256 : bytes > 1024 ? 128 : 64;
  return by_type(p.dtype, (long)p.M * p.k * bytes, [&](auto t, auto stream) {
    using T = decltype(t);
    if (p.k <= 8)
      hipLaunchKernelGGL((unpermute_bwd_kernel<T, 8, stream.value>), dim3(p.M), dim3(threads), 0, s, a);
    else
      hipLaunchKernelGGL((unpermute_bwd_kernel<T, kMaxTopK, stream.value>), dim3(p.M), dim3(threads), 0, s, a);
  });
}

}  // namespace hmoe
