// Low-rank adapters of many requests beside one shared projection:
//   z[m] = A_g x[m],  y[m] = base[m] + s_g B_g z[m],  g = ids[m]   (ids outside [0, G): y = base)
// and the gradients
//   dz[m] = s_g B_g^T dy[m],  dx[m] = dbase[m] + A_g^T dz[m],
//   dA_g = sum_m dz[m] x[m]^T,  dB_g = s_g sum_m dy[m] z[m]^T   (sums over the rows of g).
//
// With ranks of 8 to 128 the products do r / 2 operations a byte of x and y, far below what
// the matrix cores could do: the kernels are bound by reading x, base and the matrices in
// use, and by writing y. So every product runs on bf16 MFMA from global memory into fragments,
// rows of one adapter are gathered into tiles of 16 to 64 (one read of its matrices each),
// and the long axis K is split over waves and blocks when there are few tiles. z stays in fp32:
// where z or dz is an MFMA operand it goes in as a sum of three bf16 parts, which hold its 24 bits.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "group_count.h"
#include "hmoe_internal.h"

namespace hmoe {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

struct __attribute__((packed, aligned(2))) Half8 {  // 8 bf16 at any element
  uint32_t w[4];
};
struct __attribute__((packed, aligned(2))) Half4 {
  uint32_t w[2];
};
constexpr int kKStep = 128;  // K elements a wave takes at a time: four MFMAs deep

__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
  const Half8 h = *reinterpret_cast<const Half8*>(p);
  return u32x4{h.w[0], h.w[1], h.w[2], h.w[3]};
}
// the same from a wave-uniform base and a 32-bit byte offset of the lane (one register)
__device__ __forceinline__ u32x4 load8(const uint16_t* base, uint32_t bytes) {
  return load8(reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(base) + bytes));
}
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// An fp32 value as a sum of three bf16 parts, 8 of its 24 bits each: a part is the upper half of
// what the parts before it leave, so every part is exact and no finite value becomes infinite. An
// infinite value leaves nothing. part[k]: a's in the low half, b's in the high one.
__device__ __forceinline__ void split_parts(float a, float b, uint32_t (&part)[3]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    part[k] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
    const float ra = a - bf16_lo(part[k]), rb = b - bf16_hi(part[k]);
    a = k == 0 && __builtin_isinf(a) ? 0.f : ra;
    b = k == 0 && __builtin_isinf(b) ? 0.f : rb;
  }
}

// Kernel arguments into scalar registers here. The compiler would read them where they are
// first used, behind the wait for a tile's rows and in the loops after it: the backward pass of
// 4001 rows, rank 16, takes 69.0 us so, and 66.8 with its second product's arguments read ahead
// (the other kernels gain nothing).
template <typename... T>
__device__ __forceinline__ void read_ahead(const T&... v) {
  auto one = [](auto u) { asm volatile("" ::"s"(u)); };
  (one(v), ...);
}

// ---- lane exchanges ----------------------------------------------------------------
//
// An MFMA operand wants lane l to hold row l % 16, but the memory pipe takes 64 bytes a
// cycle only where four neighbouring lanes lie in one 64-byte piece: 16-byte loads with one
// row a lane ran at 9.6 TB/s over the card from L2, with four lanes a row at 34 TB/s
// (measured, 1 MiB buffer). So rows are read and written four lanes a row, four rows in four
// instructions, and exchanged inside each four lanes in registers.

__device__ __forceinline__ uint32_t quad_x1(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);  // lane ^ 1
}
__device__ __forceinline__ uint32_t quad_x2(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);  // lane ^ 2
}

// lane s of each four gets v[j] = lane j's v[s]
__device__ __forceinline__ void quad_turn(u32x4 (&v)[4]) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    uint32_t a0 = v[0][d], a1 = v[1][d], a2 = v[2][d], a3 = v[3][d];
    // every lane takes part in every exchange: they stand outside the selections
    const uint32_t x0 = quad_x1(a0), x1 = quad_x1(a1), x2 = quad_x1(a2), x3 = quad_x1(a3);
    const uint32_t b0 = odd ? x1 : a0, b1 = odd ? a1 : x0;
    const uint32_t b2 = odd ? x3 : a2, b3 = odd ? a3 : x2;
    const uint32_t y0 = quad_x2(b0), y1 = quad_x2(b1), y2 = quad_x2(b2), y3 = quad_x2(b3);
    v[0][d] = high ? y2 : b0;
    v[2][d] = high ? b2 : y0;
    v[1][d] = high ? y3 : b1;
    v[3][d] = high ? b3 : y1;
  }
}

// lane group q of 16 lanes gets v[j] = group j's v[q]
__device__ __forceinline__ void group_turn(u32x4 (&v)[4]) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const auto a = __builtin_amdgcn_permlane16_swap(v[0][d], v[1][d], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(v[2][d], v[3][d], false, false);
    const auto e = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
    const auto f = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
    v[0][d] = e[0];
    v[2][d] = e[1];
    v[1][d] = f[0];
    v[3][d] = f[1];
  }
}

// 8 rows of 4 neighbouring columns (two dwords a row) turned into 4 fragments of 8 rows of
// one column each: fragment t is column t
__device__ __forceinline__ void turn_8x4(const uint32_t (&v)[8][2], u32x4 (&f)[4]) {
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int p = 0; p < 4; ++p)
      f[t][p] = __builtin_amdgcn_perm(v[2 * p + 1][t >> 1], v[2 * p][t >> 1],
                                      (t & 1) ? 0x07060302u : 0x05040100u);
}

// Which rows a block works on: entry b % tiles of the tile table, and of a tile of more than RT
// rows its part b / tiles. The table comes from a sort before the launch (kTable), or the first
// launch does without one and leaves its tiles, of RT rows, as the table for the second:
// kRow   entry b is the tile that starts at row b, if the rows of the same adapter before b fill
//        whole tiles; the entries of all other rows are idle.
// kCount every block counts all ids by adapter and so finds tile b and its rows.
// Rank 16, us of the card, kRow and kCount: 7.1 and 8.3 (1 row, 2048 -> 1536 columns), 7.5 and 8.7
// (64), 8.5 and 8.7 (200), 13.6 and 10.5 (200 rows, 4096 -> 4096), and kCount would take 16 more
// to look through the counts of 2000 adapters. kCount and kTable: 8.9 and 12.3 (257 rows of 4
// adapters, 2048 -> 1536), 10.1 and 14.7 (1000 of 30), 18.4 and 19.9 (2000 of 100), 26.0 and
// 25.6 (4000 of 64).
enum TileFind { kTable, kRow, kCount };
constexpr int kRowRows = 128;                         // most rows of kRow
constexpr int kCountRows = 2048, kCountGroups = 256;  // of kCount, with the group of no adapter
struct Tiles {
  const int32_t* ids;
  int M, G, tiles;
  TileFind find;
  int32_t* sorted;     // rows by adapter (null: no table is kept)
  SortTile* table;
};

// false: no tile. Else *g (G: rows without an adapter), s_rows[0 .. *n), *index: the tile's
// number; *n may be 0 for a part behind the first. s_rows past *n names row 0, so that whatever
// reads it stays inside the matrices.
// ROWS: most rows of kCount, whose ids the block's THREADS hold in registers (0: only kTable).
template <int RT, int ROWS, int THREADS>
__device__ __forceinline__ bool find_tile(const Tiles& t, int* g, int* n, int* index, int32_t* s_rows) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
  if (ROWS == 0 || t.find == kTable) {
    const int part = (int)blockIdx.x / t.tiles, e = (int)blockIdx.x - part * t.tiles;
    const SortTile d = t.table[e];  // an idle entry has no rows
    *g = d.group;
    *index = d.index;
    *n = max(0, min(RT, d.rows - part * RT));
    if (tid < RT) s_rows[tid] = tid < *n ? t.sorted[d.start + part * RT + tid] : 0;
    __syncthreads();
    return d.group >= 0;
  }
  if constexpr (ROWS > 0) {
    const bool put = t.sorted && blockIdx.y == 0;  // this block writes its entry
    const int e = blockIdx.x;
    SortTile d{-1, 0, 0, 0};
    if (tid < RT) s_rows[tid] = 0;
    if (t.find == kRow) {
      // all adapters' numbers into LDS with one wait, then every wave goes through them
      __shared__ int32_t s_key[kRowRows];
      for (int m = tid; m < t.M; m += THREADS) s_key[m] = sort_key(t.ids[m], t.G, t.G + 1);
      __syncthreads();
      const int mine = s_key[e];
      int seen = 0, first = -1;  // rows of `mine` so far; their number before e
      for (int m0 = 0; m0 < t.M; m0 += kWave) {
        const int m = m0 + lane;
        const uint64_t same = __ballot(m < t.M && s_key[min(m, t.M - 1)] == mine);
        if (first < 0 && e < m0 + kWave) {
          first = seen + __popcll(same & ((1ull << (e - m0)) - 1ull));
          if (first % RT) {
            if (put && tid == 0) t.table[e] = d;
            return false;
          }
        }
        const int rank = seen + __popcll(same & ((1ull << lane) - 1ull)) - first;
        if (first >= 0 && (same >> lane & 1) && rank >= 0 && rank < RT) s_rows[rank] = m;
        seen += __popcll(same);
        if (first >= 0 && seen - first >= RT) break;
      }
      d = SortTile{mine, e * RT, min(RT, seen - first), e};
    } else {
      constexpr int kIds = ROWS / THREADS, kWaves = THREADS / kWave, kRuns = kCountGroups / kWave;
      __shared__ int32_t s_cnt[kCountGroups];
      __shared__ int32_t s_wave[kWaves];
      const int groups = t.G + 1, run = (t.M + THREADS - 1) / THREADS;  // ids of a lane
      const int w0 = wave * run * kWave;
      int id[kIds];
#pragma unroll
      for (int i = 0; i < kIds; ++i)
        if (i < run) id[i] = t.ids[min(w0 + i * kWave + lane, t.M - 1)];
      for (int k = tid; k < groups; k += THREADS) s_cnt[k] = 0;
      __syncthreads();
      const int bits = group_bits(groups);
#pragma unroll
      for (int i = 0; i < kIds; ++i)
        if (i < run) {
          id[i] = w0 + i * kWave + lane < t.M ? sort_key(id[i], t.G, groups) : -1;
          count_groups(id[i], bits, s_cnt);
        }
      __syncthreads();
      // every wave for itself: tiles and rows up to each group (both below 2^16), in registers
      int upto[kRuns], all = 0;
#pragma unroll
      for (int k = 0; k < kRuns; ++k)
        if (k * kWave < groups) {
          const int c = k * kWave + lane < groups ? s_cnt[k * kWave + lane] : 0;
          int sum = (c + RT - 1) / RT << 16 | c;
#pragma unroll
          for (int o = 1; o < kWave; o <<= 1) {
            const int u = __shfl_up(sum, o);
            if (lane >= o) sum += u;
          }
          upto[k] = all + sum;
          all += __shfl(sum, kWave - 1);
        }
      // Blocks go to the 8 XCDs in turn; a run of tiles (of one adapter mostly) goes to one.
      const int total = all >> 16, per = (total + 7) / 8;
      const int tile = e / 8 < per ? (e & 7) * per + e / 8 : total;
      if (tile >= total) {
        if (put && tid == 0) t.table[e] = d;
        return false;
      }
      int first = 0;  // the tile's first row in its group
#pragma unroll
      for (int k = 0; k < kRuns; ++k)
        if (k * kWave < groups && d.group < 0) {
          const uint64_t past = __ballot((upto[k] >> 16) > tile);
          if (past) {
            const int l = __ffsll((unsigned long long)past) - 1, end = __shfl(upto[k], l);
            const int rows = s_cnt[k * kWave + l];
            first = (tile - (end >> 16) + (rows + RT - 1) / RT) * RT;
            d = SortTile{k * kWave + l, (end & 0xffff) - rows + first, min(RT, rows - first), tile};
          }
        }
      int seen = 0;
#pragma unroll
      for (int i = 0; i < kIds; ++i)
        if (i < run) seen += __popcll(__ballot(id[i] == d.group));
      if (lane == 0) s_wave[wave] = seen;
      __syncthreads();
      int rank = -first;  // of the group's next row, from this tile's first
      for (int w = 0; w < wave; ++w) rank += s_wave[w];
#pragma unroll
      for (int i = 0; i < kIds; ++i)
        if (i < run) {
          const uint64_t same = __ballot(id[i] == d.group);
          const int at = rank + __popcll(same & ((1ull << lane) - 1ull));
          if (id[i] == d.group && at >= 0 && at < d.rows) s_rows[at] = w0 + i * kWave + lane;
          rank += __popcll(same);
        }
    }
    *g = d.group;
    *index = d.index;
    *n = d.rows;
    __syncthreads();
    if (put) {
      if (tid == 0) t.table[e] = d;
      if (tid < d.rows) t.sorted[d.start + tid] = s_rows[tid];
    }
    return true;
  }
  return false;
}

// s_red = X_rows W_g^T over the steps [s0, s1) of the reduction axis K, rows x ranks. The W
// waves of the block take the steps of 128 in turn; then the upper half of the waves hands
// its sums to the lower half through LDS, and the lower half leaves its sums in s_red[wave]
// for the caller to add in wave order. In a step lane group q holds K elements 32q .. 32q + 31
// of its row for four MFMAs: the order of the reduction axis is free as long as both operands
// share it. DEPTH > 1: that many steps' loads are in flight at a time.
template <int MT, int NT, int W, int DEPTH>
__device__ __forceinline__ void shrink_tile(const uint16_t* x, long xs, const uint16_t* w, int K,
                                            int r, int n, const int32_t* s_rows, int s0, int s1,
                                            float (*s_red)[MT * NT * 256]) {
  // A scalar wave number takes addresses out of the lanes' registers, but loops of few loads then
  // wait for each: 16 rows of rank 64 win a little (35.3 to 34.4 us at 1500 rows of 50 adapters,
  // 4096 -> 4096), one row of rank 16 loses half (10 to 20 us, 6144 -> 4096), 32 rows lose 1%.
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = MT == 1 && NT == 4 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : (int)(threadIdx.x >> 6);
  const int c = lane & 15, q = lane >> 4, at = q * 32 + (c & 3) * 8;
  const uint16_t* xp[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int rr = i * 16 + (c & 12) + j;
      xp[i][j] = x + (long)s_rows[rr < n ? rr : 0] * xs;
    }
  f32x4 acc[MT][NT] = {};
  // No load stands behind a branch of a lane's own, so that a step's loads leave together. In
  // the last step of a K that is no multiple of 128, lanes past the end read the step's start
  // and their part of x is zeroed (W is finite). Ranks come in eights: four ranks of a tile all
  // exist, or the lane reads others instead.
  auto load_x = [&](u32x4 (&v)[MT][4], int st) {
    const int k = st * kKStep, o = k + at < K ? k + at : k;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = load8(xp[i][j] + o);
  };
  auto turn_x = [&](u32x4 (&v)[MT][4], int st) {
    if ((st + 1) * kKStep > K) {
      const bool in = st * kKStep + at < K;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int d = 0; d < 4; ++d) v[i][j][d] = in ? v[i][j][d] : 0u;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) quad_turn(v[i]);
  };
  auto load_w = [&](u32x4 (&v)[4], int st, int tile) {
    const int k = st * kKStep, o = k + at < K ? k + at : k, rank = tile * 16 + (c & 12);
    const uint32_t off = ((rank < r ? rank : 0) * K + o) * 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = load8(w + (long)j * K, off);
  };
  auto multiply = [&](const u32x4 (&x)[MT][4], u32x4 (&w)[4], int tile) {
    quad_turn(w);
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i][tile] = mfma(x[i][h], w[h], acc[i][tile]);
  };
  // A load behind a condition would make every later wait count on its absence, and so wait for
  // everything; the loops below load ahead without conditions and peel their ends.
  const int mine = (s1 - s0 - wave + W - 1) / W;  // steps of this wave: s0 + wave + i W
  auto step = [&](int i) { return s0 + wave + i * W; };
  if constexpr (DEPTH > 1) {
    u32x4 x[DEPTH][MT][4], v[DEPTH][NT][4];
    auto load = [&](int d, int i) {
      load_x(x[d], step(i));
#pragma unroll
      for (int t = 0; t < NT; ++t) load_w(v[d][t], step(i), t);
    };
    auto use = [&](int d, int i) {
      turn_x(x[d], step(i));
#pragma unroll
      for (int t = 0; t < NT; ++t) multiply(x[d], v[d][t], t);
    };
    int i = 0;
    if (mine >= DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) load(d, d);
      for (; i + 2 * DEPTH <= mine; i += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
          use(d, i + d);
          load(d, i + DEPTH + d);
        }
      }
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) use(d, i + d);
      i += DEPTH;
    }
    // fewer than DEPTH left
    const int left = mine - i;
#pragma unroll
    for (int d = 0; d < DEPTH - 1; ++d)
      if (d < left) load(d, i + d);
#pragma unroll
    for (int d = 0; d < DEPTH - 1; ++d)
      if (d < left) use(d, i + d);
  } else {
    // one set of W's registers, each tile of ranks loaded again as soon as it is used up, and
    // two sets of x's: a step's loads are in flight while the one before is multiplied. Past
    // rank 64 the set holds half the tiles.
    constexpr int kW = NT == 8 ? 4 : NT;
    u32x4 x[2][MT][4], v[kW][4];
    auto use = [&](int d, int i, auto ahead) {
      if constexpr (ahead.value) load_x(x[d ^ 1], step(i + 1));
      turn_x(x[d], step(i));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        multiply(x[d], v[t % kW], t);
        if (t + kW < NT) load_w(v[t % kW], step(i), t + kW);
        else if constexpr (ahead.value) load_w(v[t % kW], step(i + 1), t % kW);
      }
    };
    if (mine > 0) {
      load_x(x[0], step(0));
#pragma unroll
      for (int t = 0; t < kW; ++t) load_w(v[t], step(0), t);
      int i = 0;
      for (; i + 2 < mine; i += 2) {
        use(0, i, std::true_type{});
        use(1, i + 1, std::true_type{});
      }
      if (i + 1 < mine) {
        use(0, i, std::true_type{});
        use(1, i + 1, std::false_type{});
      } else {
        use(0, i, std::false_type{});
      }
    }
  }
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) f(acc[i][j][e], (i * 16 + q * 4 + e) * (NT * 16) + j * 16 + c);
  };
  if (wave >= W / 2) each([&](float v, int at) { s_red[wave - W / 2][at] = v; });
  __syncthreads();
  if (wave < W / 2) each([&](float v, int at) { s_red[wave][at] += v; });
  __syncthreads();
}

// W_g z of 16 rows, added to base: a wave takes 128 columns at a time. The columns are dealt
// out to the MFMAs so that lane c of a group of 16 ends up with columns 8c .. 8c + 7 of four
// rows: base and y move as 16-byte accesses, 16 lanes on 256 contiguous bytes of a row. A
// fragment of W serves all bf16 parts of z; up to rank 16 (KS = 0) the first two share one MFMA.
// TR: W is [r, N] (a lane's columns of 8 ranks are turned in registers), else [N, r].
struct ColumnArgs {
  int r, N;
  const uint16_t* w;     // matrix of the tile's adapter
  const uint16_t* base;  // may be null
  long bs;
  uint16_t* y;
  long ys;
};

// z: rows of scale z in LDS, fp32, kLd apart; a lane makes its fragments of them
template <int KS>
struct ZShape {
  static constexpr bool kPack = KS == 0;         // rank <= 16: two parts side by side
  static constexpr int kSteps = kPack ? 1 : KS;
  static constexpr int kParts = kPack ? 2 : 3;   // fragments of a rank step
  static constexpr int kLd = kSteps * 32 + 4;    // padded off the banks
};

constexpr int kCols = 128;

// The lanes' place in a tile of 16 rows and 128 columns. No load stands behind a lane's own
// branch, so that they leave together: a lane without a row, column or rank of its own reads
// another one, which then goes nowhere (ranks: meets zeros of z, W being finite). Columns and
// ranks come in eights: what a lane reads of 4 or 8 of them exists whole.
template <int KS, bool TR>
struct Columns {
  using Z = ZShape<KS>;
  const ColumnArgs& a;
  const int n, c, q;
  int row[4];   // rows this lane reads, and writes below n

  // s_rows: the 16 rows, n of them
  __device__ __forceinline__ Columns(const ColumnArgs& a, int n, const int32_t* s_rows)
      : a(a), n(n), c(threadIdx.x & 15), q((threadIdx.x & (kWave - 1)) >> 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) row[j] = s_rows[q * 4 + j < n ? q * 4 + j : 0];
  }

  __device__ __forceinline__ void load_base(u32x4 (&b)[4], int cg) const {
    const int col = cg * kCols + c * 8, o = col < a.N ? col : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = a.base ? load8(a.base + row[j] * a.bs + o) : u32x4{};
  }

  // ranks ch .. ch + 7 of fragment step ks, chunk q, or others in place of such as do not exist
  __device__ __forceinline__ int chunk(int ks, int q) const {
    const int ch = (ks * 4 + q) * 8;
    return ch < a.r ? ch : Z::kPack && ch < 2 * a.r ? ch - a.r : 0;
  }

  // half h of W's part for rank step ks as it lies
  __device__ __forceinline__ void load_w(u32x4 (&v)[4], int cg, int ks, int h) const {
    if constexpr (TR) {  // columns 8c + 4h .. + 3 of 8 ranks, two ranks a register set
      const int col = cg * kCols + c * 8 + h * 4;
      const uint32_t off = (chunk(ks, q) * a.N + (col < a.N ? col : h * 4)) * 2;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const Half4 f = *reinterpret_cast<const Half4*>(reinterpret_cast<const char*>(a.w + (long)e * a.N) + off);
        v[e >> 1][(e & 1) * 2] = f.w[0];
        v[e >> 1][(e & 1) * 2 + 1] = f.w[1];
      }
    } else {  // column 8 (c & 12) + 8e + 4h + q, ranks of chunk c & 3
      const int ch = chunk(ks, c & 3);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = cg * kCols + ((c & 12) + e) * 8;
        v[e] = load8(a.w + h * 4 * a.r, (((col < a.N ? col : 0) + q) * a.r + ch) * 2);
      }
    }
  }

  // what load_w brought, as the fragments of columns t = 4h .. 4h + 3
  __device__ __forceinline__ static void turn_w(u32x4 (&v)[4]) {
    if constexpr (TR) {
      uint32_t x[8][2];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e][0] = v[e >> 1][(e & 1) * 2];
        x[e][1] = v[e >> 1][(e & 1) * 2 + 1];
      }
      turn_8x4(x, v);
    } else {
      quad_turn(v);
      group_turn(v);
    }
  }

  // word d of a rank step's fragments of z: two ranks of row c in three bf16 parts (zeros past r)
  __device__ __forceinline__ void split_z(uint32_t (&f)[Z::kParts], const float* s_z, int ks, int d) const {
    const int ch = (ks * 4 + q) * 8;
    const float2 v = *reinterpret_cast<const float2*>(s_z + c * Z::kLd + chunk(ks, q) + 2 * d);
    uint32_t part[3];
    split_parts(v.x, v.y, part);
    if constexpr (Z::kPack) {  // [first, second], [third, zeros]
      f[0] = ch < a.r ? part[0] : ch < 2 * a.r ? part[1] : 0u;
      f[1] = ch < a.r ? part[2] : 0u;
    } else {
#pragma unroll
      for (int k = 0; k < 3; ++k) f[k] = ch < a.r ? part[k] : 0u;
    }
  }

  // fragments of z for all rank steps, by each wave for its own 16 rows
  __device__ __forceinline__ void make_z(u32x4 (&zf)[Z::kSteps][Z::kParts], const float* s_z) const {
#pragma unroll
    for (int ks = 0; ks < Z::kSteps; ++ks)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        uint32_t f[Z::kParts];
        split_z(f, s_z, ks, d);
#pragma unroll
        for (int k = 0; k < Z::kParts; ++k) zf[ks][k][d] = f[k];
      }
  }

  // the same for a block whose W waves have the same 16 rows: each makes a part for all (1000 rows
  // of 30 adapters, 2048 -> 1536, rank 64: 15.1 us, 15.5 with every wave for itself)
  template <int W>
  __device__ __forceinline__ void share_z(u32x4 (&zf)[Z::kSteps][Z::kParts], const float* s_z,
                                          uint32_t (*s_zf)[Z::kParts][kWave][4]) const {
    const int lane = threadIdx.x & (kWave - 1);
    for (int i = threadIdx.x >> 6; i < Z::kSteps * 4; i += W) {
      uint32_t f[Z::kParts];
      split_z(f, s_z, i >> 2, i & 3);
#pragma unroll
      for (int k = 0; k < Z::kParts; ++k) s_zf[i >> 2][k][lane][i & 3] = f[k];
    }
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < Z::kSteps; ++ks)
#pragma unroll
      for (int k = 0; k < Z::kParts; ++k) zf[ks][k] = *reinterpret_cast<const u32x4*>(s_zf[ks][k][lane]);
  }

  // y = base + acc (rows without an adapter: y = base)
  __device__ __forceinline__ void store(const u32x4 (&b)[4], const f32x4 (&acc)[8], bool live, int cg) const {
    const int col = cg * kCols + c * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Half8 o;
#pragma unroll
      for (int p = 0; p < 4; ++p)
        o.w[p] = live ? pack_bf16(bf16_lo(b[j][p]) + acc[2 * p][j], bf16_hi(b[j][p]) + acc[2 * p + 1][j])
                      : b[j][p];
      if (q * 4 + j < n && col < a.N) *reinterpret_cast<Half8*>(a.y + row[j] * a.ys + col) = o;
    }
  }

  // what a group of columns starts with: base, and W's part for the first rank step
  struct Load {
    u32x4 base[4], w[2][4];
  };
  __device__ __forceinline__ void load(Load& l, bool live, int cg) const {
    load_base(l.base, cg);
    if (live)
#pragma unroll
      for (int h = 0; h < 2; ++h) load_w(l.w[h], cg, 0, h);
  }

  // groups cg, cg + W, ... below g1; `l` holds the loads of group cg
  template <int W>
  __device__ __forceinline__ void run(Load& l, bool live, int cg, int g1,
                                      const u32x4 (&zf)[Z::kSteps][Z::kParts]) const {
    while (cg < g1) {
      f32x4 acc[8] = {};
      if (live) {
#pragma unroll
        for (int ks = 0; ks < Z::kSteps; ++ks) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (ks) load_w(l.w[h], cg, ks, h);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            turn_w(l.w[h]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int p = 0; p < Z::kParts; ++p) acc[h * 4 + t] = mfma(zf[ks][p], l.w[h][t], acc[h * 4 + t]);
          }
        }
      }
      store(l.base, acc, live, cg);
      cg += W;
      if (cg < g1) load(l, live, cg);
    }
  }
};

struct ShrinkArgs {
  Tiles tiles;
  const uint16_t* x;
  long xs;
  const uint16_t* w;   // [G, r, K]
  int K, r, splits;
  float* part;         // [splits, M, r]
};

constexpr int kShrinkWaves = 4;

// part[s][m] = W_g x[m] over split s of K. Bound by the way of x from HBM and of W from L2 into
// the registers, which the few steps of a wave hide only in part: 4096 rows of 8 adapters, rank
// 64, K = 6144: 22.4 us (50 MB of x, 2.2 TB/s; 17 with W held in L1, 13 with x there, 9 with both).
// Tiles of 64 rows a block, which halve W's way, were no faster.
template <int MT, int NT>
__global__ __launch_bounds__(kShrinkWaves* kWave) void lora_shrink_kernel(ShrinkArgs a) {
  __shared__ int32_t s_rows[MT * 16];
  __shared__ __align__(16) float s_red[kShrinkWaves / 2][MT * NT * 256];
  int g, n, index;
  if (!find_tile<MT * 16, MT == 1 ? kCountRows : 0, kShrinkWaves * kWave>(a.tiles, &g, &n, &index, s_rows)) return;
  if (g == a.tiles.G) return;
  const int steps = (a.K + kKStep - 1) / kKStep;
  shrink_tile<MT, NT, kShrinkWaves, (MT + NT <= 3 ? 2 : 1)>(a.x, a.xs, a.w + (long)g * a.r * a.K, a.K, a.r, n, s_rows,
                                    (int)((long)steps * blockIdx.y / a.splits),
                                    (int)((long)steps * (blockIdx.y + 1) / a.splits), s_red);
  float* out = a.part + (long)blockIdx.y * a.tiles.M * a.r;
  for (int i = threadIdx.x; i < n * NT * 4; i += kShrinkWaves * kWave) {
    const int row = i / (NT * 4), col = i % (NT * 4) * 4;
    if (col >= a.r) continue;
    float4 s = *reinterpret_cast<const float4*>(&s_red[0][i * 4]);
#pragma unroll
    for (int w = 1; w < kShrinkWaves / 2; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(&s_red[w][i * 4]);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    *reinterpret_cast<float4*>(out + (long)s_rows[row] * a.r + col) = s;
  }
}

struct ExpandArgs {
  Tiles tiles;
  const float* part;     // [splits, M, r]
  int splits;
  const float* scale;    // [G]
  float* z;              // may be null
  int col_groups;        // groups of 128 columns a block takes
  ColumnArgs c;          // w: all adapters' matrices
  // TR (backward): where the fragments of scale dz and scale z go, and z
  uint16_t* frag[2];
  const float* fz;
  int steps_per_tile;    // 32 rows each
};

constexpr int kExpandWaves = 4;

// rank / 16 rounded up to a power of two: rank tiles of the products over K and over rows
__host__ __device__ constexpr int rank_tiles(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }

// Rows RT * part, ... of a table entry of P [rows, r] (RT of them) as the MFMA fragments that
// sums over rows need: for every 32 rows, each of three bf16 parts and each 16 ranks, lane (rank
// c, row group q) holds rows 8q .. 8q + 7 of its rank, 1 KiB together. s_p: the rows, fp32, LD
// apart; rows past n and ranks past r are zeros.
template <int RT, int LD>
__device__ __forceinline__ void put_parts(const float* s_p, int part, int n, int r, uint16_t* out) {
  const int nt = rank_tiles(r);
  for (int o = threadIdx.x; o < nt * RT * 2; o += blockDim.x) {
    const int c = o & 15, row = o / 16 % (RT / 8) * 8, i = o / (RT * 2), rank = i * 16 + c;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = rank < r && row + e < n ? s_p[(row + e) * LD + rank] : 0.f;
    const int at = part * RT + row, lane = at % 32 * 2 + c;
    Half8 h[3];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t w[3];
      split_parts(v[2 * p], v[2 * p + 1], w);
#pragma unroll
      for (int k = 0; k < 3; ++k) h[k].w[p] = w[k];
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
      *reinterpret_cast<Half8*>(out + (((at / 32 * 3 + k) * nt + i) * kWave + lane) * 8) = h[k];
  }
}

// LDS of the second product: z before the columns, then what its waves share
template <int RW, int KS>
struct ExpandLds {
  using Z = ZShape<KS>;
  static constexpr bool kDouble = KS <= 2;                        // two sets of W's fragments
  static constexpr int kFrag = RW == 1 ? 0 : Z::kSteps * 8 * 1024;  // bytes of one set
  static constexpr int kZ = RW * 16 * Z::kLd * 4;
  static constexpr int kShared = std::max(kFrag * (kDouble ? 2 : 1), kZ);
};

// y = base + W_g (scale z): z's splits are added in order, scaled and put into LDS, from where
// the fragments are made that a lane keeps for the block's columns. RW = 1: 16 rows a block, each wave has columns of
// its own. RW = 4: 64 rows, a wave 16 of them; the waves share each group of columns, and each
// turns a part of W's fragments and puts it into LDS for all, which cuts W's way from L2 to a
// quarter. In the backward pass (TR) the first block of a tile also leaves scale dz as
// fragments for the weight gradients, the last one scale z. Bound by base and y in HBM behind
// the chain table, z's splits, columns: 4096 rows, rank 64, N = 4096: 25.4 us (67 MB, 2.6 TB/s;
// 37 with RW = 1); backward, 4001 rows, rank 16, K = 6144: 24.3 us (98 MB, 4.0 TB/s; 35).
template <int RW, int KS, bool TR>
__global__ __launch_bounds__(kExpandWaves* kWave, (KS <= 2 ? (RW == 1 && KS + TR < 2 ? 4 : 3) : 2))
void lora_expand_kernel(ExpandArgs a) {
  using Z = ZShape<KS>;
  using L = ExpandLds<RW, KS>;
  constexpr int RT = RW * 16, kThreads = kExpandWaves * kWave;
  __shared__ int32_t s_rows[RT];
  __shared__ __align__(16) char s_shared[L::kShared];
  __shared__ __align__(16) uint32_t s_zf[RW == 1 ? Z::kSteps : 1][Z::kParts][RW == 1 ? kWave : 1][4];
  float* s_z = reinterpret_cast<float*>(s_shared);
  u32x4* s_w = reinterpret_cast<u32x4*>(s_shared);
  read_ahead(a.part, a.splits, a.scale, a.z, a.col_groups, a.c.w, a.c.base, a.c.bs, a.c.y, a.c.ys);
  if (TR) read_ahead(a.frag[0], a.frag[1], a.fz, a.steps_per_tile);
  int g, n, index;
  if (!find_tile<RT, 0, kThreads>(a.tiles, &g, &n, &index, s_rows)) return;
  const bool live = g != a.tiles.G, head = blockIdx.y == 0;
  const int r = a.c.r, quads = r / 4, lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int mine = RW == 1 ? 0 : wave * 16;  // first of this wave's rows
  ColumnArgs ca = a.c;
  if (live) ca.w += (long)g * ca.N * r;
  const Columns<KS, TR> cols(ca, max(0, min(16, n - mine)), s_rows + mine);
  const int g0 = blockIdx.y * a.col_groups, g1 = min(g0 + a.col_groups, (ca.N + kCols - 1) / kCols);
  int cg = RW == 1 ? g0 + wave : g0;
  // the first loads are on the way while z is put together
  constexpr int kPieces = 2 * Z::kSteps, kMine = (kPieces + kExpandWaves - 1) / kExpandWaves;
  typename Columns<KS, TR>::Load first;
  u32x4 base[4], raw[kMine][4];
  auto load_pieces = [&](int cg) {  // this wave's pieces of W's fragments: (rank step, half)
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int pc = k * kExpandWaves + wave;
      if (kPieces % kExpandWaves == 0 || pc < kPieces) cols.load_w(raw[k], cg, pc >> 1, pc & 1);
    }
  };
  if (RW == 1) {
    if (cg < g1) cols.load(first, live, cg);
  } else {
    cols.load_base(base, cg);
    if (live) load_pieces(cg);
  }
  u32x4 zf[Z::kSteps][Z::kParts];
  if (live) {
    const float sc = a.scale[g];
    const long part = (long)a.tiles.M * r;
    for (int i = threadIdx.x; i < n * quads; i += kThreads) {
      const int row = i / quads, col = i % quads * 4;
      const float* p = a.part + (long)s_rows[row] * r + col;
      float v[4] = {};
      for (int s0 = 0; s0 < a.splits; s0 += 4) {   // four loads leave together
        float4 f[4];
#pragma unroll
        for (int s = 0; s < 4; ++s)
          f[s] = *reinterpret_cast<const float4*>(p + min(s0 + s, a.splits - 1) * part);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const bool in = s0 + s < a.splits;
          v[0] += in ? f[s].x : 0.f, v[1] += in ? f[s].y : 0.f;
          v[2] += in ? f[s].z : 0.f, v[3] += in ? f[s].w : 0.f;
        }
      }
      if (!TR && a.z && head)
        *reinterpret_cast<float4*>(a.z + (long)s_rows[row] * r + col) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(s_z + row * Z::kLd + col) = make_float4(v[0] * sc, v[1] * sc, v[2] * sc, v[3] * sc);
    }
    __syncthreads();
    if constexpr (RW == 1) cols.template share_z<kExpandWaves>(zf, s_z, s_zf);
    else cols.make_z(zf, s_z + mine * Z::kLd);
    if constexpr (TR) {
      const int pt = (int)blockIdx.x / a.tiles.tiles;
      const long at = (long)index * a.steps_per_tile * 3 * rank_tiles(r) * 512;
      if (head) put_parts<RT, Z::kLd>(s_z, pt, n, r, a.frag[0] + at);
      if (blockIdx.y == gridDim.y - 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < n * quads; i += kThreads) {
          const int row = i / quads, col = i % quads * 4;
          const float4 f = *reinterpret_cast<const float4*>(a.fz + (long)s_rows[row] * r + col);
          *reinterpret_cast<float4*>(s_z + row * Z::kLd + col) = make_float4(f.x * sc, f.y * sc, f.z * sc, f.w * sc);
        }
        __syncthreads();
        put_parts<RT, Z::kLd>(s_z, pt, n, r, a.frag[1] + at);
      }
    }
  } else if (!TR && a.z && head) {
    for (int i = threadIdx.x; i < n * r; i += kThreads) a.z[(long)s_rows[i / r] * r + i % r] = 0.f;
  }
  __syncthreads();
  if (!live && a.c.base == a.c.y) return;  // rows without an adapter stay
  if constexpr (RW == 1) {
    cols.template run<kExpandWaves>(first, live, cg, g1, zf);
  } else {
    for (int it = 0; cg < g1; ++cg, ++it) {
      u32x4* buf = s_w + (L::kDouble ? (it & 1) * (L::kFrag / 16) : 0);
      if (live) {
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          const int pc = k * kExpandWaves + wave;
          if (kPieces % kExpandWaves == 0 || pc < kPieces) {
            cols.turn_w(raw[k]);
#pragma unroll
            for (int t = 0; t < 4; ++t) buf[(pc * 4 + t) * kWave + lane] = raw[k][t];
          }
        }
      }
      __syncthreads();
      u32x4 next[4] = {};
      if (cg + 1 < g1) {
        if (live) load_pieces(cg + 1);
        cols.load_base(next, cg + 1);
      }
      f32x4 acc[8] = {};
      if (live) {
#pragma unroll
        for (int ks = 0; ks < Z::kSteps; ++ks) {
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const u32x4 f = buf[(ks * 8 + t) * kWave + lane];
#pragma unroll
            for (int p = 0; p < Z::kParts; ++p) acc[t] = mfma(zf[ks][p], f, acc[t]);
          }
        }
      }
      cols.store(base, acc, live, cg);
#pragma unroll
      for (int j = 0; j < 4; ++j) base[j] = next[j];
      if (!L::kDouble) __syncthreads();
    }
  }
}

struct FusedArgs {
  Tiles tiles;
  const uint16_t* x;
  long xs;
  const uint16_t* wa;    // [G, r, K]
  int K;
  const float* scale;
  float* z;              // may be null
  int col_groups;
  ColumnArgs c;
  // TR (backward): as in ExpandArgs
  uint16_t* frag[2];
  const float* fz;
};

constexpr int kFusedWaves = 8;
constexpr int kFusedRows = 1024;  // most rows of the one-launch form

// Both products of a tile of 16 rows in one block, for few rows: the waves split K, z never
// leaves LDS, then they split the block's columns. Blocks of one tile that take different
// columns repeat the first product (its matrix comes from L2 again). TR: the backward pass, as
// in the second product alone. Bound by latency: find the tile, load, multiply, add up, load,
// multiply, write. 1 row, 2048 -> 1536, rank 16: 6.9 us; 64 rows of 48 adapters, 6144 -> 4096:
// 11.5 us (13 MB).
template <int NT, int KS, bool TR>
__global__ __launch_bounds__(kFusedWaves* kWave) void lora_fused_kernel(FusedArgs a) {
  using Z = ZShape<KS>;
  constexpr int kThreads = kFusedWaves * kWave;
  __shared__ int32_t s_rows[16];
  __shared__ __align__(16) float s_red[kFusedWaves / 2][NT * 256];
  __shared__ __align__(16) float s_z[16 * Z::kLd];
  __shared__ __align__(16) uint32_t s_zf[Z::kSteps][Z::kParts][kWave][4];
  int g, n, index;
  if (!find_tile<16, TR ? 0 : kFusedRows, kThreads>(a.tiles, &g, &n, &index, s_rows)) return;
  const bool live = g != a.tiles.G, head = blockIdx.y == 0, tail = blockIdx.y == gridDim.y - 1;
  const int r = a.c.r, quads = r / 4;
  const int part = TR ? (int)blockIdx.x / a.tiles.tiles : 0;
  const long at = TR ? (long)index * 3 * rank_tiles(r) * 512 : 0;
  if (TR && n == 0) {  // an entry's empty second half: its fragments are zeros
    if (live && head)
      for (int i = 0; i < 2; ++i) put_parts<16, Z::kLd>(s_z, part, 0, r, a.frag[i] + at);
    return;
  }
  ColumnArgs ca = a.c;
  if (live) ca.w += (long)g * ca.N * r;
  const Columns<KS, TR> cols(ca, n, s_rows);
  const int g0 = blockIdx.y * a.col_groups, g1 = min(g0 + a.col_groups, (ca.N + kCols - 1) / kCols);
  const int cg = g0 + (threadIdx.x >> 6);
  typename Columns<KS, TR>::Load first;  // on the way during the first product
  if (cg < g1) cols.load(first, live, cg);
  u32x4 zf[Z::kSteps][Z::kParts];
  if (live) {
    shrink_tile<1, NT, kFusedWaves, (NT == 1 ? 4 : NT == 2 ? 2 : 1)>(
        a.x, a.xs, a.wa + (long)g * r * a.K, a.K, r, n, s_rows, 0, (a.K + kKStep - 1) / kKStep, s_red);
    const float sc = a.scale[g];
    for (int i = threadIdx.x; i < n * NT * 4; i += kThreads) {
      const int row = i / (NT * 4), col = i % (NT * 4) * 4;
      if (col >= r) continue;
      float v[4] = {};
#pragma unroll
      for (int w = 0; w < kFusedWaves / 2; ++w) {
        const float4 f = *reinterpret_cast<const float4*>(&s_red[w][i * 4]);
        v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
      }
      if (!TR && a.z && head)
        *reinterpret_cast<float4*>(a.z + (long)s_rows[row] * r + col) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(s_z + row * Z::kLd + col) = make_float4(v[0] * sc, v[1] * sc, v[2] * sc, v[3] * sc);
    }
    __syncthreads();
    cols.template share_z<kFusedWaves>(zf, s_z, s_zf);
    if (TR && head) put_parts<16, Z::kLd>(s_z, part, n, r, a.frag[0] + at);
    if (TR && tail) {
      __syncthreads();
      for (int i = threadIdx.x; i < n * quads; i += kThreads) {
        const int row = i / quads, col = i % quads * 4;
        const float4 f = *reinterpret_cast<const float4*>(a.fz + (long)s_rows[row] * r + col);
        *reinterpret_cast<float4*>(s_z + row * Z::kLd + col) = make_float4(f.x * sc, f.y * sc, f.z * sc, f.w * sc);
      }
      __syncthreads();
      put_parts<16, Z::kLd>(s_z, part, n, r, a.frag[1] + at);
    }
  } else if (!TR && a.z && head) {
    for (int i = threadIdx.x; i < n * r; i += kThreads) a.z[(long)s_rows[i / r] * r + i % r] = 0.f;
  }
  __syncthreads();
  if (!live && a.c.base == a.c.y) return;  // rows without an adapter stay
  cols.template run<kFusedWaves>(first, live, cg, g1, zf);
}

struct WgradArgs {
  const int32_t* sorted;
  const int32_t* off;
  const int32_t* tile_first;
  int steps_per_tile;
  int r;
  // two products: [0] P = scale dz, X = x, out dA [G, r, C]; [1] P = scale z, X = dy, out dB [G, C, r]
  const uint16_t* p[2];   // fragments of P, see put_parts
  const uint16_t* x[2];
  long xs[2];
  int C[2], blocks[2];
  float* out[2];
};

constexpr int kWgradThreads = 512;
constexpr int kWgradWaves = kWgradThreads / kWave;
constexpr int kWgradRows = 2048;  // row indices kept in LDS at a time

// out_g[p, c] = sum over the rows m of group g of P[m, p] X[m, c]. The reduction axis is the
// row, so both operands are needed transposed: of X a lane reads 8 rows of 4 neighbouring
// columns (8 bytes each, 128 contiguous bytes a row over 16 lanes) and turns them in registers
// into the fragments of 4 MFMAs; P lies ready as fragments, in three bf16 parts (24 bits), so
// the fp32 result carries no bf16 rounding. A wave has 64 columns and goes through the rows in
// steps of 32, the next step's loads in flight. SHARE of the block's waves have
// the same columns, take steps in turn and add up through LDS in wave order; a wave alone
// writes its registers. Rows past the group's end are zeros of P. Ranks past
// NT * 16 go to further blocks (grid z). Bound by the rows (each read once) at low ranks, by the
// way of P's parts from L2 at high ones: 4001 rows of 4 adapters, 6144 and 4096 columns, rank
// 16: 23.9 us (82 MB, 3.4 TB/s).
template <int NT, int SHARE>
__global__ __launch_bounds__(kWgradThreads) void lora_wgrad_kernel(WgradArgs a) {
  __shared__ float s_red[SHARE > 1 ? kWgradWaves : 1][16][68];
  __shared__ int32_t s_idx[kWgradRows];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // the columns' addresses stay scalar
  constexpr int kAbreast = kWgradWaves / SHARE;  // waves of a row range
  const int tile = (int)blockIdx.x * kAbreast + wave % kAbreast, phase = wave / kAbreast;
  const int side = tile >= a.blocks[0], g = blockIdx.y;
  const int c0 = (tile - (side ? a.blocks[0] : 0)) * 64;
  const int c = lane & 15, q = lane >> 4;
  const int m0 = a.off[g], m1 = a.off[g + 1];
  const int nt = NT * gridDim.z, i0 = blockIdx.z * NT;
  const uint16_t* P = a.p[side] + ((long)a.tile_first[g] * a.steps_per_tile * 3 * nt + i0) * 512 + lane * 8;
  const uint16_t* X = a.x[side];
  const long xs = a.xs[side];
  const int C = a.C[side];
  const int col = c0 + c * 4 < C ? c0 + c * 4 : 0;  // lanes past the end: columns that go nowhere
  f32x4 acc[NT][4] = {};
  struct Step {
    uint32_t x[8][2];
    u32x4 p[3][NT];
  };
  for (int mb = m0; mb < m1; mb += kWgradRows) {
    const int rows = min(kWgradRows, m1 - mb);
    __syncthreads();
    // the last step is filled up with the last row, which meets zeros of P
    for (int i = tid; i < (rows + 31) / 32 * 32; i += kWgradThreads) s_idx[i] = a.sorted[mb + min(i, rows - 1)];
    __syncthreads();
    auto load = [&](Step& v, int m) {
      const uint16_t* p = P + (long)((mb - m0 + m) >> 5) * 3 * nt * 512;
#pragma unroll
      for (int part = 0; part < 3; ++part)
#pragma unroll
        for (int i = 0; i < NT; ++i) v.p[part][i] = load8(p + (part * nt + i) * 512);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Half4 h = *reinterpret_cast<const Half4*>(X + s_idx[m + q * 8 + j] * xs + col);
        v.x[j][0] = h.w[0];
        v.x[j][1] = h.w[1];
      }
    };
    auto multiply = [&](const Step& v) {
      u32x4 xf[4];
      turn_8x4(v.x, xf);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[i][t] = mfma(v.p[part][i], xf[t], acc[i][t]);
    };
    // the next step's loads without a condition of their own (see the first product)
    constexpr int kStride = SHARE * 32;
    Step u, v;
    int m = phase * 32;
    if (m < rows) {
      load(u, m);
      for (; m + 2 * kStride < rows; m += 2 * kStride) {
        load(v, m + kStride);
        multiply(u);
        load(u, m + 2 * kStride);
        multiply(v);
      }
      if (m + kStride < rows) {
        load(v, m + kStride);
        multiply(u);
        multiply(v);
      } else {
        multiply(u);
      }
    }
  }
  // lane (c, q) holds ranks 4q .. 4q + 3 of columns 4c .. 4c + 3; columns run fastest in dA,
  // ranks in dB
  const int phases = SHARE > 1 ? min(SHARE, (m1 - m0 + 31) / 32) : 0;  // those with rows
  if (phases <= 1) {
    const int cl = c0 + c * 4;
    if (phase || tile >= a.blocks[0] + a.blocks[1] || cl >= C) return;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int rr = (i0 + i) * 16 + q * 4;
      if (rr >= a.r) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (side)
          *reinterpret_cast<float4*>(a.out[1] + ((long)g * C + cl + k) * a.r + rr) =
              make_float4(acc[i][k][0], acc[i][k][1], acc[i][k][2], acc[i][k][3]);
        else
          *reinterpret_cast<float4*>(a.out[0] + ((long)g * a.r + rr + k) * C + cl) =
              make_float4(acc[i][0][k], acc[i][1][k], acc[i][2][k], acc[i][3][k]);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    __syncthreads();
    if (phase < phases)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_red[SHARE > 1 ? wave : 0][q * 4 + e][c * 4 + t] = acc[i][t][e];
    __syncthreads();
    // the waves of a tile add its 16 x 64 sums
    for (int o = phase * kWave + lane; o < 16 * 64; o += SHARE * kWave) {
      const int pr = side ? o & 15 : o >> 6, cc = side ? o >> 4 : o & 63;
      const int rr = (i0 + i) * 16 + pr, cl = c0 + cc;
      if (rr >= a.r || cl >= C || tile >= a.blocks[0] + a.blocks[1]) continue;
      float s = 0.f;
      for (int w = 0; w < phases; ++w) s += s_red[SHARE > 1 ? w * kAbreast + wave % kAbreast : 0][pr][cc];
      a.out[side][side ? ((long)g * C + cl) * a.r + rr : ((long)g * a.r + rr) * C + cl] = s;
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

namespace {

constexpr int kFusedRank = 64;          // largest rank of the one-launch form (registers)
constexpr int kFusedMany = 800;         // rows from which on it takes a larger first matrix
constexpr int kWideRows = 3000, kWideMean = 60;  // fewest rows, in all and an adapter, of tiles of 64
static_assert(kWideRows > kCountRows && kWideRows > kFusedRows, "tiles past 16 rows come from the sort");
constexpr int kShrinkBlocks = 400;      // about this many blocks of the first product

struct Plan {
  TileFind find;
  bool fused;      // both products in one launch
  bool wide;       // the second product's waves share its matrix
  int nt;          // rank / 16, rounded up to a power of two
  int rt;          // rows of a tile
  int mt;          // rows / 16 that a block of the first product takes
  int tiles;       // most tiles
  int busy;        // how many of them can have rows
};

bool finds_by_table(int M, int G, bool backward) {
  return backward || M > kCountRows || (M > kRowRows && G >= kCountGroups);
}
// largest first matrix of the one-launch form
int fused_bytes(int M, bool backward) { return (backward ? 192 : M >= kFusedMany ? 512 : 256) << 10; }

// K: the first product's reduction axis.
//
// One launch for few rows. Us a call among others in one and in two launches (a launch costs the
// host 3 us more), first matrix of 64 KiB (2048, rank 16), 256 KiB (2048, rank 64) and 512 KiB
// (4096, rank 64): 9.0, 11.8; 10.6, 12.0; 13.9, 12.0 at 1 row, 8.8, 11.5; 12.4, 11.7; 18.4, 16.2
// at 64 rows of 48 adapters, 8.9, 12.2; 12.8, 12.1; 17.2, 13.5 at 200 of 8, 9.0, 11.8; 13.9, 13.3;
// 18.7, 17.5 at 512 of 16, 9.8, 12.8; 14.9, 17.2; 23.6, 24.5 at 1000 of 30; 256 KiB: 14.2, 14.8 at
// 200 of 60, 15.2, 17.3 at 512 of 60; 512 KiB: 25.1, 27.7 at 512 of 60, 18.6, 17.5 at 700 of 4,
// 19.4, 19.1 at 850 of 4, 22.7, 23.3 at 850 of 16; 768 KiB: 21.9, 19.3 at 512 of 16, 26.8, 26.9 at
// 1000 of 30. Backward, 192 KiB (1536, rank 64), 256 KiB (4096, rank 32) and 512 KiB: 22.3, 22.2;
// 22.5, 21.1; 30.0, 26.7 at 1 row, 20.4, 20.8; 21.2, 19.9; 27.2, 24.1 at 64 of 4, 29.9, 31.8; 29.6,
// 29.0; 39.9, 39.1 at 512 of 16, 33.6, 35.3; 33.6, 35.2; 51.6, 50.8 at 1024 of 16, 53.4, 51.5;
// 64.7, 58.4; 103, 94 at 1024 of 60.
//
// Tiles of 64 share one read of an adapter's matrices among more rows, small ones (16; 32 in the
// backward pass, the depth of its sums over rows) waste less where adapters have few and leave
// more blocks. Us a call with tiles of 16 and 64, 4096 -> 4096, ranks 16, 64 and 128: 18.5, 19.5;
// 24.9, 25.7; 33.4, 32.3 at 1500 rows of 4 adapters, 22.5, 23.6; 31.7, 32.1; 48.5, 50.0 at 2048 of
// 20, 26.5, 27.3; 38.6, 36.4; 55.5, 57.1 at 2500 of 20, 28.6, 30.5; 48.2, 44.0; 67.2, 60.5 at 3000
// of 20, 47.8, 47.5; 70.9, 63.3; 98.2, 93.0 at 4000 of 64, 37.4, 38.8; 52.3, 47.4; 68.2, 65.4 at
// 4000 of 8; rank 16 alone: 66.6, 65.1 at 8000 of 8, 97.9, 85.5 at 12000 of 60. Fewer than 60 rows
// an adapter: 33.1, 38.0 at 3000 of 60, 21.5, 25.5; 34.6, 37.2; 55.4, 58.4 at 1500 of 50, 149, 152;
// 227, 236; 345, 374 at 16000 of 400 (but 49, 55; 81, 75; 114, 105 at 4000 of 100). Tiles of
// 32 lay above the better of the two at 2048 of 20, 4000 of 64, 8 and 100, 1500 of 50 and 16000 of
// 400. Backward, 32 and 64: 35.1, 34.8; 53.4, 57.0; 75.7, 81.2 at 1500 of 4, 40.8, 40.0; 71.4,
// 72.9; 99, 108 at 2048 of 20, 54.7, 54.0; 87.4, 85.3; 128, 119 at 3000 of 20, 61.4, 58.6; 105, 92;
// 163, 146 at 4000 of 8.
//
// Past rank 64 the first product's 32 rows take all registers of a wave; its blocks take 16 until
// there are 140 of 32. Us a call with 16 and 32, rank 128, 4096 -> 4096: 61.4, 64.3 at 3000 rows of
// 20 adapters, 66.9, 65.7 at 4000 of 8, 166, 153 at 8000 of 100; backward 109, 114 at 2048 of 4,
// 119, 122 at 3000 of 20, 148, 146 at 4000 of 8, 422, 406 at 8000 of 100.
Plan plan_tiles(int M, int G, int K, int r, bool backward) {
  Plan p;
  const int mean = M / std::max(1, std::min(G, M));
  p.nt = rank_tiles(r);
  p.fused = M <= kFusedRows && r <= kFusedRank && (long)r * K * 2 <= fused_bytes(M, backward);
  p.find = finds_by_table(M, G, backward) ? kTable : M > kRowRows ? kCount : kRow;
  p.wide = M >= kWideRows && mean >= kWideMean;
  p.rt = p.wide ? 64 : backward ? 32 : 16;
  const int most = M / p.rt + std::min(G + 1, M);
  p.tiles = p.find == kRow ? M : (most + 7) / 8 * 8;  // entries are dealt out over 8 XCDs
  p.busy = std::max(1, std::min(most, M));
  p.mt = p.rt == 16 || (p.nt == 8 && (long)p.busy * p.rt < 140 * 32) ? 1 : 2;
  return p;
}

// Splits of the reduction axis: enough blocks to fill the card, at least one step for each
// wave of a block, at most 16 partial sums to add up again.
int most_splits(int K) {
  const int steps = (K + kKStep - 1) / kKStep;
  return std::min((steps + kShrinkWaves - 1) / kShrinkWaves, 16);
}
int plan_splits(const Plan& p, int K) {
  const int blocks = p.busy * (p.rt / (p.mt * 16));
  return std::min((kShrinkBlocks + blocks - 1) / blocks, most_splits(K));
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct Space {
  size_t sorted, off, counts, tile, tile_first, part, frag[2], bt, total;
};

Space plan_space(int M, int G, int K, int N, int r, bool backward) {
  Space s{};
  const Plan p = plan_tiles(M, G, backward ? N : K, r, backward);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = align256(at + bytes);
    return o;
  };
  if (p.find == kTable || !p.fused) {
    s.sorted = take((size_t)M * (p.find == kRow ? p.rt : 1) * 4);
    s.tile = take((size_t)p.tiles * sizeof(SortTile));
  }
  if (p.find == kTable) {
    s.off = take((size_t)(G + 2) * 4);
    s.counts = take(sort_count_words(M, G + 1) * 4);
    s.tile_first = take((size_t)(G + 2) * 4);
  }
  if (!p.fused) s.part = take((size_t)plan_splits(p, backward ? N : K) * M * r * 4);
  if (backward) {
    for (size_t& f : s.frag) f = take((size_t)p.tiles * (p.rt / 32) * 3 * p.nt * 1024);
    s.bt = take((size_t)G * r * N * 2);
  }
  s.total = at;
  return s;
}

// Bytes that hold the space of every call of at most M rows, so that a buffer made for the largest
// batch serves the smaller ones. The plans of fewer rows may take more of an array (other tiles,
// more splits, two launches), so each array gets a bound that only grows with M:
// splits     at most 16 and what K has; more than one only while blocks are few: there are at least
//            M / 32 of them, so splits * M < kShrinkBlocks * 32 + M
// entries    M / rt + the adapters, rt >= 16; kRow: one a row
// fragments  32-row steps: entries at rt = 32; twice the entries of 64 rows hold them too
size_t most_space(int M, int G, int K, int N, int r, bool backward) {
  const long axis = backward ? N : K, matrix = axis * r * 2, adapters = std::min(G + 1, M);
  // the most rows of a call in two launches, and of one that finds its tiles by comparing rows
  long two = M;
  if (r <= kFusedRank && M <= kFusedRows && matrix <= fused_bytes(kFusedMany, backward))
    two = matrix <= fused_bytes(1, backward) ? 0 : std::min(M, kFusedMany - 1);
  const long rows = backward ? 0 : std::min(two, (long)kRowRows);
  const bool table = finds_by_table(M, G, backward);
  auto entries = [&](int rt) { return (M / rt + adapters + 7) / 8 * 8; };
  size_t total = 0;
  auto add = [&](size_t bytes) { total += align256(bytes); };
  if (table || two) {
    add(std::max({rows * 16, two, table ? (long)M : 0}) * 4);
    add(std::max(rows, entries(backward ? 32 : 16)) * sizeof(SortTile));
  }
  if (table) {
    add((size_t)(G + 2) * 4);
    add(sort_count_words(M, G + 1) * 4);
    add((size_t)(G + 2) * 4);
  }
  add((size_t)std::min(two * most_splits(axis), two ? kShrinkBlocks * 32 + two : 0) * r * 4);
  if (backward) {
    const bool wide = M >= kWideRows && M / std::max(1, std::min(G, M)) >= kWideMean;
    const size_t steps = wide ? 2 * entries(64) : entries(32);
    for (int i = 0; i < 2; ++i) add(steps * 3 * rank_tiles(r) * 1024);
    add((size_t)G * r * N * 2);
  }
  return total;
}

hipError_t make_tiles(const int32_t* ids, int M, int G, const Plan& p, const Space& sp, char* scratch,
                      Tiles* t, const SortTranspose& turn, hipStream_t s) {
  *t = Tiles{ids, M, G, p.tiles, p.find, nullptr, nullptr};
  if (p.find == kTable || !p.fused) {
    t->sorted = reinterpret_cast<int32_t*>(scratch + sp.sorted);
    t->table = reinterpret_cast<SortTile*>(scratch + sp.tile);
  }
  if (p.find != kTable) return hipSuccess;
  GroupSort g{};
  g.ids = ids;
  g.n = M;
  g.G = G;
  g.groups = G + 1;
  g.counts = reinterpret_cast<int32_t*>(scratch + sp.counts);
  g.sorted = t->sorted;
  g.off = reinterpret_cast<int32_t*>(scratch + sp.off);
  g.tile_rows = p.rt;
  g.max_tiles = p.tiles;
  g.tile = t->table;
  g.tile_first = reinterpret_cast<int32_t*>(scratch + sp.tile_first);
  g.turn = turn;
  return launch_sort(g, s);
}

hipError_t shrink(const Plan& p, const ShrinkArgs& a, hipStream_t s) {
  const dim3 grid(p.tiles * (p.rt / (p.mt * 16)), a.splits), block(kShrinkWaves * kWave);
#define HMOE_SHRINK(MT, NT)                                                         \
  if (p.mt == MT && p.nt == NT)                                                     \
  hipLaunchKernelGGL((lora_shrink_kernel<MT, NT>), grid, block, 0, s, a)
  HMOE_SHRINK(1, 1);
  HMOE_SHRINK(2, 1);
  HMOE_SHRINK(1, 2);
  HMOE_SHRINK(2, 2);
  HMOE_SHRINK(1, 4);
  HMOE_SHRINK(2, 4);
  HMOE_SHRINK(1, 8);
  HMOE_SHRINK(2, 8);
#undef HMOE_SHRINK
  return hipGetLastError();
}

// MFMA steps of 32 ranks (0: both parts of z in one)
int z_steps(int r) { return r <= 16 ? 0 : (r + 31) / 32; }

template <int RW, bool TR>
hipError_t expand_by_rank(const Plan& p, const ExpandArgs& a, dim3 grid, hipStream_t s) {
  const dim3 block(kExpandWaves * kWave);
  switch (z_steps(a.c.r)) {
    case 0:
      hipLaunchKernelGGL((lora_expand_kernel<RW, 0, TR>), grid, block, 0, s, a);
      break;
    case 1: hipLaunchKernelGGL((lora_expand_kernel<RW, 1, TR>), grid, block, 0, s, a); break;
    case 2: hipLaunchKernelGGL((lora_expand_kernel<RW, 2, TR>), grid, block, 0, s, a); break;
    case 3: hipLaunchKernelGGL((lora_expand_kernel<RW, 3, TR>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((lora_expand_kernel<RW, 4, TR>), grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

template <bool TR>
hipError_t expand(const Plan& p, ExpandArgs a, hipStream_t s) {
  const int groups = (a.c.N + kCols - 1) / kCols;
  const int parts = p.wide ? 1 : p.rt / 16, unit = p.wide ? 1 : kExpandWaves;
  // columns a block: as few rounds of its waves as let all blocks be on the card at once
  const int ks = z_steps(a.c.r), room = 256 * (ks <= 1 ? 3 : 2);
  const int rounds = std::max(1, (int)(((long)groups * p.busy * parts + (long)room * unit - 1) / ((long)room * unit)));
  a.col_groups = std::min(rounds, (groups + unit - 1) / unit) * unit;
  a.steps_per_tile = p.rt / 32;
  const dim3 grid(p.tiles * parts, (groups + a.col_groups - 1) / a.col_groups);
  return p.wide ? expand_by_rank<4, TR>(p, a, grid, s) : expand_by_rank<1, TR>(p, a, grid, s);
}

template <bool TR>
hipError_t fused(const Plan& p, FusedArgs a, hipStream_t s) {
  const int groups = (a.c.N + kCols - 1) / kCols;
  const int blocks = p.tiles * (p.rt / 16), busy = p.busy * (p.rt / 16);
  // columns a block: a multiple of its waves' 128, about 256 blocks in all
  const int want = std::max(1, 256 / busy);
  const int rounds = std::max(1, (groups + want * kFusedWaves - 1) / (want * kFusedWaves));
  a.col_groups = rounds * kFusedWaves;
  const dim3 grid(blocks, (groups + a.col_groups - 1) / a.col_groups), block(kFusedWaves * kWave);
  switch (z_steps(a.c.r)) {
    case 0: hipLaunchKernelGGL((lora_fused_kernel<1, 0, TR>), grid, block, 0, s, a); break;
    case 1: hipLaunchKernelGGL((lora_fused_kernel<2, 1, TR>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((lora_fused_kernel<4, 2, TR>), grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace

void lora_scratch(int M, int G, int K, int N, int r, size_t* forward, size_t* backward) {
  // the bound holds the plan of M rows; were it ever short of it, a call would still not be let in
  // with less than its own layout
  auto bytes = [&](bool b) { return std::max(plan_space(M, G, K, N, r, b).total, most_space(M, G, K, N, r, b)); };
  if (forward) *forward = bytes(false);
  if (backward) *backward = bytes(true);
}

hipError_t launch_lora(const Lora& l, void* scratch, hipStream_t s) {
  char* b = static_cast<char*>(scratch);
  const Plan p = plan_tiles(l.M, l.G, l.K, l.r, false);
  const ColumnArgs c{l.r, l.N, l.B, l.base, l.bs, l.y, l.ys};
  const Space sp = plan_space(l.M, l.G, l.K, l.N, l.r, false);
  Tiles t;
  hipError_t err = make_tiles(l.ids, l.M, l.G, p, sp, b, &t, {}, s);
  if (err != hipSuccess) return err;
  if (p.fused) return fused<false>(p, FusedArgs{t, l.x, l.xs, l.A, l.K, l.scale, l.z, 0, c, {}, nullptr}, s);
  const int splits = plan_splits(p, l.K);
  float* part = reinterpret_cast<float*>(b + sp.part);
  err = shrink(p, ShrinkArgs{t, l.x, l.xs, l.A, l.K, l.r, splits, part}, s);
  if (err != hipSuccess) return err;
  t.find = kTable;
  return expand<false>(p, ExpandArgs{t, part, splits, l.scale, l.z, 0, c, {}, nullptr, 0}, s);
}

hipError_t launch_lora_backward(const LoraGrad& l, void* scratch, hipStream_t s) {
  char* b = static_cast<char*>(scratch);
  const Plan p = plan_tiles(l.M, l.G, l.N, l.r, true);
  const Space sp = plan_space(l.M, l.G, l.K, l.N, l.r, true);
  Tiles t;
  // B^T [G, r, N], which makes dy B the same product as x A^T, is laid out beside the sort
  uint16_t* Bt = reinterpret_cast<uint16_t*>(b + sp.bt);
  hipError_t err = make_tiles(l.ids, l.M, l.G, p, sp, b, &t, SortTranspose{l.B, Bt, l.N, l.r, l.G}, s);
  if (err != hipSuccess) return err;
  uint16_t* frag[2] = {reinterpret_cast<uint16_t*>(b + sp.frag[0]), reinterpret_cast<uint16_t*>(b + sp.frag[1])};
  if (l.M > 0) {
    const ColumnArgs c{l.r, l.K, l.A, l.dbase, l.dbs, l.dx, l.dxs};
    if (p.fused) {
      err = fused<true>(p, FusedArgs{t, l.dy, l.dys, Bt, l.N, l.scale, nullptr, 0, c, {frag[0], frag[1]}, l.z}, s);
    } else {
      const int splits = plan_splits(p, l.N);
      float* part = reinterpret_cast<float*>(b + sp.part);
      err = shrink(p, ShrinkArgs{t, l.dy, l.dys, Bt, l.N, l.r, splits, part}, s);
      if (err == hipSuccess)
        err = expand<true>(p, ExpandArgs{t, part, splits, l.scale, nullptr, 0, c, {frag[0], frag[1]}, l.z, 0}, s);
    }
    if (err != hipSuccess) return err;
  }
  const int32_t* off = reinterpret_cast<const int32_t*>(b + sp.off);
  const int32_t* tile_first = reinterpret_cast<const int32_t*>(b + sp.tile_first);
  WgradArgs w{t.sorted, off, tile_first, p.rt / 32, l.r, {frag[0], frag[1]}, {l.x, l.dy}, {l.xs, l.dys}, {l.K, l.N},
              {(l.K + 63) / 64, (l.N + 63) / 64}, {l.dA, l.dB}};
  // Waves share the rows of 64 columns until there are 1024 waves (a wave a SIMD), and on to
  // 4096 while each keeps enough rows for what it adds up through LDS: 200, or 50 for every 16
  // ranks, half of that where waves share already. Us a call with 1, 2, 4, 8 waves sharing, 6144
  // -> 4096: 4000 rows of 4 adapters, rank 16: 100, 78, 72, 69; of 8, rank 16: 81, 74, 73, 73; of
  // 8, rank 128: 156, 172, 188, -; 16000 of 4, rank 128: 584, 522, 472, 470; 512 of 2, rank 64:
  // -, 59, 52, 55. 2048 -> 4096, 4000 of 16, rank 64: 77, 88.
  const int tiles = w.blocks[0] + w.blocks[1], halves = p.nt == 8 ? 2 : 1;
  int share = 1;
  for (long waves = (long)tiles * l.G * halves;
       share < kWgradWaves &&
       (waves < 1024 || (waves < 4096 && l.M / l.G / (2 * share) >= (share == 1 ? 50 : 25) * std::max(4, p.nt)));
       waves *= 2)
    share *= 2;
  const int abreast = kWgradWaves / share;
  const dim3 grid((tiles + abreast - 1) / abreast, l.G, halves), block(kWgradThreads);
#define HMOE_WGRAD(NT, SHARE)         \
  if (std::min(p.nt, 4) == NT && share == SHARE) \
  hipLaunchKernelGGL((lora_wgrad_kernel<NT, SHARE>), grid, block, 0, s, w)
  HMOE_WGRAD(1, 1);
  HMOE_WGRAD(1, 2);
  HMOE_WGRAD(1, 4);
  HMOE_WGRAD(1, 8);
  HMOE_WGRAD(2, 1);
  HMOE_WGRAD(2, 2);
  HMOE_WGRAD(2, 4);
  HMOE_WGRAD(2, 8);
  HMOE_WGRAD(4, 1);
  HMOE_WGRAD(4, 2);
  HMOE_WGRAD(4, 4);
  HMOE_WGRAD(4, 8);
#undef HMOE_WGRAD
  return hipGetLastError();
}

}  // namespace hmoe
