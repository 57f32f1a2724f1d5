// Products with one matrix of 4-bit weights and group scales:
//   moe_linear           y[m, n]  = base[m, n] + sum_k x[m, k] W[n, k]
//   moe_linear_backward  dx[m, k] = dbase[m, k] + sum_n dy[m, n] W[n, k]
//
// Few rows are bound by reading W once: the packed codes go from memory into MFMA operands (packed.h),
// and the reduction is split over the waves of a block, whose sums meet in LDS in a fixed order. Many
// rows are bound by the matrix cores: W is laid out once as 16-bit numbers in scratch, a slab of it at a
// time so that the slab stays in the caches, and one tiled product (product16_kernel) serves both
// directions; the backward pass lays W out transposed.
//
// The 16-bit form of W for the tiled product is fp16 whatever the rows' type, as it keeps 11 bits where bf16
// would keep 8. It is exact: NVFP4 and MXFP4 take no more, and INT4's (q - z) s, 12 bits with bf16 scales and 15
// with fp16 ones, comes apart in one of two ways (see in_two and group_sums). So that exponents are kept, a
// column of the product has a power of two of its own (linear_prep_kernel), which holds INT4 scales down to 2^-24
// of the largest that share it, and bf16 rows enter as fp16 times a power of two of their own (exact down to
// 2^-29 of the row's largest element, and within 2^-39 of it below; 2^-27 and 2^-35 where sums of groups
// follow). Both come back in fp32.
#include <algorithm>

#include "packed.h"

namespace hmoe {

// ------------------------------------------------------------------------------------------
// few rows
// ------------------------------------------------------------------------------------------

struct LinearRows {
  Packed w;
  const uint16_t* x;
  long xs;
  int M, K, N;
  const uint16_t* base;
  long bs;
  uint16_t* y;
  long ys;
};

// Up to 16 rows, K at least 256: a wave keeps its PX pairs of steps of the rows in registers (x is
// read once a block, however many columns the block takes), and the codes of the next columns are
// requested pair by pair as those of the present ones are used up. A block takes items of 16 R
// columns, grid-strided; the waves' sums of an item meet in LDS. Bound by HBM where items are many (16
// rows, 2048 to 100001, MXFP4: 27 us, 4.1 TB/s), by latency and cold code else (1 row, 2048 to 1536: 4).
template <int F, int X, int R, int PX, bool EXACT>
__global__ __launch_bounds__(512, PX == 1 ? 4 : 2) void linear_wide_kernel(LinearRows p) {
  extern __shared__ float red[];   // [2][waves][R * 256]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int K = p.K, items = (p.N + 16 * R - 1) / (16 * R);
  const int pairs = (K + 255) / 256;
  const PairShare share = pair_share(wave, pairs, PX);
  u32x4 a[PX][2][1][4][1];
  PairCodes c[PX][R];
  StepScales<F, 2 * PX> now[R], then[R];
  // A tile that would end past N starts earlier (rows past N are stand-ins only where N < 16); the
  // columns before its own are another item's.
  const TileLane<EXACT> at = tile_lane<F, 2 * PX, EXACT>(lane, K, p.N, 2 * share.first);
  auto tile_of = [&](int item, int r) __attribute__((always_inline)) {
    return max(0, min(item * (16 * R) + 16 * r, p.N - 16));
  };
  auto scales = [&](StepScales<F, 2 * PX>(&to)[R], int item) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const TileBase t = tile_base<F>(p.w, tile_of(item, r), K, 2 * share.first);
      load_scales<F, 2 * PX, EXACT>(to[r], t.s, t.z, at);
    }
  };
  auto codes = [&](int j, int item) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      load_pair(c[j][r], tile_base<F>(p.w, tile_of(item, r), K, 2 * (share.first + j)).q, at, share.first + j == pairs - 1);
  };
  int item = blockIdx.x;
  scales(now, item);
#pragma unroll
  for (int j = 0; j < PX; ++j) codes(j, item);
  // rows past M are stand-ins: their sums are not written
  const uint16_t* x = p.x + (long)min(lane & 15, p.M - 1) * p.xs + (lane >> 4) * 8;
#pragma unroll
  for (int j = 0; j < 2 * PX; ++j) load_pair_rows<F, EXACT>(a[j >> 1][j & 1], x, 2 * share.first + j, K);
  const float g = F == kNv ? p.w.g[0] : 1.f;
  for (int buf = 0;; buf ^= 1) {
    const int next = item + gridDim.x;
    f32x4 acc[R][1];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      acc[r][0] = f32x4{0.f, 0.f, 0.f, 0.f};
      default_zeros(now[r], p.w.z);
    }
    auto products = [&](auto P) __attribute__((always_inline)) {
      constexpr int j = decltype(P)::value;
      if (share.first + j < share.own) return;
#pragma unroll
      for (int r = 0; r < R; ++r) pair_product<F, X, X, PX, j>(acc[r], c[j][r], now[r], a[j]);
    };
    // the two cases apart: a load behind a condition would make the waits count on its absence
    if (next < items) {
      scales(then, next);
      each<PX>([&](auto P) __attribute__((always_inline)) {
        products(P);
        codes(decltype(P)::value, next);
      });
#pragma unroll
      for (int r = 0; r < R; ++r) now[r] = then[r];
    } else {
      each<PX>(products);
    }
    float* sums = red + buf * (waves * R * 256);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[(wave * R + r) * 256 + i * 64 + lane] = acc[r][0][i];
    __syncthreads();
    for (int o = threadIdx.x; o < R * 256; o += blockDim.x) {
      const int l = o & 63, m = (l >> 4) * 4 + ((o >> 6) & 3);
      const int first = item * (16 * R) + 16 * (o >> 8), n = tile_of(item, o >> 8) + (l & 15);
      if (m >= p.M || n < first || n >= p.N) continue;
      float v = 0.f;
      for (int w = 0; w < waves; ++w) v += sums[w * (R * 256) + o];
      v *= g;
      if (p.base) v += to_f32<X>(p.base[m * p.bs + n]);
      p.y[m * p.ys + n] = from_f32<X>(v);
    }
    if (next >= items) return;
    item = next;
  }
}

template <int F, int X, int R, int PX, bool EXACT>
hipError_t run_wide(const LinearRows& p, hipStream_t s) {
  const int items = (p.N + 16 * R - 1) / (16 * R), waves = ((p.K + 255) / 256 + PX - 1) / PX;
  const int blocks = std::min(items, 256 * (PX == 1 ? 16 / waves : 1));
  hipLaunchKernelGGL((linear_wide_kernel<F, X, R, PX, EXACT>), dim3((unsigned)blocks), dim3((unsigned)(waves * 64)),
                     (size_t)2 * waves * R * 1024, s, p);
  return hipGetLastError();
}

// eight waves of four pairs, or of two where the last pair is partial
constexpr int wide_max_k(bool exact) { return 8 * (exact ? 4 : 2) * 256; }

template <int F, int X>
hipError_t launch_wide(const LinearRows& p, hipStream_t s) {
  const int pairs = (p.K + 255) / 256;
  const bool two = p.N >= 256 * 32;
  if (p.K % 256) return pairs <= 8 ? run_wide<F, X, 1, 1, false>(p, s) : run_wide<F, X, 1, 2, false>(p, s);
  if (pairs <= 8) return two ? run_wide<F, X, 2, 1, true>(p, s) : run_wide<F, X, 1, 1, true>(p, s);
  if (pairs <= 16) return two ? run_wide<F, X, 2, 2, true>(p, s) : run_wide<F, X, 1, 2, true>(p, s);
  if (pairs <= 24) return run_wide<F, X, 1, 3, true>(p, s);
  return run_wide<F, X, 1, 4, true>(p, s);
}

// Fewer than 256 columns: a wave takes 16 R columns n and 16 T rows m, and the one or two steps of K.
template <int F, int X, int R, int T>
__global__ __launch_bounds__(64) void linear_rows_kernel(LinearRows p) {
  const int lane = threadIdx.x;
  const int n0 = blockIdx.x * (16 * R), m0 = blockIdx.y * (16 * T);
  const int K = p.K;
  PackedRow row[R];
#pragma unroll
  for (int r = 0; r < R; ++r) row[r] = packed_row<F>(p.w, min(n0 + 16 * r + (lane & 15), p.N - 1), K, lane);
  const uint16_t* xr[T];   // rows past M are stand-ins: their sums are not written
#pragma unroll
  for (int t = 0; t < T; ++t) xr[t] = p.x + (long)min(m0 + 16 * t + (lane & 15), p.M - 1) * p.xs + (lane >> 4) * 8;
  f32x4 acc[R][T];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int step = 0; step * 128 < K; ++step) {
    const int blocks = step_blocks<false>(step, K);
    Codes<F> c[R];
    u32x4 a[1][4][T];
#pragma unroll
    for (int r = 0; r < R; ++r) load_step<F, false>(c[r], row[r], step, K, lane);
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int t = 0; t < T; ++t) {
        a[0][b][t] = load16(xr[t] + step * 128 + min(b, blocks - 1) * 32);
        if constexpr (is_int4(F)) a[0][b][t] = int4_order(a[0][b][t]);
      }
#pragma unroll
    for (int r = 0; r < R; ++r) step_product<F, X, X, T>(acc[r], c[r], a, blocks);
  }
  const float g = F == kNv ? p.w.g[0] : 1.f;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + 16 * r + (lane & 15), m = m0 + 16 * t + (lane >> 4) * 4 + i;
        if (m >= p.M || n >= p.N) continue;
        float v = acc[r][t][i] * g;
        if (p.base) v += to_f32<X>(p.base[m * p.bs + n]);
        p.y[m * p.ys + n] = from_f32<X>(v);
      }
}

// Rows of at least 256 columns: 16 R columns n and 16 T rows m a block, pairs of steps dealt to its waves.
// The rows' fragments of a step meet the codes of R tiles each; the second step's come while the first is
// multiplied. Bound by the address unit (a fragment touches 16 lines of x): 64 rows 6144 to 4096, NVFP4, 26 us.
template <int F, int X, int R, int T, bool EXACT>
__global__ __launch_bounds__(512, 2) void linear_rows_pair_kernel(LinearRows p) {
  extern __shared__ float red[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * (16 * R), m0 = blockIdx.y * (16 * T), K = p.K, pairs = (K + 255) / 256;
  auto tile_of = [&](int r) { return max(0, min(n0 + 16 * r, p.N - 16)); };   // as in linear_wide_kernel
  const uint16_t* x[T];   // rows past M are stand-ins: their sums are not written
#pragma unroll
  for (int t = 0; t < T; ++t) x[t] = p.x + (long)min(m0 + 16 * t + (lane & 15), p.M - 1) * p.xs + (lane >> 4) * 8;
  f32x4 acc[R][T];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int pair = wave; pair < pairs; pair += waves) {
    PairCodes c[R];
    StepScales<F, 2> v[R];
    const TileLane<EXACT> at = tile_lane<F, 2, EXACT>(lane, K, p.N, 2 * pair);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const TileBase b = tile_base<F>(p.w, tile_of(r), K, 2 * pair);
      load_scales<F, 2, EXACT>(v[r], b.s, b.z, at);
      load_pair(c[r], b.q, at, pair == pairs - 1);
    }
    u32x4 a[1][4][T];
    auto rows = [&](int step) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int col = step * 128 + b * 32;
#pragma unroll
        for (int t = 0; t < T; ++t)
          a[0][b][t] = EXACT ? load16(x[t] + col) : load16(x[t] + min(col, K - 32)) & (col < K ? ~0u : 0u);
      }
    };
    rows(2 * pair);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      default_zeros(v[r], p.w.z);
      split_pair(c[r]);
    }
#pragma nounroll   // once through cold code for both steps
    for (int step = 0;; ++step) {
      if constexpr (is_int4(F)) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int t = 0; t < T; ++t) a[0][b][t] = int4_order(a[0][b][t]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        Codes<F> k;
        k.q = c[r].a;
        take_scales_of<F>(k, v[r], step);
        step_product<F, X, X, T>(acc[r], k, a, 4);
      }
      if (step) break;
      rows(2 * pair + 1);
#pragma unroll
      for (int r = 0; r < R; ++r) c[r].a = c[r].b;
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[(wave * (R * T) + r * T + t) * 256 + i * 64 + lane] = acc[r][t][i];
  __syncthreads();
  const float g = F == kNv ? p.w.g[0] : 1.f;
  for (int o = threadIdx.x; o < R * T * 256; o += blockDim.x) {
    const int l = o & 63, i = (o >> 6) & 3, rt = o >> 8;
    const int first = n0 + 16 * (rt / T), n = tile_of(rt / T) + (l & 15), m = m0 + 16 * (rt % T) + (l >> 4) * 4 + i;
    if (m >= p.M || n < first || n >= p.N) continue;
    float v = 0.f;
    for (int w = 0; w < waves; ++w) v += red[w * (R * T * 256) + o];
    v *= g;
    if (p.base) v += to_f32<X>(p.base[m * p.bs + n]);
    p.y[m * p.ys + n] = from_f32<X>(v);
  }
}

template <int F, int X, int R, int T>
hipError_t run_rows_pairs(const LinearRows& p, hipStream_t s) {
  const int waves = std::min(8, (p.K + 255) / 256);
  const dim3 grid((unsigned)((p.N + 16 * R - 1) / (16 * R)), (unsigned)((p.M + 16 * T - 1) / (16 * T)));
  const size_t lds = (size_t)waves * R * T * 1024;
  if (p.K % 256 == 0)
    hipLaunchKernelGGL((linear_rows_pair_kernel<F, X, R, T, true>), grid, dim3((unsigned)(waves * 64)), lds, s, p);
  else
    hipLaunchKernelGGL((linear_rows_pair_kernel<F, X, R, T, false>), grid, dim3((unsigned)(waves * 64)), lds, s, p);
  return hipGetLastError();
}

template <int F, int X, int R, int T>
hipError_t run_rows(const LinearRows& p, hipStream_t s) {
  hipLaunchKernelGGL((linear_rows_kernel<F, X, R, T>),
                     dim3((unsigned)((p.N + 16 * R - 1) / (16 * R)), (unsigned)((p.M + 16 * T - 1) / (16 * T))), dim3(64), 0, s, p);
  return hipGetLastError();
}

// Rows of a block of the packed product past 32: what the registers hold, less where every 32 columns have
// a scale to multiply the sum by
template <int F, int X>
constexpr int rows_tile() { return F == kI32 || (F == kMx && X == kHf) ? 32 : 64; }

template <int F, int X>
hipError_t launch_rows(const LinearRows& p, hipStream_t s) {
  if (p.M <= 16 && p.K >= 256 && p.K <= wide_max_k(p.K % 256 == 0)) return launch_wide<F, X>(p, s);
  if (p.K >= 256) {
    if (p.M <= 16) return run_rows_pairs<F, X, 1, 1>(p, s);
    constexpr int T = rows_tile<F, X>() / 16;
    // one tile of columns a block where two would leave half of the CUs without one
    const bool one = (long)((p.N + 31) / 32) * ((p.M + 16 * T - 1) / (16 * T)) <= 128;
    if (p.M <= 32) return one ? run_rows_pairs<F, X, 1, 2>(p, s) : run_rows_pairs<F, X, 2, 2>(p, s);
    return one ? run_rows_pairs<F, X, 1, T>(p, s) : run_rows_pairs<F, X, 2, T>(p, s);
  }
  if (p.M <= 16) return run_rows<F, X, 1, 1>(p, s);
  if (p.M <= 32) return run_rows<F, X, 2, 2>(p, s);
  return run_rows<F, X, 2, 4>(p, s);
}

// ------------------------------------------------------------------------------------------
// many rows: operands of the tiled product
// ------------------------------------------------------------------------------------------
// Both operands are fp16 in fragment order: tiles of 16 rows by 32 of the reduction axis, 1 KiB each
// with the 16 bytes of MFMA lane l at 16 l, all blocks of a tile's rows behind one another. So a
// wave copies a tile into LDS by one contiguous load, and its reads there are contiguous too. The
// reduction axis is padded with zeros to whole blocks; rows past the last are stand-ins.
//
// Columns of the product are dealt to tiles eight apart: tile 8 g + i holds columns 128 g + 8 c + i
// for c = 0 .. 15. Then a lane's sums of eight tiles are eight neighbours of a row of y, and the
// transposed form of W comes out of 8 x 8 blocks of codes in one lane's registers.
constexpr int kBlockK = 32;
constexpr long kSlabBytes = 64l << 20;   // of the 16-bit form of W at a time, each of its parts: a quarter of the Infinity Cache
constexpr int kPrepThreads = 1024;
constexpr int kMaxSplits = 4;   // shares of the reduction axis of the tiled product
constexpr int kTickets = 8192;  // of a product: of the tiles with shares, or of 128 columns each

struct Prep {
  const uint16_t* x;   // [M, C]
  long xs;
  int M, C, blocks;    // blocks of 32 of the reduction axis
  int sums;            // blocks of sums over a group each behind them, twice (see group_sums)
  uint16_t* rows;      // fragment order
  int* ea;             // [M]
  int row_blocks;      // thread blocks for the rows; the others take exponents
  Packed w;
  int K, N;
  int* eb;             // exponents of the product's columns
  int* done;           // tickets of the products, cleared here
};

// INT4 with bf16 scales and zero points: a weight takes 12 bits, one more than fp16 has. The tiled product
// takes it apart, (q - z) s = (q - 8) s + (8 - z) s, into two of 11, and the second is the same for a group.
// Forward, it meets the sum of the group's x, so that the reduction axis goes on with the groups:
//   sum_k x[k] (q[k] - 8) s[g(k)]  +  sum_g (sum_(k of g) x[k]) (8 - z[g]) s[g]
// with the sums as two fp16 numbers 2^-kSumShift as large, in two runs of blocks. Backward, the product of dy
// and (8 - z) s is added to all columns of a group. Both scales leave room for what a sum of 128 takes. 4096
// rows 6144 to 4096, g64, take 240 us, 4001 rows of the gradient 273; rounded to fp16 234 and 255, as two numbers
// about 376 and 405.
constexpr int kSumShift = 3, kSumRowTop = 10, kSumScaleTop = 8;

// The sums over the groups of the tile's rows, behind their blocks: those of the rows times 2^-(e + kSumShift).
template <int G>
__device__ __forceinline__ void group_sums(const Prep& p, const uint16_t* x, int tile, int e, int wave, int waves) {
  const int lane = threadIdx.x & 63, groups = p.K / G;
  uint16_t* out = p.rows + ((long)tile * (p.blocks + 2 * p.sums) + p.blocks) * 512 + lane * 8;
  for (int u = wave; u < p.sums * 8; u += waves) {   // an eighth of a block: one group a lane
    const int b = u >> 3, g = b * 32 + (lane >> 4) * 8 + (u & 7);
    float sum = 0.f;
    if (g < groups)
#pragma unroll
      for (int c = 0; c < G; c += 8) {
        const u32x4 v = load16(x + (long)g * G + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = v[i];
          sum += ldexpf(bf16_lo(w), -e - kSumShift) + ldexpf(bf16_hi(w), -e - kSumShift);
        }
      }
    const uint32_t hi = pack_f16(sum, sum) & 0xFFFFu;
    const float rest = sum - fp16_to_f32(hi);
    out[(long)b * 512 + (u & 7)] = (uint16_t)hi;
    out[(long)(p.sums + b) * 512 + (u & 7)] = (uint16_t)pack_f16(rest, rest);
  }
}

// Rows of x: 16 a block. bf16 goes to fp16 times 2^-e with e of the row's largest finite |x|, which
// lands in [2^14, 2^15), or at 2^kSumRowTop where sums follow.
template <int F, int X>
__device__ __forceinline__ void prep_rows(const Prep& p, int tile, uint32_t (&part)[kPrepThreads / 64][16]) {
  constexpr int kWaves = kPrepThreads / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = tile * 16 + (lane & 15);
  const uint16_t* x = p.x + (long)min(m, p.M - 1) * p.xs;
  auto load = [&](int b) {
    const int c = b * kBlockK + (lane >> 4) * 8;
    if (c + 8 <= p.C) return load16(x + c);
    u32x4 v = {0u, 0u, 0u, 0u};
    for (int i = 0; i < 8; ++i)
      if (c + i < p.C) {
        const uint32_t h = (uint32_t)x[c + i] << (16 * (i & 1));
        v[0] |= i >> 1 == 0 ? h : 0u;
        v[1] |= i >> 1 == 1 ? h : 0u;
        v[2] |= i >> 1 == 2 ? h : 0u;
        v[3] |= i >> 1 == 3 ? h : 0u;
      }
    return v;
  };
  uint16_t* out = p.rows + (long)tile * (p.blocks + 2 * p.sums) * 512 + lane * 8;
  auto store = [&](int b, u32x4 v, int e) {
    if constexpr (X == kBf) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = v[i];
        v[i] = pack_f16(ldexpf(bf16_lo(w), -e), ldexpf(bf16_hi(w), -e));
      }
    }
    *reinterpret_cast<u32x4*>(out + (long)b * 512) = v;
  };
  // The wave's first HELD blocks stay in registers from the search for the largest to the writing.
  constexpr int HELD = 12;
  const int whole = p.C / kBlockK;   // blocks inside C
  u32x4 held[HELD];
#pragma unroll
  for (int j = 0; j < HELD; ++j)
    if (wave + j * kWaves < whole) held[j] = load16(x + (wave + j * kWaves) * kBlockK + (lane >> 4) * 8);
  int e = 0;
  if constexpr (X == kBf) {
    uint32_t top = 0;   // largest finite |x|, as bits
    auto take = [&](const u32x4& v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = v[i] & 0x7FFFu, hi = (v[i] >> 16) & 0x7FFFu;
        top = max(top, lo < 0x7F80u ? lo : 0u);
        top = max(top, hi < 0x7F80u ? hi : 0u);
      }
    };
#pragma unroll
    for (int j = 0; j < HELD; ++j)
      if (wave + j * kWaves < whole) take(held[j]);
    for (int b = wave + HELD * kWaves; b < whole; b += kWaves) take(load(b));
    if (whole < p.blocks && wave == 0) take(load(whole));
    top = max(top, xlane_u32<32>(top));
    top = max(top, xlane_u32<16>(top));
    if (lane < 16) part[wave][lane] = top;
    __syncthreads();
    top = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = max(top, part[w][lane & 15]);
    if (top) e = (int)(top >> 7) - 127 - (p.sums ? kSumRowTop : 14);
  }
#pragma unroll
  for (int j = 0; j < HELD; ++j)
    if (wave + j * kWaves < whole) store(wave + j * kWaves, held[j], e);
  for (int b = wave + HELD * kWaves; b < whole; b += kWaves) store(b, load(b), e);
  if (whole < p.blocks && wave == 0) store(whole, load(whole), e);
  if (wave == 0 && lane < 16 && m < p.M) p.ea[m] = e;
  if constexpr (is_int4(F) && X == kBf) group_sums<group_of(F)>(p, x, tile, e, wave, kWaves);
}

// The exponent of a scale where it is finite and not zero
template <int F, int S>
__device__ __forceinline__ int scale_exponent(const Packed& w, long at) {
  if constexpr (F == kMx) {
    const int b = w.s[at];
    return b < 255 ? b - 127 : -1000;
  } else {
    const float s = fabsf(to_f32<S>(reinterpret_cast<const uint16_t*>(w.s)[at]));
    return s > 0.f && s < INFINITY ? ilogbf(s) : -1000;
  }
}
// with the largest scale of a column of the product at exponent `top`, W 2^-e fits fp16: the largest
// lands in [2^10, 2^11), or at 2^12 for MXFP4, times 16, or 6, below 2^15; with sums of groups in the rows
// at 2^kSumScaleTop, as (8 - z) s enters 2^kSumShift as large
template <int F>
__device__ __forceinline__ int column_exponent(int top, bool sums) {
  return top == -1000 ? 0 : top - (F == kMx ? 12 : sums ? kSumScaleTop : 10);
}

// What the product needs besides W: its rows as fp16, an exponent for each of its columns (NVFP4 needs
// none: e2m1 * e4m3 is a number of fp16 as it is), and its tickets at zero. Forward, a column is a row
// n of W: a wave takes one. Backward it is a column k, with one exponent for its group over all n: a
// block takes 8 groups, its lanes 8 rows of them at a time.
template <int F, int X, bool BACK>
__global__ __launch_bounds__(kPrepThreads) void linear_prep_kernel(Prep p) {
  constexpr int kWaves = kPrepThreads / 64, G = group_of(F);
  __shared__ uint32_t part[kWaves][16];
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < kTickets; i += kPrepThreads) p.done[i] = 0;
  if ((int)blockIdx.x < p.row_blocks) return prep_rows<F, X>(p, blockIdx.x, part);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.x - p.row_blocks, groups = p.K / G;
  if constexpr (F == kNv) {
    return;
  } else if constexpr (!BACK) {
    const int n = b * kWaves + wave;
    if (n >= p.N) return;
    int top = -1000;
    for (int g = lane; g < groups; g += 64) top = max(top, scale_exponent<F, X>(p.w, (long)n * groups + g));
    for (int d = 32; d; d >>= 1) top = max(top, __shfl_xor(top, d));
    if (lane == 0) p.eb[n] = column_exponent<F>(top, p.sums);
  } else {
    const int g = b * 8 + (lane & 7);
    int top = -1000;
    for (int n = wave * 8 + (lane >> 3); n < p.N; n += 8 * kWaves * 8) {
      int e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        e[j] = scale_exponent<F, X>(p.w, (long)min(n + j * 8 * kWaves, p.N - 1) * groups + min(g, groups - 1));
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, e[j]);
    }
    for (int d = 32; d >= 8; d >>= 1) top = max(top, __shfl_xor(top, d));
    if (lane < 8) part[wave][lane] = (uint32_t)top;
    __syncthreads();
    static_assert(8 * G <= kPrepThreads, "a thread a column");
    if (threadIdx.x < 8 * G) {
      const int i = threadIdx.x / G, k = (b * 8 + i) * G + threadIdx.x % G;
      top = -1000;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = max(top, (int)part[w][i]);
      if (k < p.K) p.eb[k] = column_exponent<F>(top, false);
    }
  }
}

// INT4 with fp16 scales takes up to 15 bits: two fp16 numbers a weight, in blocks of the reduction axis behind
// one another. 4096 rows 6144 to 4096 take 370 us, as one number 235. With bf16 scales and z = 8 it takes 11.
template <int F, int S>
constexpr bool in_two() { return is_int4(F) && S == kHf; }

struct Weights16 {
  Packed w;
  int K, N, first, cols, blocks;   // the slab's first column of the product and their number; blocks of the rows
  const uint8_t* z;                // zero points that were taken out of w, and the blocks of their sums
  int sums;
  const int* eb;
  uint16_t* out;
};

// Eight codes times eight scales as fp16, in their order: the scales' pairs (0 1) (2 3) .. for E2M1,
// (0 4) (1 5) .. for INT4, and the zero points' 16 + z likewise. INT4 takes up to 16 bits: what fp16 leaves
// of a product goes to `low`, if it is wanted, and is exact there (its last place is that of the scale).
template <int F>
__device__ __forceinline__ u32x4 scaled_codes(uint32_t w, const uint32_t (&s)[4], const uint32_t (&z)[4], u32x4* low = nullptr) {
  auto half2 = [](uint32_t a) { return __builtin_bit_cast(f16x2, a); };
  auto bits = [](f16x2 a) { return __builtin_bit_cast(uint32_t, a); };
  const u32x4 v = is_int4(F) ? int4_operand<kHf>(w) : e2m1_operand<kHf>(w);
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t vi = v[i];
    const f16x2 c = is_int4(F) ? half2(vi) - half2(z[i]) : half2(vi), p = c * half2(s[i]);
    hi[i] = bits(p);
    lo[i] = is_int4(F) && low ? bits(__builtin_elementwise_fma(c, half2(s[i]), -p)) : 0u;
  }
  if constexpr (!is_int4(F)) return u32x4{hi[0], hi[1], hi[2], hi[3]};
  auto order = [](const uint32_t(&a)[4]) {
    return u32x4{__builtin_amdgcn_perm(a[1], a[0], 0x05040100u), __builtin_amdgcn_perm(a[3], a[2], 0x05040100u),
                 __builtin_amdgcn_perm(a[1], a[0], 0x07060302u), __builtin_amdgcn_perm(a[3], a[2], 0x07060302u)};
  };
  if (low) *low = order(lo);
  return order(hi);
}
// A group's scale times 2^-e as fp16 bits, and 16 + z
template <int F, int S>
__device__ __forceinline__ uint32_t scale16(const Packed& w, long at, int e) {
  float s;
  if constexpr (F == kNv) s = e4m3_to_f32<0>(w.s[at]);
  else if constexpr (F == kMx) s = ldexpf(e8m0_value(w.s[at]), -e);
  else s = ldexpf(to_f32<S>(reinterpret_cast<const uint16_t*>(w.s)[at]), -e);
  return pack_f16(s, s) & 0xFFFFu;
}
template <int F>
__device__ __forceinline__ uint32_t zero16(const Packed& w, long at) {
  if constexpr (!is_int4(F)) return 0u;
  else return 0x4C00u | ((w.z ? w.z[at] & 15u : 8u) << 6);
}

// (8 - z) s 2^-e of a group: at most 11 bits with a bf16 scale
template <int S>
__device__ __forceinline__ float offset_weight(const Packed& w, const uint8_t* z, long at, int e) {
  return ldexpf((8.f - (float)(z[at] & 15u)) * to_f32<S>(reinterpret_cast<const uint16_t*>(w.s)[at]), -e);
}

// The 16-bit form of rows [first, first + cols) of W, columns of the product. A wave takes one tile and
// four steps of 128 of K, or a block of groups.
template <int F, int S>
__global__ __launch_bounds__(512) void weights16_kernel(Weights16 p) {
  constexpr int G = group_of(F);
  const int lane = threadIdx.x & 63, i = threadIdx.x >> 6;
  const int col = blockIdx.x * 128 + 8 * (lane & 15) + i;
  const long n = p.first + min(col, p.cols - 1);
  const int e = F == kNv ? 0 : p.eb[n];
  const long groups = n * (p.K / G);
  constexpr int kParts = in_two<F, S>() ? 2 : 1;
  uint16_t* out = p.out + (long)(blockIdx.x * 8 + i) * (p.blocks * kParts + 2 * p.sums) * 512 + lane * 8;
  if constexpr (is_int4(F) && S == kBf)
    if (const int b = (int)blockIdx.y - (p.blocks + 15) / 16; b >= 0) {   // (8 - z) s, for both parts of the sums
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int g = b * 32 + (lane >> 4) * 8 + j;
        v[j] = g < p.K / G ? offset_weight<S>(p.w, p.z, groups + g, e - kSumShift) : 0.f;
      }
      const u32x4 h = {pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]), pack_f16(v[6], v[7])};
      *reinterpret_cast<u32x4*>(out + (long)(p.blocks + b) * 512) = h;
      *reinterpret_cast<u32x4*>(out + (long)(p.blocks + p.sums + b) * 512) = h;
      return;
    }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int b0 = (blockIdx.y * 4 + j) * 4;      // first block of the step
    if (b0 >= p.blocks) return;
    u32x4 q = *reinterpret_cast<const u32x4*>(p.w.q + n * (p.K / 2) + min(b0 + (lane >> 4), p.blocks - 1) * 16);
    turn4(q);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (b0 + t >= p.blocks) continue;
      const long g = groups + ((b0 + t) * kBlockK + (lane >> 4) * 8) / G;
      const uint32_t s1 = scale16<F, S>(p.w, g, e), z1 = zero16<F>(p.w, g);
      const uint32_t s2 = s1 | s1 << 16, z2 = z1 | z1 << 16;
      const uint32_t s[4] = {s2, s2, s2, s2}, z[4] = {z2, z2, z2, z2};
      u32x4 low;
      u32x4* to = reinterpret_cast<u32x4*>(out + (long)(b0 + t) * kParts * 512);
      to[0] = scaled_codes<F>(q[t], s, z, kParts == 2 ? &low : nullptr);
      if constexpr (kParts == 2) to[64] = low;
    }
  }
}

// An 8 x 8 block of codes turned: in, dword j holds row j's eight codes; out, dword i column i's.
__device__ __forceinline__ void turn_codes(uint32_t (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {   // halves
    const uint32_t a = v[j], b = v[j + 4];
    v[j] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    v[j + 4] = __builtin_amdgcn_perm(b, a, 0x07060302u);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)     // bytes
    if (!(j & 2)) {
      const uint32_t a = v[j], b = v[j + 2];
      v[j] = __builtin_amdgcn_perm(b, a, 0x06020400u);
      v[j + 2] = __builtin_amdgcn_perm(b, a, 0x07030501u);
    }
#pragma unroll
  for (int j = 0; j < 8; j += 2) {   // nibbles
    const uint32_t a = v[j], b = v[j + 1];
    v[j] = (a & 0x0F0F0F0Fu) | ((b & 0x0F0F0F0Fu) << 4);
    v[j + 1] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
  }
}

// 32 rows n of W, block `block` of the reduction axis, and the lane's eight columns from k on: take(i, operand,
// low) is given column k + i of rows 8 (lane >> 4) .. + 7 of the block as fp16 times 2^-e, zeros past N, and for
// INT4, if LOW, what that leaves of it. Each lane turns an 8 x 8 block of codes, and its rows' scales multiply
// what comes out.
template <int F, int S, bool LOW, typename Fn>
__device__ __forceinline__ void turned_block(const Packed& w, int K, int N, int block, int k, int e, int lane, Fn&& take) {
  constexpr int G = group_of(F);
  uint32_t v[8], s1[8], z1[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int row = block * kBlockK + (lane >> 4) * 8 + j;
    const long n = min(row, N - 1), g = n * (K / G) + k / G;
    v[j] = *reinterpret_cast<const uint32_t*>(w.q + n * (K / 2) + k / 2);
    s1[j] = scale16<F, S>(w, g, e);
    z1[j] = zero16<F>(w, g);
    if (row >= N) {   // 0, or (z - z), times 0
      v[j] = is_int4(F) ? ((z1[j] >> 6) & 15u) * 0x11111111u : 0u;
      s1[j] = 0u;
    }
  }
  turn_codes(v);
  uint32_t s[4], z[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int a = is_int4(F) ? j : 2 * j, b = is_int4(F) ? j + 4 : 2 * j + 1;
    s[j] = s1[a] | s1[b] << 16;
    z[j] = z1[a] | z1[b] << 16;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    u32x4 low;
    const u32x4 v16 = scaled_codes<F>(v[i], s, z, LOW ? &low : nullptr);
    take(i, v16, low);
  }
}

// The 16-bit form of columns [first, first + cols) of W. A wave takes a block of the reduction axis and
// 128 columns.
template <int F, int S>
__global__ __launch_bounds__(256) void weights16_turned_kernel(Weights16 p) {
  const int lane = threadIdx.x & 63, block = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (block >= p.blocks) return;
  const int k = p.first + min(blockIdx.y * 128 + 8 * (lane & 15), p.cols - 8);   // cols is a multiple of 32
  constexpr int kParts = in_two<F, S>() ? 2 : 1;
  turned_block<F, S, kParts == 2>(p.w, p.K, p.N, block, k, F == kNv ? 0 : p.eb[k], lane, [&](int i, u32x4 v, u32x4 low) {
    u32x4* to = reinterpret_cast<u32x4*>(p.out + ((long)(blockIdx.y * 8 + i) * p.blocks + block) * kParts * 512 + lane * 8);
    to[0] = v;
    if constexpr (kParts == 2) to[64] = low;
  });
}

// (8 - z) s of the groups [first, first + cols), columns of a product over n, times the 2^-e of their columns
// of W. A block takes a block of the reduction axis and 128 groups, a wave one tile of them.
template <int F>
__global__ __launch_bounds__(512) void offsets16_turned_kernel(Weights16 p) {
  constexpr int G = group_of(F);
  const int lane = threadIdx.x & 63, i = threadIdx.x >> 6, block = blockIdx.x, groups = p.K / G;
  const int g = min(p.first + (int)blockIdx.y * 128 + 8 * (lane & 15) + i, groups - 1), e = p.eb[g * G];
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int n = block * kBlockK + (lane >> 4) * 8 + j;
    v[j] = n < p.N ? offset_weight<kBf>(p.w, p.z, (long)n * groups + g, e) : 0.f;
  }
  *reinterpret_cast<u32x4*>(p.out + ((long)(blockIdx.y * 8 + i) * p.blocks + block) * 512 + lane * 8) =
      u32x4{pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]), pack_f16(v[6], v[7])};
}

// Up to 64 rows of the gradient without the 16-bit form in between: y[m, k] = base[m, k] + g 2^(ea[m] +
// eb[k]) sum_n a[m, n] W[n, k] 2^-eb[k], INT4 as two fp16 numbers (24 rows 2048 to 1536, g64: 19.3 us a call, 18.9
// as one). A block takes 128 columns, 16 T rows and a share of the blocks of the reduction axis, which its waves take in turn; the last block of the columns to finish adds
// the shares up in their order.
struct TurnedRows {
  Packed w;
  const uint16_t* a;    // M rows, fragment order
  const int* ea;
  const int* eb;        // null: 0
  int M, K, N, blocks;
  const uint16_t* base;
  long bs;
  uint16_t* y;
  long ys;
  int splits;
  float* sums;          // [splits][thread blocks][16 T * 128]
  int* done;
};
constexpr int kMaxTurnedSplits = 8;

template <int F, int X, int T>
__global__ __launch_bounds__(256) void linear_turned_kernel(TurnedRows p) {
  constexpr int kSums = 16 * T * 128;
  extern __shared__ float red[];   // [4][kSums]
  __shared__ int s_last;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k = min(blockIdx.x * 128 + 8 * (lane & 15), p.K - 8), e = F == kNv ? 0 : p.eb[k];
  f32x4 acc[T][8];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int tiles = (p.M + 15) / 16;
  for (int b = blockIdx.y * 4 + wave; b < p.blocks; b += p.splits * 4) {
    u32x4 a[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
      a[t] = *reinterpret_cast<const u32x4*>(p.a + ((long)min(t, tiles - 1) * p.blocks + b) * 512 + lane * 8);
    turned_block<F, X, is_int4(F)>(p.w, p.K, p.N, b, k, e, lane, [&](int i, u32x4 v, u32x4 low) {
#pragma unroll
      for (int t = 0; t < T; ++t) acc[t][i] = mfma16<kHf>(a[t], v, acc[t][i]);
      if constexpr (is_int4(F))   // the matrix cores have the time
#pragma unroll
        for (int t = 0; t < T; ++t) acc[t][i] = mfma16<kHf>(a[t], low, acc[t][i]);
    });
  }
  // [row][column]: a lane's eight sums of a row are neighbours
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f32x4* at = reinterpret_cast<f32x4*>(red + wave * kSums + (t * 16 + (lane >> 4) * 4 + j) * 128 + 8 * (lane & 15));
      at[0] = f32x4{acc[t][0][j], acc[t][1][j], acc[t][2][j], acc[t][3][j]};
      at[1] = f32x4{acc[t][4][j], acc[t][5][j], acc[t][6][j], acc[t][7][j]};
    }
  __syncthreads();
  const float g = F == kNv ? p.w.g[0] : 1.f;
  const int c0 = blockIdx.x * 128;
  auto finish = [&](int o, float v) {
    const int m = o >> 7, c = c0 + (o & 127);
    if (m >= p.M || c >= p.K) return;
    v = ldexpf(v * g, p.ea[m] + (F == kNv ? 0 : p.eb[c]));   // (g first: without it the value may lie past fp32)
    if (p.base) v += to_f32<X>(p.base[m * p.bs + c]);
    p.y[m * p.ys + c] = from_f32<X>(v);
  };
  const long share = (long)gridDim.x * kSums;
  float* sums = p.sums + (long)blockIdx.x * kSums;
  for (int o = threadIdx.x; o < p.M * 128; o += 256) {
    const float v = red[o] + red[kSums + o] + red[2 * kSums + o] + red[3 * kSums + o];
    if (p.splits == 1) finish(o, v);
    else __hip_atomic_store(sums + blockIdx.y * share + o, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (p.splits == 1) return;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    s_last = __hip_atomic_fetch_add(p.done + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.splits - 1;
  __syncthreads();
  if (!s_last) return;
#pragma nounroll
  for (int o = threadIdx.x; o < min(kSums, p.M * 128); o += 4 * 256) {   // all shares of four sums requested at once
    float u[4][kMaxTurnedSplits];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int z = 0; z < kMaxTurnedSplits; ++z)
        u[q][z] = __hip_atomic_load(sums + min(z, p.splits - 1) * share + o + q * 256, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v = 0.f;
#pragma unroll
      for (int z = 0; z < kMaxTurnedSplits; ++z) v += z < p.splits ? u[q][z] : 0.f;
      finish(o + q * 256, v);
    }
  }
}

// ------------------------------------------------------------------------------------------
// many rows: the tiled product
// ------------------------------------------------------------------------------------------

struct Product16 {
  const uint16_t* a;    // M rows, fragment order
  const int* ea;        // [M]
  const uint16_t* b;    // cols columns, fragment order
  const int* eb;        // [cols]; null: 0
  const float* g;       // NVFP4's scale of the matrix; null: 1
  int M, cols, blocks;  // blocks of the reduction axis as b has them
  const uint16_t* base; // [M, cols]; may be null
  long bs;
  uint16_t* y;
  long ys;
  int splits;           // shares of the reduction axis
  float* sums;          // [splits][thread blocks][threads][a thread's sums]
  int* done;            // a ticket a tile: zero before and after
  float* raw;           // where the sums go as they are, instead of y; null: nowhere
  const float* add;     // added to the sums: a value for each 2^add_shift columns; null: nothing
  long raw_row;         // rows of raw or add
  int add_shift;
};

template <int N>
__device__ __forceinline__ void wait_vmem_at_most() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// y[m, c] = base[m, c] + g 2^(ea[m] + eb[c]) sum_i a[m, i] b[c, i]. A wave takes TM x TN tiles, a block
// WM x WN waves. Blocks of the reduction axis pass through STAGES buffers in LDS, all but one of them in
// flight, loaded by copies that go past the registers; a wave reads the next block's fragments
// while it multiplies the present one's. With splits > 1 the block of a tile that finishes last adds the
// shares up in their order. 4096 rows 6144 to 4096 take 188 us, 1.1 PFLOP/s, near what LDS gives: a wave
// reads 12 KiB for 32 MFMAs. PARTS: blocks of b for each block of a. An output of so many rows of W that a slab is a
// few hundred columns leaves CUs without a tile: 128 rows of dy through a head of 100001 rows, 2048 columns, take
// eight slabs of 116 us.
template <int X, int TM, int TN, int WM, int WN, int STAGES, int PARTS>
__global__ __launch_bounds__(WM * WN * 64, 2) void product16_kernel(Product16 p) {
  constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
  constexpr int BM = WM * TM, BN = WN * TN, kChunks = BM + BN, kLoads = kChunks / kWaves;
  static_assert(BM % kWaves == 0 && BN % kWaves == 0, "a copy is of rows or of columns for all waves");
  __shared__ u32x4 buffer[STAGES][kChunks * 64];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  // A thread block runs on XCD (its number mod 8): each XCD gets a run of tiles, column tiles of the
  // same rows behind one another, so that its L2 holds their operands.
  const int tiles_b = (p.cols + 127) / 128 * 8, tiles_n = (tiles_b + BN - 1) / BN, tiles = gridDim.x;
  const int per = (tiles + 7) / 8, id = (int)blockIdx.x;
  int tile = (id & 7) * per + (id >> 3);
  const int full = tiles % 8 ? tiles % 8 : 8;     // XCDs with `per` tiles; the others have one less
  if ((id & 7) > full) tile -= (id & 7) - full;
  const int t_m = tile / tiles_n, t_n = tile % tiles_n;
  const int m0 = t_m * BM * 16;
  const int per_split = (p.blocks + p.splits - 1) / p.splits;
  const int from = blockIdx.y * per_split, to = min(p.blocks, from + per_split);
  // this wave's copies: chunk wave + i * kWaves of the stage, rows' tiles first
  const uint16_t* src[kLoads];
  uint32_t dst[kLoads];
  const int tiles_a = (p.M + 15) / 16;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int chunk = wave + i * kWaves;
    const long t = i * kWaves < BM ? min(t_m * BM + chunk, tiles_a - 1) : min(t_n * BN + chunk - BM, tiles_b - 1);
    src[i] = i * kWaves < BM ? p.a + t * (p.blocks / PARTS) * 512 : p.b + t * p.blocks * 512;
    dst[i] = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)&buffer[0][chunk * 64];
  }
  auto copy = [&](int block, int slot) {   // past the last: a stand-in that nobody reads, so that the waits can count
    block = min(block, to - 1);
    const long at_a = (long)(block / PARTS) * 512, at_b = (long)block * 512;
    const uint32_t off = (uint32_t)slot * (kChunks * 1024);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      // (a load into LDS may read m0 one wait state after it was written)
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst[i] + off), "v"(lane * 16),
                   "s"(src[i] + (i * kWaves < BM ? at_a : at_b))
                   : "memory", "m0");
  };
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 a[2][TM], b[2][TN];
  int slot = 0;   // of the block whose arrival was waited for last
  auto read = [&](u32x4(&fa)[TM], u32x4(&fb)[TN]) __attribute__((always_inline)) {
    const u32x4* s = buffer[slot];
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[i] = s[(wm * TM + i) * 64 + lane];
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[j] = s[(BM + wn * TN + j) * 64 + lane];
  };
  auto multiply = [&](const u32x4(&fa)[TM], const u32x4(&fb)[TN]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma16<kHf>(fa[i], fb[j], acc[i][j]);
  };
  // Block k is in LDS once each wave has waited for its own copies of it and all have met. The buffer
  // that is then filled held block k - 1, whose fragments every wave had before the meeting.
  auto arrive = [&](int block) __attribute__((always_inline)) {
    wait_vmem_at_most<(STAGES - 2) * kLoads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const int before = slot;
    slot = block == from ? 0 : slot + 1 == STAGES ? 0 : slot + 1;
    copy(block + STAGES - 1, block == from ? STAGES - 1 : before);
  };
  if (from < to) {
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) copy(from + i, i);
    arrive(from);
    read(a[0], b[0]);
    for (int k = from; k < to; k += 2) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // this block's fragments, before their buffer goes
      arrive(k + 1);
      read(a[1], b[1]);
      multiply(a[0], b[0]);
      if (k + 1 >= to) break;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      arrive(k + 2);
      read(a[0], b[0]);
      multiply(a[1], b[1]);
    }
    wait_vmem_at_most<0>();
  }
  // The sums go through LDS, so that what follows is a loop (unrolled over the registers it would be
  // 30 to 100 KB of code that each wave runs once): DI rows of tiles at a time, in the wave's own part.
  __syncthreads();
  constexpr int DI = TM * TN <= kChunks * STAGES / kWaves ? TM : TM / 2;
  f32x4* dump = reinterpret_cast<f32x4*>(&buffer[0][0]) + wave * (DI * TN * 64);
  const float g = p.g ? *p.g : 1.f;
  constexpr int kRun = TN < 8 ? TN : 8;      // neighbouring columns a lane has
  struct __attribute__((packed, aligned(2))) Run { uint16_t h[kRun]; };
#pragma unroll
  for (int i0 = 0; i0 < TM; i0 += DI) {
#pragma unroll
    for (int i = 0; i < DI; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) dump[(i * TN + j) * 64 + lane] = acc[i0 + i][j];
    if (DI == TM && p.splits > 1) {
      constexpr int kTiles = TM * TN;
      const long share = (long)gridDim.x * (kThreads * kTiles * 4);
      float* sums = p.sums + ((long)tile * kWaves + wave) * (kTiles * 256) + lane;
      float* own = sums + blockIdx.y * share;
#pragma nounroll
      for (int t = 0; t < kTiles; ++t) {
        const f32x4 v = dump[t * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          __hip_atomic_store(own + t * 256 + e * 64, v[e], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      wait_vmem_at_most<0>();
      __syncthreads();
      if (threadIdx.x == 0)
        s_last = __hip_atomic_fetch_add(p.done + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.splits - 1;
      __syncthreads();
      if (!s_last) return;
      if (threadIdx.x == 0) __hip_atomic_store(p.done + tile, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma nounroll
      for (int t = 0; t < kTiles; t += 4) {   // all shares of four tiles requested at once, added in their order
        float u[kMaxSplits][4][4];
#pragma unroll
        for (int z = 0; z < kMaxSplits; ++z)
#pragma unroll
          for (int q = 0; q < 16; ++q)
            u[z][q >> 2][q & 3] = __hip_atomic_load(sums + min(z, p.splits - 1) * share + t * 256 + q * 64,
                                                    __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int z = 0; z < kMaxSplits; ++z)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += z < p.splits ? u[z][q][e] : 0.f;
          dump[(t + q) * 64 + lane] = v;
        }
      }
    }
#pragma nounroll
    for (int j0 = 0; j0 < TN; j0 += kRun) {
      const int t = t_n * BN + wn * TN + j0, c = (t >> 3) * 128 + 8 * (lane & 15) + (t & 7);
      if (c >= p.cols) continue;
      int eb[kRun];
#pragma unroll
      for (int j = 0; j < kRun; ++j) eb[j] = p.eb ? p.eb[min(c + j, p.cols - 1)] : 0;
#pragma nounroll
      for (int r = 0; r < DI * 4; ++r) {
        const int m = m0 + (wm * TM + i0 + (r >> 2)) * 16 + (lane >> 4) * 4 + (r & 3);
        if (m >= p.M) continue;
        const int ea = p.ea[m];
        const float* from_lds = reinterpret_cast<const float*>(dump + ((r >> 2) * TN + j0) * 64 + lane) + (r & 3);
        if (X == kBf && PARTS == 1 && p.raw) {
#pragma unroll
          for (int j = 0; j < kRun; ++j)
            if (c + j < p.cols) p.raw[m * p.raw_row + c + j] = from_lds[j * 256];
          continue;
        }
        const float more = X == kBf && PARTS == 1 && p.add ? p.add[m * p.raw_row + (c >> p.add_shift)] : 0.f;
        float v[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j) v[j] = ldexpf((from_lds[j * 256] + more) * g, ea + eb[j]);
        uint16_t* y = p.y + m * p.ys + c;
        const uint16_t* base = p.base ? p.base + m * p.bs + c : nullptr;
        if (c + kRun <= p.cols) {
          Run o;
          if (base) o = *reinterpret_cast<const Run*>(base);
#pragma unroll
          for (int j = 0; j < kRun; ++j) o.h[j] = from_f32<X>(v[j] + (base ? to_f32<X>(o.h[j]) : 0.f));
          *reinterpret_cast<Run*>(y) = o;
        } else {
#pragma unroll
          for (int j = 0; j < kRun; ++j)
            if (c + j < p.cols) y[j] = from_f32<X>(v[j] + (base ? to_f32<X>(base[j]) : 0.f));
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------------------
// host
// ------------------------------------------------------------------------------------------

namespace {

constexpr int kRowsMax = 64;   // rows that the packed product takes at least, and the turned one at most

size_t pad256(size_t v) { return (v + 255) & ~size_t(255); }
long up(long v, long to) { return (v + to - 1) / to * to; }
int cdiv(long a, long b) { return (int)((a + b - 1) / b); }

// How a product of M rows and `cols` columns over `blocks` blocks runs. Larger tiles read less of LDS and L2 a
// product; smaller ones fill the card.
enum : int { kSmall, kMiddle, kWide, kLarge };
struct Tile16 {
  int tile = kLarge, splits = 1;
  int bm() const { return tile == kSmall ? 64 : tile == kMiddle ? 128 : 256; }
  int bn() const { return tile == kSmall ? 64 : tile == kLarge ? 256 : 128; }
  int tiles(long M, long cols) const { return cdiv(M, bm()) * cdiv(up(cols, 128), bn()); }
};
Tile16 tile16(long M, long cols, int blocks) {
  Tile16 p;
  // 256 x 256 a CU at once, or two of 256 x 128, one of which alone takes 0.6 of the time of two:
  // whichever's last round is fuller (384 large tiles 262 us, as 768 wide ones 214 to 229)
  const int large = p.tiles(M, cols);
  p.tile = kWide;
  const int wide = p.tiles(M, cols), rest = wide % 512;
  const double t_large = cdiv(large, 256), t_wide = wide / 512 + (rest == 0 ? 0. : rest <= 256 ? 0.6 : 1.);
  if (large >= 192 || wide >= 256) {
    p.tile = t_wide < t_large ? kWide : kLarge;
    return p;
  }
  // shares of at least eight blocks each
  const int most = std::max(1, std::min(kMaxSplits, blocks / 8));
  p.tile = kMiddle;
  if (p.tiles(M, cols) * most < 192) p.tile = kSmall;
  p.splits = std::max(1, std::min(512 / std::max(p.tiles(M, cols), 1), most));
  return p;
}

// How the tiled product of M rows and O columns over C runs, and its scratch. parts: blocks of W's 16-bit
// form for each block of the rows; sums: blocks of groups' sums behind the rows', twice; groups: columns of the
// product of dy and the zero points.
struct Plan16 {
  Tile16 main;
  int blocks = 0, parts = 1, sums = 0;
  long slab = 0;          // output columns a slab
  size_t rows = 0, ea = 0, eb = 0, weights = 0, shares = 0, done = 0, add = 0, total = 0;
  int all_blocks() const { return blocks * parts + 2 * sums; }
};
Plan16 plan16(long M, long C, long O, int parts, int sums, long groups) {
  Plan16 p;
  p.blocks = cdiv(C, kBlockK);
  p.parts = parts;
  p.sums = sums;
  p.slab = std::max<long>(256, kSlabBytes / (p.blocks * 64l) / 256 * 256);
  p.slab = std::min(p.slab, up(O, 256));
  p.main = tile16(M, std::min(p.slab, O), p.all_blocks());
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += pad256(bytes);
    return r;
  };
  p.rows = take((size_t)up(M, 16) * (p.blocks + 2 * sums) * 64);
  p.ea = take((size_t)M * 4);
  p.eb = take((size_t)up(O, 128) * 4);
  p.weights = take((size_t)up(p.slab, 128) * p.all_blocks() * 64);
  // an upper bound, so that more rows never need less: with shares there are at most 512 thread blocks
  // of at most 128 x 128
  p.shares = take(std::min<size_t>((size_t)kMaxSplits * up(M, 128) * up(p.slab, 128) * 4, 512ul * 128 * 128 * 4));
  p.done = take(kTickets * 4);
  p.add = take((size_t)M * groups * 4);
  p.total = at;
  return p;
}
// Of a call: F and X as the kernels have them; zeros: zero points come with it.
template <int F, int X, bool BACK>
Plan16 plan16_of(long M, long K, long N, bool zeros) {
  const long groups = is_int4(F) && X == kBf && zeros ? K / group_of(F) : 0;
  return plan16(M, BACK ? N : K, BACK ? K : N, in_two<F, X>() ? 2 : 1, BACK ? 0 : cdiv(groups, 32), BACK ? groups : 0);
}
// Scratch of any call
size_t tiled_scratch(long M, long K, long N, bool back) {
  auto most = [&](auto BACK) {
    constexpr bool B = decltype(BACK)::value;
    return std::max({plan16_of<kNv, kBf, B>(M, K, N, false).total, plan16_of<kI32, kHf, B>(M, K, N, false).total,
                     plan16_of<kI32, kBf, B>(M, K, N, true).total});
  };
  return back ? most(std::true_type{}) : most(std::false_type{});
}

// The same for linear_turned_kernel
struct PlanTurned {
  int t = 1, blocks = 0, columns = 0, splits = 1;
  size_t rows = 0, ea = 0, eb = 0, sums = 0, done = 0, total = 0;
};
PlanTurned plan_turned(int M, int K, int N) {
  PlanTurned p;
  p.t = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  p.blocks = cdiv(N, kBlockK);
  p.columns = cdiv(K, 128);
  // shares: to two blocks a CU, and a block for every wave
  p.splits = std::max(1, std::min({512 / p.columns, cdiv(p.blocks, 4), kMaxTurnedSplits}));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += pad256(bytes);
    return r;
  };
  p.rows = take((size_t)p.t * 16 * p.blocks * 64);
  p.ea = take((size_t)p.t * 16 * 4);
  p.eb = take((size_t)p.columns * 128 * 4);
  p.sums = take(p.splits > 1 ? (size_t)p.splits * p.columns * p.t * 16 * 128 * 4 : 0);
  p.done = take(kTickets * 4);
  p.total = at;
  return p;
}

#define RETURN_IF(expr)                    \
  do {                                     \
    const hipError_t err_ = (expr);        \
    if (err_ != hipSuccess) return err_;   \
  } while (0)

template <int F, int X, bool BACK>
hipError_t run_prep(const Prep& p, int blocks, hipStream_t s) {
  hipLaunchKernelGGL((linear_prep_kernel<F, X, BACK>), dim3((unsigned)blocks), dim3(kPrepThreads), 0, s, p);
  return hipGetLastError();
}
// (Backward that is few blocks, each of which goes through all rows of W: 18 us for 4096 rows of 6144 columns,
// g64, but 487 for the 100001 rows of a head of 2048, MXFP4.)
template <int F, bool BACK>
int exponent_blocks(int O) {
  return F == kNv ? 0 : BACK ? cdiv(O / group_of(F), 8) : cdiv(O, kPrepThreads / 64);
}

template <int X, int PARTS>
hipError_t run_product(const Product16& q, const Tile16& t, hipStream_t s) {
  const dim3 grid((unsigned)t.tiles(q.M, q.cols), (unsigned)t.splits);
  const dim3 block(t.tile == kLarge ? 512 : 256);
  switch (t.tile) {
    case kSmall: hipLaunchKernelGGL((product16_kernel<X, 2, 2, 2, 2, 4, PARTS>), grid, block, 0, s, q); break;
    case kMiddle: hipLaunchKernelGGL((product16_kernel<X, 4, 4, 2, 2, 4, PARTS>), grid, block, 0, s, q); break;
    case kWide: hipLaunchKernelGGL((product16_kernel<X, 8, 4, 2, 2, 3, PARTS>), grid, block, 0, s, q); break;
    default: hipLaunchKernelGGL((product16_kernel<X, 8, 4, 2, 4, 4, PARTS>), grid, block, 0, s, q);
  }
  return hipGetLastError();
}

template <int F, int X, bool BACK>
hipError_t launch_tiled(const Linear& p, char* scratch, hipStream_t s) {
  constexpr int kParts = in_two<F, X>() ? 2 : 1, G = group_of(F);
  const int C = BACK ? p.N : p.K, O = BACK ? p.K : p.N;
  const bool zeros = is_int4(F) && X == kBf && p.w.z;
  const Plan16 plan = plan16_of<F, X, BACK>(p.M, p.K, p.N, zeros);
  uint16_t* rows = reinterpret_cast<uint16_t*>(scratch + plan.rows);
  int* ea = reinterpret_cast<int*>(scratch + plan.ea);
  int* eb = reinterpret_cast<int*>(scratch + plan.eb);
  int* done = reinterpret_cast<int*>(scratch + plan.done);
  uint16_t* weights = reinterpret_cast<uint16_t*>(scratch + plan.weights);
  float* shares = reinterpret_cast<float*>(scratch + plan.shares);
  float* add = BACK && zeros ? reinterpret_cast<float*>(scratch + plan.add) : nullptr;
  const int row_blocks = cdiv(p.M, 16);
  const Prep prep{p.x, p.xs, p.M, C, plan.blocks, plan.sums, rows, ea, row_blocks, p.w, p.K, p.N, eb, done};
  RETURN_IF((run_prep<F, X, BACK>(prep, row_blocks + exponent_blocks<F, BACK>(O), s)));
  Packed alone = p.w;
  if (zeros) alone.z = nullptr;
  if constexpr (BACK && is_int4(F) && X == kBf)
    if (zeros)
      for (long o = 0; o < p.K / G; o += plan.slab) {
        const int cols = (int)std::min<long>(plan.slab, p.K / G - o);
        const Weights16 w{p.w, p.K, p.N, (int)o, cols, plan.blocks, p.w.z, 0, eb, weights};
        hipLaunchKernelGGL((offsets16_turned_kernel<F>), dim3((unsigned)plan.blocks, (unsigned)cdiv(cols, 128)), dim3(512), 0,
                           s, w);
        RETURN_IF(hipGetLastError());
        const Tile16 tile = tile16(p.M, cols, plan.blocks);
        const Product16 q{rows, ea, weights, nullptr, nullptr, p.M, cols, plan.blocks, nullptr, 0, nullptr, 0,
                          tile.splits, shares, done, add + o, nullptr, p.K / G, 0};
        RETURN_IF((run_product<X, 1>(q, tile, s)));
      }
  for (long o = 0; o < O; o += plan.slab) {
    const int cols = (int)std::min<long>(plan.slab, O - o);
    const Weights16 w{alone, p.K, p.N, (int)o, cols, plan.blocks, p.w.z, plan.sums, eb, weights};
    if constexpr (BACK)
      hipLaunchKernelGGL((weights16_turned_kernel<F, X>), dim3((unsigned)cdiv(plan.blocks, 4), (unsigned)cdiv(cols, 128)),
                         dim3(256), 0, s, w);
    else
      hipLaunchKernelGGL((weights16_kernel<F, X>),
                         dim3((unsigned)cdiv(cols, 128), (unsigned)(cdiv(plan.blocks, 16) + plan.sums)), dim3(512), 0, s, w);
    RETURN_IF(hipGetLastError());
    const Product16 q{rows, ea, weights, F == kNv ? nullptr : eb + o, F == kNv ? p.w.g : nullptr, p.M, cols,
                      plan.all_blocks(), p.base ? p.base + o : nullptr, p.bs, p.y + o, p.ys, plan.main.splits, shares, done,
                      nullptr, add ? add + o / G : nullptr, p.K / G, G == 32 ? 5 : G == 64 ? 6 : 7};
    RETURN_IF((run_product<X, kParts>(q, plan.main, s)));
  }
  return hipSuccess;
}

template <int F, int X>
hipError_t launch_turned(const Linear& p, char* scratch, hipStream_t s) {
  const PlanTurned plan = plan_turned(p.M, p.K, p.N);
  uint16_t* rows = reinterpret_cast<uint16_t*>(scratch + plan.rows);
  int* ea = reinterpret_cast<int*>(scratch + plan.ea);
  int* eb = reinterpret_cast<int*>(scratch + plan.eb);
  int* done = reinterpret_cast<int*>(scratch + plan.done);
  const int row_blocks = cdiv(p.M, 16);
  const Prep prep{p.x, p.xs, p.M, p.N, plan.blocks, 0, rows, ea, row_blocks, p.w, p.K, p.N, eb, done};
  RETURN_IF((run_prep<F, X, true>(prep, row_blocks + exponent_blocks<F, true>(p.K), s)));
  const TurnedRows q{p.w, rows, ea, eb, p.M, p.K, p.N, plan.blocks, p.base, p.bs, p.y, p.ys, plan.splits,
                     reinterpret_cast<float*>(scratch + plan.sums), done};
  const dim3 grid((unsigned)plan.columns, (unsigned)plan.splits);
  const size_t lds = (size_t)4 * 16 * plan.t * 128 * 4;
  if (plan.t == 1) hipLaunchKernelGGL((linear_turned_kernel<F, X, 1>), grid, dim3(256), lds, s, q);
  else if (plan.t == 2) hipLaunchKernelGGL((linear_turned_kernel<F, X, 2>), grid, dim3(256), lds, s, q);
  else hipLaunchKernelGGL((linear_turned_kernel<F, X, 4>), grid, dim3(256), lds, s, q);
  return hipGetLastError();
}

// The most rows that the packed product takes: whole rounds of its blocks (32 columns and `tile` rows
// each, one a CU) against the tiled product's three launches, in us as measured on MI355X: a round of 64 rows and
// 6144 columns takes 29, of 32 rows 19; the tiled product 25, its passes over the 16-bit forms (3.5 TB/s), the
// product (0.9 PFLOP/s), and 8 for zero points that enter apart. parts: of a weight in the tiled product.
// 6144 to 4096, packed against tiled: NVFP4 128 rows 30 and 51, 256 57 and 64, 512 112 and 82; INT4 g32 with zero
// points, bf16, 128 rows 40 and 61, 256 77 and 75; g128, fp16, 512 rows 118 and 129. 2048 to 1536: 1024 rows 36 and 49.
int rows_most(int K, int N, int tile, int parts, bool zeros) {
  const double round = 2.0 + (tile == 32 ? 0.0028 : 0.0044) * K;
  const long columns = cdiv(N, 32);
  int most = kRowsMax;
  for (int r = 1; r <= 8; ++r) {
    const double M = (double)(256l * r / columns) * tile;
    const double tiled = 25.0 + (zeros ? 8.0 : 0.0) + (0.5 + 2.0 * parts) * K * N / 3.5e6 + 4.0 * M * K / 3.5e6 +
                         2.0 * parts * M * N * K / 0.9e9;
    if (M > most && r * round < tiled) most = (int)std::min(M, 1024.0);   // (measured up to there)
  }
  return most;
}
// the fewest of any format and type (two parts and zero points only make the tiled product longer)
int rows_most_least(int K, int N) { return std::min(rows_most(K, N, 32, 1, false), rows_most(K, N, 64, 1, false)); }

template <int F, int X>
hipError_t launch_any(const Linear& p, bool back, char* scratch, hipStream_t s) {
  if (back)
    return p.M <= kRowsMax ? launch_turned<F, X>(p, scratch, s) : launch_tiled<F, X, true>(p, scratch, s);
  const bool zeros = is_int4(F) && X == kBf && p.w.z;
  if (p.M > rows_most(p.K, p.N, rows_tile<F, X>(), in_two<F, X>() ? 2 : 1, zeros)) return launch_tiled<F, X, false>(p, scratch, s);
  return launch_rows<F, X>({p.w, p.x, p.xs, p.M, p.K, p.N, p.base, p.bs, p.y, p.ys}, s);
}

template <int X>
hipError_t launch_format(const Linear& p, bool back, char* scratch, hipStream_t s) {
  switch (p.w.format == HMOE_WEIGHT_INT4 ? p.w.group : p.w.format) {
    case HMOE_WEIGHT_NVFP4: return launch_any<kNv, X>(p, back, scratch, s);
    case HMOE_WEIGHT_MXFP4: return launch_any<kMx, X>(p, back, scratch, s);
    case 32: return launch_any<kI32, X>(p, back, scratch, s);
    case 64: return launch_any<kI64, X>(p, back, scratch, s);
    default: return launch_any<kI128, X>(p, back, scratch, s);
  }
}

}  // namespace

void linear_scratch(int M, int K, int N, size_t* forward, size_t* backward) {
  // whatever the format and type
  if (forward) *forward = M > rows_most_least(K, N) ? tiled_scratch(M, K, N, false) : 0;
  if (backward) {
    *backward = M > 0 ? plan_turned(std::min(M, kRowsMax), K, N).total : 0;
    if (M > kRowsMax) *backward = std::max(*backward, tiled_scratch(M, K, N, true));
  }
}

hipError_t launch_linear(const Linear& p, bool back, void* scratch, hipStream_t s) {
  char* ws = static_cast<char*>(scratch);
  return p.dtype == HMOE_DTYPE_FP16 ? launch_format<kHf>(p, back, ws, s) : launch_format<kBf>(p, back, ws, s);
}

}  // namespace hmoe
