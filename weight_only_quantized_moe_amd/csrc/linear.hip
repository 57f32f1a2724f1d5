// Products with one matrix of 4-bit weights and group scales:
//   moe_linear           y[m, n]  = base[m, n] + sum_k x[m, k] W[n, k]
//   moe_linear_backward  dx[m, k] = dbase[m, k] + sum_n dy[m, n] W[n, k]
//
// Few rows (linear_rows_kernel) are bound by reading W once: the packed codes go from memory into
// MFMA operands (packed.h), and the reduction is split over the waves of a block, whose sums meet
// in LDS in a fixed order. Many rows are bound by the matrix cores: W is laid out once as 16-bit
// numbers in scratch, a slab of it at a time so that the slab stays in the caches, and one tiled
// product (product16_kernel) serves both directions; the backward pass lays W out transposed.
//
// The 16-bit form of W for the tiled product is fp16 whatever the rows' type: (q - z) s needs 13
// bits in general, and fp16 keeps 11 of them where bf16 would keep 8 and add as much error again
// as the rounding of a bf16 output. So that no exponent is lost, a column of the product has a
// power of two of its own (column_exponent_kernel) and bf16 rows enter as fp16 times a power of two
// of their own (rows16_kernel; exact down to 2^-29 of the row's largest element, and 2^-39 of it
// for smaller ones). Both come back in fp32.
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

// Up to 16 rows, K a multiple of 256: a wave keeps its PX pairs of steps of the rows in registers (x is
// read once a block, however many columns the block takes), and the codes of the next columns are
// requested pair by pair as those of the present ones are used up. A block takes items of 16 R
// columns, grid-strided; the waves' sums of an item meet in LDS.
template <int F, int X, int R, int PX>
__global__ __launch_bounds__(512, PX == 1 ? 4 : 2) void linear_wide_kernel(LinearRows p) {
  extern __shared__ float red[];   // [2][waves][R * 256]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int K = p.K, items = (p.N + 16 * R - 1) / (16 * R);
  const PairShare share = pair_share(wave, K / 256, PX);
  u32x4 a[PX][2][1][4][1];
  PairCodes c[PX][R];
  StepScales<F, 2 * PX> now[R], then[R];
  // A tile that would end past N starts earlier (rows past N are stand-ins only where N < 16); the
  // columns before its own are another item's.
  const TileLane at = tile_lane<F, 2 * PX>(lane, K, p.N);
  auto tile_of = [&](int item, int r) __attribute__((always_inline)) {
    return max(0, min(item * (16 * R) + 16 * r, p.N - 16));
  };
  auto scales = [&](StepScales<F, 2 * PX>(&to)[R], int item) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const TileBase t = tile_base<F>(p.w, tile_of(item, r), K, 2 * share.first);
      load_scales(to[r], t.s, t.z, at);
    }
  };
  auto codes = [&](int j, int item) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < R; ++r) load_pair(c[j][r], tile_base<F>(p.w, tile_of(item, r), K, 2 * (share.first + j)).q, at);
  };
  int item = blockIdx.x;
  scales(now, item);
#pragma unroll
  for (int j = 0; j < PX; ++j) codes(j, item);
  // rows past M are stand-ins: their sums are not written
  const uint16_t* x = p.x + (long)min(lane & 15, p.M - 1) * p.xs + (lane >> 4) * 8;
#pragma unroll
  for (int j = 0; j < 2 * PX; ++j) load_rows<F, true>(a[j >> 1][j & 1], x, 2 * share.first + j, K);
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
      for (int r = 0; r < R; ++r) pair_product<F, X, X, PX, j, 1>(acc[r], c[j][r], now[r], a[j]);
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

template <int F, int X, int R, int PX>
hipError_t run_wide(const LinearRows& p, hipStream_t s) {
  const int items = (p.N + 16 * R - 1) / (16 * R), waves = (p.K / 256 + PX - 1) / PX;
  const int blocks = std::min(items, 256 * (PX == 1 ? 16 / waves : 1));
  hipLaunchKernelGGL((linear_wide_kernel<F, X, R, PX>), dim3((unsigned)blocks), dim3((unsigned)(waves * 64)),
                     (size_t)2 * waves * R * 1024, s, p);
  return hipGetLastError();
}

constexpr int kWideMaxK = 8 * 4 * 256;   // eight waves of four pairs

template <int F, int X>
hipError_t launch_wide(const LinearRows& p, hipStream_t s) {
  const int pairs = p.K / 256;
  const bool two = p.N >= 256 * 32;
  if (pairs <= 8) return two ? run_wide<F, X, 2, 1>(p, s) : run_wide<F, X, 1, 1>(p, s);
  if (pairs <= 16) return two ? run_wide<F, X, 2, 2>(p, s) : run_wide<F, X, 1, 2>(p, s);
  if (pairs <= 24) return run_wide<F, X, 1, 3>(p, s);
  return run_wide<F, X, 1, 4>(p, s);
}

// A block: 16 R columns n and 16 T rows m, the steps of 128 of K dealt to its waves. D: steps a
// wave loads at once.
template <int F, int X, int R, int T, int D>
__global__ __launch_bounds__(T == 1 ? 1024 : 512) void linear_rows_kernel(LinearRows p) {
  extern __shared__ float red[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * (16 * R), m0 = blockIdx.y * (16 * T);
  const int K = p.K, full = K / 128;
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

  auto products = [&](const Codes<F>(&c)[R], u32x4 (&a)[1][4][T], int blocks) {
    if constexpr (is_int4(F)) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int t = 0; t < T; ++t) a[0][b][t] = int4_order(a[0][b][t]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Codes<F> v = c[r];
      step_product<F, X, X, T, 1>(acc[r], v, a, blocks);
    }
  };

  for (int s0 = wave; s0 < full; s0 += waves * D) {
    Codes<F> c[D][R];
    u32x4 a[D][1][4][T];
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int s = min(s0 + d * waves, full - 1);
#pragma unroll
      for (int r = 0; r < R; ++r) load_codes<F, true>(c[d][r], row[r], s, K, lane);
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int t = 0; t < T; ++t) a[d][0][b][t] = load16(xr[t] + s * 128 + b * 32);
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (s0 + d * waves < full) products(c[d], a[d], 4);
  }
  if (K % 128 && wave == full % waves) {
    const int blocks = K % 128 / 32;
    Codes<F> c[R];
    u32x4 a[1][4][T];
#pragma unroll
    for (int r = 0; r < R; ++r) load_codes<F, false>(c[r], row[r], full, K, lane);
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int t = 0; t < T; ++t) a[0][b][t] = load16(xr[t] + full * 128 + min(b, blocks - 1) * 32);
    products(c, a, blocks);
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
    const int n = n0 + 16 * (rt / T) + (l & 15), m = m0 + 16 * (rt % T) + (l >> 4) * 4 + i;
    if (m >= p.M || n >= p.N) continue;
    float v = 0.f;
    for (int w = 0; w < waves; ++w) v += red[w * (R * T * 256) + o];
    v *= g;
    if (p.base) v += to_f32<X>(p.base[m * p.bs + n]);
    p.y[m * p.ys + n] = from_f32<X>(v);
  }
}

template <int F, int X, int R, int T, int D>
hipError_t run_rows(const LinearRows& p, int waves, hipStream_t s) {
  hipLaunchKernelGGL((linear_rows_kernel<F, X, R, T, D>),
                     dim3((unsigned)((p.N + 16 * R - 1) / (16 * R)), (unsigned)((p.M + 16 * T - 1) / (16 * T))),
                     dim3((unsigned)(waves * 64)), (size_t)waves * R * T * 1024, s, p);
  return hipGetLastError();
}

template <int F, int X>
hipError_t launch_rows(const LinearRows& p, hipStream_t s) {
  const int steps = std::max(1, p.K / 128);
  const int waves = std::min(8, steps);
  if (p.M <= 16 && p.K % 256 == 0 && p.K <= kWideMaxK) return launch_wide<F, X>(p, s);
  if (p.M <= 16) return run_rows<F, X, 1, 1, 2>(p, waves, s);
  if (p.M <= 32) return run_rows<F, X, 2, 2, 1>(p, waves, s);
  return run_rows<F, X, 2, 4, 1>(p, std::min(waves, 4), s);
}

// ------------------------------------------------------------------------------------------
// many rows: operands of the tiled product
// ------------------------------------------------------------------------------------------

// Tile of the product, and what its operands are padded to: rows to tiles, the reduction axis to
// steps (with zeros; rows behind the last are not written, and their sums are not read).
constexpr int kTileM = 128, kTileN = 128, kStepK = 64;
constexpr long kSlabBytes = 64l << 20;   // of the 16-bit form of W at a time: a quarter of the Infinity Cache

__device__ __forceinline__ long round_up(long v, long to) { return (v + to - 1) / to * to; }

// x [M, C] -> fp16 [M, Cp], zeros past C; rows of bf16 times 2^-e with e of the largest finite
// |x| (it lands in [2^14, 2^15)), and exponent[m] = e. One block a row.
template <int X>
__global__ __launch_bounds__(256) void rows16_kernel(const uint16_t* x, long xs, int C, int Cp, uint16_t* out,
                                                     int* exponent) {
  const long m = blockIdx.x;
  const uint16_t* row = x + m * xs;
  uint16_t* o = out + m * Cp;
  int e = 0;
  if constexpr (X == kBf) {
    __shared__ uint32_t part[4];
    uint32_t top = 0;   // largest finite |x|, as bits
    for (int c = threadIdx.x; c < C; c += 256) {
      const uint32_t v = row[c] & 0x7FFFu;
      if (v < 0x7F80u) top = max(top, v);
    }
    top = max(top, xlane_u32<32>(top));
    top = max(top, xlane_u32<16>(top));
    top = max(top, xlane_u32<8>(top));
    top = max(top, xlane_u32<4>(top));
    top = max(top, xlane_u32<2>(top));
    top = max(top, xlane_u32<1>(top));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(part[0], part[1]), max(part[2], part[3]));
    if (top) e = (int)(top >> 7) - 127 - 14;
  }
  for (int c = threadIdx.x; c < Cp; c += 256) {
    uint16_t v = 0;
    if (c < C) v = X == kHf ? row[c] : from_f32<kHf>(ldexpf(to_f32<X>(row[c]), -e));
    o[c] = v;
  }
  if (threadIdx.x == 0) exponent[m] = e;
}

// exponent[c] = e for each column c of the product, so that W 2^-e fits fp16. NVFP4: 0, without its
// g (e2m1 * e4m3 is a number of fp16 as it is). Forward: c = n, over the groups of row n. Backward:
// c = k, over the rows n of k's group.
template <int F, int S, bool BACK>
__global__ __launch_bounds__(256) void column_exponent_kernel(Packed w, int K, int N, int* exponent) {
  constexpr int G = group_of(F);
  const int c = blockIdx.x;   // forward: n, backward: group of k
  int* out = BACK ? exponent + (long)c * G : exponent + c;
  int e = 0;
  if constexpr (F != kNv) {
    __shared__ int part[4];
    const int groups = K / G, count = BACK ? N : groups;
    int top = -1000;          // exponent of the largest finite scale
    for (int i = threadIdx.x; i < count; i += 256) {
      const long at = BACK ? (long)i * groups + c : (long)c * groups + i;
      if constexpr (F == kMx) {
        const int b = w.s[at];
        if (b < 255) top = max(top, b - 127);
      } else {
        const float s = fabsf(to_f32<S>(reinterpret_cast<const uint16_t*>(w.s)[at]));
        if (s > 0.f && s < INFINITY) top = max(top, ilogbf(s));
      }
    }
    for (int b = 32; b; b >>= 1) top = max(top, __shfl_xor(top, b));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(part[0], part[1]), max(part[2], part[3]));
    // the largest scale lands in [2^10, 2^11), or at 2^12 for MXFP4: times 16, or 6, below 2^15
    if (top != -1000) e = top - (F == kMx ? 12 : 10);
  }
  const int n = BACK ? G : 1;
  for (int i = threadIdx.x; i < n; i += 256) out[i] = e;
}

// 32 codes of one row times 2^-e as fp16, in the order of the columns
template <int F, int S>
__device__ __forceinline__ void fp16_codes(const Packed& w, long n, int k, int K, int e, uint32_t (&out)[16]) {
  constexpr int G = group_of(F);
  const u32x4 q = *reinterpret_cast<const u32x4*>(w.q + n * (K / 2) + k / 2);
  const long g = n * (K / G) + k / G;
  if constexpr (F == kNv) {
    const float s0 = e4m3_to_f32<0>(w.s[g]), s1 = e4m3_to_f32<0>(w.s[g + 1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 v = nvfp4_operand<kHf>(q[i], i < 2 ? s0 : s1);
#pragma unroll
      for (int j = 0; j < 4; ++j) out[4 * i + j] = v[j];
    }
  } else {
    const float s = ldexpf(F == kMx ? e8m0_value(w.s[g]) : to_f32<S>(reinterpret_cast<const uint16_t*>(w.s)[g]), -e);
    const float z = is_int4(F) ? (w.z ? (float)(w.z[g] & 15) : 8.f) : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t b = q[i >> 2] >> (8 * (i & 3));
      if constexpr (F == kMx) {
        const f32x2 v = e2m1x2_f32<0>(b, 1.f);
        out[i] = pack_f16(v[0] * s, v[1] * s);
      } else {
        out[i] = pack_f16(((float)(b & 15u) - z) * s, ((float)((b >> 4) & 15u) - z) * s);
      }
    }
  }
}

// rows [n0, n0 + rows) of W as fp16 [rows, Kp], zeros past K: a thread takes 32 columns
template <int F, int S>
__global__ __launch_bounds__(256) void weights16_kernel(Packed w, int n0, int rows, int K, int Kp, const int* exponent,
                                                        uint16_t* out) {
  const int units = Kp / 32;
  const long u = (long)blockIdx.x * 256 + threadIdx.x;
  if (u >= (long)rows * units) return;
  const long r = u / units;
  const int k = (int)(u % units) * 32;
  uint32_t v[16] = {};
  if (k < K) fp16_codes<F, S>(w, n0 + r, k, K, exponent[n0 + r], v);
  u32x4* o = reinterpret_cast<u32x4*>(out + r * Kp + k);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = u32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
}

// columns [k0, k0 + cols) of W, transposed, as fp16 [cols, Np], zeros past N: a block turns 64 rows
// n and 128 columns k in LDS
template <int F, int S>
__global__ __launch_bounds__(256) void weights16_turned_kernel(Packed w, int k0, int cols, int K, int N, int Np,
                                                               const int* exponent, uint16_t* out) {
  constexpr int kPitch = 130;   // halves of a row in LDS: an odd number of dwords
  __shared__ uint16_t tile[64 * kPitch];
  const int n0 = blockIdx.x * 64, c0 = blockIdx.y * 128;
  {
    const int n = n0 + (threadIdx.x >> 2), k = c0 + (threadIdx.x & 3) * 32;
    uint32_t v[16] = {};
    if (n < N && k < cols) fp16_codes<F, S>(w, n, k0 + k, K, exponent[k0 + k], v);
    uint32_t* t = reinterpret_cast<uint32_t*>(tile + (threadIdx.x >> 2) * kPitch + (threadIdx.x & 3) * 32);
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = v[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 128 * 8; i += 256) {
    const int c = i >> 3, n = (i & 7) * 8;
    if (c0 + c >= cols || n0 + n >= Np) continue;
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = tile[(n + 2 * j) * kPitch + c] | (uint32_t)tile[(n + 2 * j + 1) * kPitch + c] << 16;
    *reinterpret_cast<u32x4*>(out + (long)(c0 + c) * Np + n0 + n) = v;
  }
}

// ------------------------------------------------------------------------------------------
// many rows: the tiled product
// ------------------------------------------------------------------------------------------

struct Product16 {
  const uint16_t* a;    // fp16 [M, Cp]
  const int* ea;        // [M]
  const uint16_t* b;    // fp16 [cols, Cp]
  const int* eb;        // [cols]
  const float* g;       // NVFP4's scale of the matrix; null: 1
  int M, cols, Cp;
  const uint16_t* base; // [M, cols]; may be null
  long bs;
  uint16_t* y;
  long ys;
};

// y[m, c] = base[m, c] + g 2^(ea[m] + eb[c]) sum_i a[m, i] b[c, i]. A block of four waves takes 128 x 128,
// a wave 64 x 64.
template <int X>
__global__ __launch_bounds__(256) void product16_kernel(Product16 p) {
  __shared__ u32x4 sa[2][kTileM * 8], sb[2][kTileN * 8];   // 8 pieces of 16 bytes a row and step
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m0 = blockIdx.y * kTileM, c0 = blockIdx.x * kTileN;
  const int wm = (wave & 1) * 64, wc = (wave >> 1) * 64;
  const int steps = p.Cp / kStepK;
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float g = p.g ? *p.g : 1.f;
  u32x4 ra[4], rb[4];
  auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 32 + (threadIdx.x >> 3), piece = threadIdx.x & 7;
      ra[i] = *reinterpret_cast<const u32x4*>(p.a + (long)min(m0 + r, p.M - 1) * p.Cp + s * kStepK + piece * 8);
      rb[i] = *reinterpret_cast<const u32x4*>(p.b + (long)min(c0 + r, p.cols - 1) * p.Cp + s * kStepK + piece * 8);
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 32 + (threadIdx.x >> 3), piece = (threadIdx.x & 7) ^ (r & 7);
      sa[buf][r * 8 + piece] = ra[i];
      sb[buf][r * 8 + piece] = rb[i];
    }
  };
  load(0);
  store(0);
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    const int buf = s & 1;
    if (s + 1 < steps) load(s + 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int piece = (h * 4 + (lane >> 4)) ^ (lane & 7);
        a[i] = sa[buf][(wm + i * 16 + (lane & 15)) * 8 + piece];
        b[i] = sb[buf][(wc + i * 16 + (lane & 15)) * 8 + piece];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma16<kHf>(a[i], b[j], acc[i][j]);
    }
    if (s + 1 < steps) store(buf ^ 1);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = m0 + wm + i * 16 + (lane >> 4) * 4 + e, c = c0 + wc + j * 16 + (lane & 15);
        if (m >= p.M || c >= p.cols) continue;
        float v = ldexpf(acc[i][j][e], p.ea[m] + p.eb[c]) * g;
        if (p.base) v += to_f32<X>(p.base[m * p.bs + c]);
        p.y[m * p.ys + c] = from_f32<X>(v);
      }
}

// ------------------------------------------------------------------------------------------
// host
// ------------------------------------------------------------------------------------------

namespace {

constexpr int kRowsMax = 64;   // rows the packed product takes

size_t pad256(size_t v) { return (v + 255) & ~size_t(255); }
long up(long v, long to) { return (v + to - 1) / to * to; }

// Scratch of the tiled product: reduction axis C, output columns O.
struct Plan16 {
  long Cp = 0, slab = 0;          // padded reduction axis, output columns a slab
  size_t rows = 0, ea = 0, eb = 0, weights = 0, total = 0;
};
Plan16 plan16(long M, long C, long O) {
  Plan16 p;
  p.Cp = up(C, kStepK);
  p.slab = std::max<long>(128, kSlabBytes / (p.Cp * 2) / 128 * 128);
  p.slab = std::min(p.slab, up(O, 128));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += pad256(bytes);
    return r;
  };
  p.rows = take((size_t)M * p.Cp * 2);
  p.ea = take((size_t)M * 4);
  p.eb = take((size_t)up(O, 128) * 4);
  p.weights = take((size_t)p.slab * p.Cp * 2);
  p.total = at;
  return p;
}

#define RETURN_IF(expr)                    \
  do {                                     \
    const hipError_t err_ = (expr);        \
    if (err_ != hipSuccess) return err_;   \
  } while (0)

template <int F, int X, bool BACK>
hipError_t launch_tiled(const Linear& p, char* scratch, hipStream_t s) {
  const int C = BACK ? p.N : p.K, O = BACK ? p.K : p.N;
  const Plan16 plan = plan16(p.M, C, O);
  uint16_t* rows = reinterpret_cast<uint16_t*>(scratch + plan.rows);
  int* ea = reinterpret_cast<int*>(scratch + plan.ea);
  int* eb = reinterpret_cast<int*>(scratch + plan.eb);
  uint16_t* weights = reinterpret_cast<uint16_t*>(scratch + plan.weights);
  const int Cp = (int)plan.Cp;
  hipLaunchKernelGGL((rows16_kernel<X>), dim3((unsigned)p.M), dim3(256), 0, s, p.x, p.xs, C, Cp, rows, ea);
  RETURN_IF(hipGetLastError());
  hipLaunchKernelGGL((column_exponent_kernel<F, X, BACK>), dim3((unsigned)(BACK ? O / group_of(F) : O)), dim3(256), 0, s,
                     p.w, p.K, p.N, eb);
  RETURN_IF(hipGetLastError());
  for (long o = 0; o < O; o += plan.slab) {
    const int cols = (int)std::min<long>(plan.slab, O - o);
    if constexpr (BACK)
      hipLaunchKernelGGL((weights16_turned_kernel<F, X>), dim3((unsigned)(Cp / 64), (unsigned)((cols + 127) / 128)),
                         dim3(256), 0, s, p.w, (int)o, cols, p.K, p.N, Cp, eb, weights);
    else
      hipLaunchKernelGGL((weights16_kernel<F, X>), dim3((unsigned)(((long)cols * (Cp / 32) + 255) / 256)), dim3(256), 0,
                         s, p.w, (int)o, cols, p.K, Cp, eb, weights);
    RETURN_IF(hipGetLastError());
    const Product16 q{rows, ea, weights, eb + o, F == kNv ? p.w.g : nullptr, p.M, cols, Cp, p.base ? p.base + o : nullptr, p.bs, p.y + o, p.ys};
    hipLaunchKernelGGL((product16_kernel<X>), dim3((unsigned)((cols + kTileN - 1) / kTileN),
                                                   (unsigned)((p.M + kTileM - 1) / kTileM)),
                       dim3(256), 0, s, q);
    RETURN_IF(hipGetLastError());
  }
  return hipSuccess;
}

template <int F, int X>
hipError_t launch_any(const Linear& p, bool back, char* scratch, hipStream_t s) {
  if (back) return launch_tiled<F, X, true>(p, scratch, s);
  if (p.M > kRowsMax) return launch_tiled<F, X, false>(p, scratch, s);
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
  if (forward) *forward = M > kRowsMax ? plan16(M, K, N).total : 0;
  if (backward) *backward = M > 0 ? plan16(M, N, K).total : 0;
}

hipError_t launch_linear(const Linear& p, bool back, void* scratch, hipStream_t s) {
  char* ws = static_cast<char*>(scratch);
  return p.dtype == HMOE_DTYPE_FP16 ? launch_format<kHf>(p, back, ws, s) : launch_format<kBf>(p, back, ws, s);
}

}  // namespace hmoe
