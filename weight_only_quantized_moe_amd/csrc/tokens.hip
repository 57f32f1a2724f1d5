// A whole mixture-of-experts layer for a few tokens (M <= 16), experts in 4-bit weights with group
// scales (packed.h):
//   l = x R^T,  the k largest of softmax(l), renormalised: p,
//   h = silu(x Wg_e^T) * (x Wu_e^T),  y = base + sum_j p_j W2_e h_e + sigmoid(x . gate) W2_s h_s.
//
// It is bound by reading the touched experts once and, for one or two tokens, by the latency of
// its dependent steps. Three launches: the router's logits; routing and the experts' first products
// (each block routes all tokens by itself, which costs less than a launch); the second products,
// where a block owns 64 columns of y and a share of the experts' steps, and the last block of the
// columns to finish adds the shares up in their order. An expert that several tokens took is read
// once: its tokens are rows of the same MFMA.
//
// h, times its routing weight and the second matrix's own scale, is kept in fp32 and goes into the second
// product as three bf16 parts that hold all of its 24 bits: it is not rounded.
#include <algorithm>

#include "packed.h"
#include "route_common.h"

namespace hmoe {

namespace {

constexpr int kUpWaves = 8, kDownWaves = 8;
constexpr int kRouterK = 1024;     // columns a block of the router takes
constexpr int kDownCols = 64;      // columns of y a block of the second products takes
constexpr int kMaxShares = 16;     // of the experts' steps
constexpr int kMaxPairs = HMOE_TOKENS_MAX_M * kMaxTopK;   // (token, expert) pairs, so also experts in use

// What the second launch leaves for the third.
struct TokensPlan {
  int infinite;                  // whether an h is infinite (cleared by the first launch)
  int count;                     // experts in use, ascending
  int expert[kMaxPairs];
  int16_t row[kMaxPairs * 16];   // row of h of each token, -1: the token did not take this expert
};

// Scratch, as offsets.
struct TokensScratch {
  size_t logits = 0, plan = 0, h = 0, hs = 0, sums = 0, done = 0, total = 0;
  int pitch = 0, parts = 0;   // of the logits: row pitch, shares of H
  int tiles = 0, shares = 0;  // of y: tiles of columns, shares of the experts' steps
};
int cdiv(long a, long b) { return (int)((a + b - 1) / b); }
TokensScratch tokens_plan(int M, int E, int H, int I, int k, int S) {
  TokensScratch t;
  auto take = [&](size_t bytes) {
    const size_t at = t.total;
    t.total += (bytes + 255) & ~size_t(255);
    return at;
  };
  t.pitch = E + 1;
  t.parts = cdiv(H, kRouterK);
  t.logits = take((size_t)t.parts * M * t.pitch * 4);
  t.plan = take(sizeof(TokensPlan));
  t.h = take((size_t)M * k * I * 4);
  t.hs = take((size_t)M * S * 4);
  // shares for two blocks a CU, and not more than give every wave a step
  const long steps = (long)std::min(M * k, E) * cdiv(I, 128) + cdiv(S, 128);
  t.tiles = cdiv(H, kDownCols);
  t.shares = (int)std::max(1l, std::min({(long)kMaxShares, 512l / t.tiles, steps / kDownWaves}));
  t.sums = take((size_t)t.shares * t.tiles * M * kDownCols * 4);
  t.done = take((size_t)t.tiles * 4);
  return t;
}

}  // namespace

// By value: a reference to one of two kernel arguments would put both into private memory.
__device__ __forceinline__ Packed pick(bool first, const Packed& a, const Packed& b) {
  return {first ? a.q : b.q, first ? a.s : b.s, first ? a.z : b.z, first ? a.g : b.g, 0, 0};
}

struct TokensArgs {
  Tokens p;
  float* logits;  // [parts, M, pitch]
  int pitch, parts;
  TokensPlan* plan;
  float* h;       // [M k, I]
  float* hs;      // [M, S]
  float* sums;    // [shares, tiles, M, 64]
  int* done;      // [tiles]: shares that are finished
  int tiles, shares;
};

// logits[part, m, e] = x[m] . router[e] over the part's 1024 columns, and the shared expert's gate as
// row E. A block takes 16 rows and one part, a wave 128 columns.
template <int X>
__global__ __launch_bounds__(512) void tokens_router_kernel(TokensArgs a) {
  __shared__ float red[8][256];
  const Tokens& p = a.p;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (blockIdx.x == 0 && blockIdx.y == 0) {   // the third launch counts from zero
    for (int i = threadIdx.x; i < a.tiles; i += 512) a.done[i] = 0;
    if (threadIdx.x == 0) a.plan->infinite = 0;
  }
  const int e = blockIdx.x * 16 + (lane & 15), rows = p.E + (p.gate ? 1 : 0);
  const uint16_t* r = (e < p.E ? p.router + (long)e * p.H : p.gate ? p.gate : p.router) + (lane >> 4) * 8;
  const uint16_t* x = p.x + (long)min(lane & 15, p.M - 1) * p.xs + (lane >> 4) * 8;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const int c0 = blockIdx.y * kRouterK + wave * 128;
  u32x4 rv[4], xv[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int c = min(c0 + d * 32, p.H - 32);
    rv[d] = load16(r + c);
    xv[d] = load16(x + c);
  }
#pragma unroll
  for (int d = 0; d < 4; ++d)
    if (c0 + d * 32 < p.H) acc = mfma16<X>(xv[d], rv[d], acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][i * 64 + lane] = acc[i];
  __syncthreads();
  if (threadIdx.x >= 256) return;
  const int l = threadIdx.x & 63, m = (l >> 4) * 4 + (threadIdx.x >> 6), c = blockIdx.x * 16 + (l & 15);
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) v += red[w][threadIdx.x];
  if (m < p.M && c < rows) a.logits[((long)blockIdx.y * p.M + m) * a.pitch + c] = v;
}

// One logit: the sum of its parts, four of them requested at a time.
__device__ __forceinline__ float whole_logit(const TokensArgs& a, int t, int e) {
  const float* at = a.logits + (long)t * a.pitch + e;
  const long part = (long)a.p.M * a.pitch;
  float v = 0.f;
  for (int i = 0; i < a.parts; i += 4) {
    float u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = at[min(i + j, a.parts - 1) * part];
#pragma unroll
    for (int j = 0; j < 4; ++j) v += i + j < a.parts ? u[j] : 0.f;
  }
  return v;
}

// moe_route's choice for one token by one wave, with few registers beside the kernel's own: the
// logits' keys lie in LDS (keys [E]), a lane holds the best of its experts lane + 64 i, and only the
// lane whose expert was taken looks through its keys again. Lane j < k returns the j-th expert and
// its weight.
__device__ __forceinline__ int route_token(uint32_t* keys, int E, int k, int lane, float* weight) {
  uint32_t best = 0u;
  int id = 0;
  for (int e = lane; e < E; e += kWave) {
    const uint32_t key = keys[e];
    if (key > best) {
      best = key;
      id = e;
    }
  }
  int sel = 0;
  uint32_t sel_key = 0u;
  for (int r = 0; r < k; ++r) {
    uint32_t top = max(best, xlane_u32<32>(best));
    top = max(top, xlane_u32<16>(top));
    top = max(top, xlane_u32<8>(top));
    top = max(top, xlane_u32<4>(top));
    top = max(top, xlane_u32<2>(top));
    top = max(top, xlane_u32<1>(top));
    top = __builtin_amdgcn_readfirstlane(top);
    uint64_t holds = __ballot(best == top);
    int first = __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(holds));
    for (holds &= holds - 1ull; holds; holds &= holds - 1ull)   // ties go to the lower id
      first = min(first, __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(holds)));
    if (lane == r) {
      sel = first;
      sel_key = top;
    }
    if (lane == (first & 63)) {
      keys[first] = 0u;                        // below every key: not taken again, as k <= E
      best = 0u;
      for (int e = lane; e < E; e += kWave) {
        const uint32_t key = keys[e];
        if (key > best) {
          best = key;
          id = e;
        }
      }
    }
  }
  const float v = key_value(sel_key);
  const float v0 = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 0));
  const double ex = lane < k ? exp((double)v - (double)v0) : 0.0;
  double sum = ex;
  sum += xlane_d<32>(sum);
  sum += xlane_d<16>(sum);
  sum += xlane_d<8>(sum);
  sum += xlane_d<4>(sum);
  sum += xlane_d<2>(sum);
  sum += xlane_d<1>(sum);
  *weight = lane < k ? (float)(ex / sum) : 0.f;
  return sel;
}

// What a block of the first products knows of the routing, in LDS.
struct Routing {
  int id[kMaxPairs];
  float w[kMaxPairs];
  uint32_t mask[kMaxExperts];                  // tokens of each expert
  int expert[kMaxPairs], off[kMaxPairs];       // experts in use, ascending; their first rows of h
  float gate[HMOE_TOKENS_MAX_M];               // the shared expert's weights
  int count;
};

// Routes all tokens in this block. keys: LDS of kUpWaves * kMaxExperts words.
__device__ __forceinline__ void route_block(const TokensArgs& a, Routing& s, uint32_t* keys) {
  const Tokens& p = a.p;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int threads = blockDim.x, waves = threads >> 6;
  for (int e = threadIdx.x; e < p.E; e += threads) s.mask[e] = 0u;
  if (p.gate && threadIdx.x < p.M) s.gate[threadIdx.x] = 1.f / (1.f + expf(-whole_logit(a, threadIdx.x, p.E)));
  // as many tokens at a time as have a wave each
  for (int t0 = 0; t0 < p.M; t0 += waves) {
    const int n = min(waves, p.M - t0);
    if (t0) __syncthreads();
    for (int i = threadIdx.x; i < n * p.E; i += threads) {
      const int t = i / p.E, e = i - t * p.E;
      float v = whole_logit(a, t0 + t, e);
      v = v == 0.f ? 0.f : v;                   // -0 ties with +0
      keys[t * kMaxExperts + e] = v != v ? 1u : order_key(v);
    }
    __syncthreads();
    if (wave >= n) continue;
    const int t = t0 + wave;
    float w;
    const int id = route_token(keys + wave * kMaxExperts, p.E, p.k, lane, &w);
    if (lane < p.k) {
      s.id[t * p.k + lane] = id;
      s.w[t * p.k + lane] = w;
      atomicOr(&s.mask[id], 1u << t);
      if (blockIdx.x == 0) {
        if (p.topk_ids) p.topk_ids[t * p.k + lane] = id;
        if (p.topk_w) p.topk_w[t * p.k + lane] = w;
      }
    }
  }
  __syncthreads();
  if (wave == 0) {
    int count = 0, rows = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const int e = e0 + lane;
      const uint32_t mask = e < p.E ? s.mask[e] : 0u;
      const uint64_t used = __ballot(mask != 0u);
      if (!used) continue;
      int before = __popc(mask);                   // pairs of lower experts: a scan over the wave
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(before, d);
        if (lane >= d) before += o;
      }
      const int total = __shfl(before, 63);
      before -= __popc(mask);
      const int at = count + __popcll(used & ((1ull << lane) - 1ull));
      if (mask) {
        s.expert[at] = e;
        s.off[at] = rows + before;
      }
      count += __popcll(used);
      rows += total;
    }
    if (lane == 0) s.count = count;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) a.plan->count = s.count;
    for (int i = threadIdx.x; i < s.count * 16; i += threads) {
      const int d = i >> 4, m = i & 15, e = s.expert[d];
      const uint32_t mask = s.mask[e];
      if (m == 0) a.plan->expert[d] = e;
      a.plan->row[i] = (mask >> m) & 1u ? (int16_t)(s.off[d] + __popc(mask & ((1u << m) - 1u))) : (int16_t)-1;
    }
  }
}

// A work item of the first products: 16 columns of one expert's h, that is 16 gate rows and 16 up rows
// of its W13.
struct Item {
  int d, e, i0, width;
  bool shared;
  float g13, g2;   // NVFP4's scales
};
template <int F>
__device__ __forceinline__ Item item_of(const Tokens& p, const Routing& s, int item) {
  const int tiles = p.I / 16;
  Item v;
  v.d = min(item / tiles, s.count);
  v.shared = v.d == s.count;
  v.i0 = (item - v.d * tiles) * 16;
  v.e = v.shared ? 0 : __builtin_amdgcn_readfirstlane(s.expert[min(v.d, kMaxPairs - 1)]);
  v.width = v.shared ? p.S : p.I;
  v.g13 = v.g2 = 1.f;
  if constexpr (F == kNv) {
    v.g13 = (v.shared ? p.s13.g : p.w13.g)[v.e];
    v.g2 = (v.shared ? p.s2.g : p.w2.g)[v.e];
  }
  return v;
}

// The waves' sums of an item, [waves][2][256] in LDS, to h of its tokens.
template <int F>
__device__ __forceinline__ void finish_item(const TokensArgs& a, const Routing& s, const Item& v, const float* sums,
                                            int waves) {
  const Tokens& p = a.p;
  const uint32_t mask = v.shared ? (1u << p.M) - 1u : s.mask[v.e];
  for (int o = threadIdx.x; o < 256; o += blockDim.x) {
    const int l = o & 63, t = (l >> 4) * 4 + (o >> 6), i = v.i0 + (l & 15);
    if (!((mask >> t) & 1u)) continue;
    float gate = 0.f, up = 0.f;
    for (int w = 0; w < waves; ++w) {
      gate += sums[w * 512 + o];
      up += sums[w * 512 + 256 + o];
    }
    float weight = 1.f;
    if (!v.shared) {
      for (int j = 0; j < p.k; ++j)
        if (s.id[t * p.k + j] == v.e) weight = s.w[t * p.k + j];
    } else if (p.gate) {
      weight = s.gate[t];
    }
    gate *= v.g13;
    up *= v.g13;
    const float h = silu(gate) * up * (weight * v.g2);
    const long r = v.shared ? t : s.off[v.d] + __popc(mask & ((1u << t) - 1u));
    (v.shared ? a.hs : a.h)[r * v.width + i] = h;
    if (__builtin_isinf(h)) a.plan->infinite = 1;
  }
}

// Routing and the first products, H at least 256 (EXACT: a multiple of it). Every item multiplies the
// same tokens, so a wave keeps its PX pairs of steps of x in registers, and it requests the next item's
// codes pair by pair as those of the present one are used up. Bound by HBM where items are many: 749 MB in
// 132 us (eight tokens of the GLM-class layer, MXFP4); by routing (4 us) and cold code where they are few.
template <int F, int X, int PX, bool EXACT>
__global__ __launch_bounds__(kUpWaves * 64, PX == 1 ? 4 : 2) void tokens_up_kernel(TokensArgs a) {
  __shared__ Routing s;
  __shared__ float red[2][kUpWaves][2][256];        // the waves' sums; before, the waves' keys
  static_assert(sizeof(red) >= kUpWaves * kMaxExperts * 4, "keys of every wave");
  const Tokens& p = a.p;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int H = p.H;
  const int pairs = (H + 255) / 256;
  const PairShare share = pair_share(wave, pairs, PX);
  u32x4 xv[PX][2][1][4][1];
  const uint16_t* x = p.x + (long)min(lane & 15, p.M - 1) * p.xs + (lane >> 4) * 8;
#pragma unroll
  for (int j = 0; j < 2 * PX; ++j) load_pair_rows<F, EXACT>(xv[j >> 1][j & 1], x, 2 * share.first + j, H);
  route_block(a, s, reinterpret_cast<uint32_t*>(&red[0][0][0][0]));
  const int items = s.count * (p.I / 16) + p.S / 16;
  int item = blockIdx.x;
  if (item >= items) return;
  __syncthreads();   // the keys have been read

  PairCodes c[PX][2];
  StepScales<F, 2 * PX> now[2], then[2];
  const TileLane<EXACT> at = tile_lane<F, 2 * PX, EXACT>(lane, H, 16, 2 * share.first);
  TileBase gate, up;
  auto rows_of = [&](const Item& v) __attribute__((always_inline)) {
    const Packed w = pick(v.shared, p.s13, p.w13);
    const long row0 = (long)v.e * 2 * v.width + v.i0;
    gate = tile_base<F>(w, row0, H, 2 * share.first);
    up = tile_base<F>(w, row0 + v.width, H, 2 * share.first);
  };
  auto scales = [&](StepScales<F, 2 * PX>(&to)[2]) __attribute__((always_inline)) {
    load_scales<F, 2 * PX, EXACT>(to[0], gate.s, gate.z, at);
    load_scales<F, 2 * PX, EXACT>(to[1], up.s, up.z, at);
  };
  auto codes = [&](int j) __attribute__((always_inline)) {
    load_pair(c[j][0], gate.q + j * 128, at, share.first + j == pairs - 1);
    load_pair(c[j][1], up.q + j * 128, at, share.first + j == pairs - 1);
  };
  Item it = item_of<F>(p, s, item);
  rows_of(it);
  scales(now);
#pragma unroll
  for (int j = 0; j < PX; ++j) codes(j);
  for (int buf = 0;; buf ^= 1) {
    const int next = item + gridDim.x;
    const Item present = it;
    f32x4 acc[2][1] = {{{0.f, 0.f, 0.f, 0.f}}, {{0.f, 0.f, 0.f, 0.f}}};
    if constexpr (is_int4(F)) {
      const bool zeros = present.shared ? p.s13.z : p.w13.z;
      default_zeros(now[0], zeros);
      default_zeros(now[1], zeros);
    }
    auto products = [&](auto P) __attribute__((always_inline)) {
      constexpr int j = decltype(P)::value;
      if (share.first + j < share.own) return;
      pair_product<F, X, X, PX, j>(acc[0], c[j][0], now[0], xv[j]);
      pair_product<F, X, X, PX, j>(acc[1], c[j][1], now[1], xv[j]);
    };
    // the two cases apart: a load behind a condition would make the waits count on its absence
    if (next < items) {
      it = item_of<F>(p, s, next);
      rows_of(it);
      scales(then);
      each<PX>([&](auto P) __attribute__((always_inline)) {
        products(P);
        codes(decltype(P)::value);
      });
      now[0] = then[0];
      now[1] = then[1];
    } else {
      each<PX>(products);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[buf][wave][r][i * 64 + lane] = acc[r][0][i];
    __syncthreads();
    finish_item<F>(a, s, present, &red[buf][0][0][0], waves);
    if (next >= items) return;
    item = next;
  }
}

// The same for every other H, narrower or wider: a step at a time, x read again for each item.
template <int F, int X>
__global__ __launch_bounds__(kUpWaves * 64, 2) void tokens_up_any_kernel(TokensArgs a) {
  __shared__ Routing s;
  __shared__ float red[2][kUpWaves][2][256];
  const Tokens& p = a.p;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int H = p.H, steps = (H + 127) / 128;
  const uint16_t* x = p.x + (long)min(lane & 15, p.M - 1) * p.xs + (lane >> 4) * 8;
  route_block(a, s, reinterpret_cast<uint32_t*>(&red[0][0][0][0]));
  __syncthreads();   // the keys have been read
  const int items = s.count * (p.I / 16) + p.S / 16;
  int buf = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x, buf ^= 1) {
    const Item v = item_of<F>(p, s, item);
    const Packed w = pick(v.shared, p.s13, p.w13);
    const long row0 = (long)v.e * 2 * v.width + v.i0 + (lane & 15);
    const PackedRow row[2] = {packed_row<F>(w, row0, H, lane), packed_row<F>(w, row0 + v.width, H, lane)};
    f32x4 acc[2][1] = {{{0.f, 0.f, 0.f, 0.f}}, {{0.f, 0.f, 0.f, 0.f}}};
    for (int s0 = wave; s0 < steps; s0 += 2 * kUpWaves) {
      Codes<F> c[2][2];
      u32x4 xv[2][1][4][1];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int step = min(s0 + j * kUpWaves, steps - 1);
#pragma unroll
        for (int r = 0; r < 2; ++r) load_step<F, false>(c[j][r], row[r], step, H, lane);
        load_rows<F, false>(xv[j], x, step, H);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int step = s0 + j * kUpWaves;
        if (step >= steps) continue;
#pragma unroll
        for (int r = 0; r < 2; ++r) step_product<F, X, X, 1>(acc[r], c[j][r], xv[j], step_blocks<false>(step, H));
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[buf][wave][r][i * 64 + lane] = acc[r][0][i];
    __syncthreads();
    finish_item<F>(a, s, v, &red[buf][0][0][0], kUpWaves);
  }
}

// y: a block takes 64 columns and one share of the units of all experts in use, which its waves take in
// turn, so that they read neighbouring lines of the same rows; four row tiles of W2 meet each piece of
// h that a wave loads. With several shares the block that finishes last adds them up in their order: a
// share is written past the caches of its own XCD, then counted. PAIRS: I and S are at least 256 (EXACT:
// multiples of it), and a unit is a pair of steps; else it is a step. h comes as fp32 and is split here,
// as three 16-bit planes of it would need 16 registers more (spills). Eight tokens of the GLM-class layer
// (MXFP4) take 116 us; two planes, 16 of h's 24 bits, took 104, and with the next pair's codes in flight
// beside, at twice the registers and half the waves, 108.
template <int F, int X, bool PAIRS, bool EXACT>
__global__ __launch_bounds__(kDownWaves * 64, 4) void tokens_down_kernel(TokensArgs a) {
  constexpr int R = kDownCols / 16, kThreads = kDownWaves * 64, kUnit = PAIRS ? 256 : 128;
  __shared__ int s_expert[kMaxPairs];
  __shared__ int16_t s_row[kMaxPairs * 16];
  __shared__ float red[kDownWaves][R * 256];
  __shared__ int s_last;
  const Tokens& p = a.p;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * kDownCols;
  // entries past the experts in use are read along: their number is not waited for
  const int most = min(p.M * p.k, p.E);
  for (int i = threadIdx.x; i < most * 16; i += kThreads) {
    s_row[i] = a.plan->row[i];
    if (i < most) s_expert[i] = a.plan->expert[i];
  }
  const int count = a.plan->count;
  const bool infinite = a.plan->infinite;
  __syncthreads();
  const int m = lane & 15;
  const int units = (p.I + kUnit - 1) / kUnit, total = count * units + (p.S + kUnit - 1) / kUnit;
  const int from = (int)((long)total * blockIdx.y / a.shares) + wave, to = (int)((long)total * (blockIdx.y + 1) / a.shares);
  f32x4 acc[R][1];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r][0] = f32x4{0.f, 0.f, 0.f, 0.f};
  // the place of a unit: expert d, unit u of its K columns
  struct Place {
    int d, u, K;
    bool shared;
  };
  auto place = [&](int d, int u) { return Place{d, u, d == count ? p.S : p.I, d == count}; };
  auto after = [&](const Place& v) {   // the wave's next unit
    int d = v.d, u = v.u + kDownWaves;
    while (d < count && u >= units) {
      u -= units;
      ++d;
    }
    return place(d, u);
  };
  auto row_of = [&](const Place& v) { return v.shared ? 0l : (long)__builtin_amdgcn_readfirstlane(s_expert[v.d]) * p.H; };
  // h of a step, zeros for tokens that did not take the expert: only the lanes of the others load, which
  // costs the address unit less than stand-ins would
  auto rows = [&](f32x4(&hv)[4][2], const Place& v, int step, int blocks) __attribute__((always_inline)) {
    const int hr = v.shared ? (m < p.M ? m : -1) : s_row[v.d * 16 + m];
    const float* h = (v.shared ? a.hs : a.h) + (long)max(hr, 0) * v.K + (lane >> 4) * 8 + step * 128;
#pragma unroll
    for (int b = 0; b < 4; ++b) hv[b][0] = hv[b][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (hr < 0) return;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (PAIRS && !EXACT && step * 128 + b * 32 >= v.K) continue;
      const float* at = h + min(b, blocks - 1) * 32;
      hv[b][0] = *reinterpret_cast<const f32x4*>(at);
      hv[b][1] = *reinterpret_cast<const f32x4*>(at + 4);
    }
  };
  if (from < to) {
    Place now = place(min(from / units, count), 0);
    now.u = from - now.d * units;
    if constexpr (PAIRS) {
      for (int f = from; f < to; f += kDownWaves) {
        PairCodes c[R];
        StepScales<F, 2> v[R];
        const Packed w = pick(now.shared, p.s2, p.w2);
        const long first = row_of(now);
        const TileLane<EXACT> at = tile_lane<F, 2, EXACT>(lane, now.K, 16, 2 * now.u);
        const bool end = !EXACT && now.K % 256 && now.u == now.K / 256;
        f32x4 hv[4][2];
        rows(hv, now, 2 * now.u, 4);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          // H is a multiple of 32: a tile is whole or past it
          const TileBase t = tile_base<F>(w, first + (n0 + 16 * r < p.H ? n0 + 16 * r : 0), now.K, 2 * now.u);
          load_scales<F, 2, EXACT>(v[r], t.s, t.z, at);
          load_pair(c[r], t.q, at, end);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          default_zeros(v[r], w.z);
          split_pair(c[r]);
        }
#pragma nounroll   // once through cold code for both steps
        for (int step = 0;; ++step) {
          Codes<F> k[R];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            k[r].q = c[r].a;
            take_scales_of<F>(k[r], v[r], step);
          }
          step_product_f32<F, X, R>(acc, k, hv, 4, infinite);
          if (step) break;
          rows(hv, now, 2 * now.u + 1, 4);
#pragma unroll
          for (int r = 0; r < R; ++r) c[r].a = c[r].b;
        }
        now = after(now);
      }
    } else {
      for (int f = from; f < to; f += kDownWaves) {
        const int blocks = step_blocks<false>(now.u, now.K);
        Codes<F> c[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
          load_step<F, false>(c[r], packed_row<F>(pick(now.shared, p.s2, p.w2), row_of(now) + min(n0 + 16 * r + m, p.H - 1),
                                                  now.K, lane), now.u, now.K, lane);
        f32x4 hv[4][2];
        rows(hv, now, now.u, blocks);
        step_product_f32<F, X, R>(acc, c, hv, blocks, infinite);
        now = after(now);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][r * 256 + i * 64 + lane] = acc[r][0][i];
  __syncthreads();
  float* sums = a.sums + (long)blockIdx.x * p.M * kDownCols;            // of share 0
  const long share = (long)a.tiles * p.M * kDownCols;
  auto finish = [&](int t, int col, float v) {
    if (p.base) v += to_f32<X>(p.base[t * p.bs + col]);
    p.y[t * p.ys + col] = from_f32<X>(v);
  };
  for (int o = threadIdx.x; o < R * 256; o += kThreads) {
    const int l = o & 63, t = (l >> 4) * 4 + ((o >> 6) & 3), cl = 16 * (o >> 8) + (l & 15);
    if (t >= p.M || n0 + cl >= p.H) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kDownWaves; ++w) v += red[w][o];
    if (a.shares == 1) finish(t, n0 + cl, v);
    else __hip_atomic_store(sums + blockIdx.y * share + t * kDownCols + cl, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (a.shares == 1) return;
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt 0: the wave's stores have been done
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __syncthreads();
  if (threadIdx.x == 0)
    s_last = __hip_atomic_fetch_add(a.done + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.shares - 1;
  __syncthreads();
  if (!s_last) return;
  for (int o = threadIdx.x; o < p.M * kDownCols; o += kThreads) {
    const int t = o / kDownCols, cl = o % kDownCols;
    if (n0 + cl >= p.H) continue;
    float v = 0.f, u[kMaxShares];   // all shares requested at once, added in their order
#pragma unroll
    for (int i = 0; i < kMaxShares; ++i)
      u[i] = __hip_atomic_load(sums + min(i, a.shares - 1) * share + o, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int i = 0; i < kMaxShares; ++i) v += i < a.shares ? u[i] : 0.f;
    finish(t, n0 + cl, v);
  }
}

namespace {

template <int F, int X>
hipError_t run_up(const TokensArgs& a, hipStream_t s) {
  const Tokens& p = a.p;
  const long items = (long)std::min(p.M * p.k, p.E) * (p.I / 16) + p.S / 16;
  const int pairs = cdiv(p.H, 256), px = cdiv(pairs, kUpWaves);   // pairs a wave takes
  const bool exact = p.H % 256 == 0;
  // A wave keeps at most three pairs of x and two tiles of codes for each (226 to 242 of its 256 registers), of
  // partial pairs two, so wider layers go a step at a time: 64 experts, 7168 to 2048, MXFP4, eight tokens take 302
  // us here, where 6144 take 101.
  if (p.H < 256 || px > (exact ? 3 : 2)) {
    const dim3 grid((unsigned)std::min<long>(items, 256));
    hipLaunchKernelGGL((tokens_up_any_kernel<F, X>), grid, dim3(kUpWaves * 64), 0, s, a);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)std::min<long>(items, px == 1 ? 512 : 256)), block((unsigned)cdiv(pairs, px) * 64);
  if (!exact && px == 1) hipLaunchKernelGGL((tokens_up_kernel<F, X, 1, false>), grid, block, 0, s, a);
  else if (!exact) hipLaunchKernelGGL((tokens_up_kernel<F, X, 2, false>), grid, block, 0, s, a);
  else if (px == 1) hipLaunchKernelGGL((tokens_up_kernel<F, X, 1, true>), grid, block, 0, s, a);
  else if (px == 2) hipLaunchKernelGGL((tokens_up_kernel<F, X, 2, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((tokens_up_kernel<F, X, 3, true>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <int F, int X>
hipError_t run_tokens(const TokensArgs& a, hipStream_t s) {
  const Tokens& p = a.p;
  const int rows = p.E + (p.gate ? 1 : 0);
  hipLaunchKernelGGL((tokens_router_kernel<X>), dim3((unsigned)((rows + 15) / 16), (unsigned)a.parts), dim3(512), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  err = run_up<F, X>(a, s);
  if (err != hipSuccess) return err;
  const dim3 down((unsigned)a.tiles, (unsigned)a.shares);
  // INT4's scales and zero points do not leave pairs the registers: with half the waves instead, eight tokens
  // of a layer of 256 experts, 6144 to 2048, g128 take 342 us against 307 by steps
  constexpr bool kPairs = !is_int4(F);
  const dim3 block(kDownWaves * 64);
  if (kPairs && p.I % 256 == 0 && p.S % 256 == 0)
    hipLaunchKernelGGL((tokens_down_kernel<F, X, kPairs, true>), down, block, 0, s, a);
  else if (kPairs && p.I >= 256 && (p.S == 0 || p.S >= 256))
    hipLaunchKernelGGL((tokens_down_kernel<F, X, kPairs, !kPairs>), down, block, 0, s, a);
  else
    hipLaunchKernelGGL((tokens_down_kernel<F, X, false, true>), down, block, 0, s, a);
  return hipGetLastError();
}

template <int X>
hipError_t run_format(const TokensArgs& a, hipStream_t s) {
  const Packed& w = a.p.w13;
  switch (w.format == HMOE_WEIGHT_INT4 ? w.group : w.format) {
    case HMOE_WEIGHT_NVFP4: return run_tokens<kNv, X>(a, s);
    case HMOE_WEIGHT_MXFP4: return run_tokens<kMx, X>(a, s);
    case 32: return run_tokens<kI32, X>(a, s);
    case 64: return run_tokens<kI64, X>(a, s);
    default: return run_tokens<kI128, X>(a, s);
  }
}

}  // namespace

size_t tokens_scratch(int M, int E, int H, int I, int k, int S) { return tokens_plan(M, E, H, I, k, S).total; }

hipError_t launch_tokens(const Tokens& p, void* scratch, hipStream_t s) {
  const TokensScratch t = tokens_plan(p.M, p.E, p.H, p.I, p.k, p.S);
  char* ws = static_cast<char*>(scratch);
  const TokensArgs a{p, reinterpret_cast<float*>(ws + t.logits), t.pitch, t.parts, reinterpret_cast<TokensPlan*>(ws + t.plan),
                     reinterpret_cast<float*>(ws + t.h), reinterpret_cast<float*>(ws + t.hs),
                     reinterpret_cast<float*>(ws + t.sums), reinterpret_cast<int*>(ws + t.done), t.tiles, t.shares};
  return p.dtype == HMOE_DTYPE_FP16 ? run_format<kHf>(a, s) : run_format<kBf>(a, s);
}

}  // namespace hmoe
