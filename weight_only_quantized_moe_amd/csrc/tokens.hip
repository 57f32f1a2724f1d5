// A whole mixture-of-experts layer for a few tokens (M <= 16), experts in 4-bit weights with group
// scales (packed.h):
//   l = x R^T,  the k largest of softmax(l), renormalised: p,
//   h = silu(x Wg_e^T) * (x Wu_e^T),  y = base + sum_j p_j W2_e h_e + sigmoid(x . gate) W2_s h_s.
//
// It is bound by reading the touched experts once and, for one or two tokens, by the latency of
// its dependent steps. Three launches: the router's logits; routing and the experts' first products
// (each block routes all tokens by itself, which costs less than a launch); the second products,
// where a block owns 16 columns of y and adds up every expert's share, so that nothing is summed
// across blocks. An expert that several tokens took is read once: its tokens are rows of the same
// MFMA.
//
// h, times its routing weight and the second matrix's own scale, goes into the second product as
// two bf16 parts (16 of its 24 bits, 2^-17 of its value off): rounding it to 16 bits once would
// add an error like that of y's own rounding, and the matrix cores have the time.
#include <algorithm>

#include "packed.h"
#include "route_common.h"

namespace hmoe {

namespace {

constexpr int kUpWaves = 8, kDownWaves = 16;
constexpr int kMaxPairs = HMOE_TOKENS_MAX_M * kMaxTopK;   // (token, expert) pairs, so also experts in use

// What the second launch leaves for the third.
struct TokensPlan {
  int count;                     // experts in use, ascending
  int expert[kMaxPairs];
  int16_t row[kMaxPairs * 16];   // row of h of each token, -1: the token did not take this expert
};

// Scratch, as offsets.
struct TokensScratch {
  size_t logits = 0, plan = 0, h = 0, hs = 0, total = 0;   // h, hs: high parts, then low parts
  int pitch = 0;                                            // of the logits
};
TokensScratch tokens_plan(int M, int E, int I, int k, int S) {
  TokensScratch t;
  auto take = [&](size_t bytes) {
    const size_t at = t.total;
    t.total += (bytes + 255) & ~size_t(255);
    return at;
  };
  t.pitch = E + 1;
  t.logits = take((size_t)M * t.pitch * 4);
  t.plan = take(sizeof(TokensPlan));
  t.h = take((size_t)M * k * I * 4);
  t.hs = take((size_t)M * S * 4);
  return t;
}

}  // namespace

struct TokensArgs {
  Tokens p;
  float* logits;
  int pitch;
  TokensPlan* plan;
  uint16_t* h;    // [2, M k, I]
  uint16_t* hs;   // [2, M, S]
};

// logits[m, e] = x[m] . router[e], and the shared expert's gate as row E. A block takes 16 rows.
template <int X>
__global__ __launch_bounds__(1024) void tokens_router_kernel(TokensArgs a) {
  __shared__ float red[16][256];
  const Tokens& p = a.p;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 16 + (lane & 15), rows = p.E + (p.gate ? 1 : 0);
  const uint16_t* r = (e < p.E ? p.router + (long)e * p.H : p.gate ? p.gate : p.router) + (lane >> 4) * 8;
  const uint16_t* x = p.x + (long)min(lane & 15, p.M - 1) * p.xs + (lane >> 4) * 8;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = wave; s < p.H / 32; s += 64) {
    u32x4 rv[4], xv[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int at = min(s + 16 * d, p.H / 32 - 1) * 32;
      rv[d] = load16(r + at);
      xv[d] = load16(x + at);
    }
#pragma unroll
    for (int d = 0; d < 4; ++d)
      if (s + 16 * d < p.H / 32) acc = mfma16<X>(xv[d], rv[d], acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][i * 64 + lane] = acc[i];
  __syncthreads();
  if (threadIdx.x >= 256) return;
  const int l = threadIdx.x & 63, m = (l >> 4) * 4 + (threadIdx.x >> 6), c = blockIdx.x * 16 + (l & 15);
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) v += red[w][threadIdx.x];
  if (m < p.M && c < rows) a.logits[m * a.pitch + c] = v;
}

// Routing, in every block, and h of the experts in use and of the shared expert. A work item is 16
// columns of one expert's h: 16 gate rows and 16 up rows of W13, the steps of K dealt to the waves.
template <int F, int X, bool FULL>
__global__ __launch_bounds__(kUpWaves * 64) void tokens_up_kernel(TokensArgs a) {
  __shared__ int s_id[kMaxPairs];
  __shared__ float s_w[kMaxPairs];
  __shared__ uint32_t s_mask[kMaxExperts];          // tokens of each expert
  __shared__ int s_expert[kMaxPairs], s_off[kMaxPairs];
  __shared__ float red[2][kUpWaves][2][256];
  __shared__ int s_count;
  const Tokens& p = a.p;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int e = threadIdx.x; e < p.E; e += kUpWaves * 64) s_mask[e] = 0u;
  __syncthreads();
  for (int t = wave; t < p.M; t += kUpWaves) {
    float w;
    const int id = route_select_any(a.logits + (long)t * a.pitch, p.E, p.k, lane, &w);
    if (lane < p.k) {
      s_id[t * p.k + lane] = id;
      s_w[t * p.k + lane] = w;
      atomicOr(&s_mask[id], 1u << t);
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
      const uint32_t mask = e < p.E ? s_mask[e] : 0u;
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
        s_expert[at] = e;
        s_off[at] = rows + before;
      }
      count += __popcll(used);
      rows += total;
    }
    if (lane == 0) s_count = count;
  }
  __syncthreads();
  const int count = s_count;
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) a.plan->count = count;
    for (int i = threadIdx.x; i < count * 16; i += kUpWaves * 64) {
      const int d = i >> 4, m = i & 15, e = s_expert[d];
      const uint32_t mask = s_mask[e];
      if (m == 0) a.plan->expert[d] = e;
      a.plan->row[i] = (mask >> m) & 1u ? (int16_t)(s_off[d] + __popc(mask & ((1u << m) - 1u))) : (int16_t)-1;
    }
  }

  const int tiles = p.I / 16, items = count * tiles + p.S / 16;
  const int steps = (p.H + 127) / 128;
  int buf = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x, buf ^= 1) {
    const int d = item / tiles;
    const bool shared = d >= count;
    const int i0 = (shared ? item - count * tiles : item - d * tiles) * 16;
    const int e = shared ? 0 : s_expert[d];
    const uint32_t mask = shared ? (1u << p.M) - 1u : s_mask[e];
    const int n = __popc(mask);
    const int width = shared ? p.S : p.I;
    const Packed& w = shared ? p.s13 : p.w13;
    const long row0 = (long)e * 2 * width + i0 + (lane & 15);
    // the lane's token: the (lane & 15)-th of the mask, or its last
    uint32_t rest = mask;
    for (int i = min(lane & 15, n - 1); i > 0; --i) rest &= rest - 1u;
    const uint16_t* x = p.x + (long)(__ffs(rest) - 1) * p.xs + (lane >> 4) * 8;
    const PackedRow row[2] = {packed_row<F>(w, row0, p.H, lane), packed_row<F>(w, row0 + width, p.H, lane)};
    f32x4 acc[2][1] = {{{0.f, 0.f, 0.f, 0.f}}, {{0.f, 0.f, 0.f, 0.f}}};
    for (int s0 = wave; s0 < steps; s0 += kUpWaves * 2) {
      Codes<F> c[2][2];
      u32x4 xv[2][4][1];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int s = min(s0 + j * kUpWaves, steps - 1);
        load_codes<F, FULL>(c[j][0], row[0], s, p.H, lane);
        load_codes<F, FULL>(c[j][1], row[1], s, p.H, lane);
#pragma unroll
        for (int b = 0; b < 4; ++b) xv[j][b][0] = load16(x + (FULL ? s * 128 + b * 32 : min(s * 128 + b * 32, p.H - 32)));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (s0 + j * kUpWaves >= steps) continue;
        const int blocks = FULL ? 4 : min(4, (p.H - (s0 + j * kUpWaves) * 128) / 32);
        if constexpr (is_int4(F)) {
#pragma unroll
          for (int b = 0; b < 4; ++b) xv[j][b][0] = int4_order(xv[j][b][0]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          turn4(c[j][r].q);
          block_product<F, X, X, 0, 1>(acc[r], c[j][r], xv[j][0], lane);
          if (blocks > 1) block_product<F, X, X, 1, 1>(acc[r], c[j][r], xv[j][1], lane);
          if (blocks > 2) block_product<F, X, X, 2, 1>(acc[r], c[j][r], xv[j][2], lane);
          if (blocks > 3) block_product<F, X, X, 3, 1>(acc[r], c[j][r], xv[j][3], lane);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[buf][wave][r][i * 64 + lane] = acc[r][0][i];
    __syncthreads();
    if (threadIdx.x < 256) {
      const int l = threadIdx.x & 63, m = (l >> 4) * 4 + (threadIdx.x >> 6), i = i0 + (l & 15);
      if (m < n) {
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int v = 0; v < kUpWaves; ++v) {
          gate += red[buf][v][0][threadIdx.x];
          up += red[buf][v][1][threadIdx.x];
        }
        float weight = 1.f;
        uint32_t left = mask;
        for (int j = 0; j < m; ++j) left &= left - 1u;
        const int t = __ffs(left) - 1;
        if (!shared) {
          for (int j = 0; j < p.k; ++j)
            if (s_id[t * p.k + j] == e) weight = s_w[t * p.k + j];
        } else if (p.gate) {
          weight = 1.f / (1.f + expf(-a.logits[(long)t * a.pitch + p.E]));
        }
        if constexpr (F == kNv) {
          gate *= w.g[e];
          up *= w.g[e];
          weight *= shared ? p.s2.g[0] : p.w2.g[e];
        }
        const float h = silu(gate) * up * weight;
        const uint32_t hi = __float_as_uint(h) & 0xFFFF0000u;
        const float lo = __builtin_isinf(h) ? 0.f : h - __uint_as_float(hi);
        const long rows = shared ? p.M : p.M * p.k;
        uint16_t* out = shared ? a.hs : a.h;
        const long at = (long)(shared ? m : s_off[d] + m) * width + i;
        out[at] = (uint16_t)(hi >> 16);
        out[rows * width + at] = from_f32<kBf>(lo);
      }
    }
  }
}

// y: a block takes 16 columns, its waves an even share of the steps of all experts in use.
template <int F, int X, bool FULL>
__global__ __launch_bounds__(kDownWaves * 64) void tokens_down_kernel(TokensArgs a) {
  __shared__ int s_expert[kMaxPairs];
  __shared__ int16_t s_row[kMaxPairs * 16];
  __shared__ float red[kDownWaves][256];
  const Tokens& p = a.p;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16, count = a.plan->count;
  for (int i = threadIdx.x; i < count * 16; i += kDownWaves * 64) {
    s_row[i] = a.plan->row[i];
    if (i < count) s_expert[i] = a.plan->expert[i];
  }
  __syncthreads();
  const int n = min(n0 + (lane & 15), p.H - 1), m = lane & 15;
  const int steps = (p.I + 127) / 128, total = count * steps + (p.S + 127) / 128;
  const int from = (int)((long)total * wave / kDownWaves), to = (int)((long)total * (wave + 1) / kDownWaves);
  f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  for (int f0 = from; f0 < to; f0 += 2) {
    Codes<F> c[2];
    u32x4 h[2][4][2];
    int blocks[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int f = min(f0 + j, to - 1);
      const int d = min(f / steps, count);
      const bool shared = d == count;
      const int s = f - d * steps, K = shared ? p.S : p.I;
      const PackedRow row = packed_row<F>(shared ? p.s2 : p.w2, (shared ? 0l : (long)s_expert[d] * p.H) + n, K, lane);
      load_codes<F, FULL>(c[j], row, s, K, lane);
      const int r = shared ? (m < p.M ? m : -1) : s_row[d * 16 + m];
      const uint16_t* hi = (shared ? a.hs : a.h) + (long)max(r, 0) * K + (lane >> 4) * 8;
      const long low = (long)(shared ? p.M : p.M * p.k) * K;
      const uint32_t keep = r < 0 ? 0u : ~0u;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int at = FULL ? s * 128 + b * 32 : min(s * 128 + b * 32, K - 32);
        h[j][b][0] = *reinterpret_cast<const u32x4*>(hi + at) & keep;
        h[j][b][1] = *reinterpret_cast<const u32x4*>(hi + low + at) & keep;
      }
      blocks[j] = FULL ? 4 : min(4, (K - s * 128) / 32);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (f0 + j >= to) continue;
      if constexpr (is_int4(F)) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          h[j][b][0] = int4_order(h[j][b][0]);
          h[j][b][1] = int4_order(h[j][b][1]);
        }
      }
      turn4(c[j].q);
      block_product<F, kBf, X, 0, 2>(acc, c[j], h[j][0], lane);
      if (blocks[j] > 1) block_product<F, kBf, X, 1, 2>(acc, c[j], h[j][1], lane);
      if (blocks[j] > 2) block_product<F, kBf, X, 2, 2>(acc, c[j], h[j][2], lane);
      if (blocks[j] > 3) block_product<F, kBf, X, 3, 2>(acc, c[j], h[j][3], lane);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][i * 64 + lane] = acc[0][i] + acc[1][i];
  __syncthreads();
  if (threadIdx.x >= 256) return;
  const int l = threadIdx.x & 63, t = (l >> 4) * 4 + (threadIdx.x >> 6), col = n0 + (l & 15);
  if (t >= p.M || col >= p.H) return;
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kDownWaves; ++w) v += red[w][threadIdx.x];
  if (p.base) v += to_f32<X>(p.base[t * p.bs + col]);
  p.y[t * p.ys + col] = from_f32<X>(v);
}

namespace {

template <int F, int X>
hipError_t run_tokens(const TokensArgs& a, hipStream_t s) {
  const Tokens& p = a.p;
  const int rows = p.E + (p.gate ? 1 : 0);
  hipLaunchKernelGGL((tokens_router_kernel<X>), dim3((unsigned)((rows + 15) / 16)), dim3(1024), 0, s, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const long items = (long)std::min(p.M * p.k, p.E) * (p.I / 16) + p.S / 16;
  const dim3 up((unsigned)std::min<long>(items, 512)), down((unsigned)((p.H + 15) / 16));
  if (p.H % 128 == 0)
    hipLaunchKernelGGL((tokens_up_kernel<F, X, true>), up, dim3(kUpWaves * 64), 0, s, a);
  else
    hipLaunchKernelGGL((tokens_up_kernel<F, X, false>), up, dim3(kUpWaves * 64), 0, s, a);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  if (p.I % 128 == 0 && p.S % 128 == 0)
    hipLaunchKernelGGL((tokens_down_kernel<F, X, true>), down, dim3(kDownWaves * 64), 0, s, a);
  else
    hipLaunchKernelGGL((tokens_down_kernel<F, X, false>), down, dim3(kDownWaves * 64), 0, s, a);
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

size_t tokens_scratch(int M, int E, int I, int k, int S) { return tokens_plan(M, E, I, k, S).total; }

hipError_t launch_tokens(const Tokens& p, void* scratch, hipStream_t s) {
  const TokensScratch t = tokens_plan(p.M, p.E, p.I, p.k, p.S);
  char* ws = static_cast<char*>(scratch);
  const TokensArgs a{p, reinterpret_cast<float*>(ws + t.logits), t.pitch, reinterpret_cast<TokensPlan*>(ws + t.plan),
                     reinterpret_cast<uint16_t*>(ws + t.h), reinterpret_cast<uint16_t*>(ws + t.hs)};
  return p.dtype == HMOE_DTYPE_FP16 ? run_format<kHf>(a, s) : run_format<kBf>(a, s);
}

}  // namespace hmoe
