// Routing kernels: softmax top-k renormalised (one 64-lane wave per token), and the
// decode variant that also writes each (token, top-k) slot's pass record and the
// expert tier map (the direct top-k addressing of the decode path,
// local-inference-lab/vllm PR #92, "How it works").
#include "route_common.h"

namespace hmoe {

constexpr int kRouteWaves = 4;  // tokens per block of the general route kernel

// route_select of one token, writing its k ids and weights
__device__ __forceinline__ int route_token_any(const float* __restrict__ row, int E, int k,
                                               int lane, int32_t* __restrict__ ids_out,
                                               float* __restrict__ w_out) {
  float w;
  const int id = route_select_any(row, E, k, lane, &w);
  if (lane < k) {
    ids_out[lane] = id;
    w_out[lane] = w;
  }
  return id;
}

__global__ __launch_bounds__(kRouteWaves * kWave) void route_kernel(
    const float* __restrict__ logits, int M, int E, int k, int32_t* __restrict__ ids,
    float* __restrict__ w) {
  const int lane = threadIdx.x & (kWave - 1);
  const int t = blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
  if (t >= M) return;
  route_token_any(logits + (size_t)t * E, E, k, lane, ids + (size_t)t * k, w + (size_t)t * k);
}

struct RouteDecodeArgs {
  const float* logits;
  int M, E, k;
  int32_t* ids;
  float* w;
  int32_t* expert_tier;
  int32_t* pass;  // [M * k, 4]: slot, tier code, token, e (slot order)
};

constexpr int kGroupThreads = kDecodeMaxM * kWave;  // one wave per decode token
constexpr int kGroupWaves = kDecodeMaxM;

// Decode routing (M <= 8): one wave per token; each slot's pass record (the direct
// top-k addressing of the decode GEMVs) and the expert tier map. No block-wide step:
// the distinct-expert grouping is built later, off the critical path, by the combine.
__global__ __launch_bounds__(kGroupThreads) void route_decode_kernel(RouteDecodeArgs a, TierMask tm) {
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x >> 6;
  if (wave < a.M) {
    const int e = route_token_any(a.logits + (size_t)wave * a.E, a.E, a.k, lane,
                                  a.ids + wave * a.k, a.w + wave * a.k);
    if (lane < a.k) {
      const int s = wave * a.k + lane;
      reinterpret_cast<int4*>(a.pass)[s] = make_int4(s, tier_code(tm, e), wave, e);
    }
  }
  for (int e = threadIdx.x; e < a.E; e += kGroupThreads) a.expert_tier[e] = tier_code(tm, e);
}

hipError_t launch_route(const float* logits, int M, int E, int k, int32_t* ids, float* w,
                        hipStream_t s) {
  if (M == 0) return hipSuccess;
  const int blocks = (M + kRouteWaves - 1) / kRouteWaves;
  hipLaunchKernelGGL(route_kernel, dim3(blocks), dim3(kRouteWaves * kWave), 0, s, logits, M, E,
                     k, ids, w);
  return hipGetLastError();
}

hipError_t launch_route_group(const Layer& L, const float* logits, int M, void* scratch,
                              hipStream_t s) {
  char* base = static_cast<char*>(scratch);
  RouteDecodeArgs a;
  a.logits = logits;
  a.M = M;
  a.E = L.E;
  a.k = L.k;
  a.ids = reinterpret_cast<int32_t*>(base + L.plan.topk_ids);
  a.w = reinterpret_cast<float*>(base + L.plan.topk_w);
  a.expert_tier = reinterpret_cast<int32_t*>(base + L.plan.expert_tier);
  a.pass = reinterpret_cast<int32_t*>(base + L.plan.d_pass);
  hipLaunchKernelGGL(route_decode_kernel, dim3(1), dim3(kGroupThreads), 0, s, a, make_tier_mask(L));
  return hipGetLastError();
}

// Gradient of the renormalised top-k weights: w = softmax over the selected logits, so
// dl[e_j] = w_j (dw_j - sum_i w_i dw_i) and every other logit's gradient is zero. Bound by
// the M * E * 4 bytes it writes. A wave takes four tokens, 16 lanes a token, so one load
// each brings their ids, weights and gradients; it then builds 256 logits a token at a time
// in LDS (zeros, then the ids' values; the slots of one id are added up in registers, in slot
// order, and its first one writes) and writes them as 16 bytes a lane: no fill before, no scatter
// to memory, no order to depend on. 16384 tokens, 256 experts (18 MB): 7.7 us, 2.4 TB/s, of
// which a launch is about 2; 8 tokens 2.1 us.
struct __attribute__((packed, aligned(4))) F32x4 {
  float v[4];
};
constexpr int kBwdTokens = 4, kBwdCols = 256;

// LDS written by some lanes of the wave is read by others: no value is carried past here in
// a register (the LDS operations themselves keep their order)
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// sum of the slots I .. k - 1 of the token that have this lane's id (a row of 16 lanes holds a
// token's slots); a lane with such a slot before its own does not write
template <int I>
__device__ __forceinline__ void add_slots(int id, float g, int j, int k, bool& writes, float& sum) {
  if constexpr (I < kMaxTopK) {
    if (I >= k) return;
    constexpr int kLane = 0x150 + I;  // lane I of each row
    const int other = __builtin_amdgcn_update_dpp(0, id, kLane, 0xF, 0xF, true);
    const float v = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(g), kLane, 0xF, 0xF, true));
    if (other == id) {
      sum += v;
      writes = writes && I >= j;
    }
    add_slots<I + 1>(id, g, j, k, writes, sum);
  }
}

__global__ __launch_bounds__(kRouteWaves * kWave) void route_bwd_kernel(
    const int32_t* __restrict__ ids, const float* __restrict__ w, const float* __restrict__ dw,
    int M, int E, int k, float* __restrict__ dl) {
  __shared__ __align__(16) float s_row[kRouteWaves][kBwdTokens][kBwdCols];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const long t0 = (blockIdx.x * (long)kRouteWaves + wave) * kBwdTokens;
  if (t0 >= M) return;
  const int j = lane & 15, mine = lane >> 4;
  const bool in = j < k && t0 + mine < M;
  const long at = (t0 + mine) * k + j;
  const int id = in ? ids[at] : -1;
  const float wj = in ? w[at] : 0.f, dj = in ? dw[at] : 0.f;
  const float g = wj * (dj - group_sum<16>(wj * dj));
  bool writes = (unsigned)id < (unsigned)E;
  float sum = 0.f;
  add_slots<0>(id, g, j, k, writes, sum);
  float(*row)[kBwdCols] = s_row[wave];
  for (int e0 = 0; e0 < E; e0 += kBwdCols) {
#pragma unroll
    for (int t = 0; t < kBwdTokens; ++t)
      *reinterpret_cast<float4*>(&row[t][lane * 4]) = make_float4(0.f, 0.f, 0.f, 0.f);
    wave_fence();
    if (writes && id >= e0 && id < e0 + kBwdCols) row[mine][id - e0] = sum;
    wave_fence();
    const int e = e0 + lane * 4;
#pragma unroll
    for (int t = 0; t < kBwdTokens; ++t) {
      if (t0 + t >= M || e >= E) continue;
      const float4 v = *reinterpret_cast<const float4*>(&row[t][lane * 4]);
      float* out = dl + (t0 + t) * E + e;
      if (e + 4 <= E) {
        *reinterpret_cast<F32x4*>(out) = F32x4{{v.x, v.y, v.z, v.w}};
      } else {
        out[0] = v.x;
        if (e + 1 < E) out[1] = v.y;
        if (e + 2 < E) out[2] = v.z;
      }
    }
    wave_fence();
  }
}

hipError_t launch_route_backward(const int32_t* ids, const float* w, const float* dw, int M, int E,
                                 int k, float* dlogits, hipStream_t s) {
  if (M == 0) return hipSuccess;
  constexpr int kTokens = kRouteWaves * kBwdTokens;
  hipLaunchKernelGGL(route_bwd_kernel, dim3((M + kTokens - 1) / kTokens), dim3(kRouteWaves * kWave), 0,
                     s, ids, w, dw, M, E, k, dlogits);
  return hipGetLastError();
}

TierMask make_tier_mask(const Layer& L) {
  TierMask m;
  for (int i = 0; i < kMaxExperts / 32; ++i) m.w[i] = L.nf3_mask[i];
  return m;
}

}  // namespace hmoe
