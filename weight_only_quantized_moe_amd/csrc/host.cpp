// C ABI of libhmoe: layer creation and validation, the scratch planner, views into
// scratch, and dispatch of the route / align / forward / dequant kernels and of the operators
// around the experts (row movements, routing gradient, adapters).
// Nothing here allocates, frees or synchronises device memory.
#include <string.h>

#include <algorithm>
#include <initializer_list>
#include <new>
#include <string>

#include "hmoe_internal.h"

struct hmoe_layer {
  hmoe::Layer L;
};

namespace {

thread_local std::string g_last_error;

hmoe_status fail(hmoe_status st, const std::string& msg) {
  g_last_error = msg;
  return st;
}

hmoe_status hip_fail(hipError_t err, const char* what) {
  return fail(HMOE_ERR_HIP, std::string(what) + ": " + hipGetErrorString(err));
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Align capacity of one tier: M*k slots plus, for every expert that can own a slot,
// up to block_m - 1 padding entries.
int tier_capacity(int tokens, int k, int experts_in_tier, int bm) {
  if (experts_in_tier == 0) return 0;
  const long ns = (long)tokens * k;
  const long touched = std::min<long>(experts_in_tier, ns);
  const long cap = ns + touched * (bm - 1);
  return (int)((cap + bm - 1) / bm * bm);
}

void plan_scratch(hmoe::Layer& L) {
  hmoe::ScratchPlan& P = L.plan;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + std::max<size_t>(bytes, 4));
    return at;
  };
  const size_t mk = (size_t)L.max_tokens * L.k;
  const size_t dec_slots = (size_t)hmoe::kDecodeMaxM * L.k;
  P.topk_ids = take(std::max(mk, dec_slots) * 4);
  P.topk_w = take(std::max(mk, dec_slots) * 4);
  P.expert_tier = take((size_t)L.E * 4);
  P.d_counts = take(2 * 4);
  P.d_experts = take((size_t)L.max_distinct * 4);
  P.d_nslots = take((size_t)L.max_distinct * 4);
  P.d_slots = take((size_t)L.max_distinct * hmoe::kDecodeMaxM * 4);
  P.d_pass = take(dec_slots * hmoe::kPassRec * 4);
  P.h_dec = take(dec_slots * L.I * 4);
  P.o_dec = take(dec_slots * L.H * 4);
  P.d_sync = take(hmoe::fused_sync_words(L.k, L.H) * 4);
  for (int t = 0; t < 2; ++t) {
    const int cap = L.cap[t];
    const int ne = t == 0 ? L.E4 : L.E3;
    P.a_slots[t] = take((size_t)cap * 4);
    P.a_bexp[t] = take((size_t)(cap / L.block_m) * 4);
    P.a_eoff[t] = take((size_t)(ne + 1) * 4);
    P.a_npad[t] = take(4);
  }
  if (L.max_tokens > hmoe::kDecodeMaxM || L.act_format == HMOE_ACT_MXFP4) {
    P.h_pre = take((size_t)(L.cap[0] + L.cap[1]) * L.I * 2);
    P.o_pre = take(mk * L.H * 4);
    P.x16_pre = take((size_t)L.max_tokens * L.H * 2);
    P.xe_pre = take((size_t)L.max_tokens * 4);
    P.pf_fac = take((size_t)(L.cap[0] + L.cap[1]) * 4);
  } else {
    P.h_pre = take(0);
    P.o_pre = take(0);
    P.x16_pre = take(0);
    P.xe_pre = take(0);
    P.pf_fac = take(0);
  }
  if (L.act_format == HMOE_ACT_MXFP4) {
    P.mx_xq = take((size_t)L.max_tokens * L.H / 2);
    P.mx_xs = take((size_t)L.max_tokens * L.H / 32);
    P.mx_h32 = take((size_t)L.cap[0] * L.I * 4);
    P.mx_hq = take((size_t)L.cap[0] * L.I / 2);
    P.mx_hs = take((size_t)L.cap[0] * L.I / 32);
  }
  P.total = off;
}

hmoe_status check_layer(const hmoe_layer* layer) {
  if (!layer) return fail(HMOE_ERR_INVALID_ARG, "layer is NULL");
  return HMOE_OK;
}

hmoe_status check_scratch(const hmoe::Layer& L, void* scratch, size_t bytes) {
  if (!scratch) return fail(HMOE_ERR_ALIGN, "scratch is NULL");
  if (!aligned(scratch, 256)) return fail(HMOE_ERR_ALIGN, "scratch must be 256-byte aligned");
  if (bytes < L.plan.total)
    return fail(HMOE_ERR_SCRATCH, "scratch has " + std::to_string(bytes) + " bytes, needs " +
                                      std::to_string(L.plan.total));
  return HMOE_OK;
}

hmoe_status check_weights(const hmoe::Layer& L, const hmoe_weights* w) {
  if (!w) return fail(HMOE_ERR_INVALID_ARG, "weights is NULL");
  if (L.E4 > 0) {
    if (!w->kept_w13_q || !w->kept_w13_s || !w->kept_w2_q || !w->kept_w2_s)
      return fail(HMOE_ERR_INVALID_ARG, "kept-tier weight or scale array is NULL");
    if (L.kept_format == HMOE_KEPT_NVFP4 && (!w->kept_w13_g || !w->kept_w2_g))
      return fail(HMOE_ERR_INVALID_ARG, "NVFP4 per-tensor scale array is NULL");
    if (!aligned(w->kept_w13_q, 16) || !aligned(w->kept_w2_q, 16) || !aligned(w->kept_w13_s, 4) ||
        !aligned(w->kept_w2_s, 4) || (w->kept_w13_g && !aligned(w->kept_w13_g, 4)) ||
        (w->kept_w2_g && !aligned(w->kept_w2_g, 4)))
      return fail(HMOE_ERR_ALIGN, "kept-tier arrays: codes need 16-byte and scales 4-byte alignment");
  }
  if (L.E3 > 0) {
    if (!w->nf3_w13_q || !w->nf3_w13_s || !w->nf3_w2_q || !w->nf3_w2_s)
      return fail(HMOE_ERR_INVALID_ARG, "NF3-tier weight or scale array is NULL");
    if (!aligned(w->nf3_w13_q, 16) || !aligned(w->nf3_w2_q, 16) || !aligned(w->nf3_w13_s, 4) ||
        !aligned(w->nf3_w2_s, 4))
      return fail(HMOE_ERR_ALIGN, "NF3-tier arrays: codes need 16-byte and scales 4-byte alignment");
  }
  return HMOE_OK;
}

// ---- operators around the experts

int element_size(int dtype) { return dtype == HMOE_DTYPE_FP32 ? 4 : 2; }

hmoe_status check_permute_shape(int32_t M, int32_t k) {
  if (M < 0) return fail(HMOE_ERR_INVALID_ARG, "M < 0");
  if (k < 1 || k > hmoe::kMaxTopK) return fail(HMOE_ERR_INVALID_ARG, "k must be in [1, 16]");
  if ((long)M * k > (1L << 24)) return fail(HMOE_ERR_UNSUPPORTED, "M * k > 2^24");
  return HMOE_OK;
}

hmoe_status check_experts(int32_t E) {
  if (E < 1 || E > hmoe::kMaxExperts) return fail(HMOE_ERR_INVALID_ARG, "E must be in [1, 1024]");
  return HMOE_OK;
}

hmoe_status check_rows(int32_t M, int32_t H, int32_t dtype) {
  if (H < 1) return fail(HMOE_ERR_INVALID_ARG, "H must be >= 1");
  if (dtype != HMOE_DTYPE_BF16 && dtype != HMOE_DTYPE_FP16 && dtype != HMOE_DTYPE_FP32)
    return fail(HMOE_ERR_INVALID_ARG, "unknown dtype");
  if (!hmoe::row_grid_fits(M, (long)H * element_size(dtype)))
    return fail(HMOE_ERR_UNSUPPORTED, "M rows of H elements are 2^24 blocks of 4 KiB or more");
  return HMOE_OK;
}

// a matrix of rows: element-aligned, rows that do not overlap
hmoe_status check_matrix(const char* name, const void* p, int64_t stride, int64_t cols, int esize) {
  if (stride < cols)
    return fail(HMOE_ERR_INVALID_ARG, std::string(name) + "'s row stride is below its row length");
  if (stride > (int64_t(1) << 40))
    return fail(HMOE_ERR_UNSUPPORTED, std::string(name) + "'s row stride is above 2^40");
  if (!p || !aligned(p, esize))
    return fail(HMOE_ERR_ALIGN, std::string(name) + " must be non-NULL and aligned to its elements");
  return HMOE_OK;
}

hmoe_status check_arrays(const char* names, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p || !aligned(p, 16))
      return fail(HMOE_ERR_ALIGN, std::string(names) + " must be non-NULL and 16-byte aligned");
  return HMOE_OK;
}

// An output that starts where an input or another output does would be written while that is read
// or written. `also`: an input of which this holds for this output, while another may be it.
struct Output {
  const char* name;
  const void* p;
  const void* also = nullptr;
};
hmoe_status check_apart(std::initializer_list<const void*> ins, std::initializer_list<Output> outs) {
  for (const Output* o = outs.begin(); o != outs.end(); ++o) {
    if (!o->p) continue;
    bool in = o->p == o->also;
    for (const void* p : ins) in = in || p == o->p;
    if (in) return fail(HMOE_ERR_INVALID_ARG, std::string(o->name) + " starts where an input does");
    for (const Output* q = outs.begin(); q != o; ++q)
      if (q->p == o->p) return fail(HMOE_ERR_INVALID_ARG, std::string(o->name) + " starts where " + q->name + " does");
  }
  return HMOE_OK;
}

hmoe_status check_op_scratch(const void* scratch, size_t have, size_t need) {
  if (have < need)
    return fail(HMOE_ERR_SCRATCH, "scratch has " + std::to_string(have) + " bytes, needs " +
                                      std::to_string(need));
  if (need && (!scratch || !aligned(scratch, 256)))
    return fail(HMOE_ERR_ALIGN, "scratch must be non-NULL and 256-byte aligned");
  return HMOE_OK;
}

size_t permute_scratch(int32_t M, int32_t k, int32_t E) {
  const int n = M * k;
  return n <= hmoe::kPermuteSmall ? 0 : align256(hmoe::sort_count_words(n, E) * 4);
}

hmoe_status check_lora(int32_t M, int32_t G, int32_t K, int32_t N, int32_t rank) {
  if (M < 0) return fail(HMOE_ERR_INVALID_ARG, "M < 0");
  if (G < 1 || K < 1 || N < 1 || rank < 1)
    return fail(HMOE_ERR_INVALID_ARG, "G, K, N and rank must be >= 1");
  if (K % 8 || N % 8 || rank % 8)
    return fail(HMOE_ERR_UNSUPPORTED, "K, N and rank must be multiples of 8");
  if (rank > hmoe::kMaxLoraRank) return fail(HMOE_ERR_UNSUPPORTED, "rank > 128");
  if (G > hmoe::kMaxGroups) return fail(HMOE_ERR_UNSUPPORTED, "G > 2048");
  if (M > (1 << 22) || K > (1 << 20) || N > (1 << 20))
    return fail(HMOE_ERR_UNSUPPORTED, "M > 2^22, or K or N > 2^20");
  return HMOE_OK;
}

hmoe_status check_base(const char* name, const uint16_t* base, int64_t bs, const uint16_t* out,
                       int64_t os, int64_t cols) {
  if (!base) return HMOE_OK;
  if (hmoe_status st = check_matrix(name, base, bs, cols, 2)) return st;
  if (base == out && bs != os)
    return fail(HMOE_ERR_INVALID_ARG, std::string(name) + " is the output itself with another stride");
  return HMOE_OK;
}

// ---- matrices of 4-bit weights

// columns K of a packed matrix: whole groups, and whole column blocks of the kernels
hmoe_status check_packed(const char* name, const hmoe_packed& w, int64_t K) {
  const std::string who = name;
  if (w.format != HMOE_WEIGHT_NVFP4 && w.format != HMOE_WEIGHT_MXFP4 && w.format != HMOE_WEIGHT_INT4)
    return fail(HMOE_ERR_INVALID_ARG, who + ": unknown format");
  const bool int4 = w.format == HMOE_WEIGHT_INT4;
  if (int4 && w.group != 32 && w.group != 64 && w.group != 128)
    return fail(HMOE_ERR_INVALID_ARG, who + ": group must be 32, 64 or 128");
  if (K % 32 || (int4 && K % w.group))
    return fail(HMOE_ERR_UNSUPPORTED, who + ": columns must be a multiple of 32 and of the group");
  if (!w.q || !aligned(w.q, 16) || !w.s || !aligned(w.s, 16))
    return fail(HMOE_ERR_ALIGN, who + ": q and s must be non-NULL and 16-byte aligned");
  if (int4 && !aligned(w.z, 16)) return fail(HMOE_ERR_ALIGN, who + ": z must be 16-byte aligned");
  if (w.format == HMOE_WEIGHT_NVFP4 && (!w.g || !aligned(w.g, 4)))
    return fail(HMOE_ERR_ALIGN, who + ": g must be non-NULL and 4-byte aligned");
  return HMOE_OK;
}

hmoe::Packed packed_of(const hmoe_packed& w) {
  const bool int4 = w.format == HMOE_WEIGHT_INT4;
  return {w.q, static_cast<const uint8_t*>(w.s), int4 ? w.z : nullptr,
          w.format == HMOE_WEIGHT_NVFP4 ? w.g : nullptr, w.format,
          int4 ? w.group : w.format == HMOE_WEIGHT_NVFP4 ? 16 : 32};
}

hmoe_status check_linear_shape(int32_t M, int32_t K, int32_t N) {
  if (M < 0 || K < 1 || N < 1) return fail(HMOE_ERR_INVALID_ARG, "M must be >= 0, K and N >= 1");
  if (K % 32) return fail(HMOE_ERR_UNSUPPORTED, "K must be a multiple of 32");
  if (M > (1 << 22) || K > (1 << 20) || N > (1 << 20))
    return fail(HMOE_ERR_UNSUPPORTED, "M > 2^22, or K or N > 2^20");
  return HMOE_OK;
}

hmoe_status check_half(int32_t dtype) {
  if (dtype != HMOE_DTYPE_BF16 && dtype != HMOE_DTYPE_FP16)
    return fail(HMOE_ERR_INVALID_ARG, "dtype must be bf16 or fp16");
  return HMOE_OK;
}

// an addend of rows: null, the output itself, a matrix, or one row for all (stride 0)
hmoe_status check_addend(const char* name, const void* base, int64_t bs, const void* out, int64_t os,
                         int64_t cols) {
  if (!base) return HMOE_OK;
  if (hmoe_status st = check_matrix(name, base, bs == 0 ? cols : bs, cols, 2)) return st;
  if (base == out && bs != os)
    return fail(HMOE_ERR_INVALID_ARG, std::string(name) + " is the output itself with another stride");
  return HMOE_OK;
}

hmoe_status run_linear(const char* in_name, const void* x, int64_t xs, const hmoe_packed* w, int32_t M,
                       int32_t K, int32_t N, int32_t dtype, const char* base_name, const void* base,
                       int64_t bs, const char* out_name, void* y, int64_t ys, void* scratch,
                       size_t scratch_bytes, bool back, hipStream_t stream) {
  if (hmoe_status st = check_linear_shape(M, K, N)) return st;
  if (hmoe_status st = check_half(dtype)) return st;
  if (!w) return fail(HMOE_ERR_INVALID_ARG, "w is NULL");
  if (hmoe_status st = check_packed("w", *w, K)) return st;
  if (M == 0) return HMOE_OK;
  const int in = back ? N : K, out = back ? K : N;
  if (hmoe_status st = check_matrix(in_name, x, xs, in, 2)) return st;
  if (hmoe_status st = check_matrix(out_name, y, ys, out, 2)) return st;
  if (hmoe_status st = check_addend(base_name, base, bs, y, ys, out)) return st;
  size_t need;
  hmoe::linear_scratch(M, K, N, back ? nullptr : &need, back ? &need : nullptr);
  if (hmoe_status st = check_op_scratch(scratch, scratch_bytes, need)) return st;
  const hmoe::Packed m = packed_of(*w);
  if (hmoe_status st = check_apart({x, m.q, m.s, m.z, m.g}, {{out_name, y}})) return st;
  const hmoe::Linear p{m, dtype, static_cast<const uint16_t*>(x), xs, M, K, N,
                       static_cast<const uint16_t*>(base), bs, static_cast<uint16_t*>(y), ys};
  hipError_t err = hmoe::launch_linear(p, back, scratch, stream);
  if (err != hipSuccess) return hip_fail(err, back ? "linear backward launch" : "linear launch");
  return HMOE_OK;
}

hmoe_status check_tokens_shape(int32_t M, int32_t E, int32_t H, int32_t I, int32_t k, int32_t S) {
  if (M < 0) return fail(HMOE_ERR_INVALID_ARG, "M < 0");
  if (hmoe_status st = check_experts(E)) return st;
  if (k < 1 || k > std::min(hmoe::kMaxTopK, (int)E))
    return fail(HMOE_ERR_INVALID_ARG, "k must be in [1, min(16, E)]");
  if (H < 1 || I < 1 || S < 0) return fail(HMOE_ERR_INVALID_ARG, "hidden and inter must be >= 1, shared_inter >= 0");
  if (H % 32 || I % 32 || S % 32)
    return fail(HMOE_ERR_UNSUPPORTED, "hidden, inter and shared_inter must be multiples of 32");
  if (H > (1 << 20) || I > (1 << 20) || S > (1 << 20))
    return fail(HMOE_ERR_UNSUPPORTED, "hidden, inter or shared_inter > 2^20");
  if (M > HMOE_TOKENS_MAX_M) return fail(HMOE_ERR_CAPACITY, "M > HMOE_TOKENS_MAX_M");
  return HMOE_OK;
}

}  // namespace

extern "C" {

// Prefill rows per expert block when the caller leaves it to the library: from the mean
// number of slots per expert at max_tokens, t = max_tokens * k / E. The GEMM runs an
// expert's last, partly padded block as a 16-, 32- or 64-row tile, so a large block_m
// costs little for small experts; but its LDS stage allows two blocks per CU where a
// 32-row block_m allows three. Measured on the GLM-class layer on MI355X, skewed and
// unskewed routing: 16 rows are fastest below t = 4, 32 below t = 24 and 128 above.
static int auto_block_m(long max_tokens, long k, long E) {
  const long t = max_tokens * k;
  if (t < 4 * E) return 16;
  if (t < 24 * E) return 32;
  return 128;
}

hmoe_status moe_layer_create(const hmoe_layer_desc* d, hmoe_layer** out) {
  if (!d || !out) return fail(HMOE_ERR_INVALID_ARG, "desc and out must not be NULL");
  *out = nullptr;
  if (d->num_experts < 1) return fail(HMOE_ERR_INVALID_ARG, "num_experts must be >= 1");
  if (d->top_k < 1 || d->top_k > d->num_experts)
    return fail(HMOE_ERR_INVALID_ARG, "top_k must be in [1, num_experts]");
  if (d->max_tokens < 1) return fail(HMOE_ERR_INVALID_ARG, "max_tokens must be >= 1");
  if (d->hidden < 1 || d->inter < 1) return fail(HMOE_ERR_INVALID_ARG, "hidden and inter must be >= 1");
  if (d->kept_format != HMOE_KEPT_NVFP4 && d->kept_format != HMOE_KEPT_MXFP4)
    return fail(HMOE_ERR_INVALID_ARG, "unknown kept_format");
  if (d->block_m != 0 && d->block_m != 16 && d->block_m != 32 && d->block_m != 64 && d->block_m != 128)
    return fail(HMOE_ERR_INVALID_ARG, "block_m must be 0, 16, 32, 64 or 128");
  if (d->decode_launch != HMOE_DECODE_STAGED && d->decode_launch != HMOE_DECODE_SINGLE_LAUNCH)
    return fail(HMOE_ERR_INVALID_ARG, "unknown decode_launch");
  if (d->act_format != HMOE_ACT_16BIT && d->act_format != HMOE_ACT_MXFP4)
    return fail(HMOE_ERR_INVALID_ARG, "unknown act_format");
  if (d->act_format == HMOE_ACT_MXFP4 && (!d->bit_map || d->kept_format != HMOE_KEPT_MXFP4))
    return fail(HMOE_ERR_INVALID_ARG, "W4A4 needs a bit map and an MXFP4 kept tier");
  if (d->act_format == HMOE_ACT_MXFP4 && d->decode_launch != HMOE_DECODE_STAGED)
    return fail(HMOE_ERR_INVALID_ARG, "the single-launch decode runs W4A16 only");
  if (d->num_experts > hmoe::kMaxExperts) return fail(HMOE_ERR_UNSUPPORTED, "num_experts > 1024");
  if (d->top_k > hmoe::kMaxTopK) return fail(HMOE_ERR_UNSUPPORTED, "top_k > 16");
  if (d->hidden % 128 || d->inter % 128)
    return fail(HMOE_ERR_UNSUPPORTED, "hidden and inter must be multiples of 128");
  if ((long)d->max_tokens * d->top_k > (1L << 24))
    return fail(HMOE_ERR_UNSUPPORTED, "max_tokens * top_k > 2^24");
  if (d->bit_map) {
    for (int e = 0; e < d->num_experts; ++e)
      if (d->bit_map[e] != 3 && d->bit_map[e] != 4)
        return fail(HMOE_ERR_INVALID_ARG, "bit_map[" + std::to_string(e) + "] = " +
                                              std::to_string(d->bit_map[e]) + ", expected 3 or 4");
  }
  hmoe_layer* h = new (std::nothrow) hmoe_layer;
  if (!h) return fail(HMOE_ERR_INVALID_ARG, "out of host memory");
  hmoe::Layer& L = h->L;
  L.E = d->num_experts;
  L.H = d->hidden;
  L.I = d->inter;
  L.k = d->top_k;
  L.max_tokens = d->max_tokens;
  L.has_map = d->bit_map != nullptr;
  L.kept_format = L.has_map ? d->kept_format : HMOE_KEPT_NVFP4;
  L.block_m = d->block_m ? d->block_m : auto_block_m(d->max_tokens, d->top_k, d->num_experts);
  L.act_format = d->act_format;
  L.bit_map.assign(L.E, 4);
  if (L.has_map) memcpy(L.bit_map.data(), d->bit_map, L.E);
  for (int e = 0; e < L.E; ++e) {
    if (L.bit_map[e] == 3) {
      ++L.E3;
      L.nf3_mask[e >> 5] |= 1u << (e & 31);
    } else {
      ++L.E4;
    }
  }
  L.max_distinct = std::min(hmoe::kDecodeMaxM * L.k, L.E);
  L.cap[0] = tier_capacity(L.max_tokens, L.k, L.E4, L.block_m);
  L.cap[1] = tier_capacity(L.max_tokens, L.k, L.E3, L.block_m);
  // the prefill GEMMs address activation rows with 32-bit element offsets
  if ((long)L.max_tokens * L.H >= (1L << 31) || (long)(L.cap[0] + L.cap[1]) * L.I >= (1L << 31)) {
    delete h;
    return fail(HMOE_ERR_UNSUPPORTED, "max_tokens too large for this layer's prefill buffers");
  }
  // the prefill GEMMs run (expert blocks of both tiers, rounded up to 64) x (column
  // tiles) blocks on a 1-D grid
  if (((long)(L.cap[0] + L.cap[1]) / L.block_m + 64) * std::max(L.I / 64, L.H / 128) >=
      (1L << 31)) {
    delete h;
    return fail(HMOE_ERR_UNSUPPORTED, "max_tokens * top_k / block_m too large for the prefill "
                                      "grid: use a larger block_m");
  }
  const bool tiled = hmoe::plan_gemv(L.H, &L.w13) && hmoe::plan_gemv(L.I, &L.w2) &&
                     L.I % ((64 / L.w13.lr) * L.w13.ri) == 0 && L.H % ((64 / L.w2.lr) * L.w2.ri) == 0;
  if (!tiled) {
    delete h;
    return fail(HMOE_ERR_UNSUPPORTED, "no decode GEMV tiling for H=" + std::to_string(d->hidden) +
                                          ", I=" + std::to_string(d->inter));
  }
  L.single_available = hmoe::fused_decode_available(L);
  if (d->decode_launch == HMOE_DECODE_SINGLE_LAUNCH && !L.single_available) {
    delete h;
    return fail(HMOE_ERR_UNSUPPORTED, "no single-launch decode for H=" + std::to_string(d->hidden) +
                                          ", I=" + std::to_string(d->inter));
  }
  L.fused_decode = d->decode_launch == HMOE_DECODE_SINGLE_LAUNCH;
  plan_scratch(L);
  *out = h;
  return HMOE_OK;
}

void moe_layer_destroy(hmoe_layer* layer) { delete layer; }

hmoe_status moe_layer_query(const hmoe_layer* layer, hmoe_layer_info* out) {
  if (hmoe_status st = check_layer(layer)) return st;
  if (!out) return fail(HMOE_ERR_INVALID_ARG, "out is NULL");
  const hmoe::Layer& L = layer->L;
  out->num_experts = L.E;
  out->hidden = L.H;
  out->inter = L.I;
  out->top_k = L.k;
  out->max_tokens = L.max_tokens;
  out->kept_format = L.kept_format;
  out->num_kept = L.E4;
  out->num_nf3 = L.E3;
  out->block_m = L.block_m;
  out->max_distinct = L.max_distinct;
  out->cap_kept = L.cap[0];
  out->cap_nf3 = L.cap[1];
  out->fused_decode = L.fused_decode ? 1 : 0;
  out->single_launch_available = L.single_available ? 1 : 0;
  out->act_format = L.act_format;
  return HMOE_OK;
}

hmoe_status moe_scratch_bytes(const hmoe_layer* layer, size_t* bytes) {
  if (hmoe_status st = check_layer(layer)) return st;
  if (!bytes) return fail(HMOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = layer->L.plan.total;
  return HMOE_OK;
}

hmoe_status moe_route(const float* logits, int32_t M, int32_t E, int32_t k, int32_t* topk_ids,
                      float* topk_w, hipStream_t stream) {
  if (M < 0) return fail(HMOE_ERR_INVALID_ARG, "M < 0");
  if (E < 1 || E > hmoe::kMaxExperts) return fail(HMOE_ERR_INVALID_ARG, "E must be in [1, 1024]");
  if (k < 1 || k > std::min(hmoe::kMaxTopK, (int)E))
    return fail(HMOE_ERR_INVALID_ARG, "k must be in [1, min(16, E)]");
  if (M == 0) return HMOE_OK;
  if (!logits || !topk_ids || !topk_w || !aligned(logits, 16) || !aligned(topk_ids, 16) ||
      !aligned(topk_w, 16))
    return fail(HMOE_ERR_ALIGN, "logits, topk_ids and topk_w must be non-NULL and 16-byte aligned");
  hipError_t err = hmoe::launch_route(logits, M, E, k, topk_ids, topk_w, stream);
  if (err != hipSuccess) return hip_fail(err, "route launch");
  return HMOE_OK;
}

hmoe_status moe_align(const hmoe_layer* layer, const int32_t* topk_ids, int32_t M, void* scratch,
                      size_t scratch_bytes, hipStream_t stream) {
  if (hmoe_status st = check_layer(layer)) return st;
  const hmoe::Layer& L = layer->L;
  if (M < 0) return fail(HMOE_ERR_INVALID_ARG, "M < 0");
  if (M > L.max_tokens) return fail(HMOE_ERR_CAPACITY, "M exceeds max_tokens");
  if (hmoe_status st = check_scratch(L, scratch, scratch_bytes)) return st;
  if (!topk_ids || !aligned(topk_ids, 16))
    return fail(HMOE_ERR_ALIGN, "topk_ids must be non-NULL and 16-byte aligned");
  hipError_t err = hmoe::launch_align(L, topk_ids, M, scratch, stream);
  if (err != hipSuccess) return hip_fail(err, "align launch");
  return HMOE_OK;
}

hmoe_status moe_align_view(const hmoe_layer* layer, void* scratch, int32_t tier,
                           hmoe_align_view* out) {
  if (hmoe_status st = check_layer(layer)) return st;
  if (!scratch || !out || (tier != 0 && tier != 1))
    return fail(HMOE_ERR_INVALID_ARG, "scratch/out NULL or tier not 0/1");
  const hmoe::Layer& L = layer->L;
  char* b = static_cast<char*>(scratch);
  out->sorted_slots = reinterpret_cast<int32_t*>(b + L.plan.a_slots[tier]);
  out->block_expert = reinterpret_cast<int32_t*>(b + L.plan.a_bexp[tier]);
  out->expert_off = reinterpret_cast<int32_t*>(b + L.plan.a_eoff[tier]);
  out->num_padded = reinterpret_cast<int32_t*>(b + L.plan.a_npad[tier]);
  out->capacity = L.cap[tier];
  out->num_experts_tier = tier == 0 ? L.E4 : L.E3;
  return HMOE_OK;
}

hmoe_status moe_decode_view(const hmoe_layer* layer, void* scratch, hmoe_decode_view* out) {
  if (hmoe_status st = check_layer(layer)) return st;
  if (!scratch || !out) return fail(HMOE_ERR_INVALID_ARG, "scratch/out NULL");
  const hmoe::Layer& L = layer->L;
  char* b = static_cast<char*>(scratch);
  out->counts = reinterpret_cast<int32_t*>(b + L.plan.d_counts);
  out->experts = reinterpret_cast<int32_t*>(b + L.plan.d_experts);
  out->num_slots = reinterpret_cast<int32_t*>(b + L.plan.d_nslots);
  out->slots = reinterpret_cast<int32_t*>(b + L.plan.d_slots);
  out->expert_tier = reinterpret_cast<int32_t*>(b + L.plan.expert_tier);
  out->passes = reinterpret_cast<int32_t*>(b + L.plan.d_pass);
  out->max_distinct = L.max_distinct;
  out->sync_timeouts = reinterpret_cast<int32_t*>(b + L.plan.d_sync) + 16;
  return HMOE_OK;
}

hmoe_status moe_topk_view(const hmoe_layer* layer, void* scratch, int32_t** topk_ids, float** topk_w) {
  if (hmoe_status st = check_layer(layer)) return st;
  if (!scratch || !topk_ids || !topk_w) return fail(HMOE_ERR_INVALID_ARG, "NULL argument");
  char* b = static_cast<char*>(scratch);
  *topk_ids = reinterpret_cast<int32_t*>(b + layer->L.plan.topk_ids);
  *topk_w = reinterpret_cast<float*>(b + layer->L.plan.topk_w);
  return HMOE_OK;
}

hmoe_status hybrid_moe_forward_stage(const hmoe_layer* layer, const hmoe_weights* weights,
                                     const uint16_t* x, const float* router_logits, int32_t M,
                                     uint16_t* y, void* scratch, size_t scratch_bytes,
                                     int32_t stage, hipStream_t stream) {
  if (hmoe_status st = check_layer(layer)) return st;
  const hmoe::Layer& L = layer->L;
  if (stage < HMOE_STAGE_ROUTE || stage > HMOE_STAGE_COMBINE)
    return fail(HMOE_ERR_INVALID_ARG, "unknown stage");
  if (M < 0) return fail(HMOE_ERR_INVALID_ARG, "M < 0");
  if (M > L.max_tokens) return fail(HMOE_ERR_CAPACITY, "M exceeds max_tokens");
  if (hmoe_status st = check_weights(L, weights)) return st;
  if (M == 0) return HMOE_OK;
  if (hmoe_status st = check_scratch(L, scratch, scratch_bytes)) return st;
  if (!x || !router_logits || !y || !aligned(x, 16) || !aligned(router_logits, 16) || !aligned(y, 16))
    return fail(HMOE_ERR_ALIGN, "x, router_logits and y must be non-NULL and 16-byte aligned");
  const bool w4a4 = L.act_format == HMOE_ACT_MXFP4;
  const bool decode = M <= hmoe::kDecodeMaxM && !w4a4;
  hipError_t err;
  if (stage == HMOE_STAGE_ROUTE) {
    if (decode) {
      err = hmoe::launch_route_group(L, router_logits, M, scratch, stream);
    } else {
      char* b = static_cast<char*>(scratch);
      int32_t* ids = reinterpret_cast<int32_t*>(b + L.plan.topk_ids);
      err = hmoe::launch_route(router_logits, M, L.E, L.k, ids,
                               reinterpret_cast<float*>(b + L.plan.topk_w), stream);
      if (err == hipSuccess) err = hmoe::launch_align(L, ids, M, scratch, stream);
      if (err == hipSuccess) err = hmoe::launch_prefill_x16(L, x, M, scratch, stream);
      if (err == hipSuccess && w4a4) err = hmoe::launch_w4a4(L, *weights, x, M, scratch, stage, stream);
    }
  } else if (decode) {
    err = hmoe::launch_decode(L, *weights, x, M, y, scratch, stage, stream);
  } else {
    // W4A4: the GEMM launches run both tiers (kept tier on MX matrix cores); the W13
    // stage then rounds the kept tier's h to MXFP4
    err = hmoe::launch_prefill(L, *weights, x, M, y, scratch, stage, stream, w4a4);
    if (err == hipSuccess && w4a4 && stage == HMOE_STAGE_W13)
      err = hmoe::launch_w4a4(L, *weights, x, M, scratch, stage, stream);
  }
  if (err != hipSuccess) return hip_fail(err, "kernel launch");
  return HMOE_OK;
}

hmoe_status hybrid_moe_forward(const hmoe_layer* layer, const hmoe_weights* weights,
                               const uint16_t* x, const float* router_logits, int32_t M,
                               uint16_t* y, void* scratch, size_t scratch_bytes,
                               hipStream_t stream) {
  if (layer && layer->L.fused_decode && M > 0 && M <= hmoe::kDecodeMaxM) {
    const hmoe::Layer& L = layer->L;
    if (M > L.max_tokens) return fail(HMOE_ERR_CAPACITY, "M exceeds max_tokens");
    if (hmoe_status st = check_weights(L, weights)) return st;
    if (hmoe_status st = check_scratch(L, scratch, scratch_bytes)) return st;
    if (!x || !router_logits || !y || !aligned(x, 16) || !aligned(router_logits, 16) ||
        !aligned(y, 16))
      return fail(HMOE_ERR_ALIGN, "x, router_logits and y must be non-NULL and 16-byte aligned");
    hipError_t err = hmoe::launch_decode_fused(L, *weights, x, router_logits, M, y, scratch, stream);
    if (err != hipSuccess) return hip_fail(err, "decode launch");
    return HMOE_OK;
  }
  for (int32_t stage = HMOE_STAGE_ROUTE; stage <= HMOE_STAGE_COMBINE; ++stage) {
    const hmoe_status st = hybrid_moe_forward_stage(layer, weights, x, router_logits, M, y, scratch,
                                                    scratch_bytes, stage, stream);
    if (st != HMOE_OK) return st;
  }
  return HMOE_OK;
}

hmoe_status hybrid_moe_forward_static(const hmoe_layer* layer, const hmoe_weights* weights,
                                      const uint16_t* x, const float* router_logits, int32_t M,
                                      uint16_t* y, hipStream_t stream) {
  if (hmoe_status st = check_layer(layer)) return st;
  const size_t need = layer->L.plan.total, have = hmoe::static_scratch_bytes();
  if (need > have)
    return fail(HMOE_ERR_SCRATCH, "the layer needs " + std::to_string(need) +
                                      " bytes of scratch, the static scratch holds " +
                                      std::to_string(have) + ": use hybrid_moe_forward");
  void* scratch = nullptr;
  hipError_t err = hmoe::static_scratch(&scratch);
  if (err != hipSuccess) return hip_fail(err, "static scratch address");
  // every layer on this GPU shares the array, so the single-launch decode's counters may
  // hold another call's data: they are cleared first (a fill kernel, capturable)
  const hmoe::Layer& L = layer->L;
  if (L.fused_decode && M > 0 && M <= hmoe::kDecodeMaxM && M <= L.max_tokens) {
    err = hmoe::launch_sync_clear(L, scratch, stream);
    if (err != hipSuccess) return hip_fail(err, "static scratch counter clear");
  }
  return hybrid_moe_forward(layer, weights, x, router_logits, M, y, scratch, have, stream);
}

hmoe_status moe_scratch_init(const hmoe_layer* layer, void* scratch, size_t scratch_bytes,
                             hipStream_t stream) {
  if (hmoe_status st = check_layer(layer)) return st;
  if (hmoe_status st = check_scratch(layer->L, scratch, scratch_bytes)) return st;
  hipError_t err = hmoe::launch_sync_clear(layer->L, scratch, stream);
  if (err != hipSuccess) return hip_fail(err, "scratch init launch");
  return HMOE_OK;
}

hmoe_status moe_dequant(const hmoe_layer* layer, const hmoe_weights* weights, int32_t expert,
                        int32_t tensor, float* out_f32, uint16_t* out_bf16, hipStream_t stream) {
  if (hmoe_status st = check_layer(layer)) return st;
  const hmoe::Layer& L = layer->L;
  if (expert < 0 || expert >= L.E) return fail(HMOE_ERR_INVALID_ARG, "expert out of range");
  if (tensor != HMOE_TENSOR_W13 && tensor != HMOE_TENSOR_W2)
    return fail(HMOE_ERR_INVALID_ARG, "tensor must be HMOE_TENSOR_W13 or HMOE_TENSOR_W2");
  if (!out_f32 && !out_bf16) return fail(HMOE_ERR_INVALID_ARG, "both outputs are NULL");
  if ((out_f32 && !aligned(out_f32, 16)) || (out_bf16 && !aligned(out_bf16, 16)))
    return fail(HMOE_ERR_ALIGN, "outputs must be 16-byte aligned");
  if (hmoe_status st = check_weights(L, weights)) return st;
  hipError_t err = hmoe::launch_dequant(L, *weights, expert, tensor, out_f32, out_bf16, stream);
  if (err != hipSuccess) return hip_fail(err, "dequant launch");
  return HMOE_OK;
}

hmoe_status moe_repack(const hmoe_layer* layer, const hmoe_expert_src* experts,
                       const hmoe_weights* dst, hipStream_t stream) {
  if (hmoe_status st = check_layer(layer)) return st;
  const hmoe::Layer& L = layer->L;
  if (!experts) return fail(HMOE_ERR_INVALID_ARG, "experts is NULL");
  if (hmoe_status st = check_weights(L, dst)) return st;
  const bool nv = L.kept_format == HMOE_KEPT_NVFP4;
  struct Tensor {
    long rows;
    int K;
  };
  const Tensor ts[2] = {{2L * L.I, L.H}, {(long)L.H, L.I}};
  // validate every expert before the first copy
  for (int e = 0; e < L.E; ++e) {
    const hmoe_expert_src& s = experts[e];
    const bool nf3 = (L.nf3_mask[e >> 5] >> (e & 31)) & 1u;
    if (!s.w13_q || !s.w13_s || !s.w2_q || !s.w2_s)
      return fail(HMOE_ERR_INVALID_ARG, "expert " + std::to_string(e) + ": a code or scale pointer is NULL");
    if (nf3 && (!s.w13_hi || !s.w2_hi))
      return fail(HMOE_ERR_INVALID_ARG, "NF3 expert " + std::to_string(e) + ": a high code plane is NULL");
    if (nf3 && (!aligned(s.w13_q, 4) || !aligned(s.w13_hi, 4) || !aligned(s.w2_q, 4) ||
                !aligned(s.w2_hi, 4)))
      return fail(HMOE_ERR_ALIGN, "NF3 expert " + std::to_string(e) + ": code planes need 4-byte alignment");
    if (!nf3 && nv && (!s.w13_g || !s.w2_g))
      return fail(HMOE_ERR_INVALID_ARG, "NVFP4 expert " + std::to_string(e) + ": a per-tensor scale is NULL");
  }
  uint8_t* kq[2] = {const_cast<uint8_t*>(dst->kept_w13_q), const_cast<uint8_t*>(dst->kept_w2_q)};
  uint8_t* ks[2] = {const_cast<uint8_t*>(dst->kept_w13_s), const_cast<uint8_t*>(dst->kept_w2_s)};
  float* kg[2] = {const_cast<float*>(dst->kept_w13_g), const_cast<float*>(dst->kept_w2_g)};
  uint8_t* nq[2] = {const_cast<uint8_t*>(dst->nf3_w13_q), const_cast<uint8_t*>(dst->nf3_w2_q)};
  uint16_t* ns[2] = {const_cast<uint16_t*>(dst->nf3_w13_s), const_cast<uint16_t*>(dst->nf3_w2_s)};
  int below[2] = {0, 0};  // experts of each tier so far: the tier-local index
  hmoe::RepackBatch batch{};
  auto add = [&](const void* src, const void* hi, void* out, long n, int kind) -> hipError_t {
    batch.job[batch.njobs++] = {src, hi, out, n, kind, 0};
    if (batch.njobs < hmoe::kRepackJobs) return hipSuccess;
    hipError_t err = hmoe::launch_repack(batch, stream);
    batch.njobs = 0;
    return err;
  };
  for (int e = 0; e < L.E; ++e) {
    const hmoe_expert_src& s = experts[e];
    const int tier = ((L.nf3_mask[e >> 5] >> (e & 31)) & 1u) ? 1 : 0;
    const long loc = below[tier]++;
    const uint8_t* sq[2] = {s.w13_q, s.w2_q};
    const uint8_t* shi[2] = {s.w13_hi, s.w2_hi};
    const void* ss[2] = {s.w13_s, s.w2_s};
    const float* sg[2] = {s.w13_g, s.w2_g};
    for (int t = 0; t < 2; ++t) {
      const long rows = ts[t].rows;
      const int K = ts[t].K;
      hipError_t err = hipSuccess;
      if (tier == 0) {
        const long qb = rows * (K / 2), sb = rows * (K / (nv ? 16 : 32));
        err = add(sq[t], nullptr, kq[t] + loc * qb, qb, hmoe::kRepackCopy);
        if (err == hipSuccess) err = add(ss[t], nullptr, ks[t] + loc * sb, sb, hmoe::kRepackCopy);
        if (err == hipSuccess && nv && kg[t])
          err = add(sg[t], nullptr, kg[t] + loc, (long)sizeof(float), hmoe::kRepackCopy);
      } else {
        const long qb = rows * (3L * K / 8), sn = rows * (K / 64);
        err = add(sq[t], shi[t], nq[t] + loc * qb, rows * (K / 32), hmoe::kRepackNf3);
        if (err == hipSuccess) err = add(ss[t], nullptr, ns[t] + loc * sn, sn * 2, hmoe::kRepackCopy);
      }
      if (err != hipSuccess) return hip_fail(err, "repack");
    }
  }
  if (batch.njobs > 0) {
    hipError_t err = hmoe::launch_repack(batch, stream);
    if (err != hipSuccess) return hip_fail(err, "repack");
  }
  return HMOE_OK;
}

hmoe_status moe_quantize_mxfp4(const float* in, int32_t rows, int32_t K, uint8_t* codes,
                               uint8_t* scales, hipStream_t stream) {
  if (rows < 0 || K <= 0 || K % 32) return fail(HMOE_ERR_INVALID_ARG, "rows >= 0 and K a positive multiple of 32");
  if (rows == 0) return HMOE_OK;
  if (!in || !codes || !scales || !aligned(in, 16) || !aligned(codes, 16))
    return fail(HMOE_ERR_ALIGN, "in, codes and scales must be non-NULL, in and codes 16-byte aligned");
  hipError_t err = hmoe::launch_mx_quant(in, false, rows, K, nullptr, codes, scales, stream);
  if (err != hipSuccess) return hip_fail(err, "quantise launch");
  return HMOE_OK;
}

hmoe_status moe_permute_scratch_bytes(int32_t M, int32_t k, int32_t E, size_t* bytes) {
  if (hmoe_status st = check_permute_shape(M, k)) return st;
  if (hmoe_status st = check_experts(E)) return st;
  if (!bytes) return fail(HMOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = permute_scratch(M, k, E);
  return HMOE_OK;
}

hmoe_status moe_permute(const void* x, int64_t x_stride, const int32_t* topk_ids, int32_t M,
                        int32_t k, int32_t E, int32_t H, int32_t dtype, void* rows,
                        int64_t rows_stride, int32_t* sorted_slots, int32_t* slot_row,
                        int32_t* expert_off, void* scratch, size_t scratch_bytes,
                        hipStream_t stream) {
  if (hmoe_status st = check_permute_shape(M, k)) return st;
  if (hmoe_status st = check_experts(E)) return st;
  if (hmoe_status st = check_rows(M, H, dtype)) return st;
  const int es = element_size(dtype);
  if (hmoe_status st = check_arrays("expert_off", {expert_off})) return st;
  if (M > 0) {
    if (hmoe_status st = check_matrix("x", x, x_stride, H, es)) return st;
    if (hmoe_status st = check_matrix("rows", rows, rows_stride, H, es)) return st;
    if (hmoe_status st = check_arrays("topk_ids, sorted_slots and slot_row",
                                      {topk_ids, sorted_slots, slot_row}))
      return st;
    if (hmoe_status st = check_op_scratch(scratch, scratch_bytes, permute_scratch(M, k, E))) return st;
    if (hmoe_status st = check_apart({x, topk_ids}, {{"rows", rows}, {"sorted_slots", sorted_slots},
                                                     {"slot_row", slot_row}, {"expert_off", expert_off}}))
      return st;
  }
  const hmoe::PermuteRows p{x, x_stride, rows, rows_stride, slot_row, M, k, H, dtype, es};
  hipError_t err = hmoe::launch_permute(p, topk_ids, E, sorted_slots, expert_off,
                                        static_cast<int32_t*>(scratch), stream);
  if (err != hipSuccess) return hip_fail(err, "permute launch");
  return HMOE_OK;
}

hmoe_status moe_permute_backward(const void* drows, int64_t drows_stride, const int32_t* slot_row,
                                 int32_t M, int32_t k, int32_t H, int32_t dtype, void* dx,
                                 int64_t dx_stride, hipStream_t stream) {
  if (hmoe_status st = check_permute_shape(M, k)) return st;
  if (hmoe_status st = check_rows(M, H, dtype)) return st;
  if (M == 0) return HMOE_OK;
  const int es = element_size(dtype);
  if (hmoe_status st = check_matrix("drows", drows, drows_stride, H, es)) return st;
  if (hmoe_status st = check_matrix("dx", dx, dx_stride, H, es)) return st;
  if (hmoe_status st = check_arrays("slot_row", {slot_row})) return st;
  if (hmoe_status st = check_apart({drows, slot_row}, {{"dx", dx}})) return st;
  const hmoe::PermuteRows p{drows, drows_stride, dx, dx_stride, slot_row, M, k, H, dtype, es};
  hipError_t err = hmoe::launch_combine(p, nullptr, stream);
  if (err != hipSuccess) return hip_fail(err, "permute backward launch");
  return HMOE_OK;
}

hmoe_status moe_unpermute(const void* rows, int64_t rows_stride, const int32_t* slot_row,
                          const float* topk_w, int32_t M, int32_t k, int32_t H, int32_t dtype,
                          void* y, int64_t y_stride, hipStream_t stream) {
  if (hmoe_status st = check_permute_shape(M, k)) return st;
  if (hmoe_status st = check_rows(M, H, dtype)) return st;
  if (M == 0) return HMOE_OK;
  const int es = element_size(dtype);
  if (hmoe_status st = check_matrix("rows", rows, rows_stride, H, es)) return st;
  if (hmoe_status st = check_matrix("y", y, y_stride, H, es)) return st;
  if (hmoe_status st = check_arrays("slot_row and topk_w", {slot_row, topk_w})) return st;
  if (hmoe_status st = check_apart({rows, slot_row, topk_w}, {{"y", y}})) return st;
  const hmoe::PermuteRows p{rows, rows_stride, y, y_stride, slot_row, M, k, H, dtype, es};
  hipError_t err = hmoe::launch_combine(p, topk_w, stream);
  if (err != hipSuccess) return hip_fail(err, "unpermute launch");
  return HMOE_OK;
}

hmoe_status moe_unpermute_backward(const void* dy, int64_t dy_stride, const void* rows,
                                   int64_t rows_stride, const int32_t* slot_row,
                                   const float* topk_w, int32_t M, int32_t k, int32_t H,
                                   int32_t dtype, void* drows, int64_t drows_stride, float* dw,
                                   hipStream_t stream) {
  if (hmoe_status st = check_permute_shape(M, k)) return st;
  if (hmoe_status st = check_rows(M, H, dtype)) return st;
  if (M == 0) return HMOE_OK;
  const int es = element_size(dtype);
  if (hmoe_status st = check_matrix("dy", dy, dy_stride, H, es)) return st;
  if (hmoe_status st = check_matrix("rows", rows, rows_stride, H, es)) return st;
  if (hmoe_status st = check_matrix("drows", drows, drows_stride, H, es)) return st;
  if (hmoe_status st = check_arrays("slot_row, topk_w and dw", {slot_row, topk_w, dw})) return st;
  if (hmoe_status st = check_apart({dy, rows, slot_row, topk_w}, {{"drows", drows}, {"dw", dw}})) return st;
  const hmoe::PermuteRows p{dy, dy_stride, drows, drows_stride, slot_row, M, k, H, dtype, es};
  hipError_t err = hmoe::launch_unpermute_bwd(p, rows, rows_stride, topk_w, dw, stream);
  if (err != hipSuccess) return hip_fail(err, "unpermute backward launch");
  return HMOE_OK;
}

hmoe_status moe_route_backward(const int32_t* topk_ids, const float* topk_w, const float* dw,
                               int32_t M, int32_t E, int32_t k, float* dlogits,
                               hipStream_t stream) {
  if (M < 0) return fail(HMOE_ERR_INVALID_ARG, "M < 0");
  if (hmoe_status st = check_experts(E)) return st;
  if (k < 1 || k > std::min(hmoe::kMaxTopK, (int)E))
    return fail(HMOE_ERR_INVALID_ARG, "k must be in [1, min(16, E)]");
  if (M == 0) return HMOE_OK;
  if (hmoe_status st = check_arrays("topk_ids, topk_w, dw and dlogits", {topk_ids, topk_w, dw, dlogits}))
    return st;
  if (hmoe_status st = check_apart({topk_ids, topk_w, dw}, {{"dlogits", dlogits}})) return st;
  hipError_t err = hmoe::launch_route_backward(topk_ids, topk_w, dw, M, E, k, dlogits, stream);
  if (err != hipSuccess) return hip_fail(err, "route backward launch");
  return HMOE_OK;
}

hmoe_status moe_lora_scratch_bytes(int32_t M, int32_t G, int32_t K, int32_t N, int32_t rank,
                                   size_t* forward_bytes, size_t* backward_bytes) {
  if (hmoe_status st = check_lora(M, G, K, N, rank)) return st;
  if (!forward_bytes || !backward_bytes) return fail(HMOE_ERR_INVALID_ARG, "bytes is NULL");
  hmoe::lora_scratch(M, G, K, N, rank, forward_bytes, backward_bytes);
  return HMOE_OK;
}

hmoe_status moe_lora(const uint16_t* x, int64_t x_stride, const int32_t* ids, const uint16_t* A,
                     const uint16_t* B, const float* scale, int32_t M, int32_t G, int32_t K,
                     int32_t N, int32_t rank, const uint16_t* base, int64_t base_stride,
                     uint16_t* y, int64_t y_stride, float* z, void* scratch, size_t scratch_bytes,
                     hipStream_t stream) {
  if (hmoe_status st = check_lora(M, G, K, N, rank)) return st;
  if (M == 0) return HMOE_OK;
  if (hmoe_status st = check_matrix("x", x, x_stride, K, 2)) return st;
  if (hmoe_status st = check_matrix("y", y, y_stride, N, 2)) return st;
  if (hmoe_status st = check_base("base", base, base_stride, y, y_stride, N)) return st;
  if (hmoe_status st = check_arrays("ids, A, B and scale", {ids, A, B, scale})) return st;
  if (!aligned(z, 16)) return fail(HMOE_ERR_ALIGN, "z must be 16-byte aligned");
  size_t need;
  hmoe::lora_scratch(M, G, K, N, rank, &need, nullptr);
  if (hmoe_status st = check_op_scratch(scratch, scratch_bytes, need)) return st;
  if (hmoe_status st = check_apart({x, ids, A, B, scale}, {{"y", y}, {"z", z, base}})) return st;
  const hmoe::Lora p{x, x_stride, ids, A, B, scale, M, G, K, N, rank, base, base_stride, y, y_stride, z};
  hipError_t err = hmoe::launch_lora(p, scratch, stream);
  if (err != hipSuccess) return hip_fail(err, "adapter launch");
  return HMOE_OK;
}

hmoe_status moe_lora_backward(const uint16_t* dy, int64_t dy_stride, const uint16_t* x,
                              int64_t x_stride, const float* z, const int32_t* ids,
                              const uint16_t* A, const uint16_t* B, const float* scale, int32_t M,
                              int32_t G, int32_t K, int32_t N, int32_t rank,
                              const uint16_t* dbase, int64_t dbase_stride, uint16_t* dx,
                              int64_t dx_stride, float* dA, float* dB, void* scratch,
                              size_t scratch_bytes, hipStream_t stream) {
  if (hmoe_status st = check_lora(M, G, K, N, rank)) return st;
  if (hmoe_status st = check_arrays("A, B, scale, dA and dB", {A, B, scale, dA, dB})) return st;
  if (M > 0) {
    if (hmoe_status st = check_matrix("dy", dy, dy_stride, N, 2)) return st;
    if (hmoe_status st = check_matrix("x", x, x_stride, K, 2)) return st;
    if (hmoe_status st = check_matrix("dx", dx, dx_stride, K, 2)) return st;
    if (hmoe_status st = check_base("dbase", dbase, dbase_stride, dx, dx_stride, K)) return st;
    if (hmoe_status st = check_arrays("ids and z", {ids, z})) return st;
  }
  size_t need;
  hmoe::lora_scratch(M, G, K, N, rank, nullptr, &need);
  if (hmoe_status st = check_op_scratch(scratch, scratch_bytes, need)) return st;
  if (hmoe_status st = check_apart({dy, x, z, ids, A, B, scale}, {{"dx", dx}, {"dA", dA, dbase}, {"dB", dB, dbase}}))
    return st;
  const hmoe::LoraGrad p{dy, dy_stride, x, x_stride, z, ids, A, B, scale, M, G, K, N, rank,
                         dbase, dbase_stride, dx, dx_stride, dA, dB};
  hipError_t err = hmoe::launch_lora_backward(p, scratch, stream);
  if (err != hipSuccess) return hip_fail(err, "adapter backward launch");
  return HMOE_OK;
}

hmoe_status moe_linear_scratch_bytes(int32_t M, int32_t K, int32_t N, size_t* forward_bytes,
                                     size_t* backward_bytes) {
  if (hmoe_status st = check_linear_shape(M, K, N)) return st;
  if (!forward_bytes || !backward_bytes) return fail(HMOE_ERR_INVALID_ARG, "bytes is NULL");
  hmoe::linear_scratch(M, K, N, forward_bytes, backward_bytes);
  return HMOE_OK;
}

hmoe_status moe_linear(const void* x, int64_t x_stride, const hmoe_packed* w, int32_t M, int32_t K,
                       int32_t N, int32_t dtype, const void* base, int64_t base_stride, void* y,
                       int64_t y_stride, void* scratch, size_t scratch_bytes, hipStream_t stream) {
  return run_linear("x", x, x_stride, w, M, K, N, dtype, "base", base, base_stride, "y", y, y_stride,
                    scratch, scratch_bytes, false, stream);
}

hmoe_status moe_linear_backward(const void* dy, int64_t dy_stride, const hmoe_packed* w, int32_t M,
                                int32_t K, int32_t N, int32_t dtype, const void* dbase,
                                int64_t dbase_stride, void* dx, int64_t dx_stride, void* scratch,
                                size_t scratch_bytes, hipStream_t stream) {
  return run_linear("dy", dy, dy_stride, w, M, K, N, dtype, "dbase", dbase, dbase_stride, "dx", dx,
                    dx_stride, scratch, scratch_bytes, true, stream);
}

hmoe_status moe_tokens_scratch_bytes(int32_t M, int32_t E, int32_t H, int32_t I, int32_t k,
                                     int32_t shared_inter, size_t* bytes) {
  if (hmoe_status st = check_tokens_shape(M, E, H, I, k, shared_inter)) return st;
  if (!bytes) return fail(HMOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = hmoe::tokens_scratch(M, E, H, I, k, shared_inter);
  return HMOE_OK;
}

hmoe_status moe_tokens(const hmoe_tokens* layer, const void* x, int64_t x_stride, int32_t M,
                       const void* base, int64_t base_stride, void* y, int64_t y_stride,
                       int32_t* topk_ids, float* topk_w, void* scratch, size_t scratch_bytes,
                       hipStream_t stream) {
  if (!layer) return fail(HMOE_ERR_INVALID_ARG, "layer is NULL");
  const hmoe_tokens& t = *layer;
  const int H = t.hidden, I = t.inter, S = t.shared_inter;
  if (hmoe_status st = check_tokens_shape(M, t.num_experts, H, I, t.top_k, S)) return st;
  if (hmoe_status st = check_half(t.dtype)) return st;
  if (hmoe_status st = check_packed("w13", t.w13, H)) return st;
  if (hmoe_status st = check_packed("w2", t.w2, I)) return st;
  if (S > 0) {
    if (hmoe_status st = check_packed("shared_w13", t.shared_w13, H)) return st;
    if (hmoe_status st = check_packed("shared_w2", t.shared_w2, S)) return st;
  }
  const bool int4 = t.w13.format == HMOE_WEIGHT_INT4;
  auto same = [&](const hmoe_packed& w) { return w.format == t.w13.format && (!int4 || w.group == t.w13.group); };
  if (!same(t.w2) || (S > 0 && (!same(t.shared_w13) || !same(t.shared_w2))))
    return fail(HMOE_ERR_INVALID_ARG, "the layer's matrices must have one format and group");
  if (hmoe_status st = check_arrays("router", {t.router})) return st;
  if (S > 0 && !aligned(t.shared_gate, 16)) return fail(HMOE_ERR_ALIGN, "shared_gate must be 16-byte aligned");
  if (M == 0) return HMOE_OK;
  if (hmoe_status st = check_matrix("x", x, x_stride, H, 2)) return st;
  if (hmoe_status st = check_matrix("y", y, y_stride, H, 2)) return st;
  if (hmoe_status st = check_addend("base", base, base_stride, y, y_stride, H)) return st;
  if (!aligned(topk_ids, 16) || !aligned(topk_w, 16))
    return fail(HMOE_ERR_ALIGN, "topk_ids and topk_w must be 16-byte aligned");
  if (hmoe_status st = check_op_scratch(scratch, scratch_bytes, hmoe::tokens_scratch(M, t.num_experts, H, I, t.top_k, S)))
    return st;
  const hmoe::Packed none{}, w13 = packed_of(t.w13), w2 = packed_of(t.w2);
  const hmoe::Packed s13 = S > 0 ? packed_of(t.shared_w13) : none, s2 = S > 0 ? packed_of(t.shared_w2) : none;
  const void* gate = S > 0 ? t.shared_gate : nullptr;
  if (hmoe_status st = check_apart({x, t.router, gate, w13.q, w13.s, w13.z, w13.g, w2.q, w2.s, w2.z, w2.g,
                                    s13.q, s13.s, s13.z, s13.g, s2.q, s2.s, s2.z, s2.g},
                                   {{"y", y}, {"topk_ids", topk_ids, base}, {"topk_w", topk_w, base}}))
    return st;
  const hmoe::Tokens p{t.dtype, static_cast<const uint16_t*>(x), x_stride, static_cast<const uint16_t*>(t.router),
                       static_cast<const uint16_t*>(gate), w13, w2, s13, s2, M, t.num_experts, H, I, t.top_k, S,
                       static_cast<const uint16_t*>(base), base_stride, static_cast<uint16_t*>(y), y_stride, topk_ids, topk_w};
  hipError_t err = hmoe::launch_tokens(p, scratch, stream);
  if (err != hipSuccess) return hip_fail(err, "tokens launch");
  return HMOE_OK;
}

const char* moe_status_string(hmoe_status s) {
  switch (s) {
    case HMOE_OK: return "HMOE_OK";
    case HMOE_ERR_INVALID_ARG: return "HMOE_ERR_INVALID_ARG";
    case HMOE_ERR_UNSUPPORTED: return "HMOE_ERR_UNSUPPORTED";
    case HMOE_ERR_ALIGN: return "HMOE_ERR_ALIGN";
    case HMOE_ERR_CAPACITY: return "HMOE_ERR_CAPACITY";
    case HMOE_ERR_SCRATCH: return "HMOE_ERR_SCRATCH";
    case HMOE_ERR_HIP: return "HMOE_ERR_HIP";
  }
  return "HMOE_ERR_UNKNOWN";
}

const char* moe_last_error(void) { return g_last_error.c_str(); }

}  // extern "C"
