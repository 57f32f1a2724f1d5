// Internal declarations of libhmoe: the layer object, the scratch plan and the
// kernel launchers each kernel file provides. Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <string>
#include <vector>

#include "hmoe.h"

namespace hmoe {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 16;
constexpr int kDecodeMaxM = HMOE_DECODE_MAX_M;
// decode pass record (int4), one per (token, top-k) slot, in slot order: slot, tier
// code, token, expert id (written by the routing stage, read by the GEMVs)
constexpr int kPassRec = 4;

// Byte offsets of every scratch region (each 256-byte aligned).
struct ScratchPlan {
  size_t topk_ids = 0, topk_w = 0, expert_tier = 0;
  size_t d_counts = 0, d_experts = 0, d_nslots = 0, d_slots = 0, d_pass = 0;
  size_t h_dec = 0, o_dec = 0;
  size_t d_sync = 0;                       // single-launch decode counters (zero between calls)
  size_t a_counts = 0;                     // int32 [E] slot counts per expert
  size_t a_slots[2] = {0, 0}, a_bexp[2] = {0, 0}, a_eoff[2] = {0, 0}, a_npad[2] = {0, 0};
  size_t h_pre = 0, o_pre = 0, x16_pre = 0, xe_pre = 0;
  size_t pf_fac = 0;                       // fp32 [cap0 + cap1]: W2 output factor per h row
  size_t mx_xq = 0, mx_xs = 0, mx_h32 = 0, mx_hq = 0, mx_hs = 0;   // W4A4 kept tier
  size_t total = 0;
};

// GEMV tiling of one weight tensor on the decode path: lanes per row (LR), units of
// 32 K-elements per lane (KU), rows (or row pairs) per lane per chunk (RI).
struct GemvTiling {
  int lr = 0, ku = 0, ri = 0;
};

struct Layer {
  int E = 0, H = 0, I = 0, k = 0, max_tokens = 0;
  int kept_format = HMOE_KEPT_NVFP4;  // effective
  int act_format = HMOE_ACT_16BIT;    // HMOE_ACT_MXFP4: the kept tier runs W4A4
  int block_m = 32;
  bool has_map = false;
  std::vector<uint8_t> bit_map;
  int E4 = 0, E3 = 0;
  uint32_t nf3_mask[kMaxExperts / 32] = {};  // bit e set: expert e is in the NF3 tier
  int max_distinct = 0;                        // min(8k, E)
  int cap[2] = {0, 0};                         // align capacity per tier
  GemvTiling w13, w2;
  bool fused_decode = false;                   // the forward runs decode as one launch
  bool single_available = false;               // a single-launch decode exists for H, I
  ScratchPlan plan;
};

// Expert-tier bit mask passed by value to the kernels that need the tier map.
struct TierMask {
  uint32_t w[kMaxExperts / 32];
};

// ---- launchers (each returns hipGetLastError() of its launch) -------------------

// route.hip
hipError_t launch_route(const float* logits, int M, int E, int k, int32_t* ids, float* w,
                        hipStream_t s);
hipError_t launch_route_group(const Layer& L, const float* logits, int M, void* scratch,
                              hipStream_t s);

// align.hip
hipError_t launch_align(const Layer& L, const int32_t* ids, int M, void* scratch, hipStream_t s);

// decode.hip: one stage (HMOE_STAGE_W13 / _W2 / _COMBINE) of the decode path
hipError_t launch_decode(const Layer& L, const hmoe_weights& W, const uint16_t* x, int M,
                         uint16_t* y, void* scratch, int stage, hipStream_t s);

// decode.hip: the whole decode forward in one launch (only for the layer shapes
// fused_decode_available accepts), the size of its sync region, and its zero fill
bool fused_decode_available(const Layer& L);
size_t fused_sync_words(int k, int H);
hipError_t launch_decode_fused(const Layer& L, const hmoe_weights& W, const uint16_t* x,
                               const float* logits, int M, uint16_t* y, void* scratch,
                               hipStream_t s);
hipError_t launch_sync_clear(const Layer& L, void* scratch, hipStream_t s);

// prefill.hip: one stage (HMOE_STAGE_W13 / _W2 / _COMBINE) of the prefill path;
// nf3_only (W4A4 layers): the W4A16 GEMM covers the NF3 tier and the same launch runs
// the kept tier on MX matrix cores
hipError_t launch_prefill(const Layer& L, const hmoe_weights& W, const uint16_t* x, int M,
                          uint16_t* y, void* scratch, int stage, hipStream_t s,
                          bool nf3_only = false);

// w4a4.hip: the W4A4 kept tier's quantisation around the GEMM launches (ROUTE: x to
// MXFP4; W13: h to MXFP4), and the MXFP4 activation quantiser (rows x K, bf16 or fp32
// input; rows at or past *nrows skipped when nrows is given)
hipError_t launch_w4a4(const Layer& L, const hmoe_weights& W, const uint16_t* x, int M,
                       void* scratch, int stage, hipStream_t s);
hipError_t launch_mx_quant(const void* in, bool bf16, int rows, int K, const int32_t* nrows,
                           uint8_t* codes, uint8_t* scales, hipStream_t s);

// prefill.hip: tokens to fp16 with a per-token power-of-two scale (prefill input)
hipError_t launch_prefill_x16(const Layer& L, const uint16_t* x, int M, void* scratch,
                              hipStream_t s);

// route.hip: gradient of the top-k weights with respect to the logits
hipError_t launch_route_backward(const int32_t* ids, const float* w, const float* dw, int M, int E,
                                 int k, float* dlogits, hipStream_t s);

// permute.hip: stable counting sort of n ids over G groups. groups = G drops ids outside
// [0, G); groups = G + 1 makes them the last group. counts holds sort_count_words words;
// slot_row may be null. tile_rows > 0 also cuts every group's run into tiles of that many
// rows, described by tile [max_tiles] (group -1 for none, index: number of the tile in sorted
// order), and writes each group's first tile to tile_first [groups + 1].
constexpr int kMaxGroups = HMOE_MAX_GROUPS;
struct SortTile {
  int32_t group, start, rows, index;
};
// A transposition [G, N, r] -> [G, r, N] of 16-bit values (N and r multiples of 8) that blocks
// of the sort's last launch do beside it (in null: none).
struct SortTranspose {
  const uint16_t* in;
  uint16_t* out;
  int N, r, G;
};
struct GroupSort {
  const int32_t* ids;
  int n, G, groups;
  int32_t* counts;
  int32_t* sorted;
  int32_t* slot_row;
  int32_t* off;
  int tile_rows, max_tiles;
  SortTile* tile;
  int32_t* tile_first;
  SortTranspose turn;
};
size_t sort_count_words(int n, int groups);
hipError_t launch_sort(const GroupSort& g, hipStream_t s);

// permute.hip: the row movements between token order and expert order (strides in
// elements); up to kPermuteSmall ids one launch ranks and copies. Every block compares its
// token's slots with all ids there: on MI355X, 8 slots a token, 2048 ids take 7.3 us (rows of
// 2048 bf16) and 10.8 (6144) in one launch, 9.3 and 12.4 with a sort before the copy; 4096 ids
// 12.2 and 26.4 against 12.9 and 18.6.
constexpr int kPermuteSmall = 2048;
struct PermuteRows {
  const void* src;
  long src_stride;
  void* dst;
  long dst_stride;
  const int32_t* slot_row;
  int M, k, H;
  int dtype, esize;
};
// whether M rows of `bytes` bytes fit one launch (2^24 blocks of 256 threads)
bool row_grid_fits(long M, long bytes);
hipError_t launch_permute(const PermuteRows& p, const int32_t* ids, int E, int32_t* sorted,
                          int32_t* off, int32_t* counts, hipStream_t s);
hipError_t launch_combine(const PermuteRows& p, const float* w, hipStream_t s);
hipError_t launch_unpermute_bwd(const PermuteRows& p, const void* rows, long rows_stride,
                                const float* w, float* dw, hipStream_t s);

// lora.hip: adapters beside a shared projection
constexpr int kMaxLoraRank = 128;
struct Lora {
  const uint16_t* x;        // [M, K], stride xs
  long xs;
  const int32_t* ids;       // [M]
  const uint16_t* A;        // [G, r, K]
  const uint16_t* B;        // [G, N, r]
  const float* scale;       // [G]
  int M, G, K, N, r;
  const uint16_t* base;     // [M, N], stride bs; may be null
  long bs;
  uint16_t* y;              // [M, N], stride ys
  long ys;
  float* z;                 // [M, r]; may be null
};
struct LoraGrad {
  const uint16_t* dy;       // [M, N]
  long dys;
  const uint16_t* x;        // [M, K]
  long xs;
  const float* z;           // [M, r]
  const int32_t* ids;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  int M, G, K, N, r;
  const uint16_t* dbase;    // [M, K]; may be null
  long dbs;
  uint16_t* dx;             // [M, K]
  long dxs;
  float* dA;                // [G, r, K]
  float* dB;                // [G, N, r]
};
void lora_scratch(int M, int G, int K, int N, int r, size_t* forward, size_t* backward);
hipError_t launch_lora(const Lora& p, void* scratch, hipStream_t s);
hipError_t launch_lora_backward(const LoraGrad& p, void* scratch, hipStream_t s);

// packed.h: a matrix of 4-bit weights with group scales, or several behind one another
struct Packed {
  const uint8_t* q;
  const uint8_t* s;
  const uint8_t* z;   // INT4 zero points; null: 8
  const float* g;     // NVFP4: a scale per matrix
  int format, group;
};

// linear.hip: products with a packed matrix W [N, K], and the gradient of their rows
struct Linear {
  Packed w;
  int dtype;
  const uint16_t* x;     // [M, K]; backward: dy [M, N]
  long xs;
  int M, K, N;
  const uint16_t* base;  // [M, N]; backward: dbase [M, K]; may be null
  long bs;
  uint16_t* y;           // [M, N]; backward: dx [M, K]
  long ys;
};
void linear_scratch(int M, int K, int N, size_t* forward, size_t* backward);
hipError_t launch_linear(const Linear& p, bool back, void* scratch, hipStream_t s);

// tokens.hip: a whole layer for a few tokens
struct Tokens {
  int dtype;
  const uint16_t* x;      // [M, H]
  long xs;
  const uint16_t* router; // [E, H]
  const uint16_t* gate;   // [H]; null: the shared expert's weight is 1
  Packed w13, w2;         // [E][2 I, H] and [E][H, I]
  Packed s13, s2;         // [2 S, H] and [H, S]
  int M, E, H, I, k, S;
  const uint16_t* base;   // [M, H]; may be null
  long bs;
  uint16_t* y;
  long ys;
  int32_t* topk_ids;      // [M, k]; may be null
  float* topk_w;
};
size_t tokens_scratch(int M, int E, int H, int I, int k, int S);
hipError_t launch_tokens(const Tokens& p, void* scratch, hipStream_t s);

// dequant.hip
hipError_t launch_dequant(const Layer& L, const hmoe_weights& W, int expert, int tensor,
                          float* out_f32, uint16_t* out_bf16, hipStream_t s);

// repack.hip: a batch of copy jobs (n bytes) and NF3 plane-to-stream jobs (n units of
// 32 elements: src = low plane, src_hi = high plane, dst = stream), one launch
constexpr int kRepackThreads = 256;
constexpr int kRepackJobs = 24;
enum : int { kRepackCopy = 0, kRepackNf3 = 1 };
struct RepackJob {
  const void* src;
  const void* src_hi;
  void* dst;
  long n;
  int kind;
  int blocks;
};
struct RepackBatch {
  RepackJob job[kRepackJobs];
  int first_block[kRepackJobs];
  int njobs;
};
hipError_t launch_repack(RepackBatch& b, hipStream_t s);

TierMask make_tier_mask(const Layer& L);

// noalloc.hip: this device's file-scope scratch array (address looked up once per
// device) and its size
hipError_t static_scratch(void** out);
size_t static_scratch_bytes();

bool plan_gemv(int K, GemvTiling* t);

}  // namespace hmoe
