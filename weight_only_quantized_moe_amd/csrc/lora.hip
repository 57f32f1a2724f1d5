// Low-rank adapters of many requests beside one shared projection:
//   z[m] = A_g x[m],  y[m] = base[m] + s_g B_g z[m],  g = ids[m]   (ids outside [0, G): y = base)
// and the gradients
//   dz[m] = s_g B_g^T dy[m],  dx[m] = dbase[m] + A_g^T dz[m],
//   dA_g = sum_m dz[m] x[m]^T,  dB_g = s_g sum_m dy[m] z[m]^T   (sums over the rows of g).
//
// With ranks of 8 to 128 the products do r / 2 operations a byte of x and y, far below what
// the matrix cores could do: the kernels are bound by reading x, base and the matrices in
// use, and by writing y. So every product runs on bf16 MFMA straight from global memory into
// fragments (no LDS staging: nothing but the small matrices is read twice), rows of one
// adapter are gathered into tiles of 16, 32 or 64, and the long axis K is split over waves
// and blocks when there are few tiles. z stays in fp32: where it is an MFMA operand it goes
// in as a sum of bf16 parts (two where the result is rounded to bf16, three where it stays
// fp32), so it is not rounded to 8 bits on the way.
#include <algorithm>

#include "device_common.h"
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
struct __attribute__((packed, aligned(4))) Int4 {
  int32_t v[4];
};

constexpr int kLoraThreads = 256;
constexpr int kLoraWaves = kLoraThreads / kWave;
constexpr int kKStep = 64;        // K elements a wave takes at a time: two MFMAs deep

__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
  const Half8 h = *reinterpret_cast<const Half8*>(p);
  return u32x4{h.w[0], h.w[1], h.w[2], h.w[3]};
}
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Which rows a block works on. With a tile table (many rows) it is looked up; without one,
// block b is the tile that starts at row b if the rows of the same adapter before b fill
// whole tiles, and has nothing to do otherwise.
struct Tiles {
  const int32_t* ids;
  int M, G;
  const int32_t* sorted;      // null: no table
  const int32_t* off;
  const int32_t* tile_group;
  const int32_t* tile_start;
};

// false: no tile. Else *g (G: rows without an adapter), s_rows[0 .. *n).
template <int RT>
__device__ __forceinline__ bool find_tile(const Tiles& t, int* g, int* n, int32_t* s_rows) {
  const int b = blockIdx.x;
  if (t.sorted) {
    const int grp = t.tile_group[b];
    if (grp < 0) return false;
    const int start = t.tile_start[b];
    *g = grp;
    *n = min(RT, t.off[grp + 1] - start);
    if ((int)threadIdx.x < *n) s_rows[threadIdx.x] = t.sorted[start + threadIdx.x];
    __syncthreads();
    return true;
  }
  const int lane = threadIdx.x & (kWave - 1);
  auto key = [&](int m) {
    const int id = t.ids[m];
    return (unsigned)id < (unsigned)t.G ? id : t.G;
  };
  const int mine = key(b);
  int seen = 0, first = -1;  // rows of `mine` so far; their number before b
  for (int m0 = 0; m0 < t.M; m0 += kWave) {
    const int m = m0 + lane;
    const uint64_t same = __ballot(m < t.M && key(min(m, t.M - 1)) == mine);
    if (first < 0 && b < m0 + kWave) {
      first = seen + __popcll(same & ((1ull << (b - m0)) - 1ull));
      if (first % RT) return false;
    }
    const int rank = seen + __popcll(same & ((1ull << lane) - 1ull)) - first;
    if (first >= 0 && (same >> lane & 1) && rank >= 0 && rank < RT) s_rows[rank] = m;
    seen += __popcll(same);
    if (first >= 0 && seen - first >= RT) break;
  }
  *g = mine;
  *n = min(RT, seen - first);
  __syncthreads();
  return true;
}

struct ShrinkArgs {
  Tiles tiles;
  const uint16_t* x;
  long xs;
  const uint16_t* w;   // [G, r, K]
  int K, r, splits;
  float* part;         // [splits, M, r]
};

// part[s][m] = W_g x[m] over split s of K. The four waves of a block take the split's steps
// of 64 in turn (512 contiguous bytes of a row together) and add up through LDS in wave
// order. Within a step lane group q holds K elements 16q .. 16q + 15 of its row for two
// MFMAs: the order of the reduction axis is free as long as both operands share it, and so
// every lane reads 32 contiguous bytes.
template <int MT, int NT>
__global__ __launch_bounds__(kLoraThreads) void lora_shrink_kernel(ShrinkArgs a) {
  constexpr int RT = MT * 16;
  __shared__ int32_t s_rows[RT];
  __shared__ float s_red[kLoraWaves][RT * NT * 16];
  int g, n;
  if (!find_tile<RT>(a.tiles, &g, &n, s_rows)) return;
  if (g == a.tiles.G) return;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int c = lane & 15, q = lane >> 4;
  const uint16_t* xp[MT];
  const uint16_t* wp[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int rr = i * 16 + c;
    xp[i] = a.x + (long)s_rows[rr < n ? rr : 0] * a.xs + q * 16;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int rr = i * 16 + c;
    wp[i] = a.w + ((long)g * a.r + (rr < a.r ? rr : 0)) * a.K + q * 16;
  }
  f32x4 acc[MT][NT] = {};
  const int steps = (a.K + kKStep - 1) / kKStep;
  const int s0 = (int)((long)steps * blockIdx.y / a.splits);
  const int s1 = (int)((long)steps * (blockIdx.y + 1) / a.splits);
  for (int st = s0 + wave; st < s1; st += kLoraWaves) {
    const int k = st * kKStep;
    u32x4 vx[MT][2] = {}, vw[NT][2] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (k + q * 16 + h * 8 < a.K) {
#pragma unroll
        for (int i = 0; i < MT; ++i) vx[i][h] = load8(xp[i] + k + h * 8);
#pragma unroll
        for (int i = 0; i < NT; ++i) vw[i][h] = load8(wp[i] + k + h * 8);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma(vx[i][h], vw[j][h], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s_red[wave][(i * 16 + q * 4 + e) * (NT * 16) + j * 16 + c] = acc[i][j][e];
  __syncthreads();
  float* out = a.part + (long)blockIdx.y * a.tiles.M * a.r;
  for (int i = threadIdx.x; i < n * NT * 16; i += kLoraThreads) {
    const int row = i / (NT * 16), col = i % (NT * 16);
    if (col >= a.r) continue;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kLoraWaves; ++w) s += s_red[w][i];
    out[(long)s_rows[row] * a.r + col] = s;
  }
}

struct ExpandArgs {
  Tiles tiles;
  const float* part;     // [splits, M, r]
  int splits, r, N;
  const uint16_t* w;     // [G, N, r]
  const float* scale;    // [G]
  const uint16_t* base;  // may be null
  long bs;
  uint16_t* y;
  long ys;
  float* z;              // may be null
  bool scaled_z;         // z receives scale * z
  int col_groups;        // groups of 64 columns a block takes
};

// bf16 parts of an fp32 value: hi + lo (+ lo2) with the residue of each rounded next. A
// value beyond bf16's range (infinite hi) has no residue.
__device__ __forceinline__ float bf16_round(float v) { return bf16_lo(pack_bf16(v, 0.f)); }
__device__ __forceinline__ float bf16_rest(float v, float hi) {
  return (__float_as_uint(hi) & 0x7F800000u) == 0x7F800000u ? 0.f : v - hi;
}

// y = base + W_g (scale z): z's splits are added in order, scaled, split into two bf16 parts
// and kept in LDS; each wave then takes 64 columns at a time. The small matrix is the MFMA's
// first operand with its rows dealt out so that a lane ends up with 16 consecutive columns
// of one row of y: base and y move as 16-byte accesses, 128 contiguous bytes a row. A
// fragment of W serves both parts of z; up to rank 16 both parts share one MFMA.
template <int MT, int KS>
__global__ __launch_bounds__(kLoraThreads) void lora_expand_kernel(ExpandArgs a) {
  constexpr int RT = MT * 16;
  constexpr bool kPack = KS == 0;                   // rank <= 16: hi and lo side by side
  constexpr int kSteps = kPack ? 1 : KS;
  constexpr int kRow = kSteps * 32 + 8;             // LDS row, padded off the banks
  __shared__ int32_t s_rows[RT];
  __shared__ __align__(16) uint16_t s_z[kPack ? 1 : 2][RT * kRow];
  int g, n;
  if (!find_tile<RT>(a.tiles, &g, &n, s_rows)) return;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
  const int c = lane & 15, q = lane >> 4;
  const int groups = (a.N + 63) / 64;
  const int g0 = blockIdx.y * a.col_groups, g1 = min(g0 + a.col_groups, groups);
  const bool live = g != a.tiles.G;
  const long part = (long)a.tiles.M * a.r;
  if (live) {
    const float sc = a.scale ? a.scale[g] : 1.f;
    for (int i = tid; i < RT * kSteps * 32; i += kLoraThreads) {
      const int row = i / (kSteps * 32), col = i % (kSteps * 32);
      float v = 0.f;
      const int rc = kPack ? col % a.r : col;       // rank index
      const bool in = row < n && (kPack ? col < 2 * a.r : col < a.r);
      if (in) {
        const float* p = a.part + (long)s_rows[row] * a.r + rc;
        for (int s = 0; s < a.splits; ++s) v += p[s * part];
        const float sv = v * sc;
        if (a.z && blockIdx.y == 0 && col < a.r)
          a.z[(long)s_rows[row] * a.r + rc] = a.scaled_z ? sv : v;
        v = sv;
      }
      const float hi = bf16_round(v);
      if (kPack) {
        s_z[0][row * kRow + col] = (uint16_t)pack_bf16(col < a.r ? hi : bf16_rest(v, hi), 0.f);
      } else {
        s_z[0][row * kRow + col] = (uint16_t)pack_bf16(hi, 0.f);
        s_z[kPack ? 0 : 1][row * kRow + col] = (uint16_t)pack_bf16(bf16_rest(v, hi), 0.f);
      }
    }
  } else if (a.z && blockIdx.y == 0) {
    for (int i = tid; i < n * a.r; i += kLoraThreads)
      a.z[(long)s_rows[i / a.r] * a.r + i % a.r] = 0.f;
  }
  __syncthreads();
  if (!live && a.base == a.y && a.bs == a.ys) return;  // rows without an adapter stay
  u32x4 zf[MT][kSteps][kPack ? 1 : 2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
      for (int p = 0; p < (kPack ? 1 : 2); ++p)
        zf[i][ks][p] = *reinterpret_cast<const u32x4*>(&s_z[p][(i * 16 + c) * kRow + ks * 32 + q * 8]);
  const uint16_t* w = a.w + (live ? (long)g * a.N * a.r : 0);
  for (int cg = g0 + wave; cg < g1; cg += kLoraWaves) {
    const int n0 = cg * 64;
    f32x4 acc[MT][4] = {};
    if (live) {
      u32x4 wf[4][kSteps] = {};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int col = min(n0 + (c >> 2) * 16 + t * 4 + (c & 3), a.N - 1);
        const uint16_t* p = w + (long)col * a.r;
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
          const int ch = (ks * 4 + q) * 8;
          if (kPack) {
            if (ch < 2 * a.r) wf[t][ks] = load8(p + (ch < a.r ? ch : ch - a.r));
          } else if (ch < a.r) {
            wf[t][ks] = load8(p + ch);
          }
        }
      }
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int p = 0; p < (kPack ? 1 : 2); ++p)
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[i][t] = mfma(wf[t][ks], zf[i][ks][p], acc[i][t]);
    }
    const int col = n0 + q * 16;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int rr = i * 16 + c;
      if (rr >= n) continue;
      const long row = s_rows[rr];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (col + h * 8 >= a.N) continue;
        Half8 o;
        u32x4 b{};
        if (a.base) b = load8(a.base + row * a.bs + col + h * 8);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const f32x4 v = acc[i][h * 2 + (p >> 1)];
          o.w[p] = live ? pack_bf16(bf16_lo(b[p]) + v[(p & 1) * 2], bf16_hi(b[p]) + v[(p & 1) * 2 + 1])
                        : b[p];
        }
        *reinterpret_cast<Half8*>(a.y + row * a.ys + col + h * 8) = o;
      }
    }
  }
}

struct WgradArgs {
  const int32_t* sorted;
  const int32_t* off;
  int r;
  const float* scale;
  // two products: [0] P = dz (scaled), X = x, out dA [G, r, C]; [1] P = z, X = dy, out dB [G, C, r]
  const float* p[2];
  const uint16_t* x[2];
  long xs[2];
  int C[2], blocks[2];
  float* out[2];
};

constexpr int kWgradThreads = 512;
constexpr int kWgradWaves = kWgradThreads / kWave;

// out_g[p, c] = sum over the rows m of group g of P[m, p] X[m, c]. The reduction axis is the
// row, so both operands are needed transposed: a lane reads 8 rows of 4 neighbouring columns
// (8 bytes each, 128 contiguous bytes a row over 16 lanes) and pairs them up by byte
// permutes into the fragments of 4 MFMAs. P goes in as three bf16 parts (24 bits), so the
// fp32 result carries no bf16 rounding. The block's eight waves take steps of 32 rows in
// turn and add up through LDS in wave order. Rows past the group's end are zero in both
// operands.
template <int NT>
__global__ __launch_bounds__(kWgradThreads) void lora_wgrad_kernel(WgradArgs a) {
  __shared__ float s_red[kWgradWaves][16][68];
  const int side = (int)blockIdx.x >= a.blocks[0];
  const int c0 = ((int)blockIdx.x - (side ? a.blocks[0] : 0)) * 64, g = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
  const int c = lane & 15, q = lane >> 4;
  const int m0 = a.off[g], m1 = a.off[g + 1];
  const float* P = a.p[side];
  const uint16_t* X = a.x[side];
  const long xs = a.xs[side];
  const int C = a.C[side];
  const float sc = side ? a.scale[g] : 1.f;
  const int col = c0 + c * 4;
  f32x4 acc[NT][4] = {};
  for (int m = m0 + wave * 32; m < m1; m += kWgradWaves * 32) {
    int row[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) row[j] = m + q * 8 + j < m1 ? a.sorted[m + q * 8 + j] : -1;
    uint32_t xv[8][2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      xv[j][0] = xv[j][1] = 0;
      if (row[j] >= 0 && col < C) {
        const Half4 h = *reinterpret_cast<const Half4*>(X + row[j] * xs + col);
        xv[j][0] = h.w[0];
        xv[j][1] = h.w[1];
      }
    }
    u32x4 xf[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int p = 0; p < 4; ++p)
        xf[t][p] = __builtin_amdgcn_perm(xv[2 * p + 1][t >> 1], xv[2 * p][t >> 1],
                                         (t & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int rr = i * 16 + c;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = row[j] >= 0 && rr < a.r ? P[(long)row[j] * a.r + rr] * sc : 0.f;
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        u32x4 pf;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          pf[p] = pack_bf16(v[2 * p], v[2 * p + 1]);
          v[2 * p] = bf16_rest(v[2 * p], bf16_lo(pf[p]));
          v[2 * p + 1] = bf16_rest(v[2 * p + 1], bf16_hi(pf[p]));
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[i][t] = mfma(pf, xf[t], acc[i][t]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s_red[wave][q * 4 + e][c * 4 + t] = acc[i][t][e];
    __syncthreads();
    for (int o = tid; o < 16 * 64; o += kWgradThreads) {
      // columns run fastest in dA, ranks in dB
      const int pr = side ? o & 15 : o >> 6, cc = side ? o >> 4 : o & 63;
      const int rr = i * 16 + pr, cl = c0 + cc;
      if (rr >= a.r || cl >= C) continue;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWgradWaves; ++w) s += s_red[w][pr][cc];
      a.out[side][side ? ((long)g * C + cl) * a.r + rr : ((long)g * a.r + rr) * C + cl] = s;
    }
  }
}

// [R, C] -> [C, R] of every group, for both matrices in one launch: the gradients multiply
// by A^T and B^T, whose copies make them the same products as the forward's.
struct TransposeArgs {
  const uint16_t* in[2];
  uint16_t* out[2];
  int R[2], C[2], tr[2], tc[2];
};

__global__ __launch_bounds__(256) void lora_transpose_kernel(TransposeArgs a) {
  __shared__ uint16_t s_t[64][66];
  const int side = (int)blockIdx.x >= a.tr[0] * a.tc[0];
  const int b = (int)blockIdx.x - (side ? a.tr[0] * a.tc[0] : 0);
  const int R = a.R[side], C = a.C[side];
  const int r0 = b / a.tc[side] * 64, c0 = b % a.tc[side] * 64;
  const long base = (long)blockIdx.y * R * C;
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int rr = r0 + i / 64, cc = c0 + i % 64;
    if (rr < R && cc < C) s_t[i / 64][i % 64] = a.in[side][base + (long)rr * C + cc];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 64; i += 256) {
    const int cc = c0 + i / 64, rr = r0 + i % 64;
    if (rr < R && cc < C) a.out[side][base + (long)cc * R + rr] = s_t[i % 64][i / 64];
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

namespace {

constexpr int kDirectRows = 1024;  // up to this many rows a block finds its tile by itself

struct Plan {
  int mt, nt, rt, tiles;     // tile rows / 16, rank / 16 rounded up, tile rows, most tiles
  bool table;                // a sort and a tile table come first
};

// Tile rows from the mean number of rows an adapter has: 64 rows share one read of the
// adapter, but a tile with few rows wastes MFMA work and registers. Accumulators bound
// mt * nt to 8.
Plan plan_tiles(int M, int G, int r, bool sorted) {
  Plan p;
  p.nt = r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8;
  const int mean = M / std::max(1, std::min(G, M));
  p.mt = std::min(mean >= 48 ? 4 : mean >= 24 ? 2 : 1, 8 / p.nt);
  p.rt = p.mt * 16;
  p.table = sorted || M > kDirectRows;
  p.tiles = p.table ? M / p.rt + std::min(G + 1, M) : M;
  return p;
}

// Splits of the reduction axis: enough blocks to fill the card, at least four steps of 64
// for each block, at most 16 partial sums to add up again.
int plan_splits(const Plan& p, int M, int G, int K) {
  const int busy = std::max(1, p.table ? p.tiles : std::min(M, M / p.rt + std::min(G, M)));
  const int steps = (K + kKStep - 1) / kKStep;
  return std::max(1, std::min({(1024 + busy - 1) / busy, (steps + 3) / 4, 16}));
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct Space {
  size_t sorted, off, counts, tile_group, tile_start, part, dz, at, bt, total;
};

Space plan_space(int M, int G, int K, int N, int r, bool backward) {
  Space s{};
  const Plan p = plan_tiles(M, G, r, backward);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = align256(at + bytes);
    return o;
  };
  if (p.table) {
    s.sorted = take((size_t)M * 4);
    s.off = take((size_t)(G + 2) * 4);
    s.counts = take(sort_count_words(M, G + 1) * 4);
    s.tile_group = take((size_t)p.tiles * 4);
    s.tile_start = take((size_t)p.tiles * 4);
  }
  s.part = take((size_t)plan_splits(p, M, G, backward ? N : K) * M * r * 4);
  if (backward) {
    s.dz = take((size_t)M * r * 4);
    s.at = take((size_t)G * r * K * 2);
    s.bt = take((size_t)G * r * N * 2);
  }
  s.total = at;
  return s;
}

hipError_t make_tiles(const int32_t* ids, int M, int G, const Plan& p, const Space& sp, char* scratch,
                      Tiles* t, hipStream_t s) {
  *t = Tiles{ids, M, G, nullptr, nullptr, nullptr, nullptr};
  if (!p.table) return hipSuccess;
  GroupSort g{};
  g.ids = ids;
  g.n = M;
  g.G = G;
  g.groups = G + 1;
  g.counts = reinterpret_cast<int32_t*>(scratch + sp.counts);
  g.sorted = reinterpret_cast<int32_t*>(scratch + sp.sorted);
  g.off = reinterpret_cast<int32_t*>(scratch + sp.off);
  g.tile_rows = p.rt;
  g.max_tiles = p.tiles;
  g.tile_group = reinterpret_cast<int32_t*>(scratch + sp.tile_group);
  g.tile_start = reinterpret_cast<int32_t*>(scratch + sp.tile_start);
  t->sorted = g.sorted;
  t->off = g.off;
  t->tile_group = g.tile_group;
  t->tile_start = g.tile_start;
  return launch_sort(g, s);
}

hipError_t shrink(const Plan& p, const ShrinkArgs& a, hipStream_t s) {
  const dim3 grid(p.tiles, a.splits), block(kLoraThreads);
#define HMOE_SHRINK(MT, NT)                                                         \
  if (p.mt == MT && p.nt == NT)                                                     \
  hipLaunchKernelGGL((lora_shrink_kernel<MT, NT>), grid, block, 0, s, a)
  HMOE_SHRINK(1, 1);
  HMOE_SHRINK(2, 1);
  HMOE_SHRINK(4, 1);
  HMOE_SHRINK(1, 2);
  HMOE_SHRINK(2, 2);
  HMOE_SHRINK(4, 2);
  HMOE_SHRINK(1, 4);
  HMOE_SHRINK(2, 4);
  HMOE_SHRINK(1, 8);
#undef HMOE_SHRINK
  return hipGetLastError();
}

hipError_t expand(const Plan& p, ExpandArgs a, hipStream_t s) {
  const int groups = (a.N + 63) / 64;
  // columns a block: a multiple of its four waves' 64, as wide as still leaves about 1024
  // blocks, so that few blocks add up z's splits again
  const int busy = p.table ? p.tiles : std::min(a.tiles.M, a.tiles.M / p.rt + std::min(a.tiles.G, a.tiles.M));
  const int want = std::max(1, (1024 + busy - 1) / busy);
  a.col_groups = std::max(kLoraWaves, (groups + want - 1) / want);
  const dim3 grid(p.tiles, (groups + a.col_groups - 1) / a.col_groups), block(kLoraThreads);
  const int ks = a.r <= 16 ? 0 : (a.r + 31) / 32;
#define HMOE_EXPAND(MT, KS)                                                         \
  if (p.mt == MT && ks == KS)                                                       \
  hipLaunchKernelGGL((lora_expand_kernel<MT, KS>), grid, block, 0, s, a)
  HMOE_EXPAND(1, 0);
  HMOE_EXPAND(2, 0);
  HMOE_EXPAND(4, 0);
  HMOE_EXPAND(1, 1);
  HMOE_EXPAND(2, 1);
  HMOE_EXPAND(4, 1);
  HMOE_EXPAND(1, 2);
  HMOE_EXPAND(2, 2);
  HMOE_EXPAND(1, 3);
  HMOE_EXPAND(1, 4);
#undef HMOE_EXPAND
  return hipGetLastError();
}

}  // namespace

void lora_scratch(int M, int G, int K, int N, int r, size_t* forward, size_t* backward) {
  *forward = plan_space(M, G, K, N, r, false).total;
  *backward = plan_space(M, G, K, N, r, true).total;
}

hipError_t launch_lora(const Lora& l, void* scratch, hipStream_t s) {
  char* b = static_cast<char*>(scratch);
  const Plan p = plan_tiles(l.M, l.G, l.r, false);
  const Space sp = plan_space(l.M, l.G, l.K, l.N, l.r, false);
  Tiles t;
  hipError_t err = make_tiles(l.ids, l.M, l.G, p, sp, b, &t, s);
  if (err != hipSuccess) return err;
  const int splits = plan_splits(p, l.M, l.G, l.K);
  float* part = reinterpret_cast<float*>(b + sp.part);
  err = shrink(p, ShrinkArgs{t, l.x, l.xs, l.A, l.K, l.r, splits, part}, s);
  if (err != hipSuccess) return err;
  return expand(p, ExpandArgs{t, part, splits, l.r, l.N, l.B, l.scale, l.base, l.bs, l.y, l.ys, l.z,
                              false, 0}, s);
}

hipError_t launch_lora_backward(const LoraGrad& l, void* scratch, hipStream_t s) {
  char* b = static_cast<char*>(scratch);
  const Plan p = plan_tiles(l.M, l.G, l.r, true);
  const Space sp = plan_space(l.M, l.G, l.K, l.N, l.r, true);
  Tiles t;
  hipError_t err = make_tiles(l.ids, l.M, l.G, p, sp, b, &t, s);
  if (err != hipSuccess) return err;
  float* dz = reinterpret_cast<float*>(b + sp.dz);
  if (l.M > 0) {
    uint16_t* At = reinterpret_cast<uint16_t*>(b + sp.at);
    uint16_t* Bt = reinterpret_cast<uint16_t*>(b + sp.bt);
    TransposeArgs ta{{l.A, l.B}, {At, Bt}, {l.r, l.N}, {l.K, l.r}, {}, {}};
    int blocks = 0;
    for (int i = 0; i < 2; ++i) {
      ta.tr[i] = (ta.R[i] + 63) / 64;
      ta.tc[i] = (ta.C[i] + 63) / 64;
      blocks += ta.tr[i] * ta.tc[i];
    }
    hipLaunchKernelGGL(lora_transpose_kernel, dim3(blocks, l.G), dim3(256), 0, s, ta);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    const int splits = plan_splits(p, l.M, l.G, l.N);
    float* part = reinterpret_cast<float*>(b + sp.part);
    err = shrink(p, ShrinkArgs{t, l.dy, l.dys, Bt, l.N, l.r, splits, part}, s);
    if (err != hipSuccess) return err;
    err = expand(p, ExpandArgs{t, part, splits, l.r, l.K, At, l.scale, l.dbase, l.dbs, l.dx, l.dxs,
                               dz, true, 0}, s);
    if (err != hipSuccess) return err;
  }
  WgradArgs w{t.sorted, t.off, l.r, l.scale, {dz, l.z}, {l.x, l.dy}, {l.xs, l.dys}, {l.K, l.N},
              {(l.K + 63) / 64, (l.N + 63) / 64}, {l.dA, l.dB}};
  const dim3 grid(w.blocks[0] + w.blocks[1], l.G), block(kWgradThreads);
  switch (p.nt) {
    case 1: hipLaunchKernelGGL(lora_wgrad_kernel<1>, grid, block, 0, s, w); break;
    case 2: hipLaunchKernelGGL(lora_wgrad_kernel<2>, grid, block, 0, s, w); break;
    case 4: hipLaunchKernelGGL(lora_wgrad_kernel<4>, grid, block, 0, s, w); break;
    default: hipLaunchKernelGGL(lora_wgrad_kernel<8>, grid, block, 0, s, w); break;
  }
  return hipGetLastError();
}

}  // namespace hmoe
