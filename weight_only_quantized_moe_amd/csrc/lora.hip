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
// adapter are gathered into tiles of 16 or 32, and the long axis K is split over waves
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
constexpr int kKStep = 64;   // K elements a wave takes at a time: two MFMAs deep

__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
  const Half8 h = *reinterpret_cast<const Half8*>(p);
  return u32x4{h.w[0], h.w[1], h.w[2], h.w[3]};
}
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// bf16 parts of an fp32 value: hi + lo (+ lo2) with the residue of each rounded next. A
// value beyond bf16's range (infinite hi) has no residue.
__device__ __forceinline__ float bf16_round(float v) { return bf16_lo(pack_bf16(v, 0.f)); }
__device__ __forceinline__ float bf16_rest(float v, float hi) {
  return (__float_as_uint(hi) & 0x7F800000u) == 0x7F800000u ? 0.f : v - hi;
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

// Which rows a block works on. With a tile table (many rows) it is looked up; without one,
// block b is the tile that starts at row b if the rows of the same adapter before b fill
// whole tiles, and has nothing to do otherwise.
struct Tiles {
  const int32_t* ids;
  int M, G;
  const int32_t* sorted;      // null: no table
  const SortTile* table;
};

// false: no tile. Else *g (G: rows without an adapter), s_rows[0 .. *n).
template <int RT>
__device__ __forceinline__ bool find_tile(const Tiles& t, int* g, int* n, int32_t* s_rows) {
  const int b = blockIdx.x;
  if (t.sorted) {
    const SortTile d = t.table[b];
    if (d.group < 0) return false;
    *g = d.group;
    *n = d.rows;
    if ((int)threadIdx.x < d.rows) s_rows[threadIdx.x] = t.sorted[d.start + threadIdx.x];
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

// s_red = X_rows W_g^T over the steps [s0, s1) of the reduction axis K, rows x ranks. The W
// waves of the block take the steps of 64 in turn; then the upper half of the waves hands
// its sums to the lower half through LDS, and the lower half leaves its sums in s_red[wave]
// for the caller to add in wave order. DEPTH
// steps' loads are in flight at a time (as many as the registers allow).
template <int MT, int NT, int W, int DEPTH>
__device__ __forceinline__ void shrink_tile(const uint16_t* x, long xs, const uint16_t* w, int K,
                                            int r, int n, const int32_t* s_rows, int s0, int s1,
                                            float (*s_red)[MT * NT * 256]) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int c = lane & 15, q = lane >> 4;
  const uint16_t* xp[MT];
  const uint16_t* wp[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int rr = i * 16 + c;
    xp[i] = x + (long)s_rows[rr < n ? rr : 0] * xs + q * 8;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int rr = i * 16 + c;
    wp[i] = w + (long)(rr < r ? rr : 0) * K + q * 8;
  }
  f32x4 acc[MT][NT] = {};
  struct Step {
    u32x4 x[MT][2], w[NT][2];
  };
  auto load = [&](Step& v, int st) {
    const int k = st * kKStep;
    if (k + kKStep <= K) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < MT; ++i) v.x[i][h] = load8(xp[i] + k + h * 32);
#pragma unroll
        for (int i = 0; i < NT; ++i) v.w[i][h] = load8(wp[i] + k + h * 32);
      }
    } else {  // the last step of a K that is no multiple of 64
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = k + h * 32 + q * 8 < K;
#pragma unroll
        for (int i = 0; i < MT; ++i) v.x[i][h] = in ? load8(xp[i] + k + h * 32) : u32x4{};
#pragma unroll
        for (int i = 0; i < NT; ++i) v.w[i][h] = in ? load8(wp[i] + k + h * 32) : u32x4{};
      }
    }
  };
  auto multiply = [&](const Step& v) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma(v.x[i][h], v.w[j][h], acc[i][j]);
  };
  Step ring[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (s0 + wave + d * W < s1) load(ring[d], s0 + wave + d * W);
  for (int st = s0 + wave; st < s1;) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (st >= s1) break;
      multiply(ring[d]);
      if (st + DEPTH * W < s1) load(ring[d], st + DEPTH * W);
      st += W;
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

// W_g z of a tile's rows, added to base: each wave takes 64 columns at a time. The small
// matrix is the MFMA's first operand with its rows dealt out so that a lane ends up with
// columns 8q .. 8q + 7 and 32 + 8q .. 32 + 8q + 7 of one row of y: base and y move as 16-byte
// accesses, the four lanes of a row on 64 contiguous bytes. A fragment of W serves both bf16 parts of z; up to rank 16 (KS = 0) both
// parts share one MFMA. TR: W is [r, N] (its columns are neighbours, turned in registers),
// else [N, r].
struct ColumnArgs {
  int r, N;
  const uint16_t* w;     // matrix of the tile's adapter
  const uint16_t* base;  // may be null
  long bs;
  uint16_t* y;
  long ys;
};

template <int KS>
struct ZShape {
  static constexpr bool kPack = KS == 0;         // rank <= 16: hi and lo side by side
  static constexpr int kSteps = kPack ? 1 : KS;
  static constexpr int kParts = kPack ? 1 : 2;
  static constexpr int kRow = kSteps * 32 + 8;   // LDS row, padded off the banks
};

template <int MT, int KS, bool TR>
struct Columns {
  using Z = ZShape<KS>;
  const ColumnArgs& a;
  const bool live;
  const int n, c, q;
  long row[MT];

  // what one group of 64 columns reads: base, and the fragments of W (TR: as they lie)
  struct Load {
    u32x4 b[MT][2];
    u32x4 w[Z::kSteps][4];
  };

  __device__ __forceinline__ Columns(const ColumnArgs& a, bool live, int n, const int32_t* s_rows)
      : a(a), live(live), n(n), c(threadIdx.x & 15), q((threadIdx.x & (kWave - 1)) >> 4) {
#pragma unroll
    for (int i = 0; i < MT; ++i) row[i] = s_rows[i * 16 + c < n ? i * 16 + c : 0];
  }

  __device__ __forceinline__ void load(Load& l, int cg) const {
    const int n0 = cg * 64, col = n0 + q * 8;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l.b[i][h] = u32x4{};
        if (a.base && i * 16 + c < n && col + h * 32 < a.N)
          l.b[i][h] = load8(a.base + row[i] * a.bs + col + h * 32);
      }
#pragma unroll
    for (int ks = 0; ks < Z::kSteps; ++ks) {
      // ranks of this lane's fragment, of W as of z
      int ch = (ks * 4 + q) * 8;
      const bool in = live && ch < (Z::kPack ? 2 * a.r : a.r);
      if (Z::kPack && ch >= a.r) ch -= a.r;
#pragma unroll
      for (int t = 0; t < 4; ++t) l.w[ks][t] = u32x4{};
      if constexpr (TR) {
        const int wc = n0 + (c & 2) * 16 + (c >> 2) * 8 + (c & 1) * 4;
        if (in && wc < a.N) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const Half4 h = *reinterpret_cast<const Half4*>(a.w + (long)(ch + j) * a.N + wc);
            l.w[ks][j >> 1][(j & 1) * 2] = h.w[0];
            l.w[ks][j >> 1][(j & 1) * 2 + 1] = h.w[1];
          }
        }
      } else if (in) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int wc = min(n0 + (t >> 1) * 32 + (c >> 2) * 8 + (t & 1) * 4 + (c & 3), a.N - 1);
          l.w[ks][t] = load8(a.w + (long)wc * a.r + ch);
        }
      }
    }
  }

  __device__ __forceinline__ void finish(const Load& l, int cg, const u32x4 (&zf)[MT][Z::kSteps][Z::kParts]) const {
    const int col = cg * 64 + q * 8;
    f32x4 acc[MT][4] = {};
    if (live) {
#pragma unroll
      for (int ks = 0; ks < Z::kSteps; ++ks) {
        u32x4 wf[4];
        if constexpr (TR) {
          uint32_t v[8][2];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            v[j][0] = l.w[ks][j >> 1][(j & 1) * 2];
            v[j][1] = l.w[ks][j >> 1][(j & 1) * 2 + 1];
          }
          turn_8x4(v, wf);
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t) wf[t] = l.w[ks][t];
        }
#pragma unroll
        for (int p = 0; p < Z::kParts; ++p)
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[i][t] = mfma(wf[t], zf[i][ks][p], acc[i][t]);
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (i * 16 + c >= n) continue;
      // value o of the lane's 16: fragment o / 4, element o % 4 (TR: the other way round)
      auto at = [&](int o) { return TR ? acc[i][o & 3][o >> 2] : acc[i][o >> 2][o & 3]; };
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (col + h * 32 >= a.N) continue;
        Half8 o;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t bp = l.b[i][h][p];
          o.w[p] = live ? pack_bf16(bf16_lo(bp) + at(h * 8 + 2 * p), bf16_hi(bp) + at(h * 8 + 2 * p + 1))
                        : bp;
        }
        *reinterpret_cast<Half8*>(a.y + row[i] * a.ys + col + h * 32) = o;
      }
    }
  }

  // groups cg, cg + W, ... below g1; `first` holds the loads of group cg. AHEAD: a second
  // set of loads is in flight (where there are registers for it).
  template <int W, bool AHEAD>
  __device__ __forceinline__ void run(Load& first, int cg, int g1,
                                      const uint16_t (*s_z)[MT * 16 * Z::kRow]) const {
    u32x4 zf[MT][Z::kSteps][Z::kParts];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int ks = 0; ks < Z::kSteps; ++ks)
#pragma unroll
        for (int p = 0; p < Z::kParts; ++p)
          zf[i][ks][p] = *reinterpret_cast<const u32x4*>(&s_z[p][(i * 16 + c) * Z::kRow + ks * 32 + q * 8]);
    if constexpr (!AHEAD) {
      while (cg < g1) {
        finish(first, cg, zf);
        cg += W;
        if (cg < g1) load(first, cg);
      }
      return;
    }
    Load next;
    while (cg < g1) {
      if (cg + W < g1) load(next, cg + W);
      finish(first, cg, zf);
      cg += W;
      if (cg >= g1) break;
      if (cg + W < g1) load(first, cg + W);
      finish(next, cg, zf);
      cg += W;
    }
  }
};

// four ranks of one row of z into LDS as bf16 parts (col: first rank; zeros past r)
template <int KS, int N>
__device__ __forceinline__ void put_z(uint16_t (*s_z)[N], int row, int col, int r, const float (&v)[4]) {
  using Z = ZShape<KS>;
  uint32_t hi[2], lo[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    hi[p] = pack_bf16(v[2 * p], v[2 * p + 1]);
    lo[p] = pack_bf16(bf16_rest(v[2 * p], bf16_lo(hi[p])), bf16_rest(v[2 * p + 1], bf16_hi(hi[p])));
  }
  uint16_t* at = &s_z[0][row * Z::kRow + col];
  *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
  *reinterpret_cast<uint2*>(Z::kPack ? at + r : &s_z[Z::kParts - 1][row * Z::kRow + col]) =
      make_uint2(lo[0], lo[1]);
}

// zeros in the ranks of z's LDS rows that pad them to whole MFMA steps
template <int KS, int RT, int N>
__device__ __forceinline__ void pad_z(uint16_t (*s_z)[N], int r) {
  using Z = ZShape<KS>;
  const int from = Z::kPack ? 2 * r : r, pad = (Z::kSteps * 32 - from) / 4;
  for (int i = threadIdx.x; i < RT * pad; i += blockDim.x)
#pragma unroll
    for (int p = 0; p < Z::kParts; ++p)
      *reinterpret_cast<uint2*>(&s_z[p][i / pad * Z::kRow + from + i % pad * 4]) = make_uint2(0, 0);
}

struct ShrinkArgs {
  Tiles tiles;
  const uint16_t* x;
  long xs;
  const uint16_t* w;   // [G, r, K]
  int K, r, splits;
  float* part;         // [splits, M, r]
};

constexpr int kShrinkWaves = 8;

// part[s][m] = W_g x[m] over split s of K
template <int MT, int NT>
__global__ __launch_bounds__(kShrinkWaves* kWave) void lora_shrink_kernel(ShrinkArgs a) {
  __shared__ int32_t s_rows[MT * 16];
  __shared__ __align__(16) float s_red[kShrinkWaves / 2][MT * NT * 256];
  int g, n;
  if (!find_tile<MT * 16>(a.tiles, &g, &n, s_rows)) return;
  if (g == a.tiles.G) return;
  const int steps = (a.K + kKStep - 1) / kKStep;
  shrink_tile<MT, NT, kShrinkWaves, (MT + NT <= 3 ? 4 : 2)>(a.x, a.xs, a.w + (long)g * a.r * a.K, a.K, a.r, n, s_rows,
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
  bool scaled_z;         // z receives scale * z
  int col_groups;        // groups of 64 columns a block takes
  ColumnArgs c;          // w: all adapters' matrices
};

constexpr int kExpandWaves = 4;

// y = base + W_g (scale z): z's splits are added in order, scaled, split into two bf16 parts
// and kept in LDS for the block's columns
template <int MT, int KS, bool TR>
__global__ __launch_bounds__(kExpandWaves* kWave) void lora_expand_kernel(ExpandArgs a) {
  using Z = ZShape<KS>;
  constexpr int RT = MT * 16;
  __shared__ int32_t s_rows[RT];
  __shared__ __align__(16) uint16_t s_z[Z::kParts][RT * Z::kRow];
  int g, n;
  if (!find_tile<RT>(a.tiles, &g, &n, s_rows)) return;
  const bool live = g != a.tiles.G;
  const int r = a.c.r, quads = r / 4;
  ColumnArgs ca = a.c;
  if (live) ca.w += (long)g * ca.N * r;
  const Columns<MT, KS, TR> cols(ca, live, n, s_rows);
  const int g0 = blockIdx.y * a.col_groups, g1 = min(g0 + a.col_groups, (ca.N + 63) / 64);
  const int cg = g0 + (threadIdx.x >> 6);
  typename Columns<MT, KS, TR>::Load first;  // on the way while z is put together
  if (cg < g1) cols.load(first, cg);
  if (live) {
    const float sc = a.scale[g];
    const long part = (long)a.tiles.M * r;
    for (int i = threadIdx.x; i < n * quads; i += kExpandWaves * kWave) {
      const int row = i / quads, col = i % quads * 4;
      const float* p = a.part + (long)s_rows[row] * r + col;
      float v[4] = {};
#pragma unroll 4
      for (int s = 0; s < a.splits; ++s) {
        const float4 f = *reinterpret_cast<const float4*>(p + s * part);
        v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
      }
      float sv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) sv[e] = v[e] * sc;
      if (a.z && blockIdx.y == 0) {
        const float* o = a.scaled_z ? sv : v;
        *reinterpret_cast<float4*>(a.z + (long)s_rows[row] * r + col) = make_float4(o[0], o[1], o[2], o[3]);
      }
      put_z<KS>(s_z, row, col, r, sv);
    }
    pad_z<KS, RT>(s_z, r);
  } else if (a.z && blockIdx.y == 0) {
    for (int i = threadIdx.x; i < n * r; i += kExpandWaves * kWave)
      a.z[(long)s_rows[i / r] * r + i % r] = 0.f;
  }
  __syncthreads();
  if (!live && a.c.base == a.c.y) return;  // rows without an adapter stay
  cols.template run<kExpandWaves, (KS <= 2)>(first, cg, g1, s_z);
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
};

constexpr int kFusedWaves = 16;

// Both products of a tile of 16 rows in one block, for few rows: the sixteen waves split K,
// z never leaves LDS, then they split the block's columns. Blocks of one tile that take
// different columns repeat the first product (its matrix comes from L2 again).
template <int NT, int KS>
__global__ __launch_bounds__(kFusedWaves* kWave) void lora_fused_kernel(FusedArgs a) {
  using Z = ZShape<KS>;
  __shared__ int32_t s_rows[16];
  __shared__ __align__(16) float s_red[kFusedWaves / 2][NT * 256];
  __shared__ __align__(16) uint16_t s_z[Z::kParts][16 * Z::kRow];
  int g, n;
  if (!find_tile<16>(a.tiles, &g, &n, s_rows)) return;
  const bool live = g != a.tiles.G;
  const int r = a.c.r;
  ColumnArgs ca = a.c;
  if (live) ca.w += (long)g * ca.N * r;
  const Columns<1, KS, false> cols(ca, live, n, s_rows);
  const int g0 = blockIdx.y * a.col_groups, g1 = min(g0 + a.col_groups, (ca.N + 63) / 64);
  const int cg = g0 + (threadIdx.x >> 6);
  // on the way during the first product (beyond rank 32 there are no registers for that)
  typename Columns<1, KS, false>::Load first;
  if (KS < 2 && cg < g1) cols.load(first, cg);
  if (live) {
    // 1024 threads have 128 registers each
    shrink_tile<1, NT, kFusedWaves, (NT == 1 ? 3 : 1)>(a.x, a.xs, a.wa + (long)g * r * a.K, a.K, r, n, s_rows,
                                               0, (a.K + kKStep - 1) / kKStep, s_red);
    const float sc = a.scale[g];
    for (int i = threadIdx.x; i < n * NT * 4; i += kFusedWaves * kWave) {
      const int row = i / (NT * 4), col = i % (NT * 4) * 4;
      if (col >= r) continue;
      float v[4] = {};
#pragma unroll
      for (int w = 0; w < kFusedWaves / 2; ++w) {
        const float4 f = *reinterpret_cast<const float4*>(&s_red[w][i * 4]);
        v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
      }
      if (a.z && blockIdx.y == 0)
        *reinterpret_cast<float4*>(a.z + (long)s_rows[row] * r + col) = make_float4(v[0], v[1], v[2], v[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= sc;
      put_z<KS>(s_z, row, col, r, v);
    }
    pad_z<KS, 16>(s_z, r);
  } else if (a.z && blockIdx.y == 0) {
    for (int i = threadIdx.x; i < n * r; i += kFusedWaves * kWave)
      a.z[(long)s_rows[i / r] * r + i % r] = 0.f;
  }
  __syncthreads();
  if (!live && a.c.base == a.c.y) return;  // rows without an adapter stay
  if (KS >= 2 && cg < g1) cols.load(first, cg);
  cols.template run<kFusedWaves, (KS < 2)>(first, cg, g1, s_z);
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
constexpr int kWgradRows = 2048;  // row indices kept in LDS at a time

// out_g[p, c] = sum over the rows m of group g of P[m, p] X[m, c]. The reduction axis is the
// row, so both operands are needed transposed: a lane reads 8 rows of 4 neighbouring columns
// (8 bytes each, 128 contiguous bytes a row over 16 lanes) and turns them in registers into
// the fragments of 4 MFMAs. P goes in as three bf16 parts (24 bits), so the fp32 result
// carries no bf16 rounding. The block's eight waves take steps of 32 rows in turn, the next
// step's loads in flight, and add up through LDS in wave order. Rows past the group's end
// are zero in both operands. Ranks past NT * 16 go to further blocks (grid z).
template <int NT>
__global__ __launch_bounds__(kWgradThreads) void lora_wgrad_kernel(WgradArgs a) {
  __shared__ float s_red[kWgradWaves][16][68];
  __shared__ int32_t s_idx[kWgradRows];
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
  const int col = c0 + c * 4, r0 = blockIdx.z * NT * 16;
  f32x4 acc[NT][4] = {};
  struct Step {
    uint32_t x[8][2];
    float p[NT][8];
  };
  for (int mb = m0; mb < m1; mb += kWgradRows) {
    const int rows = min(kWgradRows, m1 - mb);
    __syncthreads();
    for (int i = tid; i < rows; i += kWgradThreads) s_idx[i] = a.sorted[mb + i];
    __syncthreads();
    auto load = [&](Step& v, int m) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = m + q * 8 + j;
        const bool in = at < rows;
        const long row = in ? s_idx[at] : 0;
        v.x[j][0] = v.x[j][1] = 0;
        if (in && col < C) {
          const Half4 h = *reinterpret_cast<const Half4*>(X + row * xs + col);
          v.x[j][0] = h.w[0];
          v.x[j][1] = h.w[1];
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int rr = r0 + i * 16 + c;
          v.p[i][j] = in && rr < a.r ? P[row * a.r + rr] : 0.f;
        }
      }
    };
    auto multiply = [&](Step& v) {
      u32x4 xf[4];
      turn_8x4(v.x, xf);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v.p[i][j] *= sc;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          u32x4 pf;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            float &lo = v.p[i][2 * p], &hi = v.p[i][2 * p + 1];
            pf[p] = pack_bf16(lo, hi);
            lo = bf16_rest(lo, bf16_lo(pf[p]));
            hi = bf16_rest(hi, bf16_hi(pf[p]));
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[i][t] = mfma(pf, xf[t], acc[i][t]);
        }
      }
    };
    constexpr int kStride = kWgradWaves * 32;
    Step u, v;
    int m = wave * 32;
    if (m < rows) load(u, m);
    while (m < rows) {
      if (m + kStride < rows) load(v, m + kStride);
      multiply(u);
      m += kStride;
      if (m >= rows) break;
      if (m + kStride < rows) load(u, m + kStride);
      multiply(v);
      m += kStride;
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
      const int rr = r0 + i * 16 + pr, cl = c0 + cc;
      if (rr >= a.r || cl >= C) continue;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWgradWaves; ++w) s += s_red[w][pr][cc];
      a.out[side][side ? ((long)g * C + cl) * a.r + rr : ((long)g * a.r + rr) * C + cl] = s;
    }
  }
}

// B [G, N, r] -> [G, r, N], which makes dy B the same product as x A^T. A thread turns 8
// columns of 8 ranks in registers: 16-byte reads and writes.
__global__ __launch_bounds__(256) void lora_transpose_kernel(const uint16_t* in, uint16_t* out, int N,
                                                             int r, int G) {
  const int nb = N / 8, rb = r / 8;
  const long i = blockIdx.x * 256L + threadIdx.x;
  if (i >= (long)G * rb * nb) return;
  const int b = (int)(i % nb);
  const long gr = i / nb;
  const int k = (int)(gr % rb);
  const long g = gr / rb;
  u32x4 v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = load8(in + (g * N + b * 8 + j) * r + k * 8);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    Half8 o;
#pragma unroll
    for (int p = 0; p < 4; ++p)
      o.w[p] = __builtin_amdgcn_perm(v[2 * p + 1][j >> 1], v[2 * p][j >> 1],
                                     (j & 1) ? 0x07060302u : 0x05040100u);
    *reinterpret_cast<Half8*>(out + (g * r + k * 8 + j) * N + b * 8) = o;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

namespace {

constexpr int kDirectRows = 1024;       // up to this many rows a block finds its tile by itself
constexpr int kFusedBytes = 512 << 10;  // largest first matrix of the one-launch form
constexpr int kFusedRank = 64;          // and its largest rank (registers)

struct Plan {
  int mt, nt, rt, tiles;     // tile rows / 16, rank / 16 rounded up, tile rows, most tiles
  int busy;                  // tiles that can hold rows, for the grids' second axis
  bool table;                // a sort and a tile table come first
  bool fused;                // both products in one launch
};

// Tile rows from the mean number of rows an adapter has: 32 rows share one read of the
// adapter's matrices, 16 waste less where adapters have few rows. Accumulators bound
// mt * nt to 8.
Plan plan_tiles(int M, int G, int K, int r, bool backward) {
  Plan p;
  p.nt = r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8;
  p.table = backward || M > kDirectRows;
  p.fused = !p.table && r <= kFusedRank && (long)r * K * 2 <= kFusedBytes;
  const int mean = M / std::max(1, std::min(G, M));
  p.mt = p.fused ? 1 : std::min(mean >= 24 ? 2 : 1, 8 / p.nt);
  p.rt = p.mt * 16;
  const int most = M / p.rt + std::min(G + 1, M);
  p.tiles = p.table ? (most + 7) / 8 * 8 : M;  // the table is dealt out over 8 XCDs
  p.busy = std::max(1, std::min(most, M));
  return p;
}

// Splits of the reduction axis: enough blocks to fill the card, at least one step for each
// wave of a block, at most 16 partial sums to add up again.
int plan_splits(const Plan& p, int K) {
  const int steps = (K + kKStep - 1) / kKStep;
  return std::max(1, std::min({(512 + p.busy - 1) / p.busy, (steps + kShrinkWaves - 1) / kShrinkWaves, 16}));
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

struct Space {
  size_t sorted, off, counts, tile, part, dz, bt, total;
};

Space plan_space(int M, int G, int K, int N, int r, bool backward) {
  Space s{};
  const Plan p = plan_tiles(M, G, K, r, backward);
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
    s.tile = take((size_t)p.tiles * sizeof(SortTile));
  }
  if (!p.fused) s.part = take((size_t)plan_splits(p, backward ? N : K) * M * r * 4);
  if (backward) {
    s.dz = take((size_t)M * r * 4);
    s.bt = take((size_t)G * r * N * 2);
  }
  s.total = at;
  return s;
}

hipError_t make_tiles(const int32_t* ids, int M, int G, const Plan& p, const Space& sp, char* scratch,
                      Tiles* t, hipStream_t s) {
  *t = Tiles{ids, M, G, nullptr, nullptr};
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
  g.tile = reinterpret_cast<SortTile*>(scratch + sp.tile);
  t->sorted = g.sorted;
  t->table = g.tile;
  return launch_sort(g, s);
}

hipError_t shrink(const Plan& p, const ShrinkArgs& a, hipStream_t s) {
  const dim3 grid(p.tiles, a.splits), block(kShrinkWaves * kWave);
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
#undef HMOE_SHRINK
  return hipGetLastError();
}

// MFMA steps of 32 ranks (0: both parts of z in one)
int z_steps(int r) { return r <= 16 ? 0 : (r + 31) / 32; }

template <bool TR>
hipError_t expand(const Plan& p, ExpandArgs a, hipStream_t s) {
  const int groups = (a.c.N + 63) / 64;
  // columns a block: a multiple of its four waves' 64, as wide as still leaves about 1024
  // blocks, so that few blocks add up z's splits again
  const int want = std::max(1, (1024 + p.busy - 1) / p.busy);
  const int rounds = std::max(1, (groups + want * kExpandWaves - 1) / (want * kExpandWaves));
  a.col_groups = rounds * kExpandWaves;
  const dim3 grid(p.tiles, (groups + a.col_groups - 1) / a.col_groups), block(kExpandWaves * kWave);
  const int ks = z_steps(a.c.r);
#define HMOE_EXPAND(MT, KS)                                                         \
  if (p.mt == MT && ks == KS)                                                       \
  hipLaunchKernelGGL((lora_expand_kernel<MT, KS, TR>), grid, block, 0, s, a)
  HMOE_EXPAND(1, 0);
  HMOE_EXPAND(2, 0);
  HMOE_EXPAND(1, 1);
  HMOE_EXPAND(2, 1);
  HMOE_EXPAND(1, 2);
  HMOE_EXPAND(2, 2);
  HMOE_EXPAND(1, 3);
  HMOE_EXPAND(1, 4);
#undef HMOE_EXPAND
  return hipGetLastError();
}

hipError_t fused(const Plan& p, FusedArgs a, hipStream_t s) {
  const int groups = (a.c.N + 63) / 64;
  // columns a block: a multiple of its sixteen waves' 64, about 256 blocks in all
  const int want = std::max(1, 256 / p.busy);
  const int rounds = std::max(1, (groups + want * kFusedWaves - 1) / (want * kFusedWaves));
  a.col_groups = rounds * kFusedWaves;
  const dim3 grid(p.tiles, (groups + a.col_groups - 1) / a.col_groups), block(kFusedWaves * kWave);
  switch (z_steps(a.c.r)) {
    case 0: hipLaunchKernelGGL((lora_fused_kernel<1, 0>), grid, block, 0, s, a); break;
    case 1: hipLaunchKernelGGL((lora_fused_kernel<2, 1>), grid, block, 0, s, a); break;
    default: hipLaunchKernelGGL((lora_fused_kernel<4, 2>), grid, block, 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace

void lora_scratch(int M, int G, int K, int N, int r, size_t* forward, size_t* backward) {
  if (forward) *forward = plan_space(M, G, K, N, r, false).total;
  if (backward) *backward = plan_space(M, G, K, N, r, true).total;
}

hipError_t launch_lora(const Lora& l, void* scratch, hipStream_t s) {
  char* b = static_cast<char*>(scratch);
  const Plan p = plan_tiles(l.M, l.G, l.K, l.r, false);
  const ColumnArgs c{l.r, l.N, l.B, l.base, l.bs, l.y, l.ys};
  if (p.fused)
    return fused(p, FusedArgs{Tiles{l.ids, l.M, l.G, nullptr, nullptr}, l.x, l.xs, l.A, l.K, l.scale, l.z,
                              0, c}, s);
  const Space sp = plan_space(l.M, l.G, l.K, l.N, l.r, false);
  Tiles t;
  hipError_t err = make_tiles(l.ids, l.M, l.G, p, sp, b, &t, s);
  if (err != hipSuccess) return err;
  const int splits = plan_splits(p, l.K);
  float* part = reinterpret_cast<float*>(b + sp.part);
  err = shrink(p, ShrinkArgs{t, l.x, l.xs, l.A, l.K, l.r, splits, part}, s);
  if (err != hipSuccess) return err;
  return expand<false>(p, ExpandArgs{t, part, splits, l.scale, l.z, false, 0, c}, s);
}

hipError_t launch_lora_backward(const LoraGrad& l, void* scratch, hipStream_t s) {
  char* b = static_cast<char*>(scratch);
  const Plan p = plan_tiles(l.M, l.G, l.K, l.r, true);
  const Space sp = plan_space(l.M, l.G, l.K, l.N, l.r, true);
  Tiles t;
  hipError_t err = make_tiles(l.ids, l.M, l.G, p, sp, b, &t, s);
  if (err != hipSuccess) return err;
  float* dz = reinterpret_cast<float*>(b + sp.dz);
  if (l.M > 0) {
    uint16_t* Bt = reinterpret_cast<uint16_t*>(b + sp.bt);
    const long blocks = ((long)l.G * (l.r / 8) * (l.N / 8) + 255) / 256;
    hipLaunchKernelGGL(lora_transpose_kernel, dim3((unsigned)blocks), dim3(256), 0, s, l.B, Bt, l.N, l.r,
                       l.G);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    const int splits = plan_splits(p, l.N);
    float* part = reinterpret_cast<float*>(b + sp.part);
    err = shrink(p, ShrinkArgs{t, l.dy, l.dys, Bt, l.N, l.r, splits, part}, s);
    if (err != hipSuccess) return err;
    const ColumnArgs c{l.r, l.K, l.A, l.dbase, l.dbs, l.dx, l.dxs};
    err = expand<true>(p, ExpandArgs{t, part, splits, l.scale, dz, true, 0, c}, s);
    if (err != hipSuccess) return err;
  }
  const int32_t* off = reinterpret_cast<const int32_t*>(b + sp.off);
  WgradArgs w{t.sorted, off, l.r, l.scale, {dz, l.z}, {l.x, l.dy}, {l.xs, l.dys}, {l.K, l.N},
              {(l.K + 63) / 64, (l.N + 63) / 64}, {l.dA, l.dB}};
  const dim3 grid(w.blocks[0] + w.blocks[1], l.G, p.nt == 8 ? 2 : 1), block(kWgradThreads);
  switch (p.nt) {
    case 1: hipLaunchKernelGGL(lora_wgrad_kernel<1>, grid, block, 0, s, w); break;
    case 2: hipLaunchKernelGGL(lora_wgrad_kernel<2>, grid, block, 0, s, w); break;
    default: hipLaunchKernelGGL(lora_wgrad_kernel<4>, grid, block, 0, s, w); break;
  }
  return hipGetLastError();
}

}  // namespace hmoe
