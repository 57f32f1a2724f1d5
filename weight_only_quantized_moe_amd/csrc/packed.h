// Matrices of 4-bit weights with group scales as MFMA operands (gfx950), shared by the kernels of
// moe_linear and moe_tokens.
//
//   W[n, k] = e2m1(q) * e4m3(s[n, k / 16]) * g        NVFP4
//             e2m1(q) * 2^(s[n, k / 32] - 127)        MXFP4
//             (q - z[n, k / G]) * s[n, k / G]         INT4, G = 32, 64 or 128
//
// A wave takes steps of 16 rows of W and 128 columns. Lane l loads 16 bytes of row l & 15, the 32
// codes of column block l >> 4: 64 bytes of a row lie in one load. The MFMA wants the lanes of a
// row to hold 8 columns each of the same 32, so four dwords change places among the four lanes of
// a row (v_permlane32_swap, v_permlane16_swap): then dword t of every lane belongs to column block
// t, and a group scale is one factor of the product's column n = l & 15.
//
// The codes go into the product as exact 16-bit numbers and the sums are fp32:
//   E2M1 is exact in both 16-bit types. MXFP4 scales: bf16 has every exponent and the conversion of the
//   codes applies them; fp16 has not, and they multiply the fp32 sum of their 32 columns. E4M3 times E2M1
//   has 6 significant bits and is formed before the product (its groups of 16 would halve the MFMA's depth).
//   INT4 becomes 16 + q by one shift and one and-or (the code lands in the low bits of a
//   mantissa whose unit is 1), and a second product with the constant -(16 + z) into the same sum
//   takes the offset out again: both are exact, and the matrix cores have the time. Infinite
//   activations therefore give NaN.
#pragma once

#include <type_traits>

#include "device_common.h"
#include "hmoe_internal.h"

namespace hmoe {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

// the formats as the kernels know them (INT4 by its group), and the 16-bit types
enum : int { kNv = 0, kMx = 1, kI32 = 2, kI64 = 3, kI128 = 4 };
enum : int { kBf = 0, kHf = 1 };
constexpr bool is_int4(int f) { return f >= kI32; }
constexpr int group_of(int f) { return f == kNv ? 16 : f == kMx || f == kI32 ? 32 : f == kI64 ? 64 : 128; }
// bytes of a group's scale
constexpr int scale_bytes(int f) { return is_int4(f) ? 2 : 1; }

// memory of any alignment: rows of x need only element alignment, rows of scales only byte's
struct __attribute__((packed, aligned(2))) Any16 { uint32_t w[4]; };
struct __attribute__((packed, aligned(1))) Any8 { uint32_t w[2]; };
struct __attribute__((packed, aligned(1))) Any4 { uint32_t w; };
struct __attribute__((packed, aligned(1))) Any2 { uint16_t w; };

__device__ __forceinline__ u32x4 load16(const uint16_t* p) {
  const Any16 h = *reinterpret_cast<const Any16*>(p);
  return u32x4{h.w[0], h.w[1], h.w[2], h.w[3]};
}

template <int X>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (X == kBf)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <int X>
__device__ __forceinline__ float to_f32(uint32_t bits) {
  if constexpr (X == kBf) return __uint_as_float(bits << 16);
  else return fp16_to_f32(bits);
}
template <int X>
__device__ __forceinline__ uint16_t from_f32(float v) {
  return (uint16_t)(X == kBf ? pack_bf16(v, v) : pack_f16(v, v));
}

// E8M0 byte -> fp32; 255 is NaN
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float((b << 23) | (((b + 1u) & 255u) < 2u ? 0x00400000u : 0u));
}

// dword t of the lane of column block b becomes dword b of block t (see above)
__device__ __forceinline__ void turn4(u32x4& v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  v = u32x4{(uint32_t)c[0], (uint32_t)c[1], (uint32_t)d[0], (uint32_t)d[1]};
}

// 8 INT4 codes -> 16 + q, in the order of int4_order
template <int X>
__device__ __forceinline__ u32x4 int4_operand(uint32_t w) {
  if constexpr (X == kBf) {
    constexpr uint32_t m = 0x00780078u, o = 0x41804180u;
    return u32x4{((w << 3) & m) | o, ((w >> 1) & m) | o, ((w >> 5) & m) | o, ((w >> 9) & m) | o};
  } else {
    constexpr uint32_t m = 0x03C003C0u, o = 0x4C004C00u;
    return u32x4{((w << 6) & m) | o, ((w << 2) & m) | o, ((w >> 2) & m) | o, ((w >> 6) & m) | o};
  }
}
// -(16 + z) in every element
template <int X>
__device__ __forceinline__ u32x4 int4_offset(uint32_t z) {
  z &= 15u;
  z |= z << 16;
  const uint32_t v = X == kBf ? (z << 3) | 0xC180C180u : (z << 6) | 0xCC00CC00u;
  return u32x4{v, v, v, v};
}
// eight 16-bit values in the order in which int4_operand holds its codes: 0 4 1 5 2 6 3 7
__device__ __forceinline__ u32x4 int4_order(u32x4 v) {
  return u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
               __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
}

// 8 E2M1 codes
template <int X>
__device__ __forceinline__ u32x4 e2m1_operand(uint32_t w) {
  if constexpr (X == kBf)
    return u32x4{e2m1x2_bf16<0>(w, 1.f), e2m1x2_bf16<1>(w, 1.f), e2m1x2_bf16<2>(w, 1.f), e2m1x2_bf16<3>(w, 1.f)};
  else
    return u32x4{e2m1x2_f16<0>(w, 1.f), e2m1x2_f16<1>(w, 1.f), e2m1x2_f16<2>(w, 1.f), e2m1x2_f16<3>(w, 1.f)};
}
// 8 E2M1 codes times an E4M3 scale (exact)
template <int X>
__device__ __forceinline__ u32x4 nvfp4_operand(uint32_t w, float s) {
  if constexpr (X == kBf) {
    const f32x2 a = e2m1x2_f32<0>(w, 1.f), b = e2m1x2_f32<1>(w, 1.f);
    const f32x2 c = e2m1x2_f32<2>(w, 1.f), d = e2m1x2_f32<3>(w, 1.f);
    return u32x4{pack_bf16(a[0] * s, a[1] * s), pack_bf16(b[0] * s, b[1] * s),
                 pack_bf16(c[0] * s, c[1] * s), pack_bf16(d[0] * s, d[1] * s)};
  } else {
    const f16x2 f = {(_Float16)s, (_Float16)s};
    auto times = [&](uint32_t v) {
      return __builtin_bit_cast(uint32_t, (f16x2)(__builtin_bit_cast(f16x2, v) * f));
    };
    return u32x4{times(e2m1x2_f16<0>(w, 1.f)), times(e2m1x2_f16<1>(w, 1.f)), times(e2m1x2_f16<2>(w, 1.f)),
                 times(e2m1x2_f16<3>(w, 1.f))};
  }
}

// What a lane holds of one row's 128 columns: codes, scales, zero points.
template <int F>
struct Codes {
  u32x4 q;
  uint32_t s[2];   // NV: 8 bytes; MX: 4 bytes; INT4: 4, 2 or 1 halves
  uint32_t z;      // INT4: 4, 2 or 1 bytes
};

// One row of W as the lane addresses it.
struct PackedRow {
  const uint8_t* q;   // of the lane's column block
  const uint8_t* s;
  const uint8_t* z;   // null: 8 everywhere
};

template <int F>
__device__ __forceinline__ PackedRow packed_row(const Packed& w, long row, int K, int lane) {
  constexpr int G = group_of(F);
  const long groups = row * (K / G);
  return PackedRow{w.q + row * (K / 2) + (lane >> 4) * 16, w.s + groups * scale_bytes(F),
                   is_int4(F) && w.z ? w.z + groups : nullptr};
}

// Loads step `step`; full: all 128 columns lie inside K, else the columns past K are stand-ins
// from inside the row (codes that the products leave out, and the last group's scale).
template <int F, bool FULL>
__device__ __forceinline__ void load_codes(Codes<F>& c, const PackedRow& r, int step, int K, int lane) {
  constexpr int G = group_of(F), NG = 128 / G;
  const long at = (long)step * 64;
  const uint8_t* p = r.q + at;
  if constexpr (!FULL)
    if (step * 128 + (lane >> 4) * 32 >= K) p -= (lane >> 4) * 16;
  c.q = *reinterpret_cast<const u32x4*>(p);
  c.s[0] = c.s[1] = 0u;
  c.z = 0x08080808u;
  const uint8_t* s = r.s + (long)step * (NG * scale_bytes(F));
  const uint8_t* z = r.z ? r.z + (long)step * NG : nullptr;
  if constexpr (FULL) {
    if constexpr (NG * scale_bytes(F) == 8) {
      const Any8 v = *reinterpret_cast<const Any8*>(s);
      c.s[0] = v.w[0], c.s[1] = v.w[1];
    } else if constexpr (NG * scale_bytes(F) == 4) {
      c.s[0] = reinterpret_cast<const Any4*>(s)->w;
    } else {
      c.s[0] = *reinterpret_cast<const uint16_t*>(s);
    }
    if constexpr (is_int4(F)) {
      if (z) {
        if constexpr (NG == 4) c.z = reinterpret_cast<const Any4*>(z)->w;
        else if constexpr (NG == 2) c.z = reinterpret_cast<const Any2*>(z)->w;
        else c.z = *z;
      }
    }
  } else {
    const int left = K / G - step * NG;   // groups of this row from here on
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = i < left ? i : left - 1;
      if constexpr (is_int4(F)) {
        c.s[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(s)[g] << (16 * (i & 1));
        if (z) c.z = (c.z & ~(255u << (8 * i))) | ((uint32_t)z[g] << (8 * i));
      } else {
        c.s[i >> 2] |= (uint32_t)s[g] << (8 * (i & 3));
      }
    }
  }
}

// the fp32 scale of column block T (INT4 and MXFP4); S: the 16-bit type of INT4 scales
template <int F, int S, int T>
__device__ __forceinline__ float block_scale(const Codes<F>& c) {
  if constexpr (F == kMx) return e8m0_value((c.s[0] >> (8 * T)) & 255u);
  constexpr int i = T * 32 / group_of(F);
  return to_f32<S>((c.s[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
}

// acc[t] += the products of column blocks T to T + N - 1, one group or part of one, with the activations
// a[t] (in int4_order for INT4) of 16 rows each, which may come as PARTS that add up to them. X: type
// of the activations.
template <int F, int X, int S, int T, int N, int NT, int PARTS>
__device__ __forceinline__ void block_product(f32x4 (&acc)[NT], const Codes<F>& c, const u32x4 (&a)[PARTS][4][NT]) {
  if constexpr (F == kNv) {
    static_assert(N == 1, "two groups a block");
    // the dword's 8 columns lie in group 2 T + (lane >= 32)
    const uint32_t v = c.s[T >> 1] >> (16 * (T & 1));
    const float s = e4m3_to_f32<0>(threadIdx.x & 32 ? v >> 8 : v);
    const u32x4 b = nvfp4_operand<X>(c.q[T], s);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < PARTS; ++i) acc[t] = mfma16<X>(a[i][T][t], b, acc[t]);
  } else if constexpr (F == kMx && X == kBf) {
    // bf16 has every exponent: the conversion applies the scale (the mantissa bit makes byte 0
    // 2^-127 and 255 NaN, and is not applied otherwise)
    static_assert(N == 1, "a group a block");
    const uint32_t v = T == 3 ? c.s[0] >> 1 : c.s[0] << (23 - 8 * T);
    const float s = __uint_as_float((v & 0x7F800000u) | 0x00400000u);
    const uint32_t w = c.q[T];
    const u32x4 b{e2m1x2_bf16<0>(w, s), e2m1x2_bf16<1>(w, s), e2m1x2_bf16<2>(w, s), e2m1x2_bf16<3>(w, s)};
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < PARTS; ++i) acc[t] = mfma16<X>(a[i][T][t], b, acc[t]);
  } else {
    const float s = block_scale<F, S, T>(c);
    u32x4 o;
    if constexpr (is_int4(F)) o = int4_offset<X>(c.z >> (8 * (T * 32 / group_of(F))));
    f32x4 p[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) p[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const u32x4 b = F == kMx ? e2m1_operand<X>(c.q[T + n]) : int4_operand<X>(c.q[T + n]);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
          if constexpr (is_int4(F)) p[t] = mfma16<X>(a[i][T + n][t], o, p[t]);
          p[t] = mfma16<X>(a[i][T + n][t], b, p[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(s, p[t][i], acc[t][i]);
  }
}

// The four column blocks of a step against 16 NT rows of activations in registers; blocks: those
// inside K (four unless the step is a row's last). The codes' dwords are turned in place.
template <int F, int X, int S, int NT>
__device__ __forceinline__ void step_product(f32x4 (&acc)[NT], Codes<F>& c, const u32x4 (&a)[1][4][NT], int blocks) {
  turn4(c.q);
  constexpr int N = group_of(F) <= 32 ? 1 : group_of(F) / 32;   // blocks of a group
  block_product<F, X, S, 0, N, NT, 1>(acc, c, a);
  if constexpr (N == 1)
    if (blocks > 1) block_product<F, X, S, 1, N, NT, 1>(acc, c, a);
  if constexpr (N <= 2)
    if (blocks > 2) block_product<F, X, S, 2, N, NT, 1>(acc, c, a);
  if constexpr (N == 1)
    if (blocks > 3) block_product<F, X, S, 3, N, NT, 1>(acc, c, a);
}

// Eight fp32 values as three bf16 operands whose sum they are (24 bits, eight a part), in the order the
// format takes. What is left of an infinity is nothing, but for INT4, whose offset makes it NaN in any case;
// infinite: there may be one.
template <int F>
__device__ __forceinline__ void f32_operands(u32x4 (&a)[3], const f32x4 (&h)[2], bool infinite) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = is_int4(F) ? h[i & 1][i >> 1] : h[i >> 2][i & 3];
#pragma unroll
  for (int part = 0; part < 3; ++part)
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint32_t lo = __float_as_uint(v[i]), hi = __float_as_uint(v[i + 1]);
      a[part][i >> 1] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);   // the high halves
      v[i] -= __uint_as_float(lo & 0xFFFF0000u);
      v[i + 1] -= __uint_as_float(hi & 0xFFFF0000u);
    }
  if (!is_int4(F) && infinite)   // (the same for all waves, and rare)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = a[0][i];
      const uint32_t keep = ((w & 0x7FFFu) == 0x7F80u ? 0u : 0xFFFFu) | ((w & 0x7FFF0000u) == 0x7F800000u ? 0u : 0xFFFF0000u);
      a[1][i] &= keep;
      a[2][i] &= keep;
    }
}

// The four column blocks of a step of R tiles against 16 rows of fp32 values: as step_product, block by
// block, so that a block's parts are made once for all tiles. INT4's offsets meet the sum of the block's
// values, which is the same for all tiles too. S: the 16-bit type of INT4 scales.
template <int F, int S, int T, int R>
__device__ __forceinline__ void blocks_product_f32(f32x4 (&acc)[R][1], const Codes<F> (&c)[R], const f32x4 (&h)[4][2],
                                                   int blocks, bool infinite) {
  if constexpr (T < 4) {
    if (blocks <= T) return;
    u32x4 parts[3];
    f32_operands<F>(parts, h[T], infinite);
    if constexpr (is_int4(F)) {
      f32x4 sum = {0.f, 0.f, 0.f, 0.f};
      const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
      for (int i = 0; i < 3; ++i) sum = mfma16<kBf>(parts[i], ones, sum);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float s = block_scale<F, S, T>(c[r]);
        const float z = (float)(16u + ((c[r].z >> (8 * (T * 32 / group_of(F)))) & 15u));
        const u32x4 b = int4_operand<kBf>(c[r].q[T]);
        f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 3; ++i) p = mfma16<kBf>(parts[i], b, p);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][0][i] = fmaf(s, fmaf(-z, sum[i], p[i]), acc[r][0][i]);
      }
    } else {
      u32x4 a[3][4][1];
#pragma unroll
      for (int i = 0; i < 3; ++i) a[i][T][0] = parts[i];
#pragma unroll
      for (int r = 0; r < R; ++r) block_product<F, kBf, S, T, 1, 1, 3>(acc[r], c[r], a);
    }
    blocks_product_f32<F, S, T + 1, R>(acc, c, h, blocks, infinite);
  }
}
template <int F, int S, int R>
__device__ __forceinline__ void step_product_f32(f32x4 (&acc)[R][1], Codes<F> (&c)[R], const f32x4 (&h)[4][2], int blocks,
                                                 bool infinite) {
#pragma unroll
  for (int r = 0; r < R; ++r) turn4(c[r].q);
  blocks_product_f32<F, S, 0, R>(acc, c, h, blocks, infinite);
}

// load_codes where only the last step of a row can be partial (ALL: none is)
template <int F, bool ALL>
__device__ __forceinline__ void load_step(Codes<F>& c, const PackedRow& r, int step, int K, int lane) {
  if constexpr (ALL) {
    load_codes<F, true>(c, r, step, K, lane);
  } else {
    if ((step + 1) * 128 <= K) load_codes<F, true>(c, r, step, K, lane);
    else load_codes<F, false>(c, r, step, K, lane);
  }
}
template <bool ALL>
__device__ __forceinline__ int step_blocks(int step, int K) {
  return ALL ? 4 : min(4, (K - step * 128) / 32);
}

// A step of a row of activations, in the order the format takes; p points at the lane's 8 columns of
// the step's first block
template <int F, bool ALL>
__device__ __forceinline__ void load_rows(u32x4 (&a)[1][4][1], const uint16_t* p, int step, int K) {
  const int last = step_blocks<ALL>(step, K) - 1;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    a[0][b][0] = load16(p + (long)step * 128 + min(b, last) * 32);
    if constexpr (is_int4(F)) a[0][b][0] = int4_order(a[0][b][0]);
  }
}

// ------------------------------------------------------------------------------------------
// Pairs of steps: rows of at least 256 columns
// ------------------------------------------------------------------------------------------
// A pair of steps covers whole 128-byte lines of codes: one load takes rows 0 to 7 of the tile, the
// other rows 8 to 15, and two lanes eight apart exchange what is the other's. The scales of a wave's
// steps come in one load a row: each of the row's four lanes takes Q steps, and a step's scales are
// spread from their lane when they are needed. On MI355X the experts' first products of eight
// tokens (256 experts, 6144 to 2048, MXFP4) take 181 us with a load of 64 bytes a row and a load of
// scales a step, 143 without the scales (wrong results), 124 with whole lines as well.
template <int F>
constexpr int step_scale_bytes() { return 128 / group_of(F) * scale_bytes(F); }   // 8, 4 or 2
template <int F>
constexpr int step_zero_bytes() { return is_int4(F) ? 128 / group_of(F) : 0; }

struct PairCodes {
  u32x4 a, b;   // as loaded; after split_pair, the first and second step's
};

// The lane's places in a tile of 16 rows, as 32-bit offsets from the tile's first row, so that a load
// takes a scalar base and one register: of its piece of rows 0 to 7 (lo) and 8 to 15 (hi), and of its
// row's scales and zero points. Rows at and past `rows` are stand-ins. Where K is not a multiple of 256
// (EXACT false), the last pair is partial: pieces past K are stand-ins too (lo_end, hi_end), whose
// columns meet zeros of x, and scales that would reach past the row are loaded from further in front
// and shifted, zeros coming in.
template <bool EXACT>
struct TileLane {
  uint32_t lo, hi, s, z;
};
template <>
struct TileLane<false> {
  uint32_t lo, hi, s, z, lo_end, hi_end;
  int s_shift, z_shift;    // bits
};

template <bool EXACT>
__device__ __forceinline__ void load_pair(PairCodes& c, const uint8_t* tile, const TileLane<EXACT>& at, bool end) {
  uint32_t lo = at.lo, hi = at.hi;
  if constexpr (!EXACT) {
    lo = end ? at.lo_end : lo;
    hi = end ? at.hi_end : hi;
  }
  c.a = *reinterpret_cast<const u32x4*>(tile + lo);
  c.b = *reinterpret_cast<const u32x4*>(tile + hi);
}
__device__ __forceinline__ void split_pair(PairCodes& c) {
  const bool up = threadIdx.x & 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = c.a[i], b = c.b[i], give = up ? a : b;
    const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0x128, 0xF, 0xF, true);   // row_ror:8
    c.a[i] = up ? got : a;
    c.b[i] = up ? b : got;
  }
}

// The scales and zero points of STEPS steps of the lane's row, Q of them in this lane.
template <int F, int STEPS>
struct StepScales {
  static constexpr int Q = STEPS > 4 ? 2 : 1;
  static constexpr int kBytes = Q * step_scale_bytes<F>(), kZeros = Q * step_zero_bytes<F>();
  uint32_t s[(kBytes + 3) / 4 > 1 ? (kBytes + 3) / 4 : 2], z[kZeros > 4 ? 2 : 1];
};

template <int N>
__device__ __forceinline__ void load_bytes(uint32_t* out, const uint8_t* p) {
  if constexpr (N == 16) {
    const Any8 v = *reinterpret_cast<const Any8*>(p), w = *reinterpret_cast<const Any8*>(p + 8);
    out[0] = v.w[0], out[1] = v.w[1], out[2] = w.w[0], out[3] = w.w[1];
  } else if constexpr (N == 8) {
    const Any8 v = *reinterpret_cast<const Any8*>(p);
    out[0] = v.w[0], out[1] = v.w[1];
  } else if constexpr (N == 4) {
    out[0] = reinterpret_cast<const Any4*>(p)->w;
  } else if constexpr (N == 2) {
    out[0] = reinterpret_cast<const Any2*>(p)->w;
  } else {
    out[0] = *p;
  }
}

// first: the first of the wave's steps (in pairs, so even)
template <int F, int STEPS, bool EXACT>
__device__ __forceinline__ TileLane<EXACT> tile_lane(int lane, int K, int rows, int first) {
  using T = StepScales<F, STEPS>;
  constexpr int Q = T::Q;
  const int place = (lane >> 4) + ((lane >> 3) & 1) * 4, half = K / 2, groups = K / group_of(F);
  const int step = first + min(lane >> 4, STEPS / Q - 1) * Q, row = min(lane & 15, rows - 1);
  const int lo = min(lane & 7, rows - 1) * half, hi = min(8 + (lane & 7), rows - 1) * half;
  const int s = step * step_scale_bytes<F>(), z = step * step_zero_bytes<F>();
  TileLane<EXACT> t;
  t.lo = lo + place * 16;
  t.hi = hi + place * 16;
  t.s = row * groups * scale_bytes(F) + s;
  t.z = row * groups + z;
  if constexpr (!EXACT) {
    const bool inside = K / 256 * 128 + place * 16 < half;
    t.lo_end = lo + (inside ? place * 16 : 0);
    t.hi_end = hi + (inside ? place * 16 : 0);
    static_assert(T::kBytes <= 8 && T::kZeros <= 8, "partial pairs: a lane loads one step's scales");
    // how far the load reaches past the row's end
    t.s_shift = 8 * max(0, s + T::kBytes - groups * scale_bytes(F));
    t.z_shift = 8 * max(0, z + T::kZeros - groups);
  }
  return t;
}

// N bytes (at most 8) at p that reach `shift` bits past what may be read: those come as zeros
template <int N>
__device__ __forceinline__ void load_shifted(uint32_t* out, const uint8_t* p, int shift) {
  uint32_t w[2] = {0u, 0u};
  load_bytes<N>(w, p - shift / 8);
  uint64_t v = (uint64_t)w[1] << 32 | w[0];
  v = shift < 8 * N ? v >> shift : 0ull;
  out[0] = (uint32_t)v;
  if constexpr (N == 8) out[1] = (uint32_t)(v >> 32);
}

// s, z: the tile's first row; z null: 8 everywhere (the load then takes scales instead, which are no
// fewer bytes, so that no load stands behind a condition)
template <int F, int STEPS, bool EXACT>
__device__ __forceinline__ void load_scales(StepScales<F, STEPS>& v, const uint8_t* s, const uint8_t* z,
                                            const TileLane<EXACT>& at) {
  using T = StepScales<F, STEPS>;
  if constexpr (EXACT) {
    load_bytes<T::kBytes>(v.s, s + at.s);
    if constexpr (is_int4(F)) load_bytes<T::kZeros>(v.z, (z ? z : s) + at.z);
  } else {
    load_shifted<T::kBytes>(v.s, s + at.s, at.s_shift);
    if constexpr (is_int4(F)) load_shifted<T::kZeros>(v.z, (z ? z : s) + at.z, at.z_shift);
  }
}
template <int F, int STEPS>
__device__ __forceinline__ void default_zeros(StepScales<F, STEPS>& v, bool given) {
  if constexpr (is_int4(F)) {
    v.z[0] = given ? v.z[0] : 0x08080808u;
    if constexpr (StepScales<F, STEPS>::kZeros > 4) v.z[1] = given ? v.z[1] : 0x08080808u;
  }
}

// A tile's first row, n rows into the matrix: its codes at a step, its scales and zero points.
struct TileBase {
  const uint8_t* q;
  const uint8_t* s;
  const uint8_t* z;
};
template <int F>
__device__ __forceinline__ TileBase tile_base(const Packed& w, long n, int K, int step) {
  const long groups = n * (K / group_of(F));
  return {w.q + n * (K / 2) + step * 64, w.s + groups * scale_bytes(F), is_int4(F) && w.z ? w.z + groups : nullptr};
}

// the value that lane quarter Q of the row holds, in all four
template <int Q>
__device__ __forceinline__ uint32_t spread(uint32_t v) {
  const uint32_t h = __builtin_amdgcn_permlane32_swap(v, v, false, false)[Q >> 1];
  return __builtin_amdgcn_permlane16_swap(h, h, false, false)[Q & 1];
}

// Step J's scales into c
template <int F, int STEPS, int J>
__device__ __forceinline__ void take_scales(Codes<F>& c, const StepScales<F, STEPS>& v) {
  constexpr int Q = StepScales<F, STEPS>::Q, sub = J % Q, lane4 = J / Q;
  constexpr int bytes = step_scale_bytes<F>(), zeros = step_zero_bytes<F>();
  c.s[1] = 0u;
  if constexpr (bytes == 8) {
    c.s[0] = spread<lane4>(v.s[2 * sub]);
    c.s[1] = spread<lane4>(v.s[2 * sub + 1]);
  } else if constexpr (bytes == 4) {
    c.s[0] = spread<lane4>(v.s[sub]);
  } else {
    c.s[0] = spread<lane4>(v.s[0]) >> (16 * sub);
  }
  c.z = 0u;
  if constexpr (zeros == 4) c.z = spread<lane4>(v.z[sub]);
  else if constexpr (zeros > 0) c.z = spread<lane4>(v.z[0]) >> (8 * zeros * sub);
}

// The same for the first or second step of two, as a loop over them takes it
template <int F>
__device__ __forceinline__ void take_scales_of(Codes<F>& c, const StepScales<F, 2>& v, bool second) {
  auto part = [&](uint32_t x) { return second ? spread<1>(x) : spread<0>(x); };
  c.s[0] = part(v.s[0]);
  c.s[1] = step_scale_bytes<F>() == 8 ? part(v.s[1]) : 0u;
  c.z = is_int4(F) ? part(v.z[0]) : 0u;
}

// Pair P of a wave's PX: both steps' products.
template <int F, int X, int S, int PX, int P>
__device__ __forceinline__ void pair_product(f32x4 (&acc)[1], PairCodes& q, const StepScales<F, 2 * PX>& v,
                                             const u32x4 (&a)[2][1][4][1]) {
  split_pair(q);
  Codes<F> c;
  c.q = q.a;
  take_scales<F, 2 * PX, 2 * P>(c, v);
  step_product<F, X, S, 1>(acc, c, a[0], 4);
  c.q = q.b;
  take_scales<F, 2 * PX, 2 * P + 1>(c, v);
  step_product<F, X, S, 1>(acc, c, a[1], 4);
}

// for (P = 0; P < N; ++P) f(P) with P a constant
template <int N, int P = 0, typename Fn>
__device__ __forceinline__ void each(Fn&& f) {
  if constexpr (P < N) {
    f(std::integral_constant<int, P>{});
    each<N, P + 1>(f);
  }
}

// The wave's share of `pairs` pairs among `waves` waves of PX each: its first pair, and from which on
// they are its own (the last wave starts early rather than reach past the row).
struct PairShare {
  int first, own;
};
__device__ __forceinline__ PairShare pair_share(int wave, int pairs, int PX) {
  return {min(wave * PX, pairs - PX), wave * PX};
}

// load_rows of a step that may lie past K in part or in whole: zeros there
template <int F, bool EXACT>
__device__ __forceinline__ void load_pair_rows(u32x4 (&a)[1][4][1], const uint16_t* p, int step, int K) {
  if constexpr (EXACT) {
    load_rows<F, true>(a, p, step, K);
  } else {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int c = step * 128 + b * 32;
      a[0][b][0] = load16(p + min(c, K - 32)) & (c < K ? ~0u : 0u);
      if constexpr (is_int4(F)) a[0][b][0] = int4_order(a[0][b][0]);
    }
  }
}

}  // namespace hmoe
