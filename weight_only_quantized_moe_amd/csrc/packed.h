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
//   E2M1 is exact in both 16-bit types. MXFP4 scales multiply the fp32 sum of their 32 columns,
//   which holds for every exponent in either type. E4M3 times E2M1 has 6 significant bits and is
//   formed before the product (its groups of 16 would halve the MFMA's depth).
//   INT4 becomes 16 + q by one shift and one and-or (the code lands in the low bits of a
//   mantissa whose unit is 1), and a second product with the constant -(16 + z) into the same sum
//   takes the offset out again: both are exact, and the matrix cores have the time. Infinite
//   activations therefore give NaN.
#pragma once

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

// acc[tt] += the products of column block T with the activations a[tt] (in int4_order for INT4)
// of 16 rows each. X: type of the activations.
template <int F, int X, int S, int T, int NT>
__device__ __forceinline__ void block_product(f32x4 (&acc)[NT], const Codes<F>& c, const u32x4 (&a)[NT], int lane) {
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  const uint32_t w = c.q[T];
  if constexpr (F == kNv) {
    // the dword's 8 columns lie in group 2 T + (lane >= 32)
    const float s = (T & 1) ? ((lane & 32) ? e4m3_to_f32<3>(c.s[T >> 1]) : e4m3_to_f32<2>(c.s[T >> 1]))
                            : ((lane & 32) ? e4m3_to_f32<1>(c.s[T >> 1]) : e4m3_to_f32<0>(c.s[T >> 1]));
    const u32x4 b = nvfp4_operand<X>(w, s);
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = mfma16<X>(a[t], b, acc[t]);
  } else {
    const float s = block_scale<F, S, T>(c);
    u32x4 b, o;
    if constexpr (F == kMx) {
      b = e2m1_operand<X>(w);
    } else {
      b = int4_operand<X>(w);
      o = int4_offset<X>(c.z >> (8 * (T * 32 / group_of(F))));
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 p = zero;
      if constexpr (is_int4(F)) p = mfma16<X>(a[t], o, p);
      p = mfma16<X>(a[t], b, p);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(s, p[i], acc[t][i]);
    }
  }
}

}  // namespace hmoe
