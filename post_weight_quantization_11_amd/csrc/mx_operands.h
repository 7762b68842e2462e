// Operands of the 16-bit matrix instructions from microscaled weights and 16-bit
// activations: conversions, and loads at the ends of rows.
#pragma once

#include "mx.h"

namespace gptq {

// Eight codes (one word) as eight 16-bit values times the scale.
template <int XT> __device__ inline u32x4 widen8(uint32_t w, float s);
template <> __device__ inline u32x4 widen8<GPTQ_F16>(uint32_t w, float s) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3))};
}
template <> __device__ inline u32x4 widen8<GPTQ_BF16>(uint32_t w, float s) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
}

template <int XT> __device__ inline floatx4 mfma16(u32x4 a, u32x4 b, floatx4 c);
template <> __device__ inline floatx4 mfma16<GPTQ_F16>(u32x4 a, u32x4 b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8, a), __builtin_bit_cast(halfx8, b), c, 0, 0,
                                                0);
}
template <> __device__ inline floatx4 mfma16<GPTQ_BF16>(u32x4 a, u32x4 b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

// Float16 holds an e2m1 value times 2^(byte - 127) exactly for bytes 104
// (0.5 * 2^-23, the smallest subnormal) to 140 (6 * 2^13), and the conversion
// makes the NaN byte a NaN.  A unit of columns with any other scale is
// multiplied in bfloat16, which holds every value that float32 holds: X, of 11
// significant bits, is the sum of two bfloat16 numbers (its first 8 bits and
// the rest), so the products stay exact and the unit costs twice the
// instructions.
constexpr uint32_t kF16Lo = 104, kF16Span = 37;
__device__ inline bool f16_exact(uint32_t byte) { return byte - kF16Lo < kF16Span || byte == kMxScaleNan; }

// Eight float16 numbers as bfloat16 sums hi + lo (an infinity has lo = 0, a
// NaN is in lo).
__device__ inline void split8(u32x4 x, u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    uint32_t h2 = 0u, l2 = 0u;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float f = (float)__builtin_bit_cast(_Float16, (uint16_t)(x[d] >> (16 * e)));
      const uint32_t top = __float_as_uint(f) & 0xFFFF0000u;
      const bool inf = (__float_as_uint(f) & 0x7FFFFFFFu) == 0x7F800000u;
      const uint32_t rest = inf ? 0u : __float_as_uint(f - __uint_as_float(top));
      h2 |= e ? top : top >> 16;
      l2 |= e ? rest & 0xFFFF0000u : rest >> 16;
    }
    hi[d] = h2;
    lo[d] = l2;
  }
}

// Guarded loads of a row's last columns (n >= 1).  Where the row is long enough,
// one load that ends at the row's end, shifted down to the columns asked for, so
// that all of them are in flight together; what lies past the end is replaced.
// Eight columns of 16-bit X from column k, zeros past the end.
__device__ inline u32x4 load_x8_tail(const uint16_t* row, int k, int n) {
  if (n >= 8) {
    const int at = min(k, n - 8), s = k - at;
    const u32x4 v = *reinterpret_cast<const u32x4_a2*>(row + at);
    uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
    if (s & 4) {
      lo = hi;
      hi = 0;
    }
    const int bits = 16 * (s & 3);
    lo = lo >> bits | hi << 1 << (63 - bits);
    hi >>= bits;
    if (s >= 8) lo = hi = 0;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
  u32x4 v;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int c = k + 2 * d;
    const uint32_t lo = row[min(c, n - 1)], hi = row[min(c + 1, n - 1)];
    v[d] = (c < n ? lo : 0u) | (c + 1 < n ? hi << 16 : 0u);
  }
  return v;
}
// Four words of codes from word k; codes past column n are 0.
__device__ inline u32x4 load_w4_tail(const uint32_t* row, int k, int n) {
  const int nw = (n + 7) >> 3;
  u32x4 v;
  if (nw >= 4) {
    const int at = min(k, nw - 4), s = k - at;
    const u32x4 l = *reinterpret_cast<const u32x4_a4*>(row + at);
    v[0] = s == 0 ? l[0] : s == 1 ? l[1] : s == 2 ? l[2] : l[3];
    v[1] = s == 0 ? l[1] : s == 1 ? l[2] : l[3];
    v[2] = s == 0 ? l[2] : l[3];
    v[3] = l[3];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = row[min(k + i, nw - 1)];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = n - 8 * (k + i);        // columns that this word holds
    if (left < 8) v[i] &= (1u << (4 * max(left, 0))) - 1u;
  }
  return v;
}
// Scale bytes of four blocks; blocks past the row's end have scale 1.
__device__ inline uint32_t load_scales4(const uint8_t* srow, int blk, int n) {
  const int nb = (n + kMxBlock - 1) >> 5;
  uint32_t v = 0u;
  if (nb >= 4) {
    const int at = min(blk, nb - 4);
    v = *reinterpret_cast<const u32_a1*>(srow + at) >> (8 * min(blk - at, 3));
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i) v |= (uint32_t)srow[min(blk + i, nb - 1)] << (8 * i);
  }
  const int left = nb - blk;                 // blocks there are
  if (left >= 4) return v;
  const uint32_t there = (1u << (8 * max(left, 0))) - 1u;
  return (v & there) | (kMxScaleOne * 0x01010101u & ~there);
}

// 4 x 4 transpose over the lane quarters: register j of quarter q becomes
// register q of quarter j, i.e. word q of block j.
__device__ inline u32x4 transpose_quarters(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v[0], v[1], false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(v[2], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  return u32x4{c[0], d[0], c[1], d[1]};
}

// Whether four scale bytes are exact in float16, tested for 104 .. 135 only:
// the result is 0 if and only if each byte - 104 is below 32 (a byte below 104
// sets its own top bits before it can borrow from the next).
__device__ inline uint32_t f16_inexact4(uint32_t bytes) { return (bytes - 0x68686868u) & 0xE0E0E0E0u; }

}  // namespace gptq
