// Device helpers shared by the 8-bit float kernels.
//
// Format: e4m3 codes (bit 7 the sign, bits 3-6 the exponent with bias 7, bits
// 0-2 the mantissa; 448 the largest value, 0x7F and 0xFF NaN, no infinities),
// one byte each, and float32 scales for blocks of 128 columns: of one row
// (activations) or of 128 rows (weights).
#pragma once

#include "mx.h"

namespace gptq {

constexpr int kFp8Block = 128;               // columns (and rows of a weight block) that share a scale
constexpr float kFp8Max = 448.f;
constexpr int64_t kFp8MaxCols = 1 << 20;     // keeps in-row offsets far below 32 bits

// Eight codes (a half of four words) as bfloat16 numbers, which hold them exactly.
__device__ inline bf16x8 fp8_widen8(u32x4 v, int half) {
  const uint32_t lo = v[2 * half], hi = v[2 * half + 1];
  return __builtin_bit_cast(bf16x8,
                            u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false)),
                                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true)),
                                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false)),
                                  __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true))});
}

// Sixteen codes of a row from column k, zeros past column n (n >= 1, k < n or
// beyond): where the row is long enough one load that ends at the row's end,
// shifted down to the columns asked for.
__device__ inline u32x4 fp8_load16_tail(const uint8_t* row, int k, int n) {
  if (n >= 16) {
    const int at = min(k, n - 16), s = k - at;
    const u32x4 v = *reinterpret_cast<const u32x4_a1*>(row + at);
    uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
    if (s & 8) {
      lo = hi;
      hi = 0;
    }
    const int bits = 8 * (s & 7);
    lo = lo >> bits | hi << 1 << (63 - bits);
    hi >>= bits;
    if (s >= 16) lo = hi = 0;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
  u32x4 v;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    uint32_t w = 0u;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int c = k + 4 * d + b;
      w |= (c < n ? (uint32_t)row[min(c, n - 1)] : 0u) << (8 * b);
    }
    v[d] = w;
  }
  return v;
}

}  // namespace gptq
