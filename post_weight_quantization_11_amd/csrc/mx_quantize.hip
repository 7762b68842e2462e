// Microscaled quantization: rows of W to e2m1 codes and one power-of-two
// scale for every 32 columns, round to nearest.
//
//   scale = 2^(floor(log2 max|w|) - 2)   (6 = 1.5 * 2^2 is e2m1's largest value)
//   code  = the e2m1 value nearest to w / scale, ties to the even code,
//           saturating at 6
//
// The division by a power of two is exact and the conversion instructions
// round once (nearest even, saturating), from each input type and over the
// whole range of scale bytes: checked against the thresholds 0.25, 0.75,
// 1.25, 1.75, 2.5, 3.5 and 5 on the values around them and on every 16-bit
// pattern.
//
// One pass: a thread takes 8 columns (one packed word), four neighbouring
// threads a block; the block maximum is an integer maximum of the absolute
// bit patterns (monotonic in |w|, with infinities and NaN above every finite
// pattern), two steps across the four lanes.  Reads, packed words and Wq are
// contiguous over a wave.  Bound by memory: 49152 x 12288 float16 with Wq 436 us
// for 2.74 GB (6.3 TB/s), without Wq 279 us for 1.53 GB (5.5 TB/s); 256 x 256
// float32 2.8 us, a launch.
#include "mx.h"

namespace gptq {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxSlabGroups = (int64_t)1 << 30;   // groups of 8 columns per launch

// Eight elements as loaded, the largest absolute bit pattern among them, the
// scale byte of a block maximum, the packed word and the dequantized values.
template <int DT> struct Mx8;

template <> struct Mx8<GPTQ_F32> {
  static constexpr int kVecs = 2;
  __device__ static uint32_t amax(const u32x4 (&v)[2]) {
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, v[i >> 2][i & 3] & 0x7FFFFFFFu);
    return a;
  }
  // Exponent field - 2; fields 0 (subnormal) to 2 give the smallest scale.
  __device__ static uint32_t byte(uint32_t a) {
    if (a == 0u) return kMxScaleOne;
    const uint32_t e = a >> 23;
    return e == 255u ? kMxScaleNan : (e > 2u ? e - 2u : 0u);
  }
  __device__ static uint32_t encode(const u32x4 (&v)[2], float s) {
    uint32_t w = 0u;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(v[0][0]), __uint_as_float(v[0][1]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(v[0][2]), __uint_as_float(v[0][3]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(v[1][0]), __uint_as_float(v[1][1]), s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(v[1][2]), __uint_as_float(v[1][3]), s, 3);
    return w;
  }
  __device__ static void decode(uint32_t w, float s, u32x4 (&o)[2]) {
    const floatx2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
    const floatx2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
    const floatx2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
    const floatx2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
    o[0] = u32x4{__float_as_uint(p0[0]), __float_as_uint(p0[1]), __float_as_uint(p1[0]), __float_as_uint(p1[1])};
    o[1] = u32x4{__float_as_uint(p2[0]), __float_as_uint(p2[1]), __float_as_uint(p3[0]), __float_as_uint(p3[1])};
  }
};

__device__ inline uint32_t amax_pairs(const u32x4 (&v)[1]) {
  uint32_t a = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) a = max(a, max(v[0][i] & 0x7FFFu, (v[0][i] >> 16) & 0x7FFFu));
  return a;
}

template <> struct Mx8<GPTQ_F16> {
  static constexpr int kVecs = 1;
  __device__ static uint32_t amax(const u32x4 (&v)[1]) { return amax_pairs(v); }
  // floor(log2 a) - 2 + 127: from the exponent field, or from the leading
  // bit of a subnormal a 2^-24.
  __device__ static uint32_t byte(uint32_t a) {
    if (a == 0u) return kMxScaleOne;
    const uint32_t e = a >> 10;
    if (e == 31u) return kMxScaleNan;
    return e == 0u ? (uint32_t)(31 - __clz((int)a)) + 101u : e + 110u;
  }
  __device__ static uint32_t encode(const u32x4 (&v)[1], float s) {
    uint32_t w = 0u;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(halfx2, (uint32_t)v[0][0]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(halfx2, (uint32_t)v[0][1]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(halfx2, (uint32_t)v[0][2]), s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(halfx2, (uint32_t)v[0][3]), s, 3);
    return w;
  }
  // Exact: the values are multiples of 2^-24 wherever the inputs were.
  __device__ static void decode(uint32_t w, float s, u32x4 (&o)[1]) {
    o[0] = u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3))};
  }
};

template <> struct Mx8<GPTQ_BF16> {
  static constexpr int kVecs = 1;
  __device__ static uint32_t amax(const u32x4 (&v)[1]) { return amax_pairs(v); }
  __device__ static uint32_t byte(uint32_t a) {
    if (a == 0u) return kMxScaleOne;
    const uint32_t e = a >> 7;
    return e == 255u ? kMxScaleNan : (e > 2u ? e - 2u : 0u);
  }
  __device__ static uint32_t encode(const u32x4 (&v)[1], float s) {
    uint32_t w = 0u;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, (uint32_t)v[0][0]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, (uint32_t)v[0][1]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, (uint32_t)v[0][2]), s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, (uint32_t)v[0][3]), s, 3);
    return w;
  }
  __device__ static void decode(uint32_t w, float s, u32x4 (&o)[1]) {
    o[0] = u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
  }
};

// groups: groups of 8 columns in this launch, `per_row` (a multiple of 4: whole
// blocks) to a row.  Packed words that start at or past column n and scale
// bytes of such blocks do not exist and are not written.
template <int DT>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(
    const typename Elem<DT>::type* __restrict__ W, int n, int64_t ldw, uint32_t* __restrict__ packed, int64_t ldp,
    uint8_t* __restrict__ scales, int64_t lds, typename Elem<DT>::type* __restrict__ Wq, int64_t ldwq,
    uint32_t groups, uint32_t per_row, GroupDiv div) {
  typedef typename Elem<DT>::type elem;
  typedef typename Elem<DT>::vec vec_a;
  constexpr int V = Mx8<DT>::kVecs;
  constexpr int kPer = 4 / sizeof(elem);     // elements per 32-bit word
  const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
  // groups is a multiple of 4, so a block's four lanes leave together.
  if (g >= groups) return;
  const int64_t r = (int64_t)(((uint64_t)g * div.mul) >> div.shift);
  const int k0 = (int)(g - (uint32_t)r * per_row) * 8;
  const elem* src = W + r * ldw + k0;
  const int cnt = n - k0;                    // columns left (<= 0 past the row's end)
  u32x4 v[V];
  if (cnt >= 8) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = reinterpret_cast<const vec_a*>(src)[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int e = (4 * i + d) * kPer;
        uint32_t x = e < cnt ? (uint32_t)src[e] : 0u;
        if (kPer == 2 && e + 1 < cnt) x |= (uint32_t)src[e + 1] << 16;
        v[i][d] = x;
      }
  }
  uint32_t a = Mx8<DT>::amax(v);
  a = max(a, (uint32_t)__shfl_xor((int)a, 1, 64));
  a = max(a, (uint32_t)__shfl_xor((int)a, 2, 64));
  const uint32_t byte = Mx8<DT>::byte(a);
  const float s = mx_scale_operand(byte);
  // A block with a NaN or an infinity holds code 0 under the NaN scale: every
  // value it stands for is NaN.
  const uint32_t w = byte == kMxScaleNan ? 0u : Mx8<DT>::encode(v, s);
  if (cnt > 0) {
    packed[r * ldp + (k0 >> 3)] = w;
    if ((k0 & (kMxBlock - 1)) == 0) scales[r * lds + (k0 >> 5)] = (uint8_t)byte;
    if (Wq != nullptr) {
      u32x4 o[V];
      Mx8<DT>::decode(w, s, o);
      elem* dst = Wq + r * ldwq + k0;
      if (cnt >= 8) {
#pragma unroll
        for (int i = 0; i < V; ++i) reinterpret_cast<vec_a*>(dst)[i] = o[i];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const int e = (4 * i + d) * kPer;
            if (e < cnt) dst[e] = (elem)o[i][d];
            if (kPer == 2 && e + 1 < cnt) dst[e + 1] = (elem)(o[i][d] >> 16);
          }
      }
    }
  }
}

template <int DT>
gptq_status launch(const void* W, int64_t m, int64_t n, int64_t ldw, uint32_t* packed, int64_t ldp,
                   uint8_t* scales, int64_t lds, void* Wq, int64_t ldwq, hipStream_t st) {
  typedef typename Elem<DT>::type elem;
  const int64_t per_row = ceil_div(n, kMxBlock) * 4;
  const int64_t slab = std::max<int64_t>(1, kMaxSlabGroups / per_row);   // rows per launch
  for (int64_t r0 = 0; r0 < m; r0 += slab) {
    const int64_t rows = std::min(slab, m - r0);
    const uint32_t groups = (uint32_t)(rows * per_row);
    mx_quantize_kernel<DT><<<(unsigned)ceil_div(groups, kThreads), kThreads, 0, st>>>(
        static_cast<const elem*>(W) + r0 * ldw, (int)n, ldw, packed + r0 * ldp, ldp, scales + r0 * lds, lds,
        Wq == nullptr ? nullptr : static_cast<elem*>(Wq) + r0 * ldwq, ldwq, groups, (uint32_t)per_row,
        group_div((uint32_t)per_row));
    GPTQ_TRY_LAUNCH();
  }
  return GPTQ_OK;
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" gptq_status gptq_mx_quantize(const void* W, int w_dtype, int64_t m, int64_t n, int64_t ldw,
                                        uint32_t* packed, int64_t ld_packed, uint8_t* scales, int64_t ld_scales,
                                        void* Wq, int64_t ldwq, void* stream) {
  if (m < 0 || n < 0 || !valid_dtype(w_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (n > kMxMaxCols || m > ((int64_t)1 << 31) - 1) return GPTQ_ERR_UNSUPPORTED;
  if (m == 0 || n == 0) return GPTQ_OK;
  if (W == nullptr || packed == nullptr || scales == nullptr) return GPTQ_ERR_INVALID_ARG;
  if (ldw < n || ld_packed < ceil_div(n, 8) || ld_scales < ceil_div(n, kMxBlock)) return GPTQ_ERR_INVALID_ARG;
  if (Wq != nullptr && ldwq < n) return GPTQ_ERR_INVALID_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (w_dtype == GPTQ_F32) return launch<GPTQ_F32>(W, m, n, ldw, packed, ld_packed, scales, ld_scales, Wq, ldwq, st);
  if (w_dtype == GPTQ_F16) return launch<GPTQ_F16>(W, m, n, ldw, packed, ld_packed, scales, ld_scales, Wq, ldwq, st);
  return launch<GPTQ_BF16>(W, m, n, ldw, packed, ld_packed, scales, ld_scales, Wq, ldwq, st);
}
