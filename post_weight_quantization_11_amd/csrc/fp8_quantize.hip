// Quantization to 8-bit floats: rows of W to e4m3 codes, and one float32 scale
// for every 128 columns of a row or for every block of 128 x 128.
//
//   scale = max|w| / 448, rounded to float32; at least 2^-126, 1 for a block of zeros
//   code  = the e4m3 value nearest to the quotient w / scale, ties to the even code
//
// The quotient is not a float32 number, and rounding it to one first would put
// those within 2^-24 of a border between two codes on the border.  It is rounded
// to odd instead: the nearest float32 t, moved, where it is even and not exact,
// to the odd neighbour on the side of the remainder w - t scale (exact in one
// fused multiply-add).  Borders are even float32 numbers, so the conversion
// instruction, which rounds to the nearest even code, sees every quotient on its
// own side.  Scale and values are first multiplied by the power of two that
// brings the scale to [1, 2), so that no remainder is lost to underflow.
//
// One pass.  Blocks of a row: a thread takes 8 columns, sixteen neighbouring
// threads a block, its maximum in four steps across the lanes.  Blocks of 128 x
// 128: a workgroup takes one, 64 values a thread in registers between the
// maximum and the codes.  Reads, codes and Wq are contiguous.
#include "fp8.h"

namespace gptq {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxSlab = (int64_t)1 << 30;         // threads per launch

template <int DT> struct Fp8x8 {
  static constexpr int kVecs = DT == GPTQ_F32 ? 2 : 1;
  typedef u32x4 Vec[kVecs];

  // Largest absolute bit pattern (monotonic in |w|; infinities and NaN above
  // every finite one).
  __device__ static uint32_t amax(const Vec& v) {
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < 4 * kVecs; ++i) {
      const uint32_t x = v[i >> 2][i & 3];
      if constexpr (DT == GPTQ_F32) a = max(a, x & 0x7FFFFFFFu);
      else a = max(a, max(x & 0x7FFFu, (x >> 16) & 0x7FFFu));
    }
    return a;
  }
  __device__ static float widen(uint32_t bits) {
    if constexpr (DT == GPTQ_F32) return __uint_as_float(bits);
    else if constexpr (DT == GPTQ_BF16) return __uint_as_float(bits << 16);
    else return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  }
  __device__ static float at(const Vec& v, int i) {
    if constexpr (DT == GPTQ_F32) return widen(v[i >> 2][i & 3]);
    else return widen((v[0][i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
  }
};

// The scale of a block with this largest pattern; NaN if it is not finite.
template <int DT> __device__ inline float block_scale(uint32_t amax) {
  const float top = Fp8x8<DT>::widen(amax);
  if (amax == 0u) return 1.f;
  if (!(top < __builtin_inff())) return __builtin_nanf("");
  return fmaxf(top / kFp8Max, 0x1p-126f);
}

// What the codes of a block need of its scale: 2^exp scale in [1, 2).
struct Divisor {
  float s, r;                                // and (nearly) its reciprocal
  int exp;
};
__device__ inline Divisor divisor(float scale) {
  const int exp = 127 - (int)(__float_as_uint(scale) >> 23);
  const float s = ldexpf(scale, exp);
  return Divisor{s, __builtin_amdgcn_rcpf(s), exp};
}

// w / scale rounded to odd.
__device__ inline float quotient(float w, const Divisor& d) {
  const float a = ldexpf(fabsf(w), d.exp);
  float t = a * d.r;
  t = __builtin_fmaf(__builtin_fmaf(-t, d.s, a), d.r, t);      // the nearest float32
  const float rest = __builtin_fmaf(-t, d.s, a);
  uint32_t b = __float_as_uint(t);
  b = (rest < 0.f ? b - 1u : b) | (rest != 0.f ? 1u : 0u);     // even b: b - 1 is odd; odd b: b - 1 | 1 is b
  return __builtin_copysignf(__uint_as_float(b), w);
}

template <int DT>
__device__ inline u32x2 encode(const typename Fp8x8<DT>::Vec& v, const Divisor& d) {
  u32x2 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(Fp8x8<DT>::at(v, 4 * i), d), quotient(Fp8x8<DT>::at(v, 4 * i + 1), d),
                                        w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(Fp8x8<DT>::at(v, 4 * i + 2), d),
                                        quotient(Fp8x8<DT>::at(v, 4 * i + 3), d), w, true);
    c[i] = (uint32_t)w;
  }
  return c;
}

// code * scale, rounded to float32 and then, where w_dtype has fewer bits, to
// that.
template <int DT>
__device__ inline void decode(u32x2 c, float scale, typename Fp8x8<DT>::Vec& o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const floatx2 p = i & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i >> 1], true)
                            : __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i >> 1], false);
    const float a = p[0] * scale, b = p[1] * scale;
    if constexpr (DT == GPTQ_F32) {
      o[i >> 1][2 * (i & 1)] = __float_as_uint(a);
      o[i >> 1][2 * (i & 1) + 1] = __float_as_uint(b);
    } else if constexpr (DT == GPTQ_F16) {
      o[0][i] = __builtin_bit_cast(uint32_t, halfx2{(_Float16)a, (_Float16)b});
    } else {
      o[0][i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
    }
  }
}

// The first `cnt` of eight elements; the others are zero, or not written.
template <int DT>
__device__ inline void load8(const typename Elem<DT>::type* src, int cnt, typename Fp8x8<DT>::Vec& v) {
  constexpr int V = Fp8x8<DT>::kVecs, kPer = 4 / sizeof(typename Elem<DT>::type);
  if (cnt >= 8) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = reinterpret_cast<const typename Elem<DT>::vec*>(src)[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) {
    const int e = i * kPer;
    uint32_t x = e < cnt ? (uint32_t)src[e] : 0u;
    if (kPer == 2 && e + 1 < cnt) x |= (uint32_t)src[e + 1] << 16;
    v[i >> 2][i & 3] = x;
  }
}
template <int DT>
__device__ inline void store8(typename Elem<DT>::type* dst, int cnt, const typename Fp8x8<DT>::Vec& v) {
  typedef typename Elem<DT>::type elem;
  constexpr int V = Fp8x8<DT>::kVecs, kPer = 4 / sizeof(elem);
  if (cnt >= 8) {
#pragma unroll
    for (int i = 0; i < V; ++i) reinterpret_cast<typename Elem<DT>::vec*>(dst)[i] = v[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < 4 * V; ++i) {
    const int e = i * kPer;
    if (e < cnt) dst[e] = (elem)v[i >> 2][i & 3];
    if (kPer == 2 && e + 1 < cnt) dst[e + 1] = (elem)(v[i >> 2][i & 3] >> 16);
  }
}
__device__ inline void store_codes(uint8_t* dst, int cnt, u32x2 c) {
  if (cnt >= 8) {
    *reinterpret_cast<u32x2_a1*>(dst) = c;
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < cnt) dst[i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
}

// Strides in elements; blockIdx.y is the matrix of a stack.
template <int DT> struct QuantArgs {
  const typename Elem<DT>::type* W;
  uint8_t* codes;
  float* scales;
  typename Elem<DT>::type* Wq;
  int64_t ldw, ldc, lds, ldq, w_stride, c_stride, s_stride, q_stride;
  int n;
};

// Codes (and values) of eight elements; a block with a NaN or an infinity holds
// code 0 under the NaN scale.
template <int DT>
__device__ inline void finish8(const QuantArgs<DT>& p, int64_t e, int64_t r, int k0, float scale, const Divisor& d,
                               const typename Fp8x8<DT>::Vec& v) {
  const int cnt = p.n - k0;
  if (cnt <= 0) return;
  u32x2 c = encode<DT>(v, d);
  if (scale != scale) c = u32x2{0u, 0u};
  store_codes(p.codes + e * p.c_stride + r * p.ldc + k0, cnt, c);
  if (p.Wq != nullptr) {
    typename Fp8x8<DT>::Vec o;
    decode<DT>(c, scale, o);
    store8<DT>(p.Wq + e * p.q_stride + r * p.ldq + k0, cnt, o);
  }
}

// groups: threads with columns, `per_row` (a multiple of 16: whole blocks) to a row.
template <int DT>
__global__ __launch_bounds__(kThreads) void fp8_quantize_rows_kernel(QuantArgs<DT> p, uint32_t groups, uint32_t per_row,
                                                                     GroupDiv div) {
  const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
  // groups is a multiple of 16, so a block's lanes leave together.
  if (g >= groups) return;
  const int64_t e = blockIdx.y, r = (int64_t)(((uint64_t)g * div.mul) >> div.shift);
  const int k0 = (int)(g - (uint32_t)r * per_row) * 8;
  typename Fp8x8<DT>::Vec v;
  load8<DT>(p.W + e * p.w_stride + r * p.ldw + k0, p.n - k0, v);
  uint32_t a = Fp8x8<DT>::amax(v);
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) a = max(a, (uint32_t)__shfl_xor((int)a, x, 64));
  const float scale = block_scale<DT>(a);
  if ((threadIdx.x & 15) == 0) p.scales[e * p.s_stride + r * p.lds + (k0 >> 7)] = scale;
  finish8<DT>(p, e, r, k0, scale, divisor(scale), v);
}

// One block of 128 x 128 a workgroup; m: rows from the launch's first on.
template <int DT>
__global__ __launch_bounds__(kThreads) void fp8_quantize_blocks_kernel(QuantArgs<DT> p, int64_t m, uint32_t per_row) {
  constexpr int kRows = kThreads / 16, kPasses = kFp8Block / kRows;
  __shared__ uint32_t tops[kThreads / 64];
  const int64_t e = blockIdx.y, rb = blockIdx.x / per_row;
  const int cb = (int)(blockIdx.x - (uint32_t)rb * per_row);
  const int k0 = cb * kFp8Block + (int)(threadIdx.x & 15) * 8;
  const int64_t r0 = rb * kFp8Block + (threadIdx.x >> 4);
  typename Fp8x8<DT>::Vec v[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int64_t r = r0 + i * kRows;
    load8<DT>(p.W + e * p.w_stride + min(r, m - 1) * p.ldw + k0, p.n - k0, v[i]);
  }
  uint32_t a = 0u;                           // rows past the last repeat it
#pragma unroll
  for (int i = 0; i < kPasses; ++i) a = max(a, Fp8x8<DT>::amax(v[i]));
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) a = max(a, (uint32_t)__shfl_xor((int)a, x, 64));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = a;
  __syncthreads();
  a = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  const float scale = block_scale<DT>(a);
  if (threadIdx.x == 0) p.scales[e * p.s_stride + rb * p.lds + cb] = scale;
  const Divisor d = divisor(scale);
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int64_t r = r0 + i * kRows;
    if (r < m) finish8<DT>(p, e, r, k0, scale, d, v[i]);
  }
}

template <int DT>
gptq_status launch(QuantArgs<DT> p, int64_t experts, int64_t m, int block_rows, hipStream_t st) {
  const int64_t blocks = ceil_div(p.n, kFp8Block);
  const int64_t per_row = block_rows == 1 ? blocks * 16 : blocks;
  // Rows a launch: a multiple of the block's.
  const int64_t slab = block_rows == 1 ? std::max<int64_t>(1, kMaxSlab / per_row)
                                       : std::max<int64_t>(1, kMaxSlab / kThreads / per_row) * kFp8Block;
  for (int64_t r0 = 0; r0 < m; r0 += slab) {
    const int64_t rows = std::min(slab, m - r0);
    QuantArgs<DT> q = p;
    q.W += r0 * p.ldw;
    q.codes += r0 * p.ldc;
    q.scales += r0 / block_rows * p.lds;
    if (q.Wq != nullptr) q.Wq += r0 * p.ldq;
    if (block_rows == 1) {
      const uint32_t groups = (uint32_t)(rows * per_row);
      fp8_quantize_rows_kernel<DT><<<dim3((unsigned)ceil_div(groups, kThreads), (unsigned)experts), kThreads, 0, st>>>(
          q, groups, (uint32_t)per_row, group_div((uint32_t)per_row));
    } else {
      fp8_quantize_blocks_kernel<DT>
          <<<dim3((unsigned)(ceil_div(rows, kFp8Block) * per_row), (unsigned)experts), kThreads, 0, st>>>(
              q, rows, (uint32_t)per_row);
    }
    GPTQ_TRY_LAUNCH();
  }
  return GPTQ_OK;
}

template <int DT>
gptq_status start(const void* W, int64_t experts, int64_t m, int64_t n, int64_t ldw, int64_t stride_w, int block_rows,
                  uint8_t* codes, int64_t ld_codes, int64_t stride_codes, float* scales, int64_t ld_scales,
                  int64_t stride_scales, void* Wq, int64_t ldwq, int64_t stride_wq, hipStream_t st) {
  typedef typename Elem<DT>::type elem;
  // At most 65535 matrices along the grid's y.
  for (int64_t e = 0; e < experts; e += 32768) {
    QuantArgs<DT> p{static_cast<const elem*>(W) + e * stride_w, codes + e * stride_codes, scales + e * stride_scales,
                    Wq == nullptr ? nullptr : static_cast<elem*>(Wq) + e * stride_wq, ldw, ld_codes, ld_scales, ldwq,
                    stride_w, stride_codes, stride_scales, stride_wq, (int)n};
    const gptq_status rc = launch<DT>(p, std::min<int64_t>(experts - e, 32768), m, block_rows, st);
    if (rc != GPTQ_OK) return rc;
  }
  return GPTQ_OK;
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" gptq_status gptq_block_quantize(const void* W, int w_dtype, int64_t experts, int64_t m, int64_t n, int64_t ldw,
                                         int64_t stride_w, int block_rows, uint8_t* codes, int64_t ld_codes,
                                         int64_t stride_codes, float* scales, int64_t ld_scales, int64_t stride_scales,
                                         void* Wq, int64_t ldwq, int64_t stride_wq, void* stream) {
  if (experts < 0 || m < 0 || n < 0 || !valid_dtype(w_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != kFp8Block) return GPTQ_ERR_INVALID_ARG;
  if (n > kFp8MaxCols || m > ((int64_t)1 << 31) - 1 || experts > GPTQ_MX_MAX_EXPERTS) return GPTQ_ERR_UNSUPPORTED;
  if (experts == 0 || m == 0 || n == 0) return GPTQ_OK;
  if (W == nullptr || codes == nullptr || scales == nullptr) return GPTQ_ERR_INVALID_ARG;
  const int64_t row_blocks = ceil_div(m, block_rows), blocks = ceil_div(n, kFp8Block);
  if (ldw < n || ld_codes < n || ld_scales < blocks || (Wq != nullptr && ldwq < n)) return GPTQ_ERR_INVALID_ARG;
  constexpr int64_t kMaxLd = (int64_t)1 << 30, kMaxStride = (int64_t)1 << 45;
  if (ldw > kMaxLd || ld_codes > kMaxLd || ld_scales > kMaxLd || (Wq != nullptr && ldwq > kMaxLd))
    return GPTQ_ERR_UNSUPPORTED;
  if (experts > 1) {
    if (stride_w > kMaxStride || stride_codes > kMaxStride || stride_scales > kMaxStride ||
        (Wq != nullptr && stride_wq > kMaxStride))
      return GPTQ_ERR_UNSUPPORTED;
    // Outputs of two matrices must not lie in one another; inputs may.
    if (stride_w < 0 || stride_codes < (m - 1) * ld_codes + n || stride_scales < (row_blocks - 1) * ld_scales + blocks ||
        (Wq != nullptr && stride_wq < (m - 1) * ldwq + n))
      return GPTQ_ERR_INVALID_ARG;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
#define GPTQ_FP8_ARGS                                                                                            \
  W, experts, m, n, ldw, stride_w, block_rows, codes, ld_codes, stride_codes, scales, ld_scales, stride_scales, \
      Wq, ldwq, stride_wq, st
  if (w_dtype == GPTQ_F32) return start<GPTQ_F32>(GPTQ_FP8_ARGS);
  if (w_dtype == GPTQ_F16) return start<GPTQ_F16>(GPTQ_FP8_ARGS);
  return start<GPTQ_BF16>(GPTQ_FP8_ARGS);
#undef GPTQ_FP8_ARGS
}
