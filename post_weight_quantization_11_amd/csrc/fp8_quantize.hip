// Quantization to 8-bit floats: rows of W to e4m3 codes, and one float32 scale
// for every 128 columns of a row or for every block of 128 x 128.
//
//   scale = max|w| / 448, rounded to float32; at least 2^-126, 1 for a block of zeros
//   code  = the e4m3 value nearest to the quotient w / scale, ties to the even code
//
// The quotient is not a float32 number, and rounding it to one first would put
// those within 2^-24 of a border between two codes on the border.  Instead w times
// the reciprocal, a few units off, is rounded to 20 bits: t.  Borders have at most 5
// bits, so the only one that can lie between t and the quotient is t itself, and
// the sign of the remainder w - t scale, exact in one fused multiply-add, says on
// which side: t is moved one unit there.  The conversion instruction, which rounds
// to the nearest even code, then sees every quotient on its own side of a border.
// The remainder is a multiple of 2^-46 |w| (nearly): under scales below 2^-80 values
// and scale are multiplied by 2^60 first, so that it is not lost to underflow.
//
// One pass.  Blocks of a row: a thread takes 16 columns, eight neighbouring threads
// a block, its maximum in three steps across the lanes.  Blocks of 128 x 128: a
// workgroup takes one or four neighbouring ones, 64 values a thread in registers
// between the maximum and the codes.  Reads, codes and Wq are contiguous.
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

// What the codes of a block need of its scale.
struct Divisor {
  float up, s, r;                            // 1 or 2^60, the scale times that, nearly its reciprocal
};
__device__ inline Divisor divisor(float scale) {
  const float up = scale < 0x1p-80f ? 0x1p60f : 1.f;
  return Divisor{up, scale * up, __builtin_amdgcn_rcpf(scale * up)};
}

// w / scale on its side of every border between two codes.
__device__ inline float quotient(float w, const Divisor& d) {
  const float a = fabsf(w) * d.up;
  const uint32_t t = (__float_as_uint(a * d.r) + 8u) & ~15u;
  const int rest = (int)__float_as_uint(__builtin_fmaf(-__uint_as_float(t), d.s, a));
  int side;                                  // -1, 0 or 1 (of min and max the compiler makes compares and selects)
  asm("v_med3_i32 %0, %1, -1, 1" : "=v"(side) : "v"(rest));
  return __builtin_copysignf(__uint_as_float(t + (uint32_t)side), w);
}

template <int DT>
__device__ inline u32x2 encode(const typename Fp8x8<DT>::Vec& v, const Divisor& d) {
  auto at = [&](int i) { return quotient(Fp8x8<DT>::at(v, i), d); };
  u32x2 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(at(4 * i), at(4 * i + 1), w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(at(4 * i + 2), at(4 * i + 3), w, true);
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

// Sixteen columns a thread.  groups: threads with columns, `per_row` (a multiple of 8:
// whole blocks) to a row.
template <int DT>
__global__ __launch_bounds__(kThreads) void fp8_quantize_rows_kernel(QuantArgs<DT> p, uint32_t groups, uint32_t per_row,
                                                                     GroupDiv div) {
  const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
  // groups is a multiple of 8, so a block's lanes leave together.
  if (g >= groups) return;
  const int64_t e = blockIdx.y, r = (int64_t)(((uint64_t)g * div.mul) >> div.shift);
  const int k0 = (int)(g - (uint32_t)r * per_row) * 16;
  typename Fp8x8<DT>::Vec v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) load8<DT>(p.W + e * p.w_stride + r * p.ldw + k0 + 8 * i, p.n - k0 - 8 * i, v[i]);
  uint32_t a = max(Fp8x8<DT>::amax(v[0]), Fp8x8<DT>::amax(v[1]));
#pragma unroll
  for (int x = 1; x < 8; x <<= 1) a = max(a, (uint32_t)__shfl_xor((int)a, x, 64));
  const float scale = block_scale<DT>(a);
  if ((threadIdx.x & 7) == 0) p.scales[e * p.s_stride + r * p.lds + (k0 >> 7)] = scale;
  const Divisor d = divisor(scale);
#pragma unroll
  for (int i = 0; i < 2; ++i) finish8<DT>(p, e, r, k0 + 8 * i, scale, d, v[i]);
}

// BLOCKS neighbouring blocks of 128 x 128 a workgroup, sixteen rows at a time.  Four
// read 512 columns of a row in one go (49152 x 12288 float16 with Wq 560 us, 600 one by
// one); one gives small matrices more workgroups.  m: rows from the launch's first on;
// per_row: such groups of blocks.
template <int DT, int BLOCKS>
__global__ __launch_bounds__(256 * BLOCKS, DT == GPTQ_F32 ? 4 : 8) void fp8_quantize_blocks_kernel(
    QuantArgs<DT> p, int64_t m, uint32_t per_row) {
  constexpr int kRows = 16, kPasses = kFp8Block / kRows;
  __shared__ uint32_t tops[BLOCKS][kRows];
  const int at = (int)threadIdx.x % (16 * BLOCKS), row = (int)threadIdx.x / (16 * BLOCKS), l16 = at & 15;
  const int64_t e = blockIdx.y, rb = blockIdx.x / per_row;
  const int k0 = (int)(blockIdx.x - (uint32_t)rb * per_row) * (kFp8Block * BLOCKS) + at * 8;
  const int64_t r0 = rb * kFp8Block + row;
  typename Fp8x8<DT>::Vec v[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    load8<DT>(p.W + e * p.w_stride + min(r0 + i * kRows, m - 1) * p.ldw + k0, p.n - k0, v[i]);
  uint32_t a = 0u;                           // rows past the last repeat it
#pragma unroll
  for (int i = 0; i < kPasses; ++i) a = max(a, Fp8x8<DT>::amax(v[i]));
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) a = max(a, (uint32_t)__shfl_xor((int)a, x, 64));
  if (l16 == 0) tops[at >> 4][row] = a;
  __syncthreads();
  a = tops[at >> 4][l16];
#pragma unroll
  for (int x = 1; x < 16; x <<= 1) a = max(a, (uint32_t)__shfl_xor((int)a, x, 64));
  const float scale = block_scale<DT>(a);
  if (row == 0 && l16 == 0 && k0 < p.n) p.scales[e * p.s_stride + rb * p.lds + (k0 >> 7)] = scale;
  const Divisor d = divisor(scale);
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    if (r0 + i * kRows < m) finish8<DT>(p, e, r0 + i * kRows, k0, scale, d, v[i]);
}

// Calls part(rows of the launch, its operands) for as many rows at a time as one launch
// takes: `per` threads to a unit of `unit` rows.
template <int DT, typename Part>
gptq_status in_parts(const QuantArgs<DT>& p, int64_t m, int block_rows, int64_t unit, int64_t per, Part part) {
  const int64_t slab = std::max<int64_t>(1, kMaxSlab / per) * unit;
  for (int64_t r0 = 0; r0 < m; r0 += slab) {
    QuantArgs<DT> q = p;
    q.W += r0 * p.ldw;
    q.codes += r0 * p.ldc;
    q.scales += r0 / block_rows * p.lds;
    if (q.Wq != nullptr) q.Wq += r0 * p.ldq;
    part(std::min(slab, m - r0), q);
    GPTQ_TRY_LAUNCH();
  }
  return GPTQ_OK;
}

template <int DT, int BLOCKS>
gptq_status launch_blocks(const QuantArgs<DT>& p, int64_t experts, int64_t m, hipStream_t st) {
  const int64_t per_row = ceil_div(p.n, kFp8Block * BLOCKS);
  return in_parts<DT>(p, m, kFp8Block, kFp8Block, per_row * 256 * BLOCKS, [&](int64_t rows, const QuantArgs<DT>& q) {
    fp8_quantize_blocks_kernel<DT, BLOCKS>
        <<<dim3((unsigned)(ceil_div(rows, kFp8Block) * per_row), (unsigned)experts), 256 * BLOCKS, 0, st>>>(
            q, rows, (uint32_t)per_row);
  });
}

template <int DT>
gptq_status launch(const QuantArgs<DT>& p, int64_t experts, int64_t m, int block_rows, hipStream_t st) {
  const int64_t blocks = ceil_div(p.n, kFp8Block);
  if (block_rows != 1) {
    // Four blocks a workgroup where that still gives two workgroups a CU.
    if (ceil_div(m, kFp8Block) * blocks * experts >= 4 * 512) return launch_blocks<DT, 4>(p, experts, m, st);
    return launch_blocks<DT, 1>(p, experts, m, st);
  }
  const int64_t per_row = blocks * 8;
  return in_parts<DT>(p, m, 1, 1, per_row, [&](int64_t rows, const QuantArgs<DT>& q) {
    const uint32_t groups = (uint32_t)(rows * per_row);
    fp8_quantize_rows_kernel<DT><<<dim3((unsigned)ceil_div(groups, kThreads), (unsigned)experts), kThreads, 0, st>>>(
        q, groups, (uint32_t)per_row, group_div((uint32_t)per_row));
  });
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
