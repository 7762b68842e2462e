// Products with microscaled weights: Y[t, r] = sum_k What[r, k] X[t, k], for
// one weight matrix or one per expert (rows of X grouped by expert), with
// 16-bit X or with X microscaled too.
//
// 16-bit X: the codes become exact f16 or bf16 values (an e2m1 value times a
// power of two) with the scaled conversion instructions, two per instruction,
// and go into v_mfma_f32_16x16x32; products are exact in float32 and summed
// there.  Microscaled X: v_mfma_scale_f32_16x16x128_f8f6f4 takes both code
// words and scale bytes as stored.
//
// Operand layout (checked with an in-bounds probe): lane l holds row l % 16;
// of a unit of 128 columns it holds the 32 columns of block l / 16, 16 bytes
// of codes.  The order of the summed columns inside an instruction is free as
// long as both operands agree, so 16-bit step j (0..3) takes codes 8j .. 8j+7
// of every lane's block: X columns 32 (l / 16) + 8j .. + 7, one 16-byte load.
// X is the first operand, so a wave's results have consecutive W rows in
// neighbouring lanes and go out in contiguous runs.
#include "mx.h"

namespace gptq {
namespace {

constexpr int kMx = 3;                       // X operand kinds: GPTQ_F16, GPTQ_BF16, microscaled

struct MxOperands {
  const uint32_t* W;                         // packed weights, m x ldp words (per expert: + e * stride)
  const uint8_t* S;
  int64_t ldp, lds, w_stride, s_stride;
  int m, n;
  const void* X;                             // 16-bit elements, or packed words
  const uint8_t* XS;                         // scales of a microscaled X
  int64_t ldx, ldxs;
  int rows;                                  // rows of X
  const int32_t* offsets;                    // experts + 1 row offsets, or NULL (one matrix, all rows)
  int experts;
  void* Y;
  int64_t ldy;
  int y_dtype;
};

__device__ inline void store_y(const MxOperands& p, int64_t at, float v) {
  if (p.y_dtype == GPTQ_F32)
    static_cast<float*>(p.Y)[at] = v;
  else if (p.y_dtype == GPTQ_F16)
    static_cast<_Float16*>(p.Y)[at] = (_Float16)v;
  else
    static_cast<__bf16*>(p.Y)[at] = (__bf16)v;
}

// One tile of at most `tile` rows of X that share a weight matrix.
struct TokenTile {
  int expert, begin, end;                    // rows [begin, end) of X
  bool valid;
};

// The slot-th tile, counting every expert's ceil(rows / tile) tiles in order.
// All 64 lanes of the calling wave take part.  Offsets are clamped to the rows
// there are, so whatever they hold no access leaves X or Y.
__device__ inline TokenTile find_tile(const MxOperands& p, int slot, int tile) {
  if (p.offsets == nullptr) return TokenTile{0, slot * tile, min(p.rows, (slot + 1) * tile), true};
  const int lane = (int)threadIdx.x & 63;
  int before = 0;                            // tiles of the experts before this round's
  for (int e0 = 0; e0 < p.experts; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < p.experts) {
      lo = min(max(p.offsets[e], 0), p.rows);
      hi = min(max(p.offsets[e + 1], lo), p.rows);
    }
    const int own = (hi - lo + tile - 1) / tile;
    int upto = own;                          // inclusive sum over the lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(upto, d, 64);
      if (lane >= d) upto += o;
    }
    const int at = slot - before - (upto - own);
    const uint64_t hit = __ballot(at >= 0 && at < own);
    if (hit != 0) {
      const int l = __builtin_ctzll(hit);
      const int begin = __shfl(lo + at * tile, l, 64), end = __shfl(hi, l, 64);
      return TokenTile{e0 + l, __builtin_amdgcn_readfirstlane(begin),
                       __builtin_amdgcn_readfirstlane(min(end, begin + tile)), true};
    }
    before += __builtin_amdgcn_readfirstlane(__shfl(upto, 63, 64));
  }
  return TokenTile{0, 0, 0, false};
}

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

typedef int intx8 __attribute__((ext_vector_type(8)));
__device__ inline intx8 fp4_operand(u32x4 v) {
  return intx8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};   // 4-bit formats use four registers
}

// Float16 holds an e2m1 value times 2^(byte - 127) exactly for bytes 104
// (0.5 * 2^-23, the smallest subnormal) to 140 (6 * 2^13).  Other scales are
// taken in windows of 37 bytes: window i (-3 .. 4; the NaN byte in window 0)
// is moved into that range by 2^(-37 i) and its products, summed apart, are
// moved back by 2^(37 i) when they are added.  bfloat16 holds every value that
// float32 holds.
constexpr uint32_t kF16Lo = 104, kF16Span = 37;
__device__ inline bool f16_exact(uint32_t byte) { return byte - kF16Lo < kF16Span || byte == kMxScaleNan; }
__device__ inline int f16_window(uint32_t byte) {
  return byte == kMxScaleNan ? 0 : (int)(byte + 3 * kF16Span - kF16Lo) / (int)kF16Span - 3;
}

// A block of a packed row: words past the row's last are 0, as are codes past
// column n in its last word, and a block past the row's end has scale 1.
__device__ inline void load_block(const uint32_t* row, const uint8_t* srow, int blk, int n, u32x4& w,
                                  uint32_t& byte) {
  const int nw = (n + 7) >> 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = 4 * blk + i;
    uint32_t v = k < nw ? row[k] : 0u;
    if (k == nw - 1 && (n & 7) != 0) v &= (1u << (4 * (n & 7))) - 1u;
    w[i] = v;
  }
  byte = blk * kMxBlock < n ? (uint32_t)srow[blk] : (uint32_t)kMxScaleOne;
}

// Rows of W in tiles of 16; a wave holds RT tiles of W rows and NT tiles of 16
// rows of X, and takes every KW-th unit of 128 columns; the waves of the
// workgroup add their sums through LDS in wave order.
template <int XT, int RT, int NT>
__global__ __launch_bounds__(512) void mx_rows_kernel(MxOperands p) {
  constexpr int kXRegs = XT == kMx ? 1 : 4;  // 16-byte registers of X per unit and tile
  extern __shared__ floatx4 red[];           // [wave][RT][NT][64]
  const int lane = (int)threadIdx.x & 63, q = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = (int)blockDim.x >> 6;
  const TokenTile tile = find_tile(p, (int)blockIdx.y, 16 * NT);
  if (!tile.valid) return;
  const int r0 = (int)blockIdx.x * 16 * RT;
  const uint32_t* wrow[RT];
  const uint8_t* srow[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int64_t r = min(r0 + 16 * rt + c16, p.m - 1);
    wrow[rt] = p.W + (int64_t)tile.expert * p.w_stride + r * p.ldp;
    srow[rt] = p.S + (int64_t)tile.expert * p.s_stride + r * p.lds;
  }
  const uint16_t* xrow[NT];
  const uint32_t* xprow[NT];
  const uint8_t* xsrow[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int64_t t = min(tile.begin + 16 * nt + c16, tile.end - 1);
    xrow[nt] = static_cast<const uint16_t*>(p.X) + t * p.ldx;
    xprow[nt] = static_cast<const uint32_t*>(p.X) + t * p.ldx;
    xsrow[nt] = p.XS + t * p.ldxs;
  }
  floatx4 acc[RT][NT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[rt][nt] = floatx4{0.f, 0.f, 0.f, 0.f};

  const int units = (p.n + 127) >> 7;
  for (int u = wave; u < units; u += waves) {
    const int blk = 4 * u + q, k0 = blk * kMxBlock;
    u32x4 w[RT], x[NT][kXRegs];
    uint32_t wb[RT], xb[NT];
    if ((u + 1) * 128 <= p.n) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        w[rt] = *reinterpret_cast<const u32x4_a4*>(wrow[rt] + 4 * blk);
        wb[rt] = srow[rt][blk];
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (XT == kMx) {
          x[nt][0] = *reinterpret_cast<const u32x4_a4*>(xprow[nt] + 4 * blk);
          xb[nt] = xsrow[nt][blk];
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[nt][j] = *reinterpret_cast<const u32x4_a2*>(xrow[nt] + k0 + 8 * j);
        }
      }
    } else {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) load_block(wrow[rt], srow[rt], blk, p.n, w[rt], wb[rt]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (XT == kMx) {
          load_block(xprow[nt], xsrow[nt], blk, p.n, x[nt][0], xb[nt]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              const int k = k0 + 8 * j + 2 * d;
              uint32_t v = k < p.n ? (uint32_t)xrow[nt][k] : 0u;
              if (k + 1 < p.n) v |= (uint32_t)xrow[nt][k + 1] << 16;
              x[nt][j][d] = v;
            }
        }
      }
    }
    if constexpr (XT == kMx) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          acc[rt][nt] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              fp4_operand(x[nt][0]), fp4_operand(w[rt]), acc[rt][nt], 4, 4, 0, (int)xb[nt], 0, (int)wb[rt]);
    } else {
      bool exact = true;
      if constexpr (XT == GPTQ_F16) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) exact = exact && f16_exact(wb[rt]);
      }
      if (XT == GPTQ_BF16 || __all(exact)) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const u32x4 wv = widen8<XT>(w[rt][j], mx_scale_operand(wb[rt]));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[rt][nt] = mfma16<XT>(x[nt][j], wv, acc[rt][nt]);
          }
      } else {
        for (int win = -3; win <= 4; ++win) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const bool in = f16_window(wb[rt]) == win;
            if (!__any(in)) continue;
            const float s = mx_scale_operand(in ? (wb[rt] == kMxScaleNan ? wb[rt] : wb[rt] - kF16Span * win)
                                                : kMxScaleOne);
            floatx4 part[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) part[nt] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const u32x4 wv = widen8<XT>(in ? w[rt][j] : 0u, s);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) part[nt] = mfma16<XT>(x[nt][j], wv, part[nt]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[rt][nt][i] += __builtin_ldexpf(part[nt][i], (int)kF16Span * win);
          }
        }
      }
    }
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) red[((wave * RT + rt) * NT + nt) * 64 + lane] = acc[rt][nt];
  __syncthreads();
  // Accumulator register i of lane l: X row 4 (l / 16) + i, W row l % 16.
  for (int o = wave; o < RT * NT; o += waves) {
    const int rt = o / NT, nt = o % NT;
    floatx4 v = red[o * 64 + lane];
    for (int w = 1; w < waves; ++w) v += red[(w * RT * NT + o) * 64 + lane];
    const int r = r0 + 16 * rt + c16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = tile.begin + 16 * nt + 4 * q + i;
      if (t < tile.end && r < p.m) store_y(p, (int64_t)t * p.ldy + r, v[i]);
    }
  }
}

// Tiles that the rows can form at most: every expert with rows may end in a
// partial tile.
inline int64_t max_tiles(const MxOperands& p, int tile) {
  const int64_t whole = ceil_div(p.rows, tile);
  return p.offsets == nullptr ? whole : p.rows / tile + std::min<int64_t>(p.experts, p.rows);
}

template <int XT>
gptq_status launch(const MxOperands& p, hipStream_t st) {
  constexpr int kRT = 1, kNT = 1, kWaves = 8;
  constexpr int64_t kMaxGridY = 65535;
  if (max_tiles(p, 16 * kNT) > kMaxGridY) return GPTQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)ceil_div(p.m, 16 * kRT), (unsigned)max_tiles(p, 16 * kNT));
  mx_rows_kernel<XT, kRT, kNT><<<grid, 64 * kWaves, kWaves * kRT * kNT * 64 * sizeof(floatx4), st>>>(p);
  GPTQ_TRY_LAUNCH();
  return GPTQ_OK;
}

// Checks shared by the products; `rows` rows of X against `experts` matrices.
gptq_status check(int64_t m, int64_t n, int64_t rows, int64_t experts, int64_t ld_packed, int64_t ld_scales,
                  int y_dtype, int64_t ldy) {
  if (m < 0 || n < 0 || rows < 0 || experts < 0 || !valid_dtype(y_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (n > kMxMaxCols || m > GPTQ_MX_MAX_ROWS || rows > GPTQ_MX_MAX_ROWS || experts > GPTQ_MX_MAX_EXPERTS)
    return GPTQ_ERR_UNSUPPORTED;
  if (ld_packed < ceil_div(n, 8) || ld_scales < ceil_div(n, kMxBlock) || ldy < m) return GPTQ_ERR_INVALID_ARG;
  return GPTQ_OK;
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" size_t gptq_mx_gemm_ws_bytes(int64_t m, int64_t n, int64_t rows, int64_t experts) {
  (void)m; (void)n; (void)rows; (void)experts;
  return 0;
}

extern "C" gptq_status gptq_mx_gemm_grouped(const uint32_t* packed, int64_t experts, int64_t m, int64_t n,
                                            int64_t ld_packed, int64_t stride_packed, const uint8_t* scales,
                                            int64_t ld_scales, int64_t stride_scales, const void* X, int x_dtype,
                                            int64_t rows, int64_t ldx, const int32_t* offsets, void* Y, int y_dtype,
                                            int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  if (x_dtype != GPTQ_F16 && x_dtype != GPTQ_BF16) return GPTQ_ERR_INVALID_ARG;
  const gptq_status rc = check(m, n, rows, experts, ld_packed, ld_scales, y_dtype, ldy);
  if (rc != GPTQ_OK) return rc;
  if (ldx < n || stride_packed < 0 || stride_scales < 0) return GPTQ_ERR_INVALID_ARG;
  if (experts > 1 && (stride_packed < m * ld_packed || stride_scales < m * ld_scales)) return GPTQ_ERR_INVALID_ARG;
  if (m == 0 || rows == 0 || experts == 0) return GPTQ_OK;
  if (offsets == nullptr || Y == nullptr) return GPTQ_ERR_INVALID_ARG;
  if (n > 0 && (packed == nullptr || scales == nullptr || X == nullptr)) return GPTQ_ERR_INVALID_ARG;
  (void)ws; (void)ws_bytes;
  const MxOperands p{packed, scales, ld_packed, ld_scales, stride_packed, stride_scales, (int)m, (int)n, X, nullptr,
                     ldx, 0, (int)rows, offsets, (int)experts, Y, ldy, y_dtype};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return x_dtype == GPTQ_F16 ? launch<GPTQ_F16>(p, st) : launch<GPTQ_BF16>(p, st);
}

extern "C" gptq_status gptq_mx_gemm(const uint32_t* packed, int64_t m, int64_t n, int64_t ld_packed,
                                    const uint8_t* scales, int64_t ld_scales, const void* X, int x_dtype,
                                    int64_t batch, int64_t ldx, void* Y, int y_dtype, int64_t ldy, void* ws,
                                    size_t ws_bytes, void* stream) {
  if (x_dtype != GPTQ_F16 && x_dtype != GPTQ_BF16) return GPTQ_ERR_INVALID_ARG;
  const gptq_status rc = check(m, n, batch, 1, ld_packed, ld_scales, y_dtype, ldy);
  if (rc != GPTQ_OK) return rc;
  if (ldx < n) return GPTQ_ERR_INVALID_ARG;
  if (m == 0 || batch == 0) return GPTQ_OK;
  if (Y == nullptr || (n > 0 && (packed == nullptr || scales == nullptr || X == nullptr)))
    return GPTQ_ERR_INVALID_ARG;
  (void)ws; (void)ws_bytes;
  const MxOperands p{packed, scales, ld_packed, ld_scales, 0, 0, (int)m, (int)n, X, nullptr,
                     ldx, 0, (int)batch, nullptr, 1, Y, ldy, y_dtype};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return x_dtype == GPTQ_F16 ? launch<GPTQ_F16>(p, st) : launch<GPTQ_BF16>(p, st);
}

extern "C" gptq_status gptq_mx_scaled_gemm(const uint32_t* packed, int64_t m, int64_t n, int64_t ld_packed,
                                           const uint8_t* scales, int64_t ld_scales, const uint32_t* x_packed,
                                           int64_t batch, int64_t ld_xpacked, const uint8_t* x_scales,
                                           int64_t ld_xscales, void* Y, int y_dtype, int64_t ldy, void* ws,
                                           size_t ws_bytes, void* stream) {
  const gptq_status rc = check(m, n, batch, 1, ld_packed, ld_scales, y_dtype, ldy);
  if (rc != GPTQ_OK) return rc;
  if (ld_xpacked < ceil_div(n, 8) || ld_xscales < ceil_div(n, kMxBlock)) return GPTQ_ERR_INVALID_ARG;
  if (m == 0 || batch == 0) return GPTQ_OK;
  if (Y == nullptr || (n > 0 && (packed == nullptr || scales == nullptr || x_packed == nullptr || x_scales == nullptr)))
    return GPTQ_ERR_INVALID_ARG;
  (void)ws; (void)ws_bytes;
  const MxOperands p{packed, scales, ld_packed, ld_scales, 0, 0, (int)m, (int)n, x_packed, x_scales,
                     ld_xpacked, ld_xscales, (int)batch, nullptr, 1, Y, ldy, y_dtype};
  return launch<kMx>(p, static_cast<hipStream_t>(stream));
}
