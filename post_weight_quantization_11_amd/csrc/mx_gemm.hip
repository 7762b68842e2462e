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

// Guarded loads of a row's last columns: every address is clamped to the row
// and what lies past its end is replaced (n >= 1), without branches.
__device__ inline uint32_t load_word(const uint32_t* row, int k, int n) {
  const int nw = (n + 7) >> 3;
  uint32_t v = row[min(k, nw - 1)];
  const int left = n - 8 * k;                // columns that this word holds
  if (left < 8) v &= (1u << (4 * max(left, 0))) - 1u;
  return v;
}
__device__ inline uint32_t load_pair(const uint16_t* row, int k, int n) {
  const uint32_t lo = row[min(k, n - 1)], hi = row[min(k + 1, n - 1)];
  return (k < n ? lo : 0u) | (k + 1 < n ? hi << 16 : 0u);
}
__device__ inline uint32_t load_scale(const uint8_t* srow, int blk, int n) {
  const uint32_t v = srow[min(blk, (n - 1) >> 5)];
  return blk * kMxBlock < n ? v : (uint32_t)kMxScaleOne;
}
__device__ inline void load_block(const uint32_t* row, const uint8_t* srow, int blk, int n, u32x4& w,
                                  uint32_t& byte) {
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = load_word(row, 4 * blk + i, n);
  byte = load_scale(srow, blk, n);
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
            for (int d = 0; d < 4; ++d) x[nt][j][d] = load_pair(xrow[nt], k0 + 8 * j + 2 * d, p.n);
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
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            u32x4 hi, lo;
            split8(x[nt][j], hi, lo);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              const u32x4 wv = widen8<GPTQ_BF16>(w[rt][j], mx_scale_operand(wb[rt]));
              acc[rt][nt] = mfma16<GPTQ_BF16>(hi, wv, acc[rt][nt]);
              acc[rt][nt] = mfma16<GPTQ_BF16>(lo, wv, acc[rt][nt]);
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

// ---------------------------------------------------------------------------
// Tiled products (many rows of X).  A workgroup owns 32 WR RB rows of W x
// 32 WC CB rows of X; its WR x WC waves own 32 RB x 32 CB each, in
// v_mfma_f32_32x32x16 (16-bit X) or v_mfma_scale_f32_32x32x64_f8f6f4
// (microscaled X).
//
// A stage is 128 bytes of every row of X (64 or 256 columns), staged in LDS in
// two buffers: while a stage is multiplied the next one arrives.  The 16-byte
// chunk c of local row r lies in slot c ^ (r % 8) of the row's eight, so the
// reads of one chunk over 32 rows touch all banks evenly.
//
// 16-bit X: the codes of W go from memory straight into registers (a row's 32
// codes of a block are 16 bytes: 1/4 of what X needs) and become operands
// there; of a stage's two blocks, lane half h takes block h, and step j the
// codes 8j .. 8j+7 of both.  Microscaled X: W's codes are staged in LDS like
// X's; step j takes blocks 2j + h.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void lds_void;

// s_waitcnt immediate (gfx9 encoding): vmcnt <= v, expcnt unconstrained, lgkmcnt = 0.
constexpr int waitcnt_vm(int v) { return (v & 15) | ((v >> 4) << 14) | (7 << 4); }

// Orders LDS accesses only: loads in flight are waited for explicitly.
__device__ inline void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <int XT> __device__ inline floatx16 mfma32(u32x4 a, u32x4 b, floatx16 c);
template <> __device__ inline floatx16 mfma32<GPTQ_F16>(u32x4 a, u32x4 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(halfx8, a), __builtin_bit_cast(halfx8, b), c, 0, 0,
                                                0);
}
template <> __device__ inline floatx16 mfma32<GPTQ_BF16>(u32x4 a, u32x4 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

constexpr int kStageRow = 128;               // bytes of a row in a stage
typedef uint64_t u64_a1 __attribute__((aligned(1)));

// Work of one launch: tiles of W rows, of X rows, and parts of the columns.
struct TileGrid {
  int row_tiles, tok_tiles, splits, stages_per_split;
  float* part;                               // [split][row of X][m] sums, when splits > 1
};

// Tiles of X rows are numbered within bands of eight, all W tiles of a band
// before the next band: the workgroups an XCD runs at a time share few rows of
// either operand in its L2.
constexpr int kTokBand = 8;

// One 16-byte chunk of a row: of a whole stage, and of a row's last columns
// (zero past its end).
template <int XT>
__device__ inline u32x4 load_chunk(const char* row, int stage, int chunk) {
  const char* at = row + (int64_t)stage * kStageRow + chunk * 16;
  if constexpr (XT == kMx) return *reinterpret_cast<const u32x4_a4*>(at);
  else return *reinterpret_cast<const u32x4_a2*>(at);
}
template <int XT>
__device__ inline u32x4 load_chunk_tail(const char* row, int stage, int chunk, int n) {
  u32x4 v;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if constexpr (XT == kMx)
      v[d] = load_word(reinterpret_cast<const uint32_t*>(row), stage * 32 + chunk * 4 + d, n);
    else
      v[d] = load_pair(reinterpret_cast<const uint16_t*>(row), stage * 64 + chunk * 8 + 2 * d, n);
  }
  return v;
}

// Scale bytes of the eight blocks of a stage of microscaled columns: byte t of
// the result belongs to block 2t + h.  Blocks past the row's end have scale 1.
__device__ inline uint32_t order_scales8(uint64_t v, int h) {
  return __builtin_amdgcn_perm((uint32_t)(v >> 32), (uint32_t)v, h ? 0x07050301u : 0x06040200u);
}
__device__ inline uint32_t load_scales8(const uint8_t* srow, int stage, int h) {
  return order_scales8(*reinterpret_cast<const u64_a1*>(srow + 8 * stage), h);
}
__device__ inline uint32_t load_scales8_tail(const uint8_t* srow, int stage, int h, int n) {
  uint64_t v = 0;
#pragma unroll 1
  for (int i = 7; i >= 0; --i) v = v << 8 | load_scale(srow, 8 * stage + i, n);
  return order_scales8(v, h);
}

// The first `left` of eight neighbouring results.
template <int YT>
__device__ inline void store8(void* Y, int64_t at, int left, floatx4 lo, floatx4 hi) {
  if constexpr (YT == GPTQ_F32) {
    float* y = static_cast<float*>(Y) + at;
    if (left >= 8) {
      typedef floatx4 floatx4_a4 __attribute__((aligned(4)));
      reinterpret_cast<floatx4_a4*>(y)[0] = lo;
      reinterpret_cast<floatx4_a4*>(y)[1] = hi;
      return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) y[i] = i < 4 ? lo[i & 3] : hi[i & 3];
  } else {
    uint16_t* y = static_cast<uint16_t*>(Y) + at;
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = i < 2 ? lo[2 * i] : hi[2 * i - 4], b = i < 2 ? lo[2 * i + 1] : hi[2 * i - 3];
      if constexpr (YT == GPTQ_F16)
        v[i] = __builtin_bit_cast(uint32_t, halfx2{(_Float16)a, (_Float16)b});
      else
        v[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
    }
    if (left >= 8) {
      *reinterpret_cast<u32x4_a2*>(y) = v;
      return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) y[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
  }
}

// One tile.  DIRECT: 16-byte aligned rows; whole stages of X (and microscaled W)
// go from memory to LDS without passing through registers.  SPLIT (float16 X):
// every product as two bfloat16 ones.  Without SPLIT a float16 tile runs as if
// all its scales were exact in float16 and says at the end whether they were
// (the same answer in the whole workgroup); if not, nothing is stored and the
// caller runs it again with SPLIT: trained weights have no such scales, and a
// branch on them in the main loop made the compiler move the accumulators.
template <int XT, int WR, int WC, int RB, int CB, bool DIRECT, bool SPLIT>
__device__ inline bool tile_product(const MxOperands& p, const TileGrid& tg, const TokenTile& tile, int r0, int split,
                                    unsigned char* smem) {
  constexpr bool MX = XT == kMx;
  constexpr int kThreads = 64 * WR * WC, kWaves = WR * WC;
  constexpr int BM = 32 * WR * RB, BN = 32 * WC * CB;
  constexpr int kLdsRows = MX ? BM + BN : BN;                 // X rows first, then W rows
  constexpr int kPerThread = kLdsRows * 8 / kThreads;         // chunks a thread stages
  constexpr int kCols = MX ? 256 : 64;                        // columns per stage
  static_assert(kLdsRows % (8 * kWaves) == 0, "a wave stages eight rows at a time");
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / WC, wc = wave % WC;
  const int stages = (p.n + kCols - 1) / kCols;
  const int s_lo = split * tg.stages_per_split, s_hi = min(stages, s_lo + tg.stages_per_split);
  const uint32_t* W = p.W + (int64_t)tile.expert * p.w_stride;
  const uint8_t* S = p.S + (int64_t)tile.expert * p.s_stride;
  const char* X = static_cast<const char*>(p.X);
  const int64_t x_pitch = p.ldx * (MX ? 4 : 2), w_pitch = p.ldp * 4;

  // Staging.  Local row r: row of X (clamped to the tile's last row: what it
  // computes is not stored) or, behind those, of W.
  const char* xbase = X + (int64_t)tile.begin * x_pitch;
  const char* wbase = reinterpret_cast<const char*>(W + (int64_t)r0 * p.ldp);
  const uint8_t* sbase = S + (int64_t)r0 * p.lds;
  auto row_offset = [&](int r) -> uint32_t {
    if (!MX || r < BN) return (uint32_t)min(r, tile.end - 1 - tile.begin) * (uint32_t)x_pitch;
    return (uint32_t)min(r - BN, p.m - 1 - r0) * (uint32_t)w_pitch;
  };
  auto row_ptr = [&](int r) -> const char* { return (!MX || r < BN ? xbase : wbase) + row_offset(r); };
  u32x4 stage_regs[DIRECT ? 1 : kPerThread];
  auto fetch = [&](int st) {                 // by registers: any alignment
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int r = (tid >> 3) + i * (kThreads / 8);
      stage_regs[DIRECT ? 0 : i] = load_chunk<XT>(row_ptr(r), st, tid & 7);
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int r = (tid >> 3) + i * (kThreads / 8);
      *reinterpret_cast<u32x4*>(smem + buf * (kLdsRows * kStageRow) + r * kStageRow + (((tid & 7) ^ (r & 7)) << 4)) =
          stage_regs[DIRECT ? 0 : i];
    }
  };
  // Directly: a wave's instruction moves eight rows, lane i the chunk that
  // belongs into slot i % 8 of row i / 8.
  uint32_t direct_offset[DIRECT ? kLdsRows / (8 * kWaves) : 1];
  if constexpr (DIRECT) {
#pragma unroll
    for (int i = 0; i < kLdsRows / (8 * kWaves); ++i)
      direct_offset[i] = row_offset((wave + i * kWaves) * 8 + (lane >> 3)) + (((lane & 7) ^ (lane >> 3)) << 4);
  }
  auto fetch_direct = [&](int st, int buf) {
#pragma unroll
    for (int i = 0; i < kLdsRows / (8 * kWaves); ++i) {
      const uint32_t dst = (uint32_t)reinterpret_cast<uintptr_t>(
          (lds_void*)(smem + buf * (kLdsRows * kStageRow) + (wave + i * kWaves) * 8 * kStageRow));
      // BN / 8 is a multiple of the waves or the other way round: one i reads one operand.
      const char* src = ((wave + i * kWaves) * 8 < BN ? xbase : wbase) + (int64_t)st * kStageRow;
      // M0 is the LDS destination; the compiler does not track the load, the
      // pipeline waits for it explicitly.
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst),
                   "v"(direct_offset[DIRECT ? i : 0]), "s"(src)
                   : "memory", "m0");
    }
  };
  // A partial last stage, element by element, into the first buffer (the loop's
  // last barrier is behind it).
  auto fill_tail = [&](int st) {
#pragma unroll 1
    for (int i = 0; i < kPerThread; ++i) {
      const int r = (tid >> 3) + i * (kThreads / 8);
      const u32x4 v = load_chunk_tail<XT>(row_ptr(r), st, tid & 7, p.n);
      *reinterpret_cast<u32x4*>(smem + r * kStageRow + (((tid & 7) ^ (r & 7)) << 4)) = v;
    }
  };

  // This lane's rows of W (16-bit X: codes and scales; microscaled: scales) and
  // of X (microscaled: scales).
  uint32_t w_at[RB], ws_at[RB], xs_at[CB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const uint32_t r = (uint32_t)min((wr * RB + rb) * 32 + l32, p.m - 1 - r0);
    w_at[rb] = r * (uint32_t)w_pitch;
    ws_at[rb] = r * (uint32_t)p.lds;
  }
  const uint8_t* xsbase = p.XS + (int64_t)tile.begin * p.ldxs;
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
    xs_at[cb] = (uint32_t)min((wc * CB + cb) * 32 + l32, tile.end - 1 - tile.begin) * (uint32_t)p.ldxs;

  struct Regs {
    u32x4 w[RB];                             // codes of this lane's block (16-bit X)
    uint32_t ws[RB];                         // scale byte, or the stage's four
    uint32_t xs[CB];
  };
  Regs cur, nxt;
  auto fetch_regs = [&](int st, Regs& g) {
    if constexpr (MX) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) g.ws[rb] = load_scales8(sbase + ws_at[rb], st, h);
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) g.xs[cb] = load_scales8(xsbase + xs_at[cb], st, h);
    } else {
      const uint32_t blk = (uint32_t)(2 * st + h);
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        g.w[rb] = *reinterpret_cast<const u32x4_a4*>(wbase + (w_at[rb] + 16u * blk));
        g.ws[rb] = sbase[ws_at[rb] + blk];
      }
    }
  };
  auto fetch_regs_tail = [&](int st, Regs& g) {
    if constexpr (MX) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) g.ws[rb] = load_scales8_tail(sbase + ws_at[rb], st, h, p.n);
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) g.xs[cb] = load_scales8_tail(xsbase + xs_at[cb], st, h, p.n);
    } else {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
        load_block(reinterpret_cast<const uint32_t*>(wbase + w_at[rb]), sbase + ws_at[rb], 2 * st + h, p.n, g.w[rb],
                   g.ws[rb]);
    }
  };

  floatx16 acc[RB][CB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) acc[rb][cb] = floatx16{};

  auto frag = [&](int buf, int row, int chunk) {             // row % 32 == l32
    return *reinterpret_cast<const u32x4*>(smem + buf * (kLdsRows * kStageRow) + row * kStageRow +
                                           ((chunk ^ (l32 & 7)) << 4));
  };
  bool exact = true;                         // this lane's scales so far
  auto multiply = [&](int buf, const Regs& g) {
    if constexpr (MX) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 x[CB], w[RB];
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) x[cb] = frag(buf, (wc * CB + cb) * 32 + l32, 2 * j + h);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) w[rb] = frag(buf, BN + (wr * RB + rb) * 32 + l32, 2 * j + h);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) {
#define GPTQ_MX_STEP(J)                                                                                          \
  case J:                                                                                                        \
    acc[rb][cb] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(x[cb]), fp4_operand(w[rb]),        \
                                                                  acc[rb][cb], 4, 4, J, (int)g.xs[cb], J,        \
                                                                  (int)g.ws[rb]);                                \
    break;
            switch (j) {
              GPTQ_MX_STEP(0)
              GPTQ_MX_STEP(1)
              GPTQ_MX_STEP(2)
              GPTQ_MX_STEP(3)
            }
#undef GPTQ_MX_STEP
          }
      }
    } else {
      if constexpr (XT == GPTQ_F16 && !SPLIT) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) exact = exact && f16_exact(g.ws[rb]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (SPLIT) {
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) {
            u32x4 hi, lo;
            split8(frag(buf, (wc * CB + cb) * 32 + l32, 4 * h + j), hi, lo);
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
              const u32x4 wv = widen8<GPTQ_BF16>(g.w[rb][j], mx_scale_operand(g.ws[rb]));
              acc[rb][cb] = mfma32<GPTQ_BF16>(hi, wv, acc[rb][cb]);
              acc[rb][cb] = mfma32<GPTQ_BF16>(lo, wv, acc[rb][cb]);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        } else {
          u32x4 x[CB];
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) x[cb] = frag(buf, (wc * CB + cb) * 32 + l32, 4 * h + j);
#pragma unroll
          for (int rb = 0; rb < RB; ++rb) {
            const u32x4 wv = widen8<XT>(g.w[rb][j], mx_scale_operand(g.ws[rb]));
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) acc[rb][cb] = mfma32<XT>(x[cb], wv, acc[rb][cb]);
          }
        }
      }
    }
  };

  // Whole stages first; a partial one at the rows' end is staged alone.
  const int s_whole = min(s_hi, p.n / kCols);
  if (s_lo < s_whole) {
    if constexpr (DIRECT) {
      fetch_direct(s_lo, 0);
    } else {
      fetch(s_lo);
      put(0);
    }
    fetch_regs(s_lo, cur);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    lds_barrier();
    for (int st = s_lo; st < s_whole; ++st) {
      const int buf = (st - s_lo) & 1;
      // The last stage fetches itself again, into the buffer no one reads any
      // more: no branch around the loads.
      const int next = min(st + 1, s_whole - 1);
      if constexpr (DIRECT) fetch_direct(next, buf ^ 1);
      else fetch(next);
      fetch_regs(next, nxt);
      multiply(buf, cur);
      if constexpr (!DIRECT) put(buf ^ 1);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
      lds_barrier();
      cur = nxt;
    }
  }
  if (s_whole < s_hi) {
    fill_tail(s_whole);
    fetch_regs_tail(s_whole, cur);
    lds_barrier();
    multiply(0, cur);
  }

  // Accumulator register i of lane l: X row 8 (i / 4) + 4 (l / 32) + i % 4, W row
  // l % 32.  Each wave passes its sums through LDS of its own, 32 rows of X x
  // 64 (32) rows of W at a time, so that a lane stores eight neighbouring ones.
  if constexpr (XT == GPTQ_F16 && !SPLIT) {
    if (!__syncthreads_and(exact)) return false;
  } else {
    lds_barrier();
  }
  constexpr int RP = RB % 2 == 0 ? 2 : 1, kPitch = 32 * RP + 4;
  static_assert(kWaves * 32 * kPitch * 4 <= 2 * kLdsRows * kStageRow, "the stages' LDS holds every wave's block");
  float* my = reinterpret_cast<float*>(smem) + wave * 32 * kPitch;
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
#pragma unroll
    for (int r2 = 0; r2 < RB; r2 += RP) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int b = 0; b < RP; ++b)
          my[(8 * (i >> 2) + 4 * h + (i & 3)) * kPitch + 32 * b + l32] = acc[r2 + b][cb][i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
      constexpr int kLanes = 4 * RP;         // lanes that share a row of X
      const int xr = lane / kLanes, c = lane % kLanes * 8;
      const int r = r0 + (wr * RB + r2) * 32 + c;
#pragma unroll 1
      for (int k = 0; k < 32; k += 64 / kLanes) {
        const int x = tile.begin + (wc * CB + cb) * 32 + k + xr;
        const floatx4 lo = *reinterpret_cast<const floatx4*>(my + (k + xr) * kPitch + c);
        const floatx4 hi = *reinterpret_cast<const floatx4*>(my + (k + xr) * kPitch + c + 4);
        if (x < tile.end && r < p.m) {
          if (tg.splits > 1)
            store8<GPTQ_F32>(tg.part, ((int64_t)split * p.rows + x) * p.m + r, p.m - r, lo, hi);
          else if (p.y_dtype == GPTQ_F32)
            store8<GPTQ_F32>(p.Y, (int64_t)x * p.ldy + r, p.m - r, lo, hi);
          else if (p.y_dtype == GPTQ_F16)
            store8<GPTQ_F16>(p.Y, (int64_t)x * p.ldy + r, p.m - r, lo, hi);
          else
            store8<GPTQ_BF16>(p.Y, (int64_t)x * p.ldy + r, p.m - r, lo, hi);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
    }
  return true;
}

template <int XT, int WR, int WC, int RB, int CB, bool DIRECT>
__global__ __launch_bounds__(64 * WR * WC) void mx_tile_kernel(MxOperands p, TileGrid tg) {
  constexpr int BM = 32 * WR * RB, BN = 32 * WC * CB;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  // Workgroup -> (split, tile of X rows, tile of W rows).
  const int64_t tiles = (int64_t)tg.row_tiles * tg.tok_tiles;
  const int64_t item = xcd_contiguous(blockIdx.x, gridDim.x);
  if (item >= tiles * tg.splits) return;
  const int split = (int)(item / tiles);
  const int t = (int)(item % tiles);
  const int band = t / (kTokBand * tg.row_tiles);
  const int in_band = min(kTokBand, tg.tok_tiles - band * kTokBand);
  const int rest = t - band * kTokBand * tg.row_tiles;
  const TokenTile tile = find_tile(p, band * kTokBand + rest % in_band, BN);
  if (!tile.valid) return;
  const int r0 = rest / in_band * BM;
  const bool done = tile_product<XT, WR, WC, RB, CB, DIRECT, false>(p, tg, tile, r0, split, smem);
  if constexpr (XT == GPTQ_F16) {
    if (!done) tile_product<XT, WR, WC, RB, CB, DIRECT, true>(p, tg, tile, r0, split, smem);
  }
}

// Adds the splits' sums in order.  Rows that belong to no expert stay.
__global__ __launch_bounds__(256) void mx_join_kernel(MxOperands p, TileGrid tg) {
  int lo = 0, hi = p.rows;
  if (p.offsets != nullptr) {
    lo = min(max(p.offsets[0], 0), p.rows);
    hi = min(max(p.offsets[p.experts], 0), p.rows);
  }
  const int64_t total = (int64_t)p.rows * p.m;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t x = i / p.m, r = i - x * p.m;
    if (x < lo || x >= hi) continue;
    float v = tg.part[i];
    for (int s = 1; s < tg.splits; ++s) v += tg.part[s * total + i];
    store_y(p, x * p.ldy + r, v);
  }
}

// Tiles that the rows can form at most: every expert with rows may end in a
// partial tile.
int64_t max_tiles(int64_t rows, int64_t experts, bool grouped, int tile) {
  return grouped ? rows / tile + std::min(experts, rows) : ceil_div(rows, tile);
}

// What a product runs on, from its sizes alone.
struct Plan {
  int kind;                                  // 0: mx_rows_kernel, else a tile shape
  int splits, stages_per_split;
  size_t ws;
};

Plan make_plan(int64_t m, int64_t n, int64_t rows, int64_t experts, bool grouped, bool mx) {
  (void)m; (void)n; (void)experts; (void)grouped; (void)mx;
  Plan pl{0, 1, 1 << 30, 0};
  if (rows > 64) pl.kind = 1;
  return pl;
}

template <int XT, int WR, int WC, int RB, int CB>
gptq_status launch_tiles(const MxOperands& p, const Plan& pl, void* ws, hipStream_t st) {
  constexpr bool MX = XT == kMx;
  constexpr int BM = 32 * WR * RB, BN = 32 * WC * CB;
  constexpr int kLds = 2 * (MX ? BM + BN : BN) * kStageRow;
  TileGrid tg{(int)ceil_div(p.m, BM), (int)max_tiles(p.rows, p.experts, p.offsets != nullptr, BN), pl.splits,
              pl.stages_per_split, static_cast<float*>(ws)};
  const int64_t items = (int64_t)tg.row_tiles * tg.tok_tiles * tg.splits;
  if (items > ((int64_t)1 << 30)) return GPTQ_ERR_UNSUPPORTED;
  const unsigned grid = (unsigned)round_up(items, kXcds);
  const int xb = MX ? 4 : 2;
  const bool direct = ((reinterpret_cast<uintptr_t>(p.X) | (uint64_t)(p.ldx * xb)) & 15) == 0 &&
                      (!MX || ((reinterpret_cast<uintptr_t>(p.W) | (uint64_t)(p.ldp * 4) | (uint64_t)(p.w_stride * 4)) &
                               15) == 0);
  auto* k = direct ? mx_tile_kernel<XT, WR, WC, RB, CB, true> : mx_tile_kernel<XT, WR, WC, RB, CB, false>;
  if (kLds > 65536)
    GPTQ_TRY_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, kLds));
  k<<<grid, 64 * WR * WC, kLds, st>>>(p, tg);
  GPTQ_TRY_LAUNCH();
  if (tg.splits > 1) {
    const int64_t wgs = std::min<int64_t>(ceil_div((int64_t)p.rows * p.m, 256), 2048);
    mx_join_kernel<<<(unsigned)wgs, 256, 0, st>>>(p, tg);
    GPTQ_TRY_LAUNCH();
  }
  return GPTQ_OK;
}

template <int XT>
gptq_status launch(const MxOperands& p, hipStream_t st) {
  Plan pl = make_plan(p.m, p.n, p.rows, p.experts, p.offsets != nullptr, XT == kMx);
  // The tile kernels address the rows of a tile with 32 bits.
  constexpr int64_t kMaxPitch = (int64_t)1 << 22;
  if (p.ldx * (XT == kMx ? 4 : 2) > kMaxPitch || p.ldp * 4 > kMaxPitch || p.lds > kMaxPitch || p.ldxs > kMaxPitch)
    pl.kind = 0;
  if (pl.kind != 0) return launch_tiles<XT, 2, 2, 4, 4>(p, pl, nullptr, st);
  constexpr int kRT = 1, kNT = 1, kWaves = 8;
  constexpr int64_t kMaxGridY = 65535;
  const int64_t toks = max_tiles(p.rows, p.experts, p.offsets != nullptr, 16 * kNT);
  if (toks > kMaxGridY) return GPTQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)ceil_div(p.m, 16 * kRT), (unsigned)toks);
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
