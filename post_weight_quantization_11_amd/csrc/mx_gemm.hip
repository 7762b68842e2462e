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
#include "mx_operands.h"
#include "product.h"

#include <type_traits>

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

__device__ inline intx8 fp4_operand(u32x4 v) {
  return intx8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};   // 4-bit formats use four registers
}

// Stores a 16 x 16 block: accumulator register i of lane l is X row 4 (l / 16) + i,
// W row l % 16.
__device__ inline void store_block16(const MxOperands& p, const TokenTile& tile, int t0, int r0, floatx4 v) {
  const int lane = (int)threadIdx.x & 63, r = r0 + (lane & 15);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + 4 * (lane >> 4) + i;
    if (t < tile.end && r < p.m) store_y(p, (int64_t)t * p.ldy + r, v[i]);
  }
}

// What a wave multiplies in one unit of 128 columns (four blocks): RT x NT
// tiles of 16 rows.  As loaded, lane quarter q holds block q of its W row; X
// likewise where it is microscaled.  16-bit X: register j holds columns 32j + 8q
// .. + 7, so that the four lanes of a row read 64 neighbouring bytes.
template <int XT, int RT, int NT>
struct Unit {
  static constexpr int kX = XT == kMx ? 1 : 4;
  u32x4 w[RT], x[NT][kX];
};

// ws, xs: the four scale bytes of the unit of each W (microscaled X) row.
// SPLIT (float16 X): every product as two bfloat16 ones.  Otherwise `inexact`
// gathers whether all scales have been exact in float16.
template <int XT, bool SPLIT, int RT, int NT>
__device__ inline void multiply_unit(const Unit<XT, RT, NT>& u, const uint32_t (&ws)[RT], const uint32_t (&xs)[NT],
                                     floatx4 (&acc)[RT][NT], uint32_t& inexact) {
  if constexpr (XT == kMx) {
    const int shift = 8 * (((int)threadIdx.x >> 4) & 3);     // this lane's block
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        acc[rt][nt] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            fp4_operand(u.x[nt][0]), fp4_operand(u.w[rt]), acc[rt][nt], 4, 4, 0, (int)(xs[nt] >> shift), 0,
            (int)(ws[rt] >> shift));
  } else {
    u32x4 w[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      w[rt] = transpose_quarters(u.w[rt]);
      if constexpr (XT == GPTQ_F16 && !SPLIT) inexact |= f16_inexact4(ws[rt]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (!SPLIT) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const u32x4 wv = widen8<XT>(w[rt][j], mx_scale_operand((ws[rt] >> (8 * j)) & 255u));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) acc[rt][nt] = mfma16<XT>(u.x[nt][j], wv, acc[rt][nt]);
        }
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          u32x4 hi, lo;
          split8(u.x[nt][j], hi, lo);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const u32x4 wv = widen8<GPTQ_BF16>(w[rt][j], mx_scale_operand((ws[rt] >> (8 * j)) & 255u));
            acc[rt][nt] = mfma16<GPTQ_BF16>(hi, wv, acc[rt][nt]);
            acc[rt][nt] = mfma16<GPTQ_BF16>(lo, wv, acc[rt][nt]);
          }
        }
      }
    }
  }
}

// Few rows of X: the waves of a workgroup share RT tiles of W rows and NT tiles
// of X rows, take every KW-th quad of units (512 columns), and add their sums
// through LDS in wave order.  X comes straight from memory.  D units are in
// flight per wave; a row's sixteen scale bytes of a quad are one load, a quad
// ahead (one byte a lane and unit cost 30 of 88 us at 49152 x 12288).  Bound by
// latency at the sizes it is chosen for: 1 x 4096 x 4096 5.6 us (8.9 MB, of which
// launch and two dependent loads are 4), 64 experts' 16 x 1024 x 2048 7.5 us (the
// tile search reads the offsets first).  Returns
// false, with nothing stored, if a float16 workgroup met scales that are not
// exact in float16 (the caller then runs it again with SPLIT).
template <int XT, int RT, int NT, int D, bool SPLIT>
__device__ inline bool rows_product(const MxOperands& p, const TokenTile& tile, int r0, floatx4* red) {
  static_assert(D == 1 || D == 2 || D == 4, "the ring's slots are the same in every quad");
  constexpr bool MX = XT == kMx;
  const int lane = (int)threadIdx.x & 63, q = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = (int)blockDim.x >> 6;
  const uint32_t* wrow[RT];
  const uint8_t* wsrow[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int64_t r = min(r0 + 16 * rt + c16, p.m - 1);
    wrow[rt] = p.W + (int64_t)tile.expert * p.w_stride + r * p.ldp;
    wsrow[rt] = p.S + (int64_t)tile.expert * p.s_stride + r * p.lds;
  }
  const char* xrow[NT];
  const uint8_t* xsrow[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int64_t t = min(tile.begin + 16 * nt + c16, tile.end - 1);
    xrow[nt] = static_cast<const char*>(p.X) + t * p.ldx * (MX ? 4 : 2);
    xsrow[nt] = p.XS + t * p.ldxs;
  }
  floatx4 acc[RT][NT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[rt][nt] = floatx4{0.f, 0.f, 0.f, 0.f};
  uint32_t inexact = 0u;

  typedef Unit<XT, RT, NT> U;
  struct Scales {
    u32x4 w[RT], x[NT];                      // a quad's sixteen bytes
  };
  const int quads = p.n >> 9;                // whole ones
  // Past the last quad that quad is loaded again (and not used).
  auto load_unit = [&](int quad, int d, U& u) {
    const int unit = 4 * min(quad, quads - 1) + d;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) u.w[rt] = *reinterpret_cast<const u32x4_a4*>(wrow[rt] + 16 * unit + 4 * q);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (MX) {
        u.x[nt][0] = *reinterpret_cast<const u32x4_a4*>(xrow[nt] + 64 * unit + 16 * q);
      } else {
#pragma unroll
        for (int j = 0; j < U::kX; ++j)
          u.x[nt][j] = *reinterpret_cast<const u32x4_a2*>(xrow[nt] + 256 * unit + 64 * j + 16 * q);
      }
    }
  };
  auto load_scales = [&](int quad, Scales& s) {
    const int at = 16 * min(quad, quads - 1);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) s.w[rt] = *reinterpret_cast<const u32x4_a1*>(wsrow[rt] + at);
    if constexpr (MX) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s.x[nt] = *reinterpret_cast<const u32x4_a1*>(xsrow[nt] + at);
    }
  };
  auto multiply = [&](int d, const U& u, const Scales& s) {
    uint32_t ws[RT], xs[NT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) ws[rt] = s.w[rt][d];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xs[nt] = MX ? s.x[nt][d] : 0u;
    multiply_unit<XT, SPLIT>(u, ws, xs, acc, inexact);
  };
  if (wave < quads) {
    U u[D];
    Scales cur, nxt;
    load_scales(wave, cur);
#pragma unroll
    for (int d = 0; d < D; ++d) load_unit(wave, d, u[d]);
    for (int quad = wave; quad < quads; quad += waves) {
      load_scales(quad + waves, nxt);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        multiply(d, u[d % D], cur);
        load_unit(d + D < 4 ? quad : quad + waves, (d + D) % 4, u[d % D]);
      }
      cur = nxt;
    }
  }
  // The columns behind the last whole quad, one unit a wave.
  const int units = (p.n + 127) >> 7;
  for (int unit = 4 * quads + (wave + waves - quads % waves) % waves; unit < units; unit += waves) {
    U u;
    Scales s;
    const int blk = 4 * unit + q;
    const bool all = (unit + 1) * 128 <= p.n;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (all) {
        u.w[rt] = *reinterpret_cast<const u32x4_a4*>(wrow[rt] + 4 * blk);
        s.w[rt][0] = *reinterpret_cast<const u32_a1*>(wsrow[rt] + 4 * unit);
      } else {
        u.w[rt] = load_w4_tail(wrow[rt], 4 * blk, p.n);
        s.w[rt][0] = load_scales4(wsrow[rt], 4 * unit, p.n);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (MX) {
        if (all) {
          u.x[nt][0] = *reinterpret_cast<const u32x4_a4*>(xrow[nt] + 16 * blk);
          s.x[nt][0] = *reinterpret_cast<const u32_a1*>(xsrow[nt] + 4 * unit);
        } else {
          u.x[nt][0] = load_w4_tail(reinterpret_cast<const uint32_t*>(xrow[nt]), 4 * blk, p.n);
          s.x[nt][0] = load_scales4(xsrow[nt], 4 * unit, p.n);
        }
      } else {
#pragma unroll
        for (int j = 0; j < U::kX; ++j) {
          const int k = 128 * unit + 32 * j + 8 * q;
          if (all)
            u.x[nt][j] = *reinterpret_cast<const u32x4_a2*>(xrow[nt] + 2 * k);
          else
            u.x[nt][j] = load_x8_tail(reinterpret_cast<const uint16_t*>(xrow[nt]), k, p.n);
        }
      }
    }
    multiply(0, u, s);
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) red[((wave * RT + rt) * NT + nt) * 64 + lane] = acc[rt][nt];
  if constexpr (XT == GPTQ_F16 && !SPLIT) {
    if (!__syncthreads_and(inexact == 0u)) return false;
  } else {
    __syncthreads();
  }
  for (int o = wave; o < RT * NT; o += waves) {
    floatx4 v = red[o * 64 + lane];
    for (int w = 1; w < waves; ++w) v += red[(w * RT * NT + o) * 64 + lane];
    store_block16(p, tile, tile.begin + 16 * (o % NT), r0 + 16 * (o / NT), v);
  }
  return true;
}

template <int XT, int RT, int NT, int D>
__global__ __launch_bounds__(512) void mx_rows_kernel(MxOperands p) {
  extern __shared__ floatx4 red[];           // [wave][RT][NT][64]
  const int row_tiles = (p.m + 16 * RT - 1) / (16 * RT);
  const int slot = (int)(blockIdx.x / row_tiles), r0 = (int)(blockIdx.x % row_tiles) * 16 * RT;
  const TokenTile tile = find_tile(p, slot, 16 * NT);
  if (!tile.valid) return;
  const bool done = rows_product<XT, RT, NT, D, false>(p, tile, r0, red);
  if constexpr (XT == GPTQ_F16) {
    if (!done) rows_product<XT, RT, NT, D, true>(p, tile, r0, red);
  }
}

// Up to four rows of 16-bit X, many rows of W: every wave owns sixteen rows of W
// for all columns, and the workgroup stages X once for its waves, a quad of
// units at a time, two in LDS, in the order the matrix instructions take it: the
// 16 bytes of lane (q, row) of step j at place row ^ (4j + q) of the four (the
// matrix instruction's other rows repeat them), so that writing along a row of X
// and reading a step both touch all banks evenly.  The packed rows stream through
// registers, a quad ahead.  Bound by W's bytes: 1 x 49152 x 12288, W from memory,
// 65 us in bfloat16 and 69 in float16, 4.9 and 4.6 TB/s (87 and 92 us on the row
// kernel, whose every wave loads X itself; 79 and 84 us on 128 x 32 tiles).
constexpr int kStreamRows = 4;
template <int XT, bool SPLIT>
__device__ inline bool stream_product(const MxOperands& p, const TokenTile& tile, int r0, u32x4* xs) {
  constexpr int kPanel = 4 * 4 * 4 * kStreamRows;             // 16-byte chunks of a quad: one a thread
  const int tid = (int)threadIdx.x, lane = tid & 63, q = lane >> 4, c16 = lane & 15;
  const int64_t r = min(r0 + c16, p.m - 1);
  const uint32_t* wrow = p.W + (int64_t)tile.expert * p.w_stride + r * p.ldp;
  const uint8_t* wsrow = p.S + (int64_t)tile.expert * p.s_stride + r * p.lds;
  const uint16_t* X = static_cast<const uint16_t*>(p.X) + (int64_t)tile.begin * p.ldx;
  const int last = tile.end - tile.begin - 1;
  floatx4 acc[1][1] = {{floatx4{0.f, 0.f, 0.f, 0.f}}};
  uint32_t inexact = 0u;
  typedef Unit<XT, 1, 1> U;
  const int quads = p.n >> 9;

  // Thread t stages chunk t along the rows of X, 64 to a row.
  const int xrow = tid >> 6, xat = tid & 63, xjq = xat & 15;
  const uint16_t* xsrc = X + (int64_t)min(xrow, last) * p.ldx + xat * 8;
  const int xslot = ((xat >> 4) * 16 + xjq) * kStreamRows + ((xrow ^ xjq) & (kStreamRows - 1));
  u32x4 xr, w[4], cur, nxt;
  auto fetch_x = [&](int quad) { xr = *reinterpret_cast<const u32x4_a2*>(xsrc + min(quad, quads - 1) * 512); };
  auto put_x = [&](int buf) { xs[buf * kPanel + xslot] = xr; };
  auto load_w = [&](int quad, int d) {
    w[d] = *reinterpret_cast<const u32x4_a4*>(wrow + 16 * (4 * min(quad, quads - 1) + d) + 4 * q);
  };
  auto load_scales = [&](int quad) {
    return *reinterpret_cast<const u32x4_a1*>(wsrow + 16 * min(quad, quads - 1));
  };
  const uint32_t no_xs[1] = {};
  if (quads > 0) {
    fetch_x(0);
    cur = load_scales(0);
#pragma unroll
    for (int d = 0; d < 4; ++d) load_w(0, d);
    put_x(0);
    lds_barrier();
    for (int quad = 0; quad < quads; ++quad) {
      fetch_x(quad + 1);
      nxt = load_scales(quad + 1);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        U u;
        const uint32_t ws[1] = {cur[d]};
        u.w[0] = w[d];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          u.x[0][j] = xs[(quad & 1) * kPanel + (d * 16 + 4 * j + q) * kStreamRows + ((c16 ^ q) & (kStreamRows - 1))];
        multiply_unit<XT, SPLIT>(u, ws, no_xs, acc, inexact);
        load_w(quad + 1, d);
      }
      put_x((quad + 1) & 1);
      lds_barrier();
      cur = nxt;
    }
  }
  // The columns behind the last whole quad, X from memory.
  for (int unit = 4 * quads; unit < (p.n + 127) >> 7; ++unit) {
    U u;
    u.w[0] = load_w4_tail(wrow, 16 * unit + 4 * q, p.n);
    const uint32_t ws[1] = {load_scales4(wsrow, 4 * unit, p.n)};
    const uint16_t* x = X + (int64_t)min(c16, last) * p.ldx;
#pragma unroll
    for (int j = 0; j < 4; ++j) u.x[0][j] = load_x8_tail(x, 128 * unit + 32 * j + 8 * q, p.n);
    multiply_unit<XT, SPLIT>(u, ws, no_xs, acc, inexact);
  }
  if constexpr (XT == GPTQ_F16 && !SPLIT) {
    if (!__syncthreads_and(inexact == 0u)) return false;
  }
  store_block16(p, tile, tile.begin, r0, acc[0][0]);
  return true;
}

template <int XT>
__global__ __launch_bounds__(256) void mx_stream_kernel(MxOperands p) {
  __shared__ u32x4 xs[2 * 64 * kStreamRows]; // [2][unit][step][quarter][row]
  const int r0 = (int)blockIdx.x * 64 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) * 16;
  const TokenTile tile{0, 0, p.rows, true};  // never grouped by expert, at most kStreamRows rows
  const bool done = stream_product<XT, false>(p, tile, r0, xs);
  if constexpr (XT == GPTQ_F16) {
    if (!done) stream_product<XT, true>(p, tile, r0, xs);
  }
}

// ---------------------------------------------------------------------------
// Tiled products (many rows of X).  A workgroup owns 32 WR RB rows of W x
// 32 WC CB rows of X; its WR x WC waves own 32 RB x 32 CB each, in
// v_mfma_f32_32x32x16 (16-bit X) or v_mfma_scale_f32_32x32x64_f8f6f4
// (microscaled X).
//
// A panel is 128 bytes of every row of X (64 or 256 columns), a stage one or
// more panels, staged in LDS in two buffers: while a stage is multiplied the
// next one arrives.  The 16-byte chunk c of a panel's local row r lies in slot
// c ^ r % 8 ^ r / 8 % 2 of the row's eight: sixteen neighbouring rows' chunks c
// cover all 64 banks (with c ^ r % 8 alone rows r and r + 8 share theirs, which
// doubled the cycles LDS was busy).
//
// 16-bit X: the codes of W (a row's 32 codes of a block are 16 bytes: 1/4 of what
// X needs) become operands in the registers of the lanes that use them, loaded
// there or staged in LDS first; of a panel's two blocks, lane half h takes block
// h, and step j the codes 8j .. 8j+7 of both.  Microscaled X: W's codes are staged
// in LDS like X's; step j takes blocks 2j + h.
//
// Measured: 16 x 49152 x 12288 83 us (128 x 32; 324 MB, 3.9 TB/s: bound by W's
// bytes, 384 workgroups on 256 CUs), 77 x 4099 x 11007 20 us (five splits: a
// chain of 9 stages, 16 us, and the join, 4), 64 experts' 1531 x 1030 x 2044 32 us
// (84 MB: eight stages a workgroup, first loads and the stores), 2048 x 11008 x
// 4096 148 us (256 x 128; 1.24 PFLOP/s), 4096 x 8192 x 8192 374 us (256 x 256;
// 1.47 PFLOP/s, the matrix cores 80% busy at 1.7 GHz: power).  Microscaled: 4096 x
// 12288 x 12288 290 us (4.3 PFLOP/s, the matrix cores 57% busy at 1.8 GHz; with
// the loads from memory taken out 275: LDS reads, six 16-byte ones a lane for
// eight products, and the products do not overlap fully.  Four waves of 128 x 128
// read a third less but took 306, one wave a SIMD).
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void lds_void;

template <int XT> __device__ inline floatx16 mfma32(u32x4 a, u32x4 b, floatx16 c);
template <> __device__ inline floatx16 mfma32<GPTQ_F16>(u32x4 a, u32x4 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(halfx8, a), __builtin_bit_cast(halfx8, b), c, 0, 0,
                                                0);
}
template <> __device__ inline floatx16 mfma32<GPTQ_BF16>(u32x4 a, u32x4 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

constexpr int kPanelRow = 128;               // bytes of a row in a panel
__device__ inline int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// Floats per row of X in a wave's output block: two (one) row blocks of W, and
// four so that neighbouring rows start in different banks.
constexpr int out_pitch(int row_blocks) { return (row_blocks % 2 == 0 ? 64 : 32) + 4; }

// LDS of a tile: two buffers of staged rows, later the waves' output blocks.
// Behind the buffers the microscaled scales of eight stages, or (WL) the codes of
// W of two.
template <int XT, int WR, int WC, int RB, int CB, int PB, bool WL>
constexpr int tile_lds() {
  const int rows = 32 * (WC * CB + (XT == kMx ? WR * RB : 0));
  const int behind = XT == kMx ? 8 * rows * 8 : WL ? 2 * 32 * WR * RB * 32 * PB : 0;
  return std::max(2 * PB * rows * kPanelRow + behind, WR * WC * 32 * out_pitch(RB) * 4);
}

// One 16-byte chunk of a row: of a whole panel, and of a row's last columns
// (zero past its end).
template <int XT>
__device__ inline u32x4 load_chunk(const char* row, int panel, int chunk) {
  const char* at = row + (int64_t)panel * kPanelRow + chunk * 16;
  if constexpr (XT == kMx) return *reinterpret_cast<const u32x4_a4*>(at);
  else return *reinterpret_cast<const u32x4_a2*>(at);
}
template <int XT>
__device__ inline u32x4 load_chunk_tail(const char* row, int panel, int chunk, int n) {
  if constexpr (XT == kMx) return load_w4_tail(reinterpret_cast<const uint32_t*>(row), panel * 32 + chunk * 4, n);
  else return load_x8_tail(reinterpret_cast<const uint16_t*>(row), panel * 64 + chunk * 8, n);
}

// The scale bytes of the eight blocks of a microscaled stage as the lane halves
// use them: word h holds blocks h, 2 + h, 4 + h and 6 + h.
__device__ inline u32x2 order_scales8(uint32_t lo, uint32_t hi) {
  return u32x2{__builtin_amdgcn_perm(hi, lo, 0x06040200u), __builtin_amdgcn_perm(hi, lo, 0x07050301u)};
}
__device__ inline uint32_t load_scales8_tail(const uint8_t* srow, int stage, int h, int n) {
  return order_scales8(load_scales4(srow, 8 * stage, n), load_scales4(srow, 8 * stage + 4, n))[h];
}

// Step `step` of a microscaled stage: byte `step` of the scales.
__device__ inline floatx16 mfma_mx(int step, u32x4 x, uint32_t xs, u32x4 w, uint32_t ws, floatx16 c) {
  const intx8 a = fp4_operand(x), b = fp4_operand(w);
  switch (step) {                            // the byte is an immediate
    case 0: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, 0, (int)xs, 0, (int)ws);
    case 1: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, 1, (int)xs, 1, (int)ws);
    case 2: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, 2, (int)xs, 2, (int)ws);
    default: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, 3, (int)xs, 3, (int)ws);
  }
}

// Stores a workgroup's sums.  Accumulator register i of lane l: X row 8 (i / 4) +
// 4 (l / 32) + i % 4, W row l % 32.  Each wave passes its sums through LDS of its
// own (the stages are no longer read), 32 rows of X x 64 (32) rows of W at a
// time, so that a lane stores eight neighbouring ones.
template <int WR, int WC, int RB, int CB>
__device__ inline void store_tile(const MxOperands& p, const TileGrid& tg, const TokenTile& tile, int r0, int split,
                                  const floatx16 (&acc)[RB][CB], unsigned char* smem) {
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / WC, wc = wave % WC;
  constexpr int RP = RB % 2 == 0 ? 2 : 1, kPitch = out_pitch(RB);
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
}

// One tile.  PB: panels of 128 bytes per row in a stage.  DIRECT: 16-byte
// aligned rows; whole stages of X (and microscaled W) go from memory to LDS
// without passing through registers.  WL (16-bit X, 16-byte aligned rows of W):
// so do W's codes, 32 PB bytes of a row at a time, where the lanes that use them
// would load 32 (64 x 11008 x 4096 on 128 x 32 tiles 20 -> 14.5 us).  SPLIT (float16
// X): every product as two bfloat16 ones.  Without SPLIT a float16 tile runs as if all its scales were
// exact in float16 and says at the end whether they were (the same answer in
// the whole workgroup); if not, nothing is stored and the caller runs it again
// with SPLIT: trained weights have no such scales, and a branch on them in the
// main loop made the compiler move the accumulators.
//
// Pipeline, 16-bit X: a step's operands are read from LDS while the step before
// it multiplies.  The one barrier of a stage stands in its last step, between the
// two halves of that step's products: every wave then holds the step's operands,
// so the other buffer is complete (its loads were waited for) and this one is
// free, and the next stage's first reads overlap the second half.
// Microscaled X, whose steps take half as long: operands are read two steps
// ahead, so the barrier stands in the middle of the stage, and behind it the
// stage after the next is fetched (512 x 4096 x 11008 36 -> 32 us, 256 x 12288 x
// 12288 47 -> 42; the 256 x 256 tiles, at half the matrix cores' rate, lose 1%).
template <int XT, int WR, int WC, int RB, int CB, int PB, bool DIRECT, bool WL, bool SPLIT>
__device__ inline bool tile_product(const MxOperands& p, const TileGrid& tg, const TokenTile& tile, int r0, int split,
                                    unsigned char* smem) {
  constexpr bool MX = XT == kMx;
  static_assert(MX ? PB == 1 && !WL : PB == 2 || PB == 4, "microscaled stages are one panel, with W's");
  constexpr int kThreads = 64 * WR * WC, kWaves = WR * WC;
  constexpr int BM = 32 * WR * RB, BN = 32 * WC * CB;
  constexpr int kLdsRows = MX ? BM + BN : BN;                 // X rows first, then W rows
  constexpr int kPanel = kLdsRows * kPanelRow, kBuf = PB * kPanel;
  constexpr int kPerThread = PB * kLdsRows * 8 / kThreads;    // chunks a thread stages
  constexpr int kRowStep = kThreads / 8;                      // rows that the threads' chunks cover at once
  constexpr int kDirect = PB * kLdsRows / (8 * kWaves);       // direct loads a wave issues per stage
  constexpr int kCols = MX ? 256 : 64 * PB;                   // columns per stage
  constexpr int kSteps = 4 * PB;
  static_assert(kLdsRows % (8 * kWaves) == 0, "a wave stages eight rows at a time");
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / WC, wc = wave % WC;
  const int stages = (p.n + kCols - 1) / kCols;
  const int per_split = tg.cols_per_split / kCols;
  const int s_lo = split * per_split, s_hi = min(stages, s_lo + per_split);
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
  // Chunk i of this thread: panel and local row.
  auto my_panel = [&](int i) { return i / (kPerThread / PB); };
  auto my_row = [&](int i) { return (tid >> 3) + i % (kPerThread / PB) * kRowStep; };
  auto my_slot = [&](int buf, int i) {
    const int r = my_row(i);
    return reinterpret_cast<u32x4*>(smem + buf * kBuf + my_panel(i) * kPanel + r * kPanelRow +
                                    (((tid & 7) ^ swizzle(r)) << 4));
  };
  u32x4 stage_regs[DIRECT ? 1 : kPerThread];
  auto fetch = [&](int st) {                 // by registers: any alignment
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      stage_regs[DIRECT ? 0 : i] = load_chunk<XT>(row_ptr(my_row(i)), st * PB + my_panel(i), tid & 7);
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) *my_slot(buf, i) = stage_regs[DIRECT ? 0 : i];
  };
  // Directly: a wave's instruction moves eight rows, lane i the chunk that
  // belongs into slot i % 8 of row i / 8.  (Eight-row groups alternate between
  // the waves, so a wave's are all even or all odd.)
  static_assert(kWaves % 2 == 0, "a wave's eight-row groups have one parity");
  uint32_t direct_offset[DIRECT ? kDirect / PB : 1];
  if constexpr (DIRECT) {
#pragma unroll
    for (int i = 0; i < kDirect / PB; ++i)
      direct_offset[i] =
          row_offset((wave + i * kWaves) * 8 + (lane >> 3)) + (((lane & 7) ^ swizzle(wave * 8 + (lane >> 3))) << 4);
  }
  auto fetch_direct = [&](int st, int buf, int i) {
    const int rows8 = wave + i % (kDirect / PB) * kWaves, panel = i / (kDirect / PB);
    const uint32_t dst = (uint32_t)reinterpret_cast<uintptr_t>(
        (lds_void*)(smem + buf * kBuf + panel * kPanel + rows8 * 8 * kPanelRow));
    const char* src = (!MX || rows8 * 8 < BN ? xbase : wbase) + (int64_t)(st * PB + panel) * kPanelRow;
    // M0 is the LDS destination; the compiler does not track the load, the
    // pipeline waits for it explicitly.
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst),
                 "v"(direct_offset[DIRECT ? i % (kDirect / PB) : 0]), "s"(src)
                 : "memory", "m0");
  };
  // A partial last stage, element by element, into the first buffer (the loop's
  // last barrier is behind it).
  auto fill_tail = [&](int st) {
#pragma unroll 4
    for (int i = 0; i < kPerThread; ++i)
      *my_slot(0, i) = load_chunk_tail<XT>(row_ptr(my_row(i)), st * PB + my_panel(i), tid & 7, p.n);
  };

  // Microscaled: the scale bytes of four stages (a group: 32 bytes of every
  // local row) are staged together, four lanes to a row, in the order the lanes
  // use them: [two groups][stage][row][half].  Each stage of a group fetches a
  // quarter of the rows of the next group, so the loop has no branch (one made
  // the compiler copy the accumulators).  Loaded by the lanes that use them,
  // eight bytes a row and stage, the scales cost a third of the kernel's time.
  constexpr int kQuarter = kLdsRows / 4;
  constexpr int kScaleLoads = MX ? (kQuarter * 4 + kThreads - 1) / kThreads : 1;
  uint32_t* scale_lds = reinterpret_cast<uint32_t*>(smem + 2 * kBuf);
  u32x2 scale_regs[kScaleLoads];
  const int s_whole = min(s_hi, p.n / kCols);
  auto scale_row = [&](int quarter, int i) {
    return quarter * kQuarter + min((tid + i * kThreads) >> 2, kQuarter - 1);
  };
  auto fetch_scales = [&](int group, int quarter) {
    const int st = min(s_lo + 4 * group + (tid & 3), s_whole - 1);
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) {
      const int r = scale_row(quarter, i);
      const uint8_t* row = r < BN ? p.XS + (int64_t)min(tile.begin + r, tile.end - 1) * p.ldxs
                                  : S + (int64_t)min(r0 + r - BN, p.m - 1) * p.lds;
      scale_regs[i] = *reinterpret_cast<const u32x2_a1*>(row + 8 * st);
    }
  };
  auto put_scales = [&](int group, int quarter) {
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i)
      *reinterpret_cast<u32x2*>(scale_lds + ((4 * (group & 1) + (tid & 3)) * kLdsRows + scale_row(quarter, i)) * 2) =
          order_scales8(scale_regs[i][0], scale_regs[i][1]);
  };

  // This lane's rows of W (16-bit X: codes and scales).
  uint32_t w_at[RB], ws_at[RB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const uint32_t r = (uint32_t)min((wr * RB + rb) * 32 + l32, p.m - 1 - r0);
    w_at[rb] = r * (uint32_t)w_pitch;
    ws_at[rb] = r * (uint32_t)p.lds;
  }
  constexpr int kWRow = 32 * PB, kWLanes = 2 * PB, kWRows = 64 / kWLanes;    // a row, its lanes, rows a load
  constexpr int kWLoads = WL ? BM / (kWRows * kWaves) : 1;    // a wave's per stage
  static_assert(!WL || BM % (kWRows * kWaves) == 0, "every wave loads whole rows");
  unsigned char* w_lds = smem + 2 * kBuf;    // [2][BM][kWRow]
  auto w_swizzle = [](int row) { return PB == 4 ? swizzle(row) : (row >> 2) & 3; };
  uint32_t w_direct[kWLoads], w_frag[WL ? PB : 1];
  if constexpr (WL) {
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) {
      const int r = (wave + i * kWaves) * kWRows + lane / kWLanes;
      w_direct[i] = (uint32_t)min(r, p.m - 1 - r0) * (uint32_t)w_pitch + (((lane % kWLanes) ^ w_swizzle(r)) << 4);
    }
#pragma unroll
    for (int u = 0; u < PB; ++u)
      w_frag[u] = (uint32_t)((wr * RB * 32 + l32) * kWRow + (((2 * u + h) ^ w_swizzle(l32)) << 4));
  }
  auto fetch_codes = [&](int st, int buf) {
    if constexpr (WL) {
#pragma unroll
      for (int i = 0; i < kWLoads; ++i) {
        const uint32_t dst = (uint32_t)reinterpret_cast<uintptr_t>(
            (lds_void*)(w_lds + buf * (BM * kWRow) + (wave + i * kWaves) * kWRows * kWRow));
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst), "v"(w_direct[i]),
                     "s"(wbase + (int64_t)st * kWRow)
                     : "memory", "m0");
      }
    }
  };

  struct Regs {
    u32x4 w[MX ? 1 : PB][RB];                // codes of this lane's block of each panel (16-bit X)
    uint32_t ws[(PB + 1) / 2][RB];           // scale bytes of two panels' blocks; microscaled: of the stage's four
    uint32_t xs[CB];
  };
  Regs cur, nxt;
  auto fetch_regs = [&](int st, Regs& g) {
    if constexpr (!MX) {
      if constexpr (!WL) {
#pragma unroll
        for (int u = 0; u < PB; ++u)
#pragma unroll
          for (int rb = 0; rb < RB; ++rb) {
            const uint32_t blk = (uint32_t)(2 * (st * PB + u) + h);
            g.w[u][rb] = *reinterpret_cast<const u32x4_a4*>(wbase + (w_at[rb] + 16u * blk));
          }
      }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        const uint8_t* at = sbase + (ws_at[rb] + 2u * PB * st);
#pragma unroll
        for (int i = 0; i < PB / 2; ++i) g.ws[i][rb] = reinterpret_cast<const u32_a1*>(at)[i];
      }
    }
  };
  // What of a stage's registers comes from LDS.
  auto read_regs = [&](int st, int buf, Regs& g) {
    if constexpr (WL) {
#pragma unroll
      for (int u = 0; u < PB; ++u)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
          g.w[u][rb] = *reinterpret_cast<const u32x4*>(w_lds + buf * (BM * kWRow) + w_frag[u] + rb * 32 * kWRow);
    }
    if constexpr (MX) {
      const uint32_t* at = scale_lds + ((st - s_lo) & 7) * kLdsRows * 2 + l32 * 2 + h;
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) g.xs[cb] = at[(wc * CB + cb) * 64];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) g.ws[0][rb] = at[(BN + (wr * RB + rb) * 32) * 2];
    }
  };
  auto fetch_regs_tail = [&](int st, Regs& g) {
    if constexpr (MX) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
        g.ws[0][rb] = load_scales8_tail(S + (int64_t)min(r0 + (wr * RB + rb) * 32 + l32, p.m - 1) * p.lds, st, h, p.n);
#pragma unroll
      for (int cb = 0; cb < CB; ++cb)
        g.xs[cb] = load_scales8_tail(
            p.XS + (int64_t)min(tile.begin + (wc * CB + cb) * 32 + l32, tile.end - 1) * p.ldxs, st, h, p.n);
    } else {
#pragma unroll
      for (int u = 0; u < PB; ++u)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          const int blk = 2 * (st * PB + u) + h;
          g.w[u][rb] = load_w4_tail(reinterpret_cast<const uint32_t*>(wbase + w_at[rb]), 4 * blk, p.n);
          if (u % 2 == 0) g.ws[u / 2][rb] = load_scales4(sbase + ws_at[rb], 2 * (st * PB + u), p.n);
        }
    }
  };

  floatx16 acc[RB][CB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) acc[rb][cb] = floatx16{};

  // The operands of one step that come from LDS.
  struct Frags {
    u32x4 x[CB], w[MX ? RB : 1];
  };
  Frags f[MX ? 4 : 2];
  // This lane's address of chunk j in the wave's first X row block (and, the
  // constant w_off further, its first W row block).
  uint32_t frag_at[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    frag_at[j] = (uint32_t)((wc * CB * 32 + l32) * kPanelRow + (((MX ? 2 * j + h : 4 * h + j) ^ swizzle(l32)) << 4));
  const uint32_t w_off = (uint32_t)((BN + (wr * RB - wc * CB) * 32) * kPanelRow);
  auto load_frags = [&](int buf, int step, Frags& o) {
    const unsigned char* at = smem + buf * kBuf + (MX ? 0 : step / 4) * kPanel + frag_at[step % 4];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) o.x[cb] = *reinterpret_cast<const u32x4*>(at + cb * 32 * kPanelRow);
    if constexpr (MX) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) o.w[rb] = *reinterpret_cast<const u32x4*>(at + w_off + rb * 32 * kPanelRow);
    }
  };
  // This lane's scale byte in panel u.
  auto scale_byte = [&](const Regs& g, int u, int rb) { return (g.ws[u / 2][rb] >> (16 * (u % 2) + 8 * h)) & 255u; };
  // Products of one step, row blocks [lo, hi).
  auto products = [&](int step, const Frags& o, const Regs& g, int lo, int hi) {
    if constexpr (SPLIT) {
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        u32x4 top, rest;
        split8(o.x[cb], top, rest);
#pragma unroll
        for (int rb = lo; rb < hi; ++rb) {
          const u32x4 wv = widen8<GPTQ_BF16>(g.w[step / 4][rb][step % 4], mx_scale_operand(scale_byte(g, step / 4, rb)));
          acc[rb][cb] = mfma32<GPTQ_BF16>(top, wv, acc[rb][cb]);
          acc[rb][cb] = mfma32<GPTQ_BF16>(rest, wv, acc[rb][cb]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int rb = lo; rb < hi; ++rb) {
        if constexpr (MX) {
#pragma unroll
          for (int cb = 0; cb < CB; ++cb)
            acc[rb][cb] = mfma_mx(step, o.x[cb], g.xs[cb], o.w[rb], g.ws[0][rb], acc[rb][cb]);
        } else {
          const u32x4 wv = widen8<XT>(g.w[step / 4][rb][step % 4], mx_scale_operand(scale_byte(g, step / 4, rb)));
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) acc[rb][cb] = mfma32<XT>(o.x[cb], wv, acc[rb][cb]);
        }
      }
    }
  };
  // Asks the scheduler for one LDS read and up to two conversions behind each of
  // `count` products.
  auto interleave = [&](int count) {
    if constexpr (!SPLIT) {
#pragma unroll
      for (int i = 0; i < count; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
        __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);   // two VALU
      }
    }
  };
  bool exact = true;                         // this lane's scales so far
  auto check_scales = [&](const Regs& g) {
    if constexpr (XT == GPTQ_F16 && !SPLIT) {
#pragma unroll
      for (int u = 0; u < PB; ++u)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) exact = exact && f16_exact(scale_byte(g, u, rb));
    }
  };

  // Whole stages first; a partial one at the rows' end is staged alone.
  if constexpr (MX) {
    if (s_lo < s_whole) {
      // The last stages fetch the last one again, into buffers no one reads any
      // more: no branch around the loads.
      auto stage = [&](int st, int buf) {
        if constexpr (DIRECT) {
#pragma unroll
          for (int i = 0; i < kDirect; ++i) fetch_direct(min(st, s_whole - 1), buf, i);
        } else {
          fetch(min(st, s_whole - 1));
        }
      };
      stage(s_lo, 0);
      if constexpr (!DIRECT) put(0);
      stage(s_lo + 1, 1);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        fetch_scales(0, q);
        put_scales(0, q);
      }
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
      lds_barrier();
      load_frags(0, 0, f[0]);
      load_frags(0, 1, f[1]);
      read_regs(s_lo, 0, cur);
      fetch_scales(1, 0);
      for (int st = s_lo; st < s_whole; ++st) {
        const int buf = (st - s_lo) & 1;
#pragma unroll
        for (int step = 0; step < 2; ++step) {
          load_frags(buf, step + 2, f[step + 2]);
          products(step, f[step], cur, 0, RB);
          interleave(RB * CB);
        }
        if constexpr (!DIRECT) put(buf ^ 1);
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        put_scales(((st - s_lo) >> 2) + 1, (st - s_lo) & 3);
        lds_barrier();
        stage(st + 2, buf);
        fetch_scales(((st + 1 - s_lo) >> 2) + 1, (st + 1 - s_lo) & 3);
        __builtin_amdgcn_sched_barrier(0);   // the loads are issued before the products
        read_regs(min(st + 1, s_whole - 1), buf ^ 1, nxt);
#pragma unroll
        for (int step = 2; step < 4; ++step) {
          load_frags(buf ^ 1, step - 2, f[step - 2]);
          products(step, f[step], cur, 0, RB);
          interleave(RB * CB);
        }
        cur = nxt;
      }
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));   // none is left in flight to the buffers
    }
  } else if (s_lo < s_whole) {
    if constexpr (DIRECT) {
#pragma unroll
      for (int i = 0; i < kDirect; ++i) fetch_direct(s_lo, 0, i);
    } else {
      fetch(s_lo);
      put(0);
    }
    fetch_codes(s_lo, 0);
    fetch_regs(s_lo, cur);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    lds_barrier();
    load_frags(0, 0, f[0]);
    read_regs(s_lo, 0, cur);
    for (int st = s_lo; st < s_whole; ++st) {
      const int buf = (st - s_lo) & 1;
      // The last stage fetches itself again, into the buffer no one reads any
      // more: no branch around the loads.
      const int next = min(st + 1, s_whole - 1);
      if constexpr (DIRECT) {
#pragma unroll
        for (int i = 0; i < kDirect; ++i) fetch_direct(next, buf ^ 1, i);
      } else {
        fetch(next);
      }
      fetch_codes(next, buf ^ 1);
      fetch_regs(next, nxt);
      __builtin_amdgcn_sched_barrier(0);     // the loads are issued before the products
      check_scales(cur);
#pragma unroll
      for (int step = 0; step < kSteps - 1; ++step) {
        load_frags(buf, step + 1, f[(step + 1) & 1]);
        products(step, f[step & 1], cur, 0, RB);
        interleave(RB * CB);
      }
      products(kSteps - 1, f[1], cur, 0, RB / 2);
      interleave(RB / 2 * CB);
      if constexpr (!DIRECT) put(buf ^ 1);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
      lds_barrier();
      load_frags(buf ^ 1, 0, f[0]);
      read_regs(next, buf ^ 1, nxt);
      products(kSteps - 1, f[1], cur, RB / 2, RB);
      interleave((RB - RB / 2) * CB);
      cur = nxt;
    }
  }
  if (s_lo <= s_whole && s_whole < s_hi) {
    lds_barrier();                           // the loop's last reads are done
    fill_tail(s_whole);
    fetch_regs_tail(s_whole, cur);
    check_scales(cur);
    lds_barrier();
#pragma unroll
    for (int step = 0; step < kSteps; ++step) {
      load_frags(0, step, f[0]);
      products(step, f[0], cur, 0, RB);
    }
  }

  if constexpr (XT == GPTQ_F16 && !SPLIT) {
    if (!__syncthreads_and(exact)) return false;
  } else {
    lds_barrier();
  }
  store_tile<WR, WC, RB, CB>(p, tg, tile, r0, split, acc, smem);
  return true;
}

// One large tile of 16-bit X with 16-byte aligned rows of both operands.  As
// tile_product, but the codes of W are staged in LDS too, a super-stage of SP
// panels (64 SP columns: 32 SP bytes of a row) at a time, and its scale bytes
// with them: loaded into registers by the lanes that use them, 32 bytes of a row
// at a time, codes and scales took 59 and 56 of 433 us at 4096 x 8192 x 8192.  A
// stage of X is one panel; each of the SP stages of a super-stage fetches its
// share of the next one's W, and each super-stage a quarter of the rows of the
// next four super-stages' scales (no branch in the loop).
template <int XT, int WR, int WC, int RB, int CB, int SP>
constexpr int big_tile_lds() {
  const int x = 32 * WC * CB, w = 32 * WR * RB;
  return std::max(2 * x * kPanelRow + 2 * w * 32 * SP + 8 * w * 2 * SP, WR * WC * 32 * out_pitch(RB) * 4);
}

template <int XT, int WR, int WC, int RB, int CB, int SP, bool SPLIT>
__device__ inline bool big_tile_product(const MxOperands& p, const TileGrid& tg, const TokenTile& tile, int r0,
                                        int split, unsigned char* smem) {
  static_assert(SP == 2 || SP == 4, "64 or 128 bytes of a row");
  constexpr int kThreads = 64 * WR * WC, kWaves = WR * WC;
  constexpr int BM = 32 * WR * RB, BN = 32 * WC * CB, kCols = 64 * SP;
  constexpr int kWRow = 32 * SP, kWLanes = 2 * SP, kWRows = 64 / kWLanes;    // of W: a row, its lanes, rows a load
  constexpr int kX = BN * kPanelRow, kW = BM * kWRow;         // bytes of a buffer
  constexpr int kXLoads = BN / (8 * kWaves), kWLoads = BM / (32 * kWaves);   // a wave's per stage
  static_assert(BN % (8 * kWaves) == 0 && BM % (32 * kWaves) == 0 && kWaves % 2 == 0, "every wave loads whole rows");
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / WC, wc = wave % WC;
  unsigned char* xs = smem;                  // [2][BN][128]
  unsigned char* wsm = smem + 2 * kX;        // [2][BM][kWRow]
  unsigned char* ssm = wsm + 2 * kW;         // [8 super-stages][BM][2 SP]
  const int64_t x_pitch = p.ldx * 2, w_pitch = p.ldp * 4;
  const char* xbase = static_cast<const char*>(p.X) + (int64_t)tile.begin * x_pitch;
  const char* wbase = reinterpret_cast<const char*>(p.W + (int64_t)tile.expert * p.w_stride + (int64_t)r0 * p.ldp);
  const uint8_t* sbase = p.S + (int64_t)tile.expert * p.s_stride + (int64_t)r0 * p.lds;
  auto x_row = [&](int r) { return (uint32_t)min(r, tile.end - 1 - tile.begin) * (uint32_t)x_pitch; };
  auto w_row = [&](int r) { return (uint32_t)min(r, p.m - 1 - r0) * (uint32_t)w_pitch; };
  // Slot of a row's chunk of W: sixteen neighbouring rows' cover all banks.
  auto w_swizzle = [](int row) { return SP == 4 ? swizzle(row) : (row >> 2) & 3; };

  // Super-stages [lo, hi) of this split; whole ones below `whole`.
  const int per_split = tg.cols_per_split / kCols;
  const int lo = split * per_split, hi = min((p.n + kCols - 1) / kCols, lo + per_split), whole = min(hi, p.n / kCols);
  uint32_t x_at[kXLoads], w_at[SP * kWLoads];
#pragma unroll
  for (int i = 0; i < kXLoads; ++i)          // source chunk of the lane's slot
    x_at[i] = x_row((wave + i * kWaves) * 8 + (lane >> 3)) + (((lane & 7) ^ swizzle(wave * 8 + (lane >> 3))) << 4);
#pragma unroll
  for (int i = 0; i < SP * kWLoads; ++i) {
    const int r = (wave + i * kWaves) * kWRows + lane / kWLanes;
    w_at[i] = w_row(r) + (((lane % kWLanes) ^ w_swizzle(r)) << 4);
  }
  auto direct = [&](unsigned char* dst, const char* src, uint32_t offset) {
    // As in tile_product: M0 is the LDS destination, waited for explicitly.
    const uint32_t d = (uint32_t)reinterpret_cast<uintptr_t>((lds_void*)dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(d), "v"(offset), "s"(src)
                 : "memory", "m0");
  };
  auto fetch_x = [&](int panel, int buf) {
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
      direct(xs + buf * kX + (wave + i * kWaves) * 8 * kPanelRow, xbase + (int64_t)panel * kPanelRow, x_at[i]);
  };
  auto fetch_w = [&](int super, int share) {
#pragma unroll
    for (int i = share * kWLoads; i < (share + 1) * kWLoads; ++i)
      direct(wsm + (super & 1) * kW + (wave + i * kWaves) * kWRows * kWRow,
             wbase + (int64_t)min(super, whole - 1) * kWRow, w_at[i]);
  };
  // Scale bytes: four lanes to a row, one for each super-stage of the group (of
  // four); the threads beyond a quarter's rows write the same values again.
  typedef std::conditional_t<SP == 4, u32x2, uint32_t> Scale;
  typedef std::conditional_t<SP == 4, u32x2_a1, u32_a1> ScaleA1;
  auto s_row = [&](int quarter) { return quarter * (BM / 4) + (tid >> 2) % (BM / 4); };
  Scale sreg;
  auto fetch_s = [&](int group, int quarter) {
    const int super = min(lo + 4 * group + (tid & 3), whole - 1);
    const uint8_t* row = sbase + (int64_t)min(s_row(quarter), p.m - 1 - r0) * p.lds;
    sreg = *reinterpret_cast<const ScaleA1*>(row + 2 * SP * super);
  };
  auto put_s = [&](int group, int quarter) {
    Scale* at = reinterpret_cast<Scale*>(ssm) + (4 * (group & 1) + (tid & 3)) * BM + s_row(quarter);
    if constexpr (SP == 4) *at = order_scales8(sreg[0], sreg[1]);
    else *at = sreg;
  };

  floatx16 acc[RB][CB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) acc[rb][cb] = floatx16{};
  uint32_t frag_x[4], frag_w[SP];            // this lane's addresses of step j, of stage u's codes
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    frag_x[j] = (uint32_t)((wc * CB * 32 + l32) * kPanelRow + (((4 * h + j) ^ swizzle(l32)) << 4));
    if (j < SP) frag_w[j] = (uint32_t)((wr * RB * 32 + l32) * kWRow + (((2 * j + h) ^ w_swizzle(l32)) << 4));
  }
  u32x4 x[2][CB], w[2][RB];
  uint32_t sc[RB], inexact = 0u;
  auto load_x = [&](int buf, int step, u32x4 (&o)[CB]) {
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
      o[cb] = *reinterpret_cast<const u32x4*>(xs + buf * kX + frag_x[step] + cb * 32 * kPanelRow);
  };
  auto load_w = [&](int super, int u, u32x4 (&o)[RB]) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
      o[rb] = *reinterpret_cast<const u32x4*>(wsm + (super & 1) * kW + frag_w[u] + rb * 32 * kWRow);
  };
  // Four scale bytes: this half's of the four stages, or both halves' of the two.
  auto load_s = [&](int super) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int at = ((super - lo) & 7) * BM + (wr * RB + rb) * 32 + l32;
      sc[rb] = reinterpret_cast<const uint32_t*>(ssm)[SP == 4 ? 2 * at + h : at];
      if constexpr (XT == GPTQ_F16 && !SPLIT) inexact |= f16_inexact4(sc[rb]);
    }
  };
  auto scale_of = [&](int u, int rb) {
    return mx_scale_operand((SP == 4 ? sc[rb] >> (8 * u) : sc[rb] >> (16 * u + 8 * h)) & 255u);
  };
  // Products of step j of stage u, row blocks [from, to).
  auto products = [&](int u, int j, const u32x4 (&xf)[CB], const u32x4 (&wf)[RB], int from, int to) {
    if constexpr (SPLIT) {
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        u32x4 top, rest;
        split8(xf[cb], top, rest);
#pragma unroll
        for (int rb = from; rb < to; ++rb) {
          const u32x4 wv = widen8<GPTQ_BF16>(wf[rb][j], scale_of(u, rb));
          acc[rb][cb] = mfma32<GPTQ_BF16>(top, wv, acc[rb][cb]);
          acc[rb][cb] = mfma32<GPTQ_BF16>(rest, wv, acc[rb][cb]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int rb = from; rb < to; ++rb) {
        const u32x4 wv = widen8<XT>(wf[rb][j], scale_of(u, rb));
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) acc[rb][cb] = mfma32<XT>(xf[cb], wv, acc[rb][cb]);
      }
#pragma unroll
      for (int i = 0; i < (to - from) * CB; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
        __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);   // two VALU
      }
    }
  };

  if (lo < whole) {
    fetch_x(SP * lo, 0);
#pragma unroll
    for (int u = 0; u < SP; ++u) fetch_w(lo, u);
#pragma unroll
    for (int quarter = 0; quarter < 4; ++quarter) {
      fetch_s(0, quarter);
      put_s(0, quarter);
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    lds_barrier();
    load_x(0, 0, x[0]);
    load_w(lo, 0, w[0]);
    load_s(lo);
    for (int super = lo; super < whole; ++super) {
      const int group = ((super - lo) >> 2) + 1, quarter = (super - lo) & 3;
#pragma unroll
      for (int u = 0; u < SP; ++u) {
        // Past the last panel that panel is fetched again, for no one.
        fetch_x(min(SP * super + u + 1, SP * whole - 1), (u + 1) & 1);
        fetch_w(super + 1, u);
        if (u == 0) fetch_s(group, quarter);
        __builtin_amdgcn_sched_barrier(0);   // the loads are issued before the products
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          load_x(u & 1, j + 1, x[(j + 1) & 1]);
          products(u, j, x[j & 1], w[u & 1], 0, RB);
        }
        products(u, 3, x[1], w[u & 1], 0, RB / 2);
        if (u == SP - 1) put_s(group, quarter);
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        lds_barrier();
        load_x((u + 1) & 1, 0, x[0]);
        load_w(super + (u == SP - 1), (u + 1) % SP, w[(u + 1) & 1]);
        products(u, 3, x[1], w[u & 1], RB / 2, RB);
        if (u == SP - 1) load_s(super + 1);
      }
    }
  }
  // The columns behind the last whole super-stage, a panel at a time.
  if (lo <= whole && whole < hi) {
#pragma unroll 1
    for (int panel = SP * whole; panel < (p.n + 63) / 64; ++panel) {
      lds_barrier();
#pragma unroll
      for (int i = 0; i < BN * 8 / kThreads; ++i) {
        const int r = (tid >> 3) + i * (kThreads / 8);
        *reinterpret_cast<u32x4*>(xs + r * kPanelRow + (((tid & 7) ^ swizzle(r)) << 4)) =
            load_x8_tail(reinterpret_cast<const uint16_t*>(xbase + x_row(r)), panel * 64 + (tid & 7) * 8, p.n);
      }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        const int r = (wr * RB + rb) * 32 + l32;
        w[0][rb] = load_w4_tail(reinterpret_cast<const uint32_t*>(wbase + w_row(r)), 8 * panel + 4 * h, p.n);
        // This half's byte in every place a stage may take it from.
        sc[rb] = ((load_scales4(sbase + (int64_t)min(r, p.m - 1 - r0) * p.lds, 2 * panel, p.n) >> (8 * h)) & 255u) *
                 0x01010101u;
        if constexpr (XT == GPTQ_F16 && !SPLIT) inexact |= f16_inexact4(sc[rb]);
      }
      lds_barrier();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        load_x(0, j, x[0]);
        products(0, j, x[0], w[0], 0, RB);
      }
    }
  }
  if constexpr (XT == GPTQ_F16 && !SPLIT) {
    if (!__syncthreads_and(inexact == 0u)) return false;
  } else {
    lds_barrier();
  }
  store_tile<WR, WC, RB, CB>(p, tg, tile, r0, split, acc, smem);
  return true;
}

// Two waves per SIMD where the accumulators leave room for them.
template <int XT, int WR, int WC, int RB, int CB, int PB, bool DIRECT, bool WL>
__global__ __launch_bounds__(64 * WR * WC, RB * CB <= 8 ? 2 : 1) void mx_tile_kernel(MxOperands p, TileGrid tg) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  int split, r0;
  TokenTile tile;
  if (!tile_of_workgroup(p, tg, 32 * WR * RB, 32 * WC * CB, split, tile, r0)) return;
  const bool done = tile_product<XT, WR, WC, RB, CB, PB, DIRECT, WL, false>(p, tg, tile, r0, split, smem);
  if constexpr (XT == GPTQ_F16) {
    if (!done) tile_product<XT, WR, WC, RB, CB, PB, DIRECT, WL, true>(p, tg, tile, r0, split, smem);
  }
}

template <int XT, int WR, int WC, int RB, int CB, int SP>
__global__ __launch_bounds__(64 * WR * WC, 2) void mx_big_tile_kernel(MxOperands p, TileGrid tg) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  int split, r0;
  TokenTile tile;
  if (!tile_of_workgroup(p, tg, 32 * WR * RB, 32 * WC * CB, split, tile, r0)) return;
  const bool done = big_tile_product<XT, WR, WC, RB, CB, SP, false>(p, tg, tile, r0, split, smem);
  if constexpr (XT == GPTQ_F16) {
    if (!done) big_tile_product<XT, WR, WC, RB, CB, SP, true>(p, tg, tile, r0, split, smem);
  }
}

__global__ __launch_bounds__(kJoinCols / 4) void mx_join_kernel(MxOperands p, TileGrid tg) { join_splits(p, tg); }

// What a product runs on, from its sizes alone.
enum Kind {
  kRows1, kRows2, kRows2x2,                  // mx_rows_kernel: tiles of W (x tiles of X)
  kStream,                                   // mx_stream_kernel: up to kStreamRows rows of X
  kTile128x32, kTile128x64, kTile128x128, kTile256x128, kTile256x256, // W rows x X rows of a tile
};
struct Plan {
  Kind kind;
  int splits;                                // of the columns, tiles only
};

// Products on tiles: the shape and the splits with the least time by the model of
// choose_tiles.  Fitted to 180 sizes of 16-bit X from
// 8 x 1024 x 2048 to 2048 x 49152 x 12288 and 50 of microscaled X: what it
// chooses takes 1.02 and 1.01 times the fastest's time in the mean, 1.3 and 1.13
// at worst.  It knows sizes only: rows that are not 16-byte aligned take longer (2448
// x 320 x 8606 28.5 us by the model, 39 measured), and so does a partial last stage
// of the large tiles (2368 x 14720 x 864: 102 us, 38 by its bytes).  Some of the
// measured pairs, the chosen first, 16-bit: 16 x 12288 x 12288 (W from memory) on
// 128 x 32 with 5 splits 26, with 4 28, with 1 54; 256 x 4096 x 4096 on 128 x 32
// 15, 128 x 64 20; 256 x 11008 x 4096 on 128 x 64 31, 128 x 32 36; 2048 x 11008 x
// 4096 on 256 x 128 150, 256 x 256 169; 4096 x 8192 x 8192 on 256 x 256 374, 256 x
// 128 433.  Microscaled: 128 x 4096 x 4096 on 128 x 32 10.5, 128 x 64 12.9; 512 x
// 4096 x 4096 on 128 x 64 13.8, 128 x 128 16.1; 2048 x 4096 x 4096 on 128 x 128
// 28, 256 x 256 32; 4096 x 12288 x 12288 on 256 x 256 286, 128 x 128 391.  128 x
// 128 tiles of 16-bit X and 256 x 128 of microscaled X were the fastest of no size
// by more than a tenth: they are not built.
constexpr TileShape kTileShapes[] = {
    {kTile128x32, 128, 32, 2, 3.3, 0.74, 1.3},
    {kTile128x64, 128, 64, 2, 3.5, 1.3, 2.2},
    {kTile256x128, 256, 128, 2, 9.2, 3.5, 6.2},
    {kTile256x256, 256, 256, 1, 5.2, 5.4, 5.4},
};
constexpr TileShape kScaledTileShapes[] = {
    {kTile128x32, 128, 32, 2, 3.0, 0.46, 0.81},
    {kTile128x64, 128, 64, 2, 2.9, 0.67, 1.0},
    {kTile128x128, 128, 128, 1, 3.9, 0.65, 0.65},
    {kTile256x256, 256, 256, 1, 6.8, 1.6, 1.6},
};
// Grouped by expert: half a tile more for every expert that can have rows, and no
// splits.  64 experts of 1024 x 2048 with 64 rows each on 128 x 32 37 us, 256 x 128
// 50, with 256 101 and 85; 8 of 11008 x 4096 with 128 143 and 147, with 256 257 and
// 239; 28 of 120 x 10624 with 196 46 and 127 (57
// workgroups); 8 of 4096 x 4096 with 375 139 and 106.  128 x 64 tiles were
// the fastest of no size by a tenth.
constexpr TileShape kGroupedTileShapes[] = {kTileShapes[0], kTileShapes[2]};
template <size_t N>
Plan tile_plan(const TileShape (&shapes)[N], int64_t m, int64_t n, int64_t rows, int64_t experts = 0) {
  // Half a tile more for every expert that can have rows.
  const auto groups = [&](int64_t w_tiles, int bn) {
    return w_tiles * (ceil_div(rows, bn) + (std::min(experts, rows) + 1) / 2);
  };
  const TileChoice c = choose_tiles(shapes, m, n, rows, experts, groups, 4.3, 0.22e-6, false);
  return Plan{(Kind)c.kind, c.splits};
}

// The row kernels, whose waves split the columns, take products small enough for
// their operands to come through L2 (32 x 4096 x 4096: 9.3 against 10.6 us on
// tiles; 64 x 4096 x 4096: 15 against 11.6; 1 x 4096 x 11008: 9.0 against 11.4;
// 4 x 11008 x 4096: 11.5 against 10.6).  Their waves load X's rows in pieces:
// rows of odd lengths slow them down (2 x 4099 x 11007: 21 against 15.6; 8 x 130
// x 1001 still 5.6 against 7.6).  Microscaled X, which is smaller, stays on them
// longer, up to 2^30 products (64 x 4096 x 4096, the last of them: 8.2 against 12.8;
// 128 x 4096 x 4096: 12.5 against 10.5; 8 x 11008 x 4096: 8.6 against 9.8; 32 x
// 11008 x 4096: 13.6 against 10.3).
// Long matrices with up to four rows of 16-bit X take the stream kernel (1 x
// 28672 x 8192: 24 against 30 on tiles; 1 x 12288 x 12288: 27 against 20).  The
// thresholds stand beside the model: 32 x 4096 x 4128, just past one, takes 12.6 on
// tiles where 32 x 4096 x 4096 takes 9.5 on the row kernel.
Plan make_plan(int64_t m, int64_t n, int64_t rows, int64_t experts, bool grouped, bool mx) {
  if (grouped) {
    // By the rows an expert has on average; the workgroups of an expert without
    // rows do not exist.  64 experts of 1024 x 2048 with 2 rows each: 18 us on the
    // row kernel, 20 on tiles; 8 of 11008 x 4096 with 4: 47 and 40.
    if (rows <= 4) return Plan{kRows1, 1};
    if (rows / experts < 4) return Plan{kRows2, 1};
    return tile_plan(kGroupedTileShapes, m, n, rows, experts);
  }
  const int64_t outputs = m * rows, products = outputs * std::max<int64_t>(n, 1);
  const bool small = m * n <= ((int64_t)1 << 24);
  if (mx) {
    if (small ? products > ((int64_t)1 << 30) : products > 500000000) return tile_plan(kScaledTileShapes, m, n, rows);
    if (outputs <= 65536 || !small) return Plan{kRows1, 1};
    return Plan{rows <= 32 ? kRows2 : kRows2x2, 1};
  }
  if (m >= 24576 && rows <= kStreamRows) return Plan{kStream, 1};
  if (rows == 1 || n % 4 == 0 || products <= 50000000) {
    if (small ? outputs <= 65536 : products <= 150000000) return Plan{kRows1, 1};
    if (small && outputs <= 131072) return Plan{kRows2, 1};
  }
  return tile_plan(kTileShapes, m, n, rows);
}

// Workspace of a plan: the splits' sums.
size_t plan_ws(const Plan& pl, int64_t m, int64_t rows) {
  return pl.splits > 1 ? align256((size_t)pl.splits * (size_t)rows * (size_t)m * sizeof(float)) : 0;
}

// A launch has fewer than 2^32 threads.  Calls launch(operands) for the rows of W in
// parts of whole tiles of bm rows, as many as fit when each tile of W takes `slots`
// workgroups (at most 2^20 / 16 + 65536 tiles of X: one tile of W always fits).
// Split columns, whose sums are laid out for all rows at once, never have more
// than one part: the plan adds splits up to 2048 workgroups.
template <typename Launch>
gptq_status in_row_parts(const MxOperands& p, int bm, int64_t slots, int threads, Launch launch) {
  const int64_t part = std::max<int64_t>(((int64_t)1 << 31) / (slots * threads), 1) * bm;
  for (int64_t r = 0; r < p.m; r += part) {
    MxOperands q = p;
    q.W += r * p.ldp;
    q.S += r * p.lds;
    q.Y = static_cast<char*>(p.Y) + r * elem_bytes(p.y_dtype);
    q.m = (int)std::min(part, p.m - r);
    launch(q);
    GPTQ_TRY_LAUNCH();
  }
  return GPTQ_OK;
}

// Runs tile kernel k (tiles of BM x BN) and, with splits, the sum over them.
gptq_status run_tiles(void (*k)(MxOperands, TileGrid), int BM, int BN, int threads, int lds, const MxOperands& p,
                      const Plan& pl, void* ws, hipStream_t st) {
  const int64_t cols = round_up(std::max<int64_t>(ceil_div(p.n, pl.splits), 1), kSplitCols);
  // Whole splits can leave fewer of them than were asked for.
  const int splits = (int)std::max<int64_t>(ceil_div(p.n, cols), 1);
  TileGrid tg{(int)ceil_div(p.m, BM), (int)max_tiles(p.rows, p.experts, p.offsets != nullptr, BN), splits,
              (int)cols, static_cast<float*>(ws)};
  const int64_t slots = (int64_t)tg.tok_tiles * tg.splits;
  if (lds > 65536)
    GPTQ_TRY_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds));
  const gptq_status rc = in_row_parts(p, BM, slots, threads, [&](const MxOperands& q) {
    tg.row_tiles = (int)ceil_div(q.m, BM);
    k<<<(unsigned)round_up(tg.row_tiles * slots, kXcds), threads, lds, st>>>(q, tg);
  });
  if (rc != GPTQ_OK) return rc;
  if (tg.splits > 1) {
    mx_join_kernel<<<(unsigned)(ceil_div(p.m, kJoinCols) * p.rows), kJoinCols / 4, 0, st>>>(p, tg);
    GPTQ_TRY_LAUNCH();
  }
  return GPTQ_OK;
}

// Whether every row of both operands starts at a 16-byte aligned address.
template <int XT>
bool aligned_x(const MxOperands& p) {
  return ((reinterpret_cast<uintptr_t>(p.X) | (uint64_t)(p.ldx * (XT == kMx ? 4 : 2))) & 15) == 0;
}
bool aligned_w(const MxOperands& p) {
  return ((reinterpret_cast<uintptr_t>(p.W) | (uint64_t)(p.ldp * 4) | (uint64_t)(p.w_stride * 4)) & 15) == 0;
}

template <int XT, int WR, int WC, int RB, int CB, int PB, bool DIRECT, bool WL>
gptq_status launch_tile(const MxOperands& p, const Plan& pl, void* ws, hipStream_t st) {
  return run_tiles(mx_tile_kernel<XT, WR, WC, RB, CB, PB, DIRECT, WL>, 32 * WR * RB, 32 * WC * CB, 64 * WR * WC,
                   tile_lds<XT, WR, WC, RB, CB, PB, WL>(), p, pl, ws, st);
}

// WL: the shape stages the codes of W in LDS where their rows allow it.
template <int XT, int WR, int WC, int RB, int CB, int PB, bool WL>
gptq_status launch_tiles(const MxOperands& p, const Plan& pl, void* ws, hipStream_t st) {
  const bool x = aligned_x<XT>(p), w = aligned_w(p);
  if constexpr (WL) {
    if (w && x) return launch_tile<XT, WR, WC, RB, CB, PB, true, true>(p, pl, ws, st);
    if (w) return launch_tile<XT, WR, WC, RB, CB, PB, false, true>(p, pl, ws, st);
  }
  if (x && (w || XT != kMx)) return launch_tile<XT, WR, WC, RB, CB, PB, true, false>(p, pl, ws, st);
  return launch_tile<XT, WR, WC, RB, CB, PB, false, false>(p, pl, ws, st);
}

template <int XT, int WR, int WC, int RB, int CB, int SP>
gptq_status launch_big_tiles(const MxOperands& p, const Plan& pl, void* ws, hipStream_t st) {
  return run_tiles(mx_big_tile_kernel<XT, WR, WC, RB, CB, SP>, 32 * WR * RB, 32 * WC * CB, 64 * WR * WC,
                   big_tile_lds<XT, WR, WC, RB, CB, SP>(), p, pl, ws, st);
}

template <int XT, int RT, int NT, int D>
gptq_status launch_rows(const MxOperands& p, int waves, hipStream_t st) {
  const int64_t slots = max_tiles(p.rows, p.experts, p.offsets != nullptr, 16 * NT);
  return in_row_parts(p, 16 * RT, slots, 64 * waves, [&](const MxOperands& q) {
    mx_rows_kernel<XT, RT, NT, D>
        <<<(unsigned)(ceil_div(q.m, 16 * RT) * slots), 64 * waves, waves * RT * NT * 64 * sizeof(floatx4), st>>>(q);
  });
}

template <int XT>
gptq_status launch_stream(const MxOperands& p, hipStream_t st) {
  mx_stream_kernel<XT><<<(unsigned)ceil_div(p.m, 64), 256, 0, st>>>(p);
  GPTQ_TRY_LAUNCH();
  return GPTQ_OK;
}

template <int XT>
gptq_status launch(const MxOperands& p, void* ws, size_t ws_bytes, hipStream_t st) {
  Plan pl = make_plan(p.m, p.n, p.rows, p.experts, p.offsets != nullptr, XT == kMx);
  // The tile kernels address the rows of a tile with 32 bits; rows further apart
  // take the row kernel, which reads both operands many times over (X's rows 4.4 MB
  // apart: 512 x 11008 x 4096 270 us instead of 64, 2048 rows 985 instead of 162).
  constexpr int64_t kMaxPitch = (int64_t)1 << 22;
  if (p.ldx * (XT == kMx ? 4 : 2) > kMaxPitch || p.ldp * 4 > kMaxPitch || p.lds > kMaxPitch || p.ldxs > kMaxPitch)
    pl = Plan{kRows2, 1};
  const size_t need = plan_ws(pl, p.m, p.rows);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return GPTQ_ERR_WORKSPACE;
  if (need > 0 && (reinterpret_cast<uintptr_t>(ws) & 3) != 0) return GPTQ_ERR_INVALID_ARG;
  constexpr bool MX = XT == kMx;
  constexpr int P2 = MX ? 1 : 2, P4 = MX ? 1 : 4;            // panels per stage
  if constexpr (!MX) {
    if (aligned_x<XT>(p) && aligned_w(p)) {
      if (pl.kind == kTile256x256) return launch_big_tiles<XT, 4, 2, 2, 4, 4>(p, pl, ws, st);
      if (pl.kind == kTile256x128) return launch_big_tiles<XT, 4, 1, 2, 4, 2>(p, pl, ws, st);
    }
  }
  switch (pl.kind) {
    // Microscaled: 128 x 64 a wave (4096 x 12288 x 12288 298 us, 310 with 64 x 128).
    case kTile256x256:
      if constexpr (MX) return launch_tiles<XT, 2, 4, 4, 2, P2, false>(p, pl, ws, st);
      else return launch_tiles<XT, 4, 2, 2, 4, P2, false>(p, pl, ws, st);
    case kTile256x128:
      if constexpr (!MX) return launch_tiles<XT, 4, 1, 2, 4, P2, false>(p, pl, ws, st);
      break;
    case kTile128x128:
      if constexpr (MX) return launch_tiles<XT, 4, 1, 1, 4, P2, false>(p, pl, ws, st);
      break;
    case kTile128x64: return launch_tiles<XT, 4, 1, 1, 2, P2, !MX>(p, pl, ws, st);
    case kTile128x32: return launch_tiles<XT, 4, 1, 1, 1, P4, !MX>(p, pl, ws, st);
    case kRows1: return launch_rows<XT, 1, 1, 4>(p, 8, st);
    case kRows2x2:
      if constexpr (MX) return launch_rows<XT, 2, 2, 2>(p, 8, st);
      break;
    case kStream:
      if constexpr (!MX) return launch_stream<XT>(p, st);
      break;
    default: break;
  }
  return launch_rows<XT, 2, 1, 2>(p, 8, st);
}

constexpr int64_t kMaxLd = (int64_t)1 << 40; // products of strides and indexes stay below 2^62

// Checks shared by the products; `rows` rows of X against `experts` matrices.
gptq_status check(int64_t m, int64_t n, int64_t rows, int64_t experts, int64_t ld_packed, int64_t ld_scales,
                  int y_dtype, int64_t ldy) {
  if (m < 0 || n < 0 || rows < 0 || experts < 0 || !valid_dtype(y_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (n > kMxMaxCols || m > GPTQ_MX_MAX_ROWS || rows > GPTQ_MX_MAX_ROWS || experts > GPTQ_MX_MAX_EXPERTS)
    return GPTQ_ERR_UNSUPPORTED;
  if (ld_packed < ceil_div(n, 8) || ld_scales < ceil_div(n, kMxBlock) || ldy < m) return GPTQ_ERR_INVALID_ARG;
  if (ld_packed > kMaxLd || ld_scales > kMaxLd || ldy > kMaxLd) return GPTQ_ERR_UNSUPPORTED;
  return GPTQ_OK;
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" size_t gptq_mx_gemm_ws_bytes(int64_t m, int64_t n, int64_t rows, int64_t experts) {
  if (m <= 0 || n < 0 || rows <= 0 || experts <= 0 || n > kMxMaxCols || m > GPTQ_MX_MAX_ROWS ||
      rows > GPTQ_MX_MAX_ROWS || experts > GPTQ_MX_MAX_EXPERTS)
    return 0;
  // Of one matrix with either kind of X; products grouped by expert need none.
  if (experts > 1) return 0;
  return std::max(plan_ws(make_plan(m, n, rows, 1, false, false), m, rows),
                  plan_ws(make_plan(m, n, rows, 1, false, true), m, rows));
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
  if (ldx > kMaxLd || stride_packed > (kMaxLd << 5) || stride_scales > (kMaxLd << 5)) return GPTQ_ERR_UNSUPPORTED;
  if (experts > 1 && (stride_packed < m * ld_packed || stride_scales < m * ld_scales)) return GPTQ_ERR_INVALID_ARG;
  if (m == 0 || rows == 0 || experts == 0) return GPTQ_OK;
  if (offsets == nullptr || Y == nullptr) return GPTQ_ERR_INVALID_ARG;
  if (n > 0 && (packed == nullptr || scales == nullptr || X == nullptr)) return GPTQ_ERR_INVALID_ARG;
  const MxOperands p{packed, scales, ld_packed, ld_scales, stride_packed, stride_scales, (int)m, (int)n, X, nullptr,
                     ldx, 0, (int)rows, offsets, (int)experts, Y, ldy, y_dtype};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return x_dtype == GPTQ_F16 ? launch<GPTQ_F16>(p, ws, ws_bytes, st) : launch<GPTQ_BF16>(p, ws, ws_bytes, st);
}

extern "C" gptq_status gptq_mx_gemm(const uint32_t* packed, int64_t m, int64_t n, int64_t ld_packed,
                                    const uint8_t* scales, int64_t ld_scales, const void* X, int x_dtype,
                                    int64_t batch, int64_t ldx, void* Y, int y_dtype, int64_t ldy, void* ws,
                                    size_t ws_bytes, void* stream) {
  if (x_dtype != GPTQ_F16 && x_dtype != GPTQ_BF16) return GPTQ_ERR_INVALID_ARG;
  const gptq_status rc = check(m, n, batch, 1, ld_packed, ld_scales, y_dtype, ldy);
  if (rc != GPTQ_OK) return rc;
  if (ldx < n) return GPTQ_ERR_INVALID_ARG;
  if (ldx > kMaxLd) return GPTQ_ERR_UNSUPPORTED;
  if (m == 0 || batch == 0) return GPTQ_OK;
  if (Y == nullptr || (n > 0 && (packed == nullptr || scales == nullptr || X == nullptr)))
    return GPTQ_ERR_INVALID_ARG;
  const MxOperands p{packed, scales, ld_packed, ld_scales, 0, 0, (int)m, (int)n, X, nullptr,
                     ldx, 0, (int)batch, nullptr, 1, Y, ldy, y_dtype};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return x_dtype == GPTQ_F16 ? launch<GPTQ_F16>(p, ws, ws_bytes, st) : launch<GPTQ_BF16>(p, ws, ws_bytes, st);
}

extern "C" gptq_status gptq_mx_scaled_gemm(const uint32_t* packed, int64_t m, int64_t n, int64_t ld_packed,
                                           const uint8_t* scales, int64_t ld_scales, const uint32_t* x_packed,
                                           int64_t batch, int64_t ld_xpacked, const uint8_t* x_scales,
                                           int64_t ld_xscales, void* Y, int y_dtype, int64_t ldy, void* ws,
                                           size_t ws_bytes, void* stream) {
  const gptq_status rc = check(m, n, batch, 1, ld_packed, ld_scales, y_dtype, ldy);
  if (rc != GPTQ_OK) return rc;
  if (ld_xpacked < ceil_div(n, 8) || ld_xscales < ceil_div(n, kMxBlock)) return GPTQ_ERR_INVALID_ARG;
  if (ld_xpacked > kMaxLd || ld_xscales > kMaxLd) return GPTQ_ERR_UNSUPPORTED;
  if (m == 0 || batch == 0) return GPTQ_OK;
  if (Y == nullptr || (n > 0 && (packed == nullptr || scales == nullptr || x_packed == nullptr || x_scales == nullptr)))
    return GPTQ_ERR_INVALID_ARG;
  const MxOperands p{packed, scales, ld_packed, ld_scales, 0, 0, (int)m, (int)n, x_packed, x_scales,
                     ld_xpacked, ld_xscales, (int)batch, nullptr, 1, Y, ldy, y_dtype};
  return launch<kMx>(p, ws, ws_bytes, static_cast<hipStream_t>(stream));
}
