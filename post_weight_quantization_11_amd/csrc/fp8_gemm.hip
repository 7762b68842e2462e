// Products of 8-bit floats with a scale for each block of 128:
//   Y[t, r] = sum_b xs[t, b] ws[r / 128, b] sum_{k in b} w[r, k] x[t, k]
// for one weight matrix or one per expert (rows of X grouped by expert).
//
// A block's 128 columns are summed from zero in the matrix cores and then added,
// times the two scales, to the running float32 sums: one fused multiply-add an
// output and block.  W is the first operand, so a lane's results belong to one
// row of X and, inside a tile's 32 or 64 rows of W, to one block of W: their
// factor xs * ws is one number a lane.
//
// The matrix instructions on 8-bit operands, of either generation
// (v_mfma_f32_32x32x64_f8f6f4 at twice the rate of the 16-bit ones, v_mfma_f32_32x32x16_fp8_fp8
// at theirs), do not sum in float32: probed, they cut each product at 2^-13 of the
// largest power of two among the eight that they add at a time (5e-5 of the result for
// codes of all magnitudes, any part of it where large terms cancel), where the 16-bit
// ones cut at 2^-24.  So codes are widened to bfloat16, which holds them exactly.
//
// Operand layout (checked with an in-bounds probe): lane l holds 8 elements of row l
// % 32 (l % 16); the order of the summed columns is free as long as both operands
// agree.  Accumulator register i of lane l is row 8 (i /
// 4) + 4 (l / 32) + i % 4 (4 (l / 16) + i) of the first operand and row l % 32 (l %
// 16) of the second.
#include "fp8.h"
#include "product.h"

namespace gptq {
namespace {

struct Fp8Operands {
  const uint8_t* W;                          // codes, m x ldw (per expert: + e * w_stride)
  const float* S;                            // scales, ceil(m / 128) x lds (+ e * s_stride)
  int64_t ldw, lds, w_stride, s_stride;
  int m, n;
  const uint8_t* X;
  const float* XS;                           // rows x ldxs
  int64_t ldx, ldxs;
  int rows;
  const int32_t* offsets;
  int experts;
  void* Y;
  int64_t ldy;
  int y_dtype;
};

__device__ inline floatx16 mfma32(bf16x8 w, bf16x8 x, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, x, c, 0, 0, 0);
}
__device__ inline floatx4 mfma16(bf16x8 w, bf16x8 x, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Few rows of X: the waves of a workgroup share RT tiles of 16 rows of W and one
// of X, take every eighth quad of blocks (512 columns) and add their sums through
// LDS in wave order.  Both operands come straight from memory, D blocks in flight a
// wave, along their rows, and are exchanged between lanes (loaded in the matrix
// instruction's order they cost the CU's cache four times the accesses: 1 x 49152 x
// 12288 139 us for 108, with rows at odd addresses 1 x 12288 x 12288 93 for 45); a
// quad's four scales are one load.  Measured: 1 x 4096 x 4096 6.7 us,
// 1 x 12288 x 12288 37 us, 1 x 49152 x 12288 108 us (5.6 TB/s), 16 x 49152 x 12288 131.
// ---------------------------------------------------------------------------
constexpr int kRowWaves = 8;
template <int RT, int CT> constexpr int rows_lds() {
  return kRowWaves * std::max(RT * CT * 64 * (int)sizeof(floatx4), kExchange);
}
template <int RT, int CT, int D>
__global__ __launch_bounds__(64 * kRowWaves) void fp8_rows_kernel(Fp8Operands p) {
  static_assert(D == 1 || D == 2 || D == 4, "the ring's slots are the same in every quad");
  extern __shared__ floatx4 red[];           // a wave's exchanges, then its sums [CT][RT][64]
  const int row_tiles = (p.m + 16 * RT - 1) / (16 * RT);
  const int slot = (int)(blockIdx.x / row_tiles), r0 = (int)(blockIdx.x % row_tiles) * 16 * RT;
  const TokenTile tile = find_tile(p, slot, 16 * CT);
  if (!tile.valid) return;
  const int lane = (int)threadIdx.x & 63, q = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  // Rows past the last repeat it: what they give is not stored.
  const uint8_t *wrow[RT], *xrow[CT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
    wrow[rt] = p.W + (int64_t)tile.expert * p.w_stride + (int64_t)min(r0 + 16 * rt + (lane >> 2), p.m - 1) * p.ldw;
  // 16 RT divides 128: the tiles lie in one block of rows.
  const float* wsrow = p.S + (int64_t)tile.expert * p.s_stride + (int64_t)(r0 >> 7) * p.lds;
  const float* xsrow[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    xrow[ct] = p.X + (int64_t)min(tile.begin + 16 * ct + (lane >> 2), tile.end - 1) * p.ldx;
    xsrow[ct] = p.XS + (int64_t)min(tile.begin + 16 * ct + c16, tile.end - 1) * p.ldxs;
  }
  constexpr int kTiles = RT * CT, kMine = rows_lds<RT, CT>() / kRowWaves / 16;
  u32x4* swap = reinterpret_cast<u32x4*>(red + wave * kMine);
  floatx4 acc[CT][RT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[ct][rt] = floatx4{0.f, 0.f, 0.f, 0.f};

  // Lane quarter q is to hold bytes 16 q .. + 15 of both halves of a block.
  struct Unit {
    u32x4 w[RT][2], x[CT][2];
  };
  struct Scales {
    floatx4 w, x[CT];                        // a quad's
  };
  const int quads = p.n >> 9;                // whole ones
  // Past the last quad that quad is loaded again (and not used).
  auto load_unit = [&](int quad, int d, Unit& u) {
    const int at = 128 * (4 * min(quad, quads - 1) + d) + 16 * (lane & 3);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) u.w[rt][h] = *reinterpret_cast<const u32x4_a1*>(wrow[rt] + at + 64 * h);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) u.x[ct][h] = *reinterpret_cast<const u32x4_a1*>(xrow[ct] + at + 64 * h);
    }
  };
  auto load_scales = [&](int quad, Scales& s) {
    const int at = 4 * min(quad, quads - 1);
    s.w = *reinterpret_cast<const floatx4_a4*>(wsrow + at);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) s.x[ct] = *reinterpret_cast<const floatx4_a4*>(xsrow[ct] + at);
  };
  auto multiply = [&](Unit& u, const float (&f)[CT]) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) exchange(u.x[ct], swap, lane);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      exchange(u.w[rt], swap, lane);
      floatx4 v[CT];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) v[ct] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bf16x8 w = fp8_widen8(u.w[rt][s >> 1], s & 1);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) v[ct] = mfma16(w, fp8_widen8(u.x[ct][s >> 1], s & 1), v[ct]);
      }
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[ct][rt][i] = __builtin_fmaf(f[ct], v[ct][i], acc[ct][rt][i]);
    }
  };
  if (wave < quads) {
    Unit u[D];
    Scales cur, nxt;
    load_scales(wave, cur);
#pragma unroll
    for (int d = 0; d < D; ++d) load_unit(wave, d, u[d]);
    for (int quad = wave; quad < quads; quad += kRowWaves) {
      load_scales(quad + kRowWaves, nxt);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        float f[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) f[ct] = cur.w[d] * cur.x[ct][d];
        multiply(u[d % D], f);
        load_unit(d + D < 4 ? quad : quad + kRowWaves, (d + D) % 4, u[d % D]);
      }
      cur = nxt;
    }
  }
  // The columns behind the last whole quad, one block a wave.
  const int blocks = (p.n + 127) >> 7;
  for (int b = 4 * quads + (wave + kRowWaves - quads % kRowWaves) % kRowWaves; b < blocks; b += kRowWaves) {
    Unit u;
    float f[CT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 128 * b + 64 * h + 16 * (lane & 3);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) u.w[rt][h] = fp8_load16_tail(wrow[rt], k, p.n);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) u.x[ct][h] = fp8_load16_tail(xrow[ct], k, p.n);
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) f[ct] = wsrow[b] * xsrow[ct][b];
    multiply(u, f);
  }
  wave_fence();
#pragma unroll
  for (int i = 0; i < kTiles; ++i) red[wave * kMine + i * 64 + lane] = acc[i / RT][i % RT];
  __syncthreads();
  if (wave < kTiles) {
    floatx4 v = red[wave * 64 + lane];
    for (int w = 1; w < kRowWaves; ++w) v += red[w * kMine + wave * 64 + lane];
    const int x = tile.begin + 16 * (wave / RT) + c16, r = r0 + 16 * (wave % RT) + 4 * q;
    if (x < tile.end) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + i < p.m) store_y(p, (int64_t)x * p.ldy + r + i, v[i]);
    }
  }
}

// ---------------------------------------------------------------------------
// Tiled products.  A workgroup owns 32 WR RB rows of W x 32 WC CB rows of X; its
// WR x WC waves own 32 RB x 32 CB each.  A stage is one block: 128 bytes of every
// row of both operands and their scales, in one of NB buffers in LDS.  The 16-byte
// chunk c of a row lies in slot c ^ r % 8 ^ r / 8 % 2 of the row's eight: sixteen
// neighbouring rows' chunks c cover all 64 banks.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kRow = kFp8Block;              // bytes of a row in a stage
__device__ inline int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// Floats per row of X in a wave's output block: two (one) row blocks of W, and
// four so that neighbouring rows start in different banks.
constexpr int out_pitch(int row_blocks) { return (row_blocks % 2 == 0 ? 64 : 32) + 4; }

// Scales of a stage: X's rows, then W's blocks of rows.
constexpr int scale_slots(int bn) { return std::max(bn, 64) + 64; }

template <int WR, int WC, int RB, int CB, int NB>
constexpr int tile_lds() {
  const int bm = 32 * WR * RB, bn = 32 * WC * CB;
  return std::max(NB * ((bm + bn) * kRow + scale_slots(bn) * 4), WR * WC * 32 * out_pitch(RB) * 4);
}

// Stores a workgroup's sums.  Each wave passes its own through LDS (the stages are
// no longer read), 32 rows of X x 64 (32) rows of W at a time, so that a lane
// stores eight neighbouring ones.  Y16: a 16-bit Y, otherwise float32.
template <bool Y16, int WR, int WC, int RB, int CB>
__device__ inline void store_tile(const Fp8Operands& p, const TileGrid& tg, const TokenTile& tile, int r0, int split,
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
      for (int b = 0; b < RP; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<floatx4*>(my + l32 * kPitch + 32 * b + 8 * g + 4 * h) =
              floatx4{acc[r2 + b][cb][4 * g], acc[r2 + b][cb][4 * g + 1], acc[r2 + b][cb][4 * g + 2],
                      acc[r2 + b][cb][4 * g + 3]};
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
          else if (!Y16)
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

// DIRECT: rows of both operands are 16-byte aligned and go from memory to LDS
// without passing through registers, NB - 1 stages ahead.  Otherwise one stage
// ahead, through registers, any alignment.
template <bool Y16, int WR, int WC, int RB, int CB, int NB, bool DIRECT>
__global__ __launch_bounds__(64 * WR * WC, 2) void fp8_tile_kernel(Fp8Operands p, TileGrid tg) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int kThreads = 64 * WR * WC, kWaves = WR * WC;
  constexpr int BM = 32 * WR * RB, BN = 32 * WC * CB, kRows = BM + BN;        // X rows first, then W rows
  constexpr int kBuf = kRows * kRow, kSlots = scale_slots(BN);
  constexpr int kLoads = kRows / (8 * kWaves);                // direct loads of codes a wave issues per stage
  constexpr int kPerThread = kRows * 8 / kThreads;            // chunks a thread stages through registers
  constexpr int kGroups = kSlots / 64, kScaleLoads = (kGroups + kWaves - 1) / kWaves;
  static_assert(kRows % (8 * kWaves) == 0 && kWaves % 2 == 0, "a wave stages eight rows at a time, all even or all odd");
  static_assert(32 * RB <= kFp8Block && BM % kFp8Block == 0, "a wave's rows of W lie in one block");
  static_assert(DIRECT || NB == 2, "through registers one stage is ahead");
  int split, r0;
  TokenTile tile;
  if (!tile_of_workgroup(p, tg, BM, BN, split, tile, r0)) return;
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / WC, wc = wave % WC;
  const int blocks = (p.n + kFp8Block - 1) / kFp8Block;
  const int per_split = tg.cols_per_split / kFp8Block;
  const int lo = split * per_split, hi = min(blocks, lo + per_split), whole = min(hi, p.n / kFp8Block);

  const uint8_t* xbase = p.X + (int64_t)tile.begin * p.ldx;
  const uint8_t* wbase = p.W + (int64_t)tile.expert * p.w_stride + (int64_t)r0 * p.ldw;
  const float* xsbase = p.XS + (int64_t)tile.begin * p.ldxs;
  const float* wsbase = p.S + (int64_t)tile.expert * p.s_stride + (int64_t)(r0 >> 7) * p.lds;
  // Rows past the tile's (matrix's) last repeat it: what they give is not stored.
  auto row_offset = [&](int r) -> uint32_t {
    if (r < BN) return (uint32_t)min(r, tile.end - 1 - tile.begin) * (uint32_t)p.ldx;
    return (uint32_t)min(r - BN, p.m - 1 - r0) * (uint32_t)p.ldw;
  };
  auto row_ptr = [&](int r) { return (r < BN ? xbase : wbase) + row_offset(r); };

  float* scale_lds = reinterpret_cast<float*>(smem + NB * kBuf);              // [NB][kSlots]
  // This wave's groups of 64 scales of a stage; groups beyond the last repeat one.
  auto group = [&](int i) { return (wave + i * kWaves) % kGroups; };
  auto sbase = [&](int i) { return group(i) == kGroups - 1 ? wsbase : xsbase; };
  uint32_t s_at[kScaleLoads];
#pragma unroll
  for (int i = 0; i < kScaleLoads; ++i)
    s_at[i] = group(i) == kGroups - 1
                  ? (uint32_t)min(lane, (p.m - 1 - r0) >> 7) * (uint32_t)p.lds
                  : (uint32_t)min(group(i) * 64 + lane, tile.end - 1 - tile.begin) * (uint32_t)p.ldxs;

  // Direct: a wave's instruction moves eight rows, lane i the chunk that belongs
  // into slot i % 8 of row i / 8.
  uint32_t direct_at[DIRECT ? kLoads : 1];
  if constexpr (DIRECT) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      direct_at[i] =
          row_offset((wave + i * kWaves) * 8 + (lane >> 3)) + (((lane & 7) ^ swizzle(wave * 8 + (lane >> 3))) << 4);
  }
  auto direct = [&](int st, int buf) {
    // M0 is the LDS destination; the compiler does not track the loads, the
    // pipeline waits for them explicitly.
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int rows8 = wave + i * kWaves;
      const uint32_t dst =
          (uint32_t)reinterpret_cast<uintptr_t>((lds_void*)(smem + buf * kBuf + rows8 * 8 * kRow));
      const uint8_t* src = (rows8 * 8 < BN ? xbase : wbase) + (int64_t)st * kRow;
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst),
                   "v"(direct_at[DIRECT ? i : 0]), "s"(src)
                   : "memory", "m0");
    }
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) {
      const uint32_t dst =
          (uint32_t)reinterpret_cast<uintptr_t>((lds_void*)(scale_lds + buf * kSlots + group(i) * 64));
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(dst), "v"(s_at[i] * 4u),
                   "s"(sbase(i) + st)
                   : "memory", "m0");
    }
  };
  // By registers: chunk i of this thread.
  auto my_row = [&](int i) { return (tid >> 3) + i * (kThreads / 8); };
  auto my_slot = [&](int buf, int i) {
    const int r = my_row(i);
    return reinterpret_cast<u32x4*>(smem + buf * kBuf + r * kRow + (((tid & 7) ^ swizzle(r)) << 4));
  };
  u32x4 regs[DIRECT ? 1 : kPerThread];
  float scale_regs[DIRECT ? 1 : kScaleLoads];
  auto fetch = [&](int st) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      regs[DIRECT ? 0 : i] = *reinterpret_cast<const u32x4_a1*>(row_ptr(my_row(i)) + (int64_t)st * kRow + (tid & 7) * 16);
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) scale_regs[DIRECT ? 0 : i] = sbase(i)[s_at[i] + (uint32_t)st];
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) *my_slot(buf, i) = regs[DIRECT ? 0 : i];
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i)
      scale_lds[buf * kSlots + group(i) * 64 + lane] = scale_regs[DIRECT ? 0 : i];
  };

  floatx16 acc[RB][CB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) acc[rb][cb] = floatx16{};

  // This lane's chunks of its row in the wave's first X (W) row block.
  uint32_t frag_at[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) frag_at[j] = (uint32_t)(l32 * kRow + (((4 * (j >> 1) + 2 * h + (j & 1)) ^ swizzle(l32)) << 4));
  auto fold = [&](floatx16& to, const floatx16& sum, float f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) to[i] = __builtin_fmaf(f, sum[i], to[i]);
  };
  // One stage: W's part widened once, then 32 rows of X at a time.  (All sums at once
  // would need as many registers again as acc.)
  auto compute = [&](int buf) {
    const unsigned char* xs = smem + buf * kBuf + wc * CB * 32 * kRow;
    const unsigned char* ws = smem + buf * kBuf + (BN + wr * RB * 32) * kRow;
    const float* sc = scale_lds + buf * kSlots;
    const float wscale = sc[kSlots - 64 + ((wr * RB * 32) >> 7)];
    bf16x8 w[RB][8];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(ws + rb * 32 * kRow + frag_at[j]);
#pragma unroll
        for (int s = 0; s < 2; ++s) w[rb][2 * j + s] = fp8_widen8(v, s);
      }
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      floatx16 sum[RB];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(xs + cb * 32 * kRow + frag_at[j]);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bf16x8 x = fp8_widen8(v, s);
#pragma unroll
          for (int rb = 0; rb < RB; ++rb) sum[rb] = mfma32(w[rb][2 * j + s], x, j + s == 0 ? floatx16{} : sum[rb]);
        }
      }
      const float f = sc[(wc * CB + cb) * 32 + l32] * wscale;
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) fold(acc[rb][cb], sum[rb], f);
    }
  };

  // Whole blocks first.  Past the last one it is fetched again, into buffers no one
  // reads any more: the number of loads in flight is the same in every stage.
  if (lo < whole) {
    if constexpr (DIRECT) {
#pragma unroll
      for (int i = 0; i < NB - 1; ++i) direct(min(lo + i, whole - 1), i);
      int buf = 0, ahead = NB - 1;
      for (int st = lo; st < whole; ++st) {
        __builtin_amdgcn_s_waitcnt(waitcnt_vm((NB - 2) * (kLoads + kScaleLoads)));
        lds_barrier();                       // the stage is there, and the one before it read
        direct(min(st + NB - 1, whole - 1), ahead);
        compute(buf);
        buf = buf + 1 == NB ? 0 : buf + 1;
        ahead = ahead + 1 == NB ? 0 : ahead + 1;
      }
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));              // none is left in flight to the buffers
    } else {
      fetch(lo);
      put(0);
      for (int st = lo; st < whole; ++st) {
        const int buf = (st - lo) & 1;
        lds_barrier();
        fetch(min(st + 1, whole - 1));
        compute(buf);
        put(buf ^ 1);
      }
    }
  }
  // The partial block at the rows' end.
  if (lo <= whole && whole < hi) {
    lds_barrier();                           // the last reads (and loads) are done
#pragma unroll 4
    for (int i = 0; i < kPerThread; ++i)
      *my_slot(0, i) = fp8_load16_tail(row_ptr(my_row(i)), whole * kRow + (tid & 7) * 16, p.n);
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i)
      scale_lds[group(i) * 64 + lane] = sbase(i)[s_at[i] + (uint32_t)whole];
    lds_barrier();
    compute(0);
  }
  lds_barrier();
  store_tile<Y16, WR, WC, RB, CB>(p, tg, tile, r0, split, acc, smem);
}

__global__ __launch_bounds__(kJoinCols / 4) void fp8_join_kernel(Fp8Operands p, TileGrid tg) { join_splits(p, tg); }

// What a product runs on, from its sizes alone.
enum Kind {
  kRows1, kRows2, kRows4x2,                  // fp8_rows_kernel: 16 or 32 rows of W, 64 with 32 of X
  kTile128x32, kTile128x64, kTile128x128, kTile256x256,     // W rows x X rows of a tile
};
struct Plan {
  Kind kind;
  int splits;                                // of the columns, tiles only
};

// Fitted to 95 sizes from 20 x 91 x 1824 to 4096 x 12288 x 12288: what the model chooses
// takes 1.005 times the fastest shape's time in the mean, 1.1 at worst (128 x 4096 x
// 4096: 19.2 us on 128 x 64 with four splits, 17.6 on 128 x 32 with two).  Some of the
// measured pairs, the chosen first: 40 x 11008 x 4096 on 128 x 64 with two splits (172
// workgroups) 20.8, with three (258, two CUs with two each) 25.9, with one 27.2; 77 x
// 4096 x 11008 on 128 x 64 with four 25.9, 128 x 128 with four 34; 512 x 4096 x 4096 on
// 128 x 64 28, 128 x 128 40; 2048 x 4096 x 4096 on 128 x 128 71, 256 x 256 116.
constexpr TileShape kTileShapes[] = {
    {kTile128x32, 128, 32, 2, 1.77, 1.07, 2.32, 3.0},
    {kTile128x64, 128, 64, 2, 3.76, 1.31, 2.37, 0.84},
    {kTile128x128, 128, 128, 2, 3.65, 2.37, 3.69, 0.49},
};
// Of a 16-bit Y (4096 x 4096 x 4096 on 256 x 256 124 us, 128 x 128 132; 4096 x 12288 x
// 12288 1051 and 1147; 2100 x 6200 x 400 26 and 29).
constexpr TileShape kTileShapes16[] = {
    {kTile128x32, 128, 32, 2, 1.77, 1.07, 2.32, 3.0},
    {kTile128x64, 128, 64, 2, 3.76, 1.31, 2.37, 0.84},
    {kTile128x128, 128, 128, 2, 3.65, 2.37, 3.69, 0.49},
    {kTile256x256, 256, 256, 1, 4.41, 6.97, 6.97, 0.72},
};
constexpr double kJoin = 3.74, kJoinBytes = 0.25e-6;

// Rows through registers.  Fitted to 27 sizes from 17 x 4099 x 4097 to 2048 x 4099 x
// 4097: 1.02 times the fastest in the mean, 1.1 at worst.
constexpr TileShape kRaggedTileShapes[] = {
    {kTile128x32, 128, 32, 2, 1.04, 1.97, 2.54, 0.1},
    {kTile128x64, 128, 64, 2, 1.09, 2.98, 3.8, 0.32},
    {kTile128x128, 128, 128, 2, 1.37, 4.05, 4.59, 0.1},
};
constexpr double kRaggedJoin = 6.35, kRaggedJoinBytes = 0.16e-6;

// The row kernels take up to 16 rows of X and whatever is small: their time goes with
// their workgroups' columns, of 32 rows of W and 16 of X each and about 700 more to
// start (us, against tiles: 32 x 11008 x 4096 18.0 / 18.7, 34 x 11008 x 4096 21.8 / 20.5, 48
// x 11008 x 4096 22.4 / 21.4; 96 x 4096 x 4096 14 / 17, 200 x 4096 x 4096 25 / 21; 17 x
// 4096 x 11008 17 / 18, 33 x 4096 x 11008 23 / 20; 24 x 12288 x 12288 52 / 41; 256 x 2048 x
// 2048 9.6 / 11.5, 512 x 2048 x 2048 17 / 12), unless short rows leave their many
// workgroups little each (24 x 8192 x 512 4.4 / 5.5, 64 x 8192 x 512 7.1 / 5.5; 256 x 1024
// x 1024 4.7 / 7.3, 512 x 1024 x 1024 7.9 / 7.6).  On the slower side are 128 x 4096 x 4096
// (19.2 on tiles, 17.1) and 640 x 300 x 8208 (20.2 on rows, 17.5).  Of rows that are not
// 16-byte aligned they take less (16 x 4099 x 4097 13 / 15, 24 x 4099 x 4097 15 / 14; 128 x
// 1030 x 2044 8.3 / 12, 256 x 1030 x 2043 13 / 14).  Two tiles of W a workgroup read X
// half as often, one gives more workgroups (16 x 4096 x 4096 7.9 and 7.2; 24 x 4096 x
// 4096 7.5 and 10.3; 16 x 49152 x 12288 131 and 159).
Plan make_plan(int64_t m, int64_t n, int64_t rows, int64_t experts, bool grouped, bool y16, bool direct) {
  const int64_t outputs = m * rows, products = outputs * std::max<int64_t>(n, 1);
  // Tiles of bn rows of X that the experts' rows form: as a geometric distribution has
  // them (all of an expert's rows in one tile where they are few, half a tile more where
  // they are many).
  const int64_t touched = std::min(experts, rows);
  const auto expert_tiles = [&](int bn) {
    return (double)touched / -std::expm1(-(double)bn * (double)touched / (double)rows);
  };
  if (grouped) {
    // By the rows that an expert has on average, and more columns than a block for each of
    // the eight waves (us, against tiles: 8 experts of 11008 x 4096 with 8 rows each 68 /
    // 99, with 14 79 / 93; 64 of 1030 x 1024 with 8 25 / 23, 1030 x 1100 31 / 35, 1030 x 1300
    // 34 / 39, 1030 x 1999 43 / 50; at odd addresses 28 / 27, 34 / 31, 37 / 37, 48 / 49 and
    // 1408 x 1536 43 / 53; 64 of 2048 x 1024 with 4 40 / 32; 100 of 512 x 512 with 8 16 /
    // 11; one of 512 x 512 3.4 / 4.2).
    constexpr int64_t kColsAll = kRowWaves * kFp8Block;
    const double row_groups = (double)ceil_div(m, 32) * expert_tiles(16);
    const Plan by_rows{row_groups < 128 ? kRows1 : kRows2, 1};
    if (rows <= 12 * experts && (rows <= 16 || n > kColsAll || touched * m * n <= ((int64_t)1 << 22))) return by_rows;
    // Thirty-two rows of X a workgroup: the weights once.  Where tiles go through registers
    // from three quads of columns on (64 experts of 1030 x 1100 with 24 rows each 50 / 46,
    // 1030 x 1300 53 / 54, 1030 x 1540 54 / 60, 1030 x 1999 63 / 72, 1408 x 4096 123 / 151),
    // where they take rows straight to LDS from eight (1408 x 2304 72 / 55, 1030 x 2560 56 /
    // 55, 1030 x 4096 73 / 84; 8 of 11008 x 4096 with 32 101 / 115).
    if (rows > 12 * experts && rows <= 32 * experts && touched * ceil_div(m, 64) >= 256 && n >= (direct ? 8 : 3) * 512)
      return Plan{kRows4x2, 1};
    // Whatever else is small, as one matrix's below, with any number of rows (2 experts of
    // 128 x 5312 with 60 rows each 6.3 / 27, at odd addresses 7.9 / 53; 20 of 172 x 9051
    // with 23 20 / 44; 3 of 3780 x 1062 with 49 18 / 11; on the slower side 5 of 1205 x 1929
    // with 73, 17 / 15, and 3 of 3634 x 8944 with 55 at odd addresses, 65 / 106).
    if (outputs <= 400 * n && row_groups * (double)(n + 700) <= 5e6) return by_rows;
  } else if (rows <= 16 || (direct ? ceil_div(m, 32) * ceil_div(rows, 16) * (n + 700) <= 4000000 && outputs <= 400 * n
                                   : products <= 400000000)) {
    return Plan{outputs <= 65536 && m < 8192 ? kRows1 : kRows2, 1};
  }
  // A quarter more than the geometric distribution's, as the fit has it.  Over 190 measured
  // pairs of sizes and alignments that take tiles, rows spread twofold, the shape chosen
  // takes 1.02 times the fastest's time in the mean, 1.4 at worst (64 experts of 1030 x 1100
  // with 20 rows each at odd addresses 45 us on 128 x 32, 33 on 128 x 64).
  const auto groups = [&](int64_t w_tiles, int bn) {
    return (int64_t)std::ceil(1.25 * (double)w_tiles * expert_tiles(bn));
  };
  const int64_t e = grouped ? experts : 0;
  const TileChoice c =
      !direct ? choose_tiles(kRaggedTileShapes, m, n, rows, e, groups, kRaggedJoin, kRaggedJoinBytes, true)
      : y16   ? choose_tiles(kTileShapes16, m, n, rows, e, groups, kJoin, kJoinBytes, true)
              : choose_tiles(kTileShapes, m, n, rows, e, groups, kJoin, kJoinBytes, true);
  return Plan{(Kind)c.kind, c.splits};
}

// Workspace of a plan: the splits' sums.
size_t plan_ws(const Plan& pl, int64_t m, int64_t rows) {
  return pl.splits > 1 ? align256((size_t)pl.splits * (size_t)rows * (size_t)m * sizeof(float)) : 0;
}

// A launch has fewer than 2^32 threads.  Calls launch(operands) for the rows of W in
// parts of whole tiles of bm rows, as many as fit when each tile of W takes `slots`
// workgroups.  A part starts at a block of rows.
template <typename Launch>
gptq_status in_row_parts(const Fp8Operands& p, int bm, int64_t slots, int threads, Launch launch) {
  const int64_t unit = std::max(bm, kFp8Block);
  const int64_t part = std::max<int64_t>(((int64_t)1 << 31) / (slots * threads * (unit / bm)), 1) * unit;
  for (int64_t r = 0; r < p.m; r += part) {
    Fp8Operands q = p;
    q.W += r * p.ldw;
    q.S += r / kFp8Block * p.lds;
    q.Y = static_cast<char*>(p.Y) + r * elem_bytes(p.y_dtype);
    q.m = (int)std::min(part, p.m - r);
    launch(q);
    GPTQ_TRY_LAUNCH();
  }
  return GPTQ_OK;
}

template <bool Y16, int WR, int WC, int RB, int CB, int NB, bool DIRECT>
gptq_status launch_tile(const Fp8Operands& p, const Plan& pl, void* ws, hipStream_t st) {
  constexpr int BM = 32 * WR * RB, BN = 32 * WC * CB, lds = tile_lds<WR, WC, RB, CB, NB>();
  const auto k = fp8_tile_kernel<Y16, WR, WC, RB, CB, NB, DIRECT>;
  const int64_t cols = round_up(std::max<int64_t>(ceil_div(p.n, pl.splits), 1), kSplitCols);
  // Whole splits can leave fewer of them than were asked for.
  const int splits = (int)std::max<int64_t>(ceil_div(p.n, cols), 1);
  TileGrid tg{(int)ceil_div(p.m, BM), (int)max_tiles(p.rows, p.experts, p.offsets != nullptr, BN), splits,
              (int)cols, static_cast<float*>(ws)};
  const int64_t slots = (int64_t)tg.tok_tiles * tg.splits;
  if (lds > 65536)
    GPTQ_TRY_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds));
  const gptq_status rc = in_row_parts(p, BM, slots, 64 * WR * WC, [&](const Fp8Operands& q) {
    tg.row_tiles = (int)ceil_div(q.m, BM);
    k<<<(unsigned)round_up(tg.row_tiles * slots, kXcds), 64 * WR * WC, lds, st>>>(q, tg);
  });
  if (rc != GPTQ_OK) return rc;
  if (tg.splits > 1) {
    fp8_join_kernel<<<(unsigned)(ceil_div(p.m, kJoinCols) * p.rows), kJoinCols / 4, 0, st>>>(p, tg);
    GPTQ_TRY_LAUNCH();
  }
  return GPTQ_OK;
}

// What the addresses of all rows have in common: the low bits that are 0.
uint64_t row_starts(const Fp8Operands& p) {
  return reinterpret_cast<uintptr_t>(p.X) | reinterpret_cast<uintptr_t>(p.W) | (uint64_t)(p.rows > 1 ? p.ldx : 0) |
         (uint64_t)(p.m > 1 ? p.ldw : 0) | (uint64_t)p.w_stride;
}

template <bool Y16, int WR, int WC, int RB, int CB, int NB>
gptq_status launch_tiles(const Fp8Operands& p, const Plan& pl, void* ws, hipStream_t st) {
  if ((row_starts(p) & 15) == 0) return launch_tile<Y16, WR, WC, RB, CB, NB, true>(p, pl, ws, st);
  return launch_tile<Y16, WR, WC, RB, CB, 2, false>(p, pl, ws, st);
}

template <int RT, int CT, int D>
gptq_status launch_rows(const Fp8Operands& p, hipStream_t st) {
  constexpr int threads = 64 * kRowWaves;
  const int64_t slots = max_tiles(p.rows, p.experts, p.offsets != nullptr, 16 * CT);
  return in_row_parts(p, 16 * RT, slots, threads, [&](const Fp8Operands& q) {
    fp8_rows_kernel<RT, CT, D>
        <<<(unsigned)(ceil_div(q.m, 16 * RT) * slots), threads, rows_lds<RT, CT>(), st>>>(q);
  });
}

template <bool Y16>
gptq_status launch(const Fp8Operands& p, void* ws, size_t ws_bytes, hipStream_t st) {
  const bool direct = (row_starts(p) & 15) == 0;
  Plan pl = make_plan(p.m, p.n, p.rows, p.experts, p.offsets != nullptr, Y16, direct);
  // The tile kernels address the rows of a tile with 32 bits; rows further apart
  // take the row kernel.
  constexpr int64_t kMaxPitch = (int64_t)1 << 22;
  if (p.ldx > kMaxPitch || p.ldw > kMaxPitch || p.lds * 4 > kMaxPitch || p.ldxs * 4 > kMaxPitch) pl = Plan{kRows2, 1};
  const size_t need = plan_ws(pl, p.m, p.rows);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return GPTQ_ERR_WORKSPACE;
  if (need > 0 && (reinterpret_cast<uintptr_t>(ws) & 3) != 0) return GPTQ_ERR_INVALID_ARG;
  switch (pl.kind) {
    case kTile256x256:
      if constexpr (Y16) return launch_tile<Y16, 4, 2, 2, 4, 2, true>(p, pl, ws, st);
      [[fallthrough]];
    case kTile128x128: return launch_tiles<Y16, 2, 2, 2, 2, 2>(p, pl, ws, st);
    case kTile128x64: return launch_tiles<Y16, 4, 1, 1, 2, 3>(p, pl, ws, st);
    case kTile128x32: return launch_tiles<Y16, 4, 1, 1, 1, 4>(p, pl, ws, st);
    case kRows1: return launch_rows<1, 1, 4>(p, st);
    case kRows4x2: return launch_rows<4, 2, 1>(p, st);
    default: return launch_rows<2, 1, 2>(p, st);
  }
}

gptq_status launch(const Fp8Operands& p, void* ws, size_t ws_bytes, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  return p.y_dtype == GPTQ_F32 ? launch<false>(p, ws, ws_bytes, st) : launch<true>(p, ws, ws_bytes, st);
}

constexpr int64_t kMaxLd = (int64_t)1 << 40; // products of strides and indexes stay below 2^62

// Checks shared by the products; `rows` rows of X against `experts` matrices.
gptq_status check(const Fp8Operands& p, int64_t m, int64_t n, int64_t rows, int64_t experts) {
  if (m < 0 || n < 0 || rows < 0 || experts < 0 || !valid_dtype(p.y_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (n > kFp8MaxCols || m > GPTQ_MX_MAX_ROWS || rows > GPTQ_MX_MAX_ROWS || experts > GPTQ_MX_MAX_EXPERTS)
    return GPTQ_ERR_UNSUPPORTED;
  const int64_t blocks = ceil_div(n, kFp8Block);
  if (p.ldw < n || p.lds < blocks || p.ldx < n || p.ldxs < blocks || p.ldy < m) return GPTQ_ERR_INVALID_ARG;
  if (p.ldw > kMaxLd || p.lds > kMaxLd || p.ldx > kMaxLd || p.ldxs > kMaxLd || p.ldy > kMaxLd)
    return GPTQ_ERR_UNSUPPORTED;
  if (m == 0 || rows == 0 || experts == 0) return GPTQ_OK;
  if (p.Y == nullptr || (n > 0 && (p.W == nullptr || p.S == nullptr || p.X == nullptr || p.XS == nullptr)))
    return GPTQ_ERR_INVALID_ARG;
  return GPTQ_OK;
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" size_t gptq_block_gemm_ws_bytes(int64_t m, int64_t n, int64_t rows, int64_t experts) {
  if (m <= 0 || n < 0 || rows <= 0 || experts <= 0 || n > kFp8MaxCols || m > GPTQ_MX_MAX_ROWS ||
      rows > GPTQ_MX_MAX_ROWS || experts > GPTQ_MX_MAX_EXPERTS)
    return 0;
  // Of one matrix with either kind of Y and rows of any alignment; products grouped
  // by expert need none.
  if (experts > 1) return 0;
  size_t need = 0;
  for (int y16 = 0; y16 < 2; ++y16)
    for (int direct = 0; direct < 2; ++direct)
      need = std::max(need, plan_ws(make_plan(m, n, rows, 1, false, y16 != 0, direct != 0), m, rows));
  return need;
}

extern "C" gptq_status gptq_block_gemm(const uint8_t* codes, int64_t m, int64_t n, int64_t ld_codes, const float* scales,
                                     int64_t ld_scales, const uint8_t* x_codes, int64_t batch, int64_t ld_xcodes,
                                     const float* x_scales, int64_t ld_xscales, void* Y, int y_dtype, int64_t ldy,
                                     void* ws, size_t ws_bytes, void* stream) {
  const Fp8Operands p{codes, scales, ld_codes, ld_scales, 0, 0, (int)m, (int)n, x_codes, x_scales,
                      ld_xcodes, ld_xscales, (int)batch, nullptr, 1, Y, ldy, y_dtype};
  const gptq_status rc = check(p, m, n, batch, 1);
  if (rc != GPTQ_OK || m == 0 || batch == 0) return rc;
  return launch(p, ws, ws_bytes, stream);
}

extern "C" gptq_status gptq_block_gemm_grouped(const uint8_t* codes, int64_t experts, int64_t m, int64_t n,
                                             int64_t ld_codes, int64_t stride_codes, const float* scales,
                                             int64_t ld_scales, int64_t stride_scales, const uint8_t* x_codes,
                                             int64_t rows, int64_t ld_xcodes, const float* x_scales, int64_t ld_xscales,
                                             const int32_t* offsets, void* Y, int y_dtype, int64_t ldy, void* ws,
                                             size_t ws_bytes, void* stream) {
  const Fp8Operands p{codes, scales, ld_codes, ld_scales, stride_codes, stride_scales, (int)m, (int)n, x_codes,
                      x_scales, ld_xcodes, ld_xscales, (int)rows, offsets, (int)experts, Y, ldy, y_dtype};
  const gptq_status rc = check(p, m, n, rows, experts);
  if (rc != GPTQ_OK) return rc;
  if (stride_codes < 0 || stride_scales < 0) return GPTQ_ERR_INVALID_ARG;
  if (stride_codes > (kMaxLd << 5) || stride_scales > (kMaxLd << 5)) return GPTQ_ERR_UNSUPPORTED;
  if (experts > 1 && (stride_codes < m * ld_codes || stride_scales < ceil_div(m, kFp8Block) * ld_scales))
    return GPTQ_ERR_INVALID_ARG;
  if (m == 0 || rows == 0 || experts == 0) return GPTQ_OK;
  if (offsets == nullptr) return GPTQ_ERR_INVALID_ARG;
  return launch(p, ws, ws_bytes, stream);
}
