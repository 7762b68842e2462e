// What the products with quantized weights share on their way from a launch to
// stored results: tiles of X rows by expert, the order of workgroups, the sum
// over split columns, stores.
//
// P is a product's operands: int m, n, rows; const int32_t* offsets (experts + 1
// row offsets, or NULL: one matrix, all rows); int experts; void* Y; int64_t
// ldy; int y_dtype.
#pragma once

#include "mx.h"

#include <cmath>
#include <limits>

namespace gptq {

typedef floatx4 floatx4_a4 __attribute__((aligned(4)));

template <class P>
__device__ inline void store_y(const P& p, int64_t at, float v) {
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
// there are, so whatever they hold no access leaves X or Y (the counts wrap where
// descending offsets count rows more than once: up to 2^16 experts of 2^16 tiles).
template <class P>
__device__ inline TokenTile find_tile(const P& p, int slot, int tile) {
  if (p.offsets == nullptr) return TokenTile{0, slot * tile, min(p.rows, (slot + 1) * tile), true};
  const int lane = (int)threadIdx.x & 63;
  uint32_t before = 0u;                      // tiles of the experts before these 64
  for (int e0 = 0; e0 < p.experts; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < p.experts) {
      lo = min(max(p.offsets[e], 0), p.rows);
      hi = min(max(p.offsets[e + 1], lo), p.rows);
    }
    const uint32_t own = (uint32_t)((hi - lo + tile - 1) / tile);
    uint32_t upto = own;                     // inclusive sum over the lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(upto, d, 64);
      if (lane >= d) upto += o;
    }
    const uint32_t at = (uint32_t)slot - before - (upto - own);
    const uint64_t hit = __ballot(at < own);
    if (hit != 0) {
      const int l = __builtin_ctzll(hit);
      const int begin = __shfl(lo + (int)at * tile, l, 64), end = __shfl(hi, l, 64);
      return TokenTile{e0 + l, __builtin_amdgcn_readfirstlane(begin),
                       __builtin_amdgcn_readfirstlane(min(end, begin + tile)), true};
    }
    before += (uint32_t)__builtin_amdgcn_readfirstlane((int)__shfl(upto, 63, 64));
  }
  return TokenTile{0, 0, 0, false};
}

// s_waitcnt immediate (gfx9 encoding): vmcnt <= v, expcnt unconstrained, lgkmcnt = 0.
constexpr int waitcnt_vm(int v) { return (v & 15) | ((v >> 4) << 14) | (7 << 4); }

// Orders LDS accesses only: loads in flight are waited for explicitly.
__device__ inline void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// What the lanes loaded, row lane / 4 and quarter lane % 4 of its 64 bytes, into the
// order of the matrix instruction, row lane % 16 and quarter lane / 16, through the
// wave's own kExchange bytes of LDS (its accesses are done in their order).  Loaded in
// the instruction's order, every lane beside another's row, a load takes 64 accesses
// of the cache for 16 (16 tokens, 64 experts 2048 x 1024 in 8 bits 71 us for 68; 1 token,
// 8 of 4096 x 11008 in 4 bits 46 for 43).
constexpr int kExchange = 2 * 64 * 16;
__device__ inline void wave_fence() {        // for the compiler alone
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}
__device__ inline void exchange(u32x4 (&w)[2], u32x4* lds, int lane) {
  wave_fence();
#pragma unroll
  for (int h = 0; h < 2; ++h) lds[64 * h + ((lane & 60) | ((lane & 3) ^ (lane >> 4)))] = w[h];
  wave_fence();
#pragma unroll
  for (int h = 0; h < 2; ++h) w[h] = lds[64 * h + (4 * (lane & 15) | ((lane >> 4) ^ (lane >> 2 & 3)))];
}

// Work of one launch: tiles of W rows, of X rows, and parts of the columns.
struct TileGrid {
  int row_tiles, tok_tiles, splits, cols_per_split;
  float* part;                               // [split][row of X][m] sums, when splits > 1
};

// Tiles of X rows are numbered within bands of eight, all W tiles of a band
// before the next band: the workgroups an XCD runs at a time share few rows of
// either operand in its L2.
constexpr int kTokBand = 8;

// The first `left` of eight neighbouring results.
template <int YT>
__device__ inline void store8(void* Y, int64_t at, int left, floatx4 lo, floatx4 hi) {
  if constexpr (YT == GPTQ_F32) {
    float* y = static_cast<float*>(Y) + at;
    if (left >= 8) {
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

// Workgroup -> (split, tile of X rows, tile of W rows); false: none.
template <class P>
__device__ inline bool tile_of_workgroup(const P& p, const TileGrid& tg, int BM, int BN, int& split,
                                         TokenTile& tile, int& r0) {
  const int64_t tiles = (int64_t)tg.row_tiles * tg.tok_tiles;
  const int64_t item = xcd_contiguous(blockIdx.x, gridDim.x);
  if (item >= tiles * tg.splits) return false;
  split = (int)(item / tiles);
  const int t = (int)(item % tiles);
  const int band = t / (kTokBand * tg.row_tiles);
  const int in_band = min(kTokBand, tg.tok_tiles - band * kTokBand);
  const int rest = t - band * kTokBand * tg.row_tiles;
  tile = find_tile(p, band * kTokBand + rest % in_band, BN);
  r0 = rest / in_band * BM;
  return tile.valid;
}

// Adds the splits' sums in order, four columns a thread and four splits' loads
// in flight (one at a time they cost a memory latency a split).  All workgroups
// lie along x, a row of X after the other: there can be more rows than a grid
// has along y (65535).  Every row has a sum: products grouped by expert are never
// split.
constexpr int kJoinCols = 1024;              // columns of Y a workgroup
template <class P>
__device__ inline void join_splits(const P& p, const TileGrid& tg) {
  const int chunks = (p.m + kJoinCols - 1) / kJoinCols;
  const int x = (int)(blockIdx.x / chunks), r = (int)(blockIdx.x % chunks) * kJoinCols + (int)threadIdx.x * 4;
  if (r >= p.m) return;
  const int64_t total = (int64_t)p.rows * p.m;
  const float* part = tg.part + (int64_t)x * p.m;
  const int left = p.m - r;
  auto load = [&](int split) {
    const float* at = part + min(split, tg.splits - 1) * total;
    if (left >= 4) return *reinterpret_cast<const floatx4_a4*>(at + r);
    return floatx4{at[r], at[min(r + 1, p.m - 1)], at[min(r + 2, p.m - 1)], 0.f};
  };
  floatx4 v = load(0);
  for (int s = 1; s < tg.splits; s += 4) {
    floatx4 t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = load(s + i);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (s + i < tg.splits) v += t[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) store_y(p, (int64_t)x * p.ldy + r + i, v[i]);
}

// Tiles that the rows can form at most: every expert with rows may end in a
// partial tile.
inline int64_t max_tiles(int64_t rows, int64_t experts, bool grouped, int tile) {
  return grouped ? rows / tile + std::min(experts, rows) : ceil_div(rows, tile);
}

// Products on tiles: the shape and the splits of the columns with the least time by
// this model, in us: a launch, 256 columns of every round of workgroups, each
// round with as many as the CUs hold at once, what a round takes beside them, and
// the join with its splits' sums (a launch, and the bytes that they move).  A round's time grows from `one` (a
// workgroup a CU) to `full` along a square root (a few CUs with two already hold
// the rest up), or at_once: it is `full` as soon as one CU has two.  experts: 0, or of
// products grouped by expert, which have no splits; expert_groups(tiles of W, rows of X
// of a tile): their workgroups.
struct TileShape {
  int kind;                                  // of the caller
  int bm, bn, per_cu;                        // rows of W and of X, workgroups a CU holds
  double launch, one, full;
  double round = 0;                          // what every round takes beside its columns
};
struct TileChoice {
  int kind, splits;
};
constexpr int kSplitCols = 256;              // a split is a multiple of this
template <size_t N, typename Groups>
TileChoice choose_tiles(const TileShape (&shapes)[N], int64_t m, int64_t n, int64_t rows, int64_t experts,
                        Groups expert_groups, double join, double join_bytes, bool at_once) {
  const int max_splits = experts > 0 ? 1 : 16;
  TileChoice best{shapes[0].kind, 1};
  double least = std::numeric_limits<double>::infinity();
  const double parts = (double)m * (double)rows * 8.0;       // bytes that a split's sums move
  for (const TileShape& s : shapes) {
    const int64_t held = 256 * s.per_cu, w_tiles = ceil_div(m, s.bm);
    const int64_t tiles = experts > 0 ? expert_groups(w_tiles, s.bn) : w_tiles * ceil_div(rows, s.bn);
    for (int splits = 1; splits <= max_splits && (splits == 1 || n >= (int64_t)splits * kSplitCols); ++splits) {
      const int64_t groups = tiles * splits, rest = groups % held;
      double t = (double)(groups / held) * s.full;
      if (rest > 256) t += at_once ? s.full : s.one + (s.full - s.one) * std::sqrt((double)(rest - 256) * (1.0 / 256));
      else if (rest > 0) t += s.one;
      t = s.launch + s.round * (double)ceil_div(groups, held) + t * (double)ceil_div(ceil_div(n, splits), kSplitCols);
      if (splits > 1) t += join + join_bytes * splits * parts;
      if (t < least) least = t, best = TileChoice{s.kind, splits};
      if (groups > 2 * held) break;          // more splits only add sums
    }
  }
  return best;
}

}  // namespace gptq
