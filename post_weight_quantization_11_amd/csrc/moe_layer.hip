// A whole layer of experts for few tokens, in two launches:
//   y_t = sum over t's experts e of p_te D_e (silu(G_e x_t) * (U_e x_t))
// with the experts and probabilities of the router, and G, U (rows of one stack)
// and D microscaled or in block-scaled 8-bit floats.
//
// First launch (moe_up_kernel): every workgroup routes all tokens itself (a wave a
// token, the experts' tokens as 64-bit masks in LDS), takes the slot-th expert that
// has any, and 16 rows of its G with the same 16 of its U; its eight waves split
// the columns.  h = silu(g) * u goes to the workspace as three bfloat16 numbers
// that add up to its float32 value (8 bits each), so that the second launch's
// products, exact in float32, lose none of it.
//
// Second launch (moe_down_kernel): a workgroup takes 64 rows of D for all experts
// and tokens; the waves of the row group's `splits` workgroups share the list of
// (expert, 128 columns) and add p h D into sums of their own, in float32, joined in
// wave order and, by the workgroup that comes last, in split order.  The first
// launch clears the counters that tell the last.
//
// Both are bound by the weights' bytes, or for small layers by latency: routing,
// one load after it, and the joins.
#include "fp8.h"
#include "moe.h"
#include "mx_operands.h"
#include "product.h"

namespace gptq {
namespace {

constexpr int kMxWeights = 0, kBlockWeights = 1;             // formats of the weights
constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kPlanes = 3;                   // bfloat16 numbers of an h
constexpr int kDownTiles = 4, kDownRows = 16 * kDownTiles;

// A stack of weights: `experts` matrices.
struct Weights {
  const void* codes;                         // packed words or bytes
  const void* scales;                        // bytes or float32
  int64_t ld, lds, stride, s_stride;         // in those
};

struct MoeArgs {
  Weights gate_up, down;
  int tokens, experts, k, renormalize, d, f, f_pad, splits;
  const void* X;
  int64_t ldx;
  const void* logits;
  int l_dtype;
  int64_t ld_logits;
  // Workspace.
  int32_t* ids;                              // tokens x k
  float* weights;
  uint32_t* arrived;                         // a counter for each group of rows of D
  uint16_t* h;                               // [plane][tokens * k][f_pad]
  float* part;                               // [split][token][d]
  void* Y;
  int64_t ldy;
  int y_dtype;
};

// What a wave multiplies of one row of weights in 128 columns.
template <int WF> struct Row;
template <> struct Row<kMxWeights> {
  const uint32_t* codes;
  const uint8_t* scales;
  u32x4 w;
  uint32_t s;
};
template <> struct Row<kBlockWeights> {
  const uint8_t* codes;
  const float* scales;
  u32x4 w[2];
  float s;
};

// Row r of expert e (clamped by the caller).
__device__ inline void point(Row<kMxWeights>& o, const Weights& w, int64_t e, int64_t r) {
  o.codes = static_cast<const uint32_t*>(w.codes) + e * w.stride + r * w.ld;
  o.scales = static_cast<const uint8_t*>(w.scales) + e * w.s_stride + r * w.lds;
}
__device__ inline void point(Row<kBlockWeights>& o, const Weights& w, int64_t e, int64_t r) {
  o.codes = static_cast<const uint8_t*>(w.codes) + e * w.stride + r * w.ld;
  o.scales = static_cast<const float*>(w.scales) + e * w.s_stride + (r >> 7) * w.lds;
}

// Lane quarter q's share of unit u (columns 128 u ..); n: columns of the row, `all`
// of the unit's there or not.
__device__ inline void load_row(Row<kMxWeights>& o, int u, int q, bool all, int n) {
  if (all) {
    o.w = *reinterpret_cast<const u32x4_a4*>(o.codes + 16 * u + 4 * q);
    o.s = *reinterpret_cast<const u32_a1*>(o.scales + 4 * u);
  } else {
    o.w = load_w4_tail(o.codes, 16 * u + 4 * q, n);
    o.s = load_scales4(o.scales, 4 * u, n);
  }
}
__device__ inline void load_row(Row<kBlockWeights>& o, int u, int q, bool all, int n) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = 128 * u + 64 * h + 16 * q;
    o.w[h] = all ? (u32x4)*reinterpret_cast<const u32x4_a1*>(o.codes + k) : fp8_load16_tail(o.codes, k, n);
  }
  o.s = o.scales[u];
}

// The column, inside a unit, of the eight that lane quarter q holds in step s.
template <int WF> __device__ inline int step_col(int s, int q) {
  return WF == kMxWeights ? 32 * s + 8 * q : 64 * (s >> 1) + 16 * q + 8 * (s & 1);
}

// Eight weights of step s as 16-bit numbers.  (w: of microscaled codes, transposed.)
template <int T> __device__ inline u32x4 widen(const Row<kMxWeights>& o, u32x4 w, int s) {
  return widen8<T>(w[s], mx_scale_operand((o.s >> (8 * s)) & 255u));
}
template <int T> __device__ inline u32x4 widen(const Row<kBlockWeights>& o, u32x4, int s) {
  if constexpr (T == GPTQ_BF16) {
    return __builtin_bit_cast(u32x4, fp8_widen8(o.w[s >> 1], s & 1));
  } else {
    const uint32_t lo = o.w[s >> 1][2 * (s & 1)], hi = o.w[s >> 1][2 * (s & 1) + 1];
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true))};
  }
}
__device__ inline u32x4 transposed(const Row<kMxWeights>& o) { return transpose_quarters(o.w); }
__device__ inline u32x4 transposed(const Row<kBlockWeights>&) { return u32x4{0u, 0u, 0u, 0u}; }

// The index of the n-th set bit (n below their count; the last one otherwise).
__device__ inline int nth_bit(uint64_t mask, int n) {
  int at = 0;
  for (int i = 0; mask != 0; ++i, mask &= mask - 1)           // the same for all lanes
    if (i <= n) at = __builtin_ctzll(mask);
  return at;
}

// The place of expert e among token t's.
__device__ inline int place_of(const int* ids, int t, int k, int e) {
  int j = 0;
  for (int i = 1; i < k; ++i)
    if (ids[t * k + i] == e) j = i;
  return j;
}

// ---------------------------------------------------------------------------
// Gate and up.
// ---------------------------------------------------------------------------
// Sums of the wave's share of the columns: 16 tokens x 16 rows of G and of U.  SPLIT
// (float16 X, microscaled weights that float16 does not hold): X as the sum of two
// bfloat16 numbers.  Otherwise `inexact` gathers whether there are such weights.
template <int WF, int XT, bool SPLIT>
__device__ inline void up_sums(const MoeArgs& p, Row<WF> (&row)[2], const uint16_t* x, floatx4 (&acc)[2],
                               uint32_t& inexact) {
  constexpr int D = 2;
  const int lane = (int)threadIdx.x & 63, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int units = (p.d + 127) >> 7, whole = p.d >> 7;
  const int lo = units * wave / kWaves, hi = units * (wave + 1) / kWaves, last = min(hi, whole);
  struct Unit {
    Row<WF> w[2];
    u32x4 x[4];
  };
  auto load = [&](int u, bool all, Unit& o) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o.w[i].codes = row[i].codes;
      o.w[i].scales = row[i].scales;
      load_row(o.w[i], u, q, all, p.d);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = 128 * u + step_col<WF>(s, q);
      o.x[s] = all ? (u32x4)*reinterpret_cast<const u32x4_a2*>(x + k) : load_x8_tail(x, k, p.d);
    }
  };
  auto multiply = [&](const Unit& o) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4 w = transposed(o.w[i]);
      floatx4 v = floatx4{0.f, 0.f, 0.f, 0.f};
      if constexpr (WF == kMxWeights) {
        v = acc[i];
        if constexpr (XT == GPTQ_F16 && !SPLIT) inexact |= f16_inexact4(o.w[i].s);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if constexpr (SPLIT) {
          u32x4 top, rest;
          split8(o.x[s], top, rest);
          const u32x4 wv = widen<GPTQ_BF16>(o.w[i], w, s);
          v = mfma16<GPTQ_BF16>(top, wv, v);
          v = mfma16<GPTQ_BF16>(rest, wv, v);
        } else {
          v = mfma16<XT>(o.x[s], widen<XT>(o.w[i], w, s), v);
        }
      }
      if constexpr (WF == kMxWeights) {
        acc[i] = v;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_fmaf(o.w[i].s, v[j], acc[i][j]);
      }
    }
  };
  if (lo < last) {
    Unit ring[D];
#pragma unroll
    for (int i = 0; i < D; ++i) load(min(lo + i, last - 1), true, ring[i]);
    for (int u = lo; u < last; u += D) {
#pragma unroll
      for (int i = 0; i < D; ++i) {
        if (u + i < last) multiply(ring[i]);
        load(min(u + i + D, last - 1), true, ring[i]);
      }
    }
  }
  if (lo < hi && whole < hi) {
    Unit o;
    load(whole, false, o);
    multiply(o);
  }
}

template <int WF, int XT>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeArgs p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  floatx4* red = reinterpret_cast<floatx4*>(smem);            // [wave][gate, up][64]
  uint64_t* masks = reinterpret_cast<uint64_t*>(red + kWaves * 2 * 64);       // tokens of each expert
  int* ids = reinterpret_cast<int*>(masks + p.experts);       // tokens x k
  const int tid = (int)threadIdx.x, lane = tid & 63, q = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = p.f_pad / 16;
  const int slot = (int)(blockIdx.x / tiles), f0 = (int)(blockIdx.x % tiles) * 16;
  const bool first = blockIdx.x == 0;

  for (int e = tid; e < p.experts; e += kThreads) masks[e] = 0u;
  __syncthreads();
  for (int t = wave; t < p.tokens; t += kWaves) {
    const Routed r = route_token(p.logits, p.l_dtype, (int64_t)t * p.ld_logits, p.experts, p.k,
                                 first && !p.renormalize);
    if (lane < p.k) {
      ids[t * p.k + lane] = r.id;
      atomicOr(reinterpret_cast<unsigned long long*>(masks + r.id), 1ull << t);
    }
    if (first) {
      const float w = route_weight(r, p.k, p.renormalize);
      if (lane < p.k) {
        p.ids[t * p.k + lane] = r.id;
        p.weights[t * p.k + lane] = w;
      }
    }
  }
  if (first)
    for (int i = tid; i < (p.d + kDownRows - 1) / kDownRows; i += kThreads) p.arrived[i] = 0u;
  __syncthreads();

  // The slot-th expert that has tokens.
  int expert = -1, before = 0;
  uint64_t mask = 0;
  for (int e0 = 0; e0 < p.experts; e0 += 64) {
    const uint64_t m = e0 + lane < p.experts ? masks[e0 + lane] : 0u;
    const uint64_t has = __ballot(m != 0);
    const int count = __popcll(has);
    if (slot < before + count) {
      expert = e0 + nth_bit(has, slot - before);
      mask = masks[expert];
      break;
    }
    before += count;
  }
  if (expert < 0) return;
  expert = __builtin_amdgcn_readfirstlane(expert);
  mask = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(mask >> 32)) << 32 |
         (uint32_t)__builtin_amdgcn_readfirstlane((int)mask);
  const int count = __popcll(mask);

  Row<WF> row[2];
  if (f0 < p.f) {
    const int r = min(f0 + c16, p.f - 1);
    point(row[0], p.gate_up, expert, r);
    point(row[1], p.gate_up, expert, p.f + r);
  }
  for (int c0 = 0; c0 < count; c0 += 16) {   // tokens, sixteen at a time
    if (f0 < p.f) {
      const int t = nth_bit(mask, c0 + c16);
      const uint16_t* x = static_cast<const uint16_t*>(p.X) + (int64_t)t * p.ldx;
      floatx4 acc[2] = {floatx4{0.f, 0.f, 0.f, 0.f}, floatx4{0.f, 0.f, 0.f, 0.f}};
      uint32_t inexact = 0u;
      up_sums<WF, XT, false>(p, row, x, acc, inexact);
      if constexpr (WF == kMxWeights && XT == GPTQ_F16) {
        if (!__syncthreads_and(inexact == 0u)) {
          acc[0] = acc[1] = floatx4{0.f, 0.f, 0.f, 0.f};
          up_sums<WF, XT, true>(p, row, x, acc, inexact);
        }
      }
      red[(wave * 2) * 64 + lane] = acc[0];
      red[(wave * 2 + 1) * 64 + lane] = acc[1];
    }
    __syncthreads();
    if (tid < 256) {
      // Register j of lane l: token 4 (l / 16) + j, row l % 16.
      const int l = tid >> 2, at = c0 + 4 * (l >> 4) + (tid & 3), r = f0 + (l & 15);
      float h = 0.f;
      if (r < p.f) {
        const float* s = reinterpret_cast<const float*>(red) + tid;
        float g = s[0], u = s[256];
        for (int w = 1; w < kWaves; ++w) {
          g += s[w * 512];
          u += s[w * 512 + 256];
        }
        h = g / (1.f + expf(-g)) * u;
      }
      if (at < count) {
        const int t = nth_bit(mask, at);
        const int64_t pairs = (int64_t)p.tokens * p.k, pair = (int64_t)t * p.k + place_of(ids, t, p.k, expert);
        uint16_t* o = p.h + pair * p.f_pad + r;
#pragma unroll
        for (int i = 0; i < kPlanes; ++i) {
          const uint32_t top = __float_as_uint(h) & 0xFFFF0000u;               // 8 bits, the rest exact
          o[i * pairs * p.f_pad] = (uint16_t)(top >> 16);
          const bool finite = (top & 0x7F800000u) != 0x7F800000u;
          h = finite ? h - __uint_as_float(top) : 0.f;
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Down.
// ---------------------------------------------------------------------------
template <int WF>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int pairs = p.tokens * p.k;
  float* sums = reinterpret_cast<float*>(smem);               // [wave][token][64 rows]
  uint64_t* masks = reinterpret_cast<uint64_t*>(sums + kWaves * p.tokens * kDownRows);
  int* ids = reinterpret_cast<int*>(masks + p.experts);
  float* weights = reinterpret_cast<float*>(ids + pairs);
  int* items = reinterpret_cast<int*>(weights + pairs);       // experts and their sixteens of tokens
  __shared__ int item_count, is_last;
  const int tid = (int)threadIdx.x, lane = tid & 63, q = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int groups = (p.d + kDownRows - 1) / kDownRows;
  const int group = (int)blockIdx.x % groups, split = (int)blockIdx.x / groups, r0 = group * kDownRows;

  for (int e = tid; e < p.experts; e += kThreads) masks[e] = 0u;
  for (int i = tid; i < pairs; i += kThreads) {
    ids[i] = p.ids[i];
    weights[i] = p.weights[i];
  }
  for (int i = tid; i < kWaves * p.tokens * kDownRows; i += kThreads) sums[i] = 0.f;
  __syncthreads();
  for (int i = tid; i < pairs; i += kThreads)
    atomicOr(reinterpret_cast<unsigned long long*>(masks + ids[i]), 1ull << (i / p.k));
  __syncthreads();
  if (wave == 0) {
    int before = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
      const int own = e0 + lane < p.experts ? (__popcll(masks[e0 + lane]) + 15) / 16 : 0;
      int upto = own;
#pragma unroll
      for (int x = 1; x < 64; x <<= 1) {
        const int o = __shfl_up(upto, x, 64);
        if (lane >= x) upto += o;
      }
      for (int i = 0; i < own; ++i) items[before + upto - own + i] = (e0 + lane) | i << 16;
      before += __shfl(upto, 63, 64);
    }
    if (lane == 0) item_count = before;
  }
  __syncthreads();

  const int per_item = p.f_pad / 128, whole = p.f >> 7;
  const int64_t total = (int64_t)item_count * per_item, parts = (int64_t)p.splits * kWaves, part = split * kWaves + wave;
  const int lo = (int)(total * part / parts), hi = (int)(total * (part + 1) / parts);
  const int64_t plane = (int64_t)pairs * p.f_pad;
  float* mine = sums + wave * p.tokens * kDownRows;

  // Lane c16's pair of an item (clamped to the last), and whether it is one.
  auto pair_of = [&](int item, bool& there) {
    const int e = items[item] & 0xFFFF, c = (items[item] >> 16) * 16 + c16;
    const uint64_t mask = masks[e];
    const int t = nth_bit((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(mask >> 32)) << 32 |
                              (uint32_t)__builtin_amdgcn_readfirstlane((int)mask),
                          c);
    there = c < __popcll(mask);
    return t * p.k + place_of(ids, t, p.k, e);
  };

  constexpr int D = 2;
  struct Unit {
    Row<WF> w[kDownTiles];
    u32x4 x[kPlanes][4];
  };
  int at_item = -1;                          // of the loads
  const uint16_t* h = p.h;
  Row<WF> row[kDownTiles];
  auto load = [&](int n, Unit& o) {
    const int item = n / per_item, u = n - item * per_item;
    if (item != at_item) {
      at_item = item;
      const int e = __builtin_amdgcn_readfirstlane(items[item] & 0xFFFF);
#pragma unroll
      for (int i = 0; i < kDownTiles; ++i) point(row[i], p.down, e, min(r0 + 16 * i + c16, p.d - 1));
      bool there;
      h = p.h + (int64_t)pair_of(item, there) * p.f_pad;
    }
    const bool all = u < whole;
#pragma unroll
    for (int i = 0; i < kDownTiles; ++i) {
      o.w[i].codes = row[i].codes;
      o.w[i].scales = row[i].scales;
      load_row(o.w[i], u, q, all, p.f);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < kPlanes; ++i)
        o.x[i][s] = *reinterpret_cast<const u32x4*>(h + i * plane + 128 * u + step_col<WF>(s, q));
  };
  floatx4 acc[kDownTiles];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < kDownTiles; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  };
  auto multiply = [&](const Unit& o) {
#pragma unroll
    for (int i = 0; i < kDownTiles; ++i) {
      const u32x4 w = transposed(o.w[i]);
      floatx4 v = WF == kMxWeights ? acc[i] : floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const u32x4 wv = widen<GPTQ_BF16>(o.w[i], w, s);
#pragma unroll
        for (int j = 0; j < kPlanes; ++j) v = mfma16<GPTQ_BF16>(wv, o.x[j][s], v);
      }
      if constexpr (WF == kMxWeights) {
        acc[i] = v;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_fmaf(o.w[i].s, v[j], acc[i][j]);
      }
    }
  };
  // Register j of lane l: row 4 (l / 16) + j, the item's token l % 16.  A weight of 0
  // leaves a token without the expert's product, whatever that is.
  auto flush = [&](int item) {
    bool there;
    const int pair = pair_of(item, there);
    const float w = weights[pair];
    if (there && w != 0.f) {
      float* to = mine + pair / p.k * kDownRows + 4 * q;
#pragma unroll
      for (int i = 0; i < kDownTiles; ++i) {
        floatx4 s = *reinterpret_cast<floatx4*>(to + 16 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = __builtin_fmaf(w, acc[i][j], s[j]);
        *reinterpret_cast<floatx4*>(to + 16 * i) = s;
      }
    }
  };
  if (lo < hi) {
    Unit ring[D];
#pragma unroll
    for (int i = 0; i < D; ++i) load(min(lo + i, hi - 1), ring[i]);
    clear();
    for (int n = lo; n < hi; n += D) {
#pragma unroll
      for (int i = 0; i < D; ++i) {
        if (n + i < hi) {
          multiply(ring[i]);
          if (n + i + 1 == hi || (n + i + 1) % per_item == 0) {
            flush((n + i) / per_item);
            clear();
          }
        }
        load(min(n + i + D, hi - 1), ring[i]);
      }
    }
  }
  __syncthreads();
  const int outputs = p.tokens * kDownRows;
  for (int i = tid; i < outputs; i += kThreads) {
    const int t = i / kDownRows, r = r0 + i % kDownRows;
    float v = sums[i];
    for (int w = 1; w < kWaves; ++w) v += sums[w * outputs + i];
    if (r >= p.d) continue;
    if (p.splits == 1) store_y(p, (int64_t)t * p.ldy + r, v);
    else p.part[((int64_t)split * p.tokens + t) * p.d + r] = v;
  }
  if (p.splits == 1) return;
  // The last workgroup of the group adds the parts, in order.
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
  __syncthreads();
  if (tid == 0)
    is_last = __hip_atomic_fetch_add(p.arrived + group, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
              (uint32_t)p.splits - 1u;
  __syncthreads();
  if (!is_last) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  for (int i = tid; i < outputs; i += kThreads) {
    const int t = i / kDownRows, r = r0 + i % kDownRows;
    if (r >= p.d) continue;
    const float* at = p.part + (int64_t)t * p.d + r;
    float v = at[0];
    for (int s = 1; s < p.splits; ++s) v += at[(int64_t)s * p.tokens * p.d];
    store_y(p, (int64_t)t * p.ldy + r, v);
  }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------
struct Workspace {
  size_t ids, weights, arrived, h, part, total;               // offsets in bytes
};
constexpr int64_t kMaxSplits = 16;

int down_splits(int64_t tokens, int64_t experts, int64_t topk, int64_t d, int64_t f) {
  // Two workgroups a CU, a unit of 128 columns a wave at least.
  const int64_t groups = ceil_div(d, kDownRows), units = std::min(experts, tokens * topk) * ceil_div(f, 128);
  return (int)std::max<int64_t>(1, std::min({kMaxSplits, 512 / groups, units / kWaves}));
}

Workspace workspace(int64_t tokens, int64_t experts, int64_t topk, int64_t d, int64_t f) {
  const size_t pairs = (size_t)(tokens * topk), f_pad = (size_t)round_up(f, 128);
  const int splits = down_splits(tokens, experts, topk, d, f);
  Workspace w;
  w.ids = 0;
  w.weights = align256(pairs * 4);
  w.arrived = w.weights + align256(pairs * 4);
  w.h = w.arrived + align256((size_t)ceil_div(d, kDownRows) * 4);
  w.part = w.h + align256(kPlanes * pairs * f_pad * 2);
  w.total = w.part + (splits > 1 ? align256((size_t)splits * (size_t)(tokens * d) * 4) : 0);
  return w;
}

bool sizes_fit(int64_t tokens, int64_t experts, int64_t topk, int64_t d, int64_t f) {
  return tokens <= GPTQ_MOE_MAX_TOKENS && experts <= kMoeMaxExperts && topk <= kMoeMaxTopk && d <= kMxMaxCols &&
         f <= kMxMaxCols / 2;
}

// One stack of weights of `rows` x `cols`: words (bytes) and scales to a row, rows of
// scales.
gptq_status check_weights(const Weights& w, int64_t experts, int64_t rows, int64_t words, int64_t scale_rows,
                          int64_t scales) {
  constexpr int64_t kMaxLd = (int64_t)1 << 40;
  if (w.codes == nullptr || w.scales == nullptr || w.ld < words || w.lds < scales) return GPTQ_ERR_INVALID_ARG;
  if (w.ld > kMaxLd || w.lds > kMaxLd) return GPTQ_ERR_UNSUPPORTED;
  if (experts == 1) return GPTQ_OK;
  if (w.stride < rows * w.ld || w.s_stride < scale_rows * w.lds) return GPTQ_ERR_INVALID_ARG;
  return w.stride > (kMaxLd << 10) || w.s_stride > (kMaxLd << 10) ? GPTQ_ERR_UNSUPPORTED : GPTQ_OK;
}

template <int WF>
gptq_status layer(MoeArgs p, int64_t experts, int64_t d, int64_t f, int x_dtype, int64_t tokens, int topk, void* ws,
                  size_t ws_bytes, void* stream) {
  if (tokens < 0 || experts < 1 || d < 0 || f < 1 || topk < 1 || topk > experts) return GPTQ_ERR_INVALID_ARG;
  if ((x_dtype != GPTQ_F16 && x_dtype != GPTQ_BF16) || !valid_dtype(p.l_dtype) || !valid_dtype(p.y_dtype))
    return GPTQ_ERR_INVALID_ARG;
  if (!sizes_fit(tokens, experts, topk, d, f)) return GPTQ_ERR_UNSUPPORTED;
  if (p.ldx < d || p.ldy < d || p.ld_logits < experts) return GPTQ_ERR_INVALID_ARG;
  constexpr int64_t kMaxLd = (int64_t)1 << 40;
  if (p.ldx > kMaxLd || p.ldy > kMaxLd || p.ld_logits > kMaxLd) return GPTQ_ERR_UNSUPPORTED;
  if (tokens == 0 || d == 0) return GPTQ_OK;
  if (p.X == nullptr || p.logits == nullptr || p.Y == nullptr) return GPTQ_ERR_INVALID_ARG;
  constexpr bool MX = WF == kMxWeights;
  gptq_status rc = MX ? check_weights(p.gate_up, experts, 2 * f, ceil_div(d, 8), 2 * f, ceil_div(d, kMxBlock))
                      : check_weights(p.gate_up, experts, 2 * f, d, ceil_div(2 * f, kFp8Block), ceil_div(d, kFp8Block));
  if (rc != GPTQ_OK) return rc;
  rc = MX ? check_weights(p.down, experts, d, ceil_div(f, 8), d, ceil_div(f, kMxBlock))
          : check_weights(p.down, experts, d, f, ceil_div(d, kFp8Block), ceil_div(f, kFp8Block));
  if (rc != GPTQ_OK) return rc;
  const Workspace w = workspace(tokens, experts, topk, d, f);
  if (ws == nullptr || ws_bytes < w.total) return GPTQ_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 15) != 0) return GPTQ_ERR_INVALID_ARG;
  char* base = static_cast<char*>(ws);
  p.ids = reinterpret_cast<int32_t*>(base + w.ids);
  p.weights = reinterpret_cast<float*>(base + w.weights);
  p.arrived = reinterpret_cast<uint32_t*>(base + w.arrived);
  p.h = reinterpret_cast<uint16_t*>(base + w.h);
  p.part = reinterpret_cast<float*>(base + w.part);
  p.tokens = (int)tokens;
  p.experts = (int)experts;
  p.k = topk;
  p.d = (int)d;
  p.f = (int)f;
  p.f_pad = (int)round_up(f, 128);
  p.splits = down_splits(tokens, experts, topk, d, f);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t pairs = tokens * topk, slots = std::min<int64_t>(experts, pairs);

  const size_t up_lds = kWaves * 2 * 64 * sizeof(floatx4) + experts * 8 + pairs * 4;
  const unsigned up_grid = (unsigned)(slots * (p.f_pad / 16));
  if (x_dtype == GPTQ_F16) moe_up_kernel<WF, GPTQ_F16><<<up_grid, kThreads, up_lds, st>>>(p);
  else moe_up_kernel<WF, GPTQ_BF16><<<up_grid, kThreads, up_lds, st>>>(p);
  GPTQ_TRY_LAUNCH();

  // An item for every expert with tokens and every sixteen tokens more.
  const size_t items = (size_t)(slots + pairs / 16);
  const int down_lds = (int)(kWaves * tokens * kDownRows * 4 + experts * 8 + pairs * 8 + items * 4);
  const auto k = moe_down_kernel<WF>;
  if (down_lds > 65536)
    GPTQ_TRY_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize,
                                     down_lds));
  k<<<(unsigned)(ceil_div(d, kDownRows) * p.splits), kThreads, down_lds, st>>>(p);
  GPTQ_TRY_LAUNCH();
  return GPTQ_OK;
}

}  // namespace
}  // namespace gptq

using namespace gptq;

extern "C" size_t gptq_moe_ws_bytes(int64_t tokens, int64_t experts, int topk, int64_t d, int64_t f) {
  if (tokens <= 0 || experts < 1 || topk < 1 || topk > experts || d <= 0 || f < 1 ||
      !sizes_fit(tokens, experts, topk, d, f))
    return 0;
  return workspace(tokens, experts, topk, d, f).total;
}

extern "C" gptq_status gptq_mx_moe(const uint32_t* gate_up, int64_t ld_gate_up, int64_t stride_gate_up,
                                   const uint8_t* gate_up_scales, int64_t ld_gate_up_scales,
                                   int64_t stride_gate_up_scales, const uint32_t* down, int64_t ld_down,
                                   int64_t stride_down, const uint8_t* down_scales, int64_t ld_down_scales,
                                   int64_t stride_down_scales, int64_t experts, int64_t d, int64_t f, const void* X,
                                   int x_dtype, int64_t tokens, int64_t ldx, const void* logits, int l_dtype,
                                   int64_t ld_logits, int topk, int renormalize, void* Y, int y_dtype, int64_t ldy,
                                   void* ws, size_t ws_bytes, void* stream) {
  MoeArgs p{};
  p.gate_up = Weights{gate_up, gate_up_scales, ld_gate_up, ld_gate_up_scales, stride_gate_up, stride_gate_up_scales};
  p.down = Weights{down, down_scales, ld_down, ld_down_scales, stride_down, stride_down_scales};
  p.X = X, p.ldx = ldx, p.logits = logits, p.l_dtype = l_dtype, p.ld_logits = ld_logits;
  p.renormalize = renormalize != 0, p.Y = Y, p.y_dtype = y_dtype, p.ldy = ldy;
  return layer<kMxWeights>(p, experts, d, f, x_dtype, tokens, topk, ws, ws_bytes, stream);
}

extern "C" gptq_status gptq_block_moe(const uint8_t* gate_up, int64_t ld_gate_up, int64_t stride_gate_up,
                                      const float* gate_up_scales, int64_t ld_gate_up_scales,
                                      int64_t stride_gate_up_scales, const uint8_t* down, int64_t ld_down,
                                      int64_t stride_down, const float* down_scales, int64_t ld_down_scales,
                                      int64_t stride_down_scales, int64_t experts, int64_t d, int64_t f, const void* X,
                                      int x_dtype, int64_t tokens, int64_t ldx, const void* logits, int l_dtype,
                                      int64_t ld_logits, int topk, int renormalize, void* Y, int y_dtype, int64_t ldy,
                                      void* ws, size_t ws_bytes, void* stream) {
  MoeArgs p{};
  p.gate_up = Weights{gate_up, gate_up_scales, ld_gate_up, ld_gate_up_scales, stride_gate_up, stride_gate_up_scales};
  p.down = Weights{down, down_scales, ld_down, ld_down_scales, stride_down, stride_down_scales};
  p.X = X, p.ldx = ldx, p.logits = logits, p.l_dtype = l_dtype, p.ld_logits = ld_logits;
  p.renormalize = renormalize != 0, p.Y = Y, p.y_dtype = y_dtype, p.ldy = ldy;
  return layer<kBlockWeights>(p, experts, d, f, x_dtype, tokens, topk, ws, ws_bytes, stream);
}
