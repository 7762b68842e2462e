// A whole layer of experts for few tokens, in two launches:
//   y_t = sum over t's experts e of p_te D_e (silu(G_e x_t) * (U_e x_t))
// with the experts and probabilities of the router, and G, U (rows of one stack)
// and D microscaled or in block-scaled 8-bit floats.
//
// Slots: an expert with tokens has one for every fifteen of them, and both launches
// read its weights once a slot.
//
// First launch (moe_up_kernel): every workgroup routes all tokens itself (a wave a
// token, the experts' tokens as 64-bit masks in LDS; more than sixteen tokens are
// routed by a launch before) and takes its share of the list of (slot, 16 rows of G
// with the same 16 of U); its eight waves split the columns, or are several teams with
// a tile each.  h = silu(g) * u goes to the workspace as three bfloat16 numbers that
// add up to its float32 value (8 bits each), so that the second launch's products,
// exact in float32, lose none of it.
//
// Second launch (moe_down_kernel): a workgroup takes 32 rows of D for all slots; the
// waves of the row group's `splits` workgroups share the list of (slot, 128 or 256
// columns).  A matrix instruction's sixteen columns are five tokens' three parts of h.
// Sums times p go to the wave's own sums of its tokens in LDS, joined in wave order
// and, by the workgroup that comes last, in split order.  The first launch clears the
// counters that tell the last.
//
// Bounds: the weights' bytes, and the accesses of the CU's cache, of which a load
// whose neighbouring lanes read different rows takes four times as many.  So a wave
// holds X from tile to tile, h lies in the order of its loads, and weights are loaded
// along their rows and exchanged between lanes.  Small layers are bound by latency:
// routing, one load after it, and the joins (5 us of the first launch, 6 to 9 of the
// second).  Measured: 1 token, 2 of 8 experts 4096 x 11008 in 4 bits 25 + 18 us (144 MB,
// 3.4 TB/s); 16 tokens, 6 of 64 experts 2048 x 1024 in 8 bits 43 + 25 us (320 MB, 4.7
// TB/s); 61 tokens, 4 of 33 experts 1030 x 2043 in 4 bits 5 + 39 + 26 us (111 MB, 1.6
// TB/s: five units of 256 columns leave some of eight waves without work).
#include "fp8.h"
#include "moe.h"
#include "mx_operands.h"
#include "product.h"

#include <type_traits>

namespace gptq {
namespace {

constexpr int kMxWeights = 0, kBlockWeights = 1;             // formats of the weights
constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kSlot = 15;                    // tokens of a slot: three parts
constexpr int kPlanes = 3;                   // bfloat16 numbers of an h
constexpr int kPart = 5;                     // tokens whose three parts are columns of one instruction
constexpr int kPadCols = 256;                // rows of h are whole units of either format
constexpr int kDownTiles = 2, kDownRows = 16 * kDownTiles;

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
  float* weights;                            // of the pairs: tokens x k
  int32_t* ids;                              // and their experts, where a launch before chose them
  bool chosen;
  int* slots;                                // their number, then the word of each
  uint32_t* slot_pairs;                      // [slot][kSlot]: pair, token in the upper half
  uint32_t* arrived;                         // a counter for each group of rows of D
  uint16_t* h;                               // [part of a slot][8 columns][token][plane][8], see h_at
  float* part;                               // [split][token][d]
  void* Y;
  int64_t ldy;
  int y_dtype;
};

// A slot's word: its expert, its tokens and how many pairs the slots before it have.
__device__ inline int slot_word(int expert, int tokens, int first) { return expert | tokens << 16 | first << 20; }
__device__ inline int slot_expert(int word) { return word & 0xFFFF; }
__device__ inline int slot_tokens(int word) { return word >> 16 & 15; }
__device__ inline int slot_first(int word) { return word >> 20; }
static_assert(kSlot < 16 && GPTQ_MOE_MAX_TOKENS * kMoeMaxTopk <= 2048);

// Slots there can be.
__host__ __device__ inline int max_slots(int tokens, int experts, int k) {
  return (experts < tokens * k ? experts : tokens * k) + tokens * k / kSlot;
}

// What a lane holds of a unit of a row of weights: 128 bytes of codes, a whole line
// of the caches, in two neighbouring loads (units of 64 bytes, half a line at a time,
// reached three quarters of the rate).
template <int WF> struct Row;
template <> struct Row<kMxWeights> {
  static constexpr int kCols = 256, kSteps = 8;
  u32x4 w[2];
  u32x2 s;
};
template <> struct Row<kBlockWeights> {
  static constexpr int kCols = 128, kSteps = 4;
  u32x4 w[2];
  float s;
};

// Lane quarter q's share of unit u of the row whose codes and scales start at `codes
// + at`, `scales + s_at` (bytes).  CLAMP: of n >= kCols columns, no multiple of a unit;
// loads end at the row's end, and the last unit's are put right by fix_row.
template <bool CLAMP>
__device__ inline void load_row(Row<kMxWeights>& o, const char* codes, uint32_t at, const char* scales, uint32_t s_at,
                                int u, int q, int n) {
  const uint32_t last = 4u * ((uint32_t)(n + 7) >> 3) - 16u, s_last = ((uint32_t)(n + 31) >> 5) - 8u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t b = 128u * u + 64u * h + 16u * q;
    o.w[h] = *reinterpret_cast<const u32x4_a4*>(codes + (at + (CLAMP ? min(b, last) : b)));
  }
  o.s = *reinterpret_cast<const u32x2_a1*>(scales + (s_at + (CLAMP ? min(8u * u, s_last) : 8u * u)));
}
template <bool CLAMP>
__device__ inline void load_row(Row<kBlockWeights>& o, const char* codes, uint32_t at, const char* scales,
                                uint32_t s_at, int u, int q, int n) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t b = 128u * u + 64u * h + 16u * q;
    o.w[h] = *reinterpret_cast<const u32x4_a1*>(codes + (at + (CLAMP ? min(b, (uint32_t)n - 16u) : b)));
  }
  o.s = *reinterpret_cast<const float*>(scales + (s_at + 4u * u));
}
// v moved `bytes` bytes down, zeros from above (bytes <= 0: v itself).
__device__ inline u32x4 shift_down(u32x4 v, int bytes) {
  const int n = max(bytes, 0), words = n >> 2;
  u32x4 o = v;
  if (words & 1) o = u32x4{o[1], o[2], o[3], 0u};
  if (words & 2) o = u32x4{o[2], o[3], 0u, 0u};
  if (words > 3) o = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __builtin_amdgcn_alignbyte(i < 3 ? o[i + 1] : 0u, o[i], n & 3);
  return o;
}
// The last unit's share after load_row<true>.  A word's codes past column n stay, for
// zeros of the other operand; scales past it are 1.
__device__ inline void fix_row(Row<kMxWeights>& o, int u, int q, int n) {
  const int from = 4 * ((n + 7) >> 3) - 16, s = 8 * (8 * u - (((n + 31) >> 5) - 8));
#pragma unroll
  for (int h = 0; h < 2; ++h) o.w[h] = shift_down(o.w[h], 128 * u + 64 * h + 16 * q - from);
  uint64_t b = (uint64_t)o.s[1] << 32 | o.s[0];
  b = b >> s | (s > 0 ? 0x0101010101010101ull * kMxScaleOne << (64 - s) : 0u);
  o.s = u32x2{(uint32_t)b, (uint32_t)(b >> 32)};
}
__device__ inline void fix_row(Row<kBlockWeights>& o, int u, int q, int n) {
#pragma unroll
  for (int h = 0; h < 2; ++h) o.w[h] = shift_down(o.w[h], 128 * u + 64 * h + 16 * q - (n - 16));
}
// The same of unit 0 of n < kCols columns.
__device__ inline void load_row_tail(Row<kMxWeights>& o, const char* codes, uint32_t at, const char* scales,
                                     uint32_t s_at, int u, int q, int n) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    o.w[h] = load_w4_tail(reinterpret_cast<const uint32_t*>(codes + at), 32 * u + 16 * h + 4 * q, n);
    o.s[h] = load_scales4(reinterpret_cast<const uint8_t*>(scales + s_at), 8 * u + 4 * h, n);
  }
}
__device__ inline void load_row_tail(Row<kBlockWeights>& o, const char* codes, uint32_t at, const char* scales,
                                     uint32_t s_at, int u, int q, int n) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    o.w[h] = fp8_load16_tail(reinterpret_cast<const uint8_t*>(codes + at), 128 * u + 64 * h + 16 * q, n);
  o.s = *reinterpret_cast<const float*>(scales + (s_at + 4u * u));
}

// Step s alone of unit 0 of n < kCols columns: eight weights as 16-bit numbers (0 past
// column n), and their scale where it is not in them.
template <int T>
__device__ inline u32x4 load_step(Row<kMxWeights>& o, const char* codes, uint32_t at, const char* scales, uint32_t s_at,
                                  int u, int s, int q, int n) {
  const int word = 32 * u + 4 * s + q, block = 8 * u + s, left = n - 8 * word;
  const uint32_t w = reinterpret_cast<const uint32_t*>(codes + at)[min(word, (n - 1) >> 3)];
  const uint32_t b = reinterpret_cast<const uint8_t*>(scales + s_at)[min(block, (n - 1) >> 5)];
  o.s[0] = left > 0 ? b : (uint32_t)kMxScaleOne;
  return widen8<T>(left >= 8 ? w : w & ((1u << (4 * max(left, 0))) - 1u), mx_scale_operand(o.s[0]));
}
template <int T>
__device__ inline u32x4 load_step(Row<kBlockWeights>& o, const char* codes, uint32_t at, const char* scales,
                                  uint32_t s_at, int u, int s, int q, int n) {
  const uint8_t* row = reinterpret_cast<const uint8_t*>(codes + at);
  const int k = 128 * u + 64 * (s >> 1) + 16 * q + 8 * (s & 1);
  uint64_t v = 0;
  if (n >= 8) {                              // one load that ends at the row's end, shifted down
    const int from = min(k, n - 8);
    const u32x2 w = *reinterpret_cast<const u32x2_a1*>(row + from);
    v = k - from < 8 ? ((uint64_t)w[1] << 32 | w[0]) >> (8 * (k - from)) : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v |= (uint64_t)(k + i < n ? row[min(k + i, n - 1)] : 0) << (8 * i);
  }
  o.s = *reinterpret_cast<const float*>(scales + (s_at + 4u * u));
  const int lo = (int)v, hi = (int)(v >> 32);
  return T == GPTQ_BF16
             ? u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true))}
             : u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true))};
}

// Where row r of a matrix has its codes and scales, in bytes from the matrix's.
template <int WF> __device__ inline uint32_t codes_at(const Weights& w, int r) {
  return (uint32_t)r * (uint32_t)w.ld * (WF == kMxWeights ? 4u : 1u);
}
template <int WF> __device__ inline uint32_t scales_at(const Weights& w, int r) {
  return WF == kMxWeights ? (uint32_t)r * (uint32_t)w.lds : (uint32_t)(r >> 7) * (uint32_t)w.lds * 4u;
}
template <int WF> __device__ inline const char* matrix_codes(const Weights& w, int e) {
  return static_cast<const char*>(w.codes) + e * w.stride * (WF == kMxWeights ? 4 : 1);
}
template <int WF> __device__ inline const char* matrix_scales(const Weights& w, int e) {
  return static_cast<const char*>(w.scales) + e * w.s_stride * (WF == kMxWeights ? 1 : 4);
}

// The column, inside a unit, of the eight that lane quarter q holds in step s.
template <int WF> __device__ inline int step_col(int s, int q) {
  return WF == kMxWeights ? 32 * s + 8 * q : 64 * (s >> 1) + 16 * q + 8 * (s & 1);
}

// Codes in the order of the steps.
__device__ inline void arrange(Row<kMxWeights>& o) {
#pragma unroll
  for (int h = 0; h < 2; ++h) o.w[h] = transpose_quarters(o.w[h]);
}
__device__ inline void arrange(Row<kBlockWeights>&) {}

// Eight weights of step s as 16-bit numbers.
template <int T> __device__ inline u32x4 widen(const Row<kMxWeights>& o, int s) {
  return widen8<T>(o.w[s >> 2][s & 3], mx_scale_operand((o.s[s >> 2] >> (8 * (s & 3))) & 255u));
}
template <int T> __device__ inline u32x4 widen(const Row<kBlockWeights>& o, int s) {
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

// h lies as the second launch's lanes read it: a part's columns of eight, in the
// order of the steps, and of each its tokens' three numbers, 16 bytes of each: a
// load's neighbouring lanes read neighbouring bytes.  (A row a token, they read rows
// far apart, 64 accesses of the cache a load: second launch of 61 tokens, 33 experts
// 1030 x 2043 37 us for 27.)
// The place of column r's eight in that order, and the first number of a part.
template <int WF> __device__ inline int h_chunk(int r) {
  return WF == kMxWeights ? r >> 3 : (r >> 7) * 16 + (r >> 6 & 1) * 8 + (r >> 3 & 1) * 4 + (r >> 4 & 3);
}
__device__ inline uint32_t h_at(int word, int part, int f_pad) {
  return (uint32_t)((slot_first(word) + kPart * part) * kPlanes) * (uint32_t)f_pad;
}
// A part's columns: its tokens' numbers.
__device__ inline int h_columns(int word, int part) { return kPlanes * min(slot_tokens(word) - kPart * part, kPart); }

// acc += f * v, v being a unit's sums (block-scaled weights).
__device__ inline void add_scaled(floatx4& acc, float f, floatx4 v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = __builtin_fmaf(f, v[j], acc[j]);
}

// ---------------------------------------------------------------------------
// Gate and up.
// ---------------------------------------------------------------------------
constexpr size_t kRedBytes = 2 * kWaves * 2 * 64 * sizeof(floatx4);        // sums of two rounds of tiles
// What a workgroup knows of the routes, in LDS.
struct Routes {
  uint64_t* masks;                           // tokens of each expert
  int* first;                                // first slot of each expert
  int* slot_words;
  uint32_t* slot_pairs;                      // as in the workspace
};
constexpr size_t routes_lds(int tokens, int experts, int k) {
  const int pairs = tokens * k, slots = (experts < pairs ? experts : pairs) + pairs / kSlot;
  return (size_t)experts * 12 + (size_t)slots * 4 * (1 + kSlot) + (size_t)pairs * 4;
}

// Routes all tokens; returns the number of slots.  Workgroup 0 writes what the
// second launch needs.
__device__ inline int route_all(const MoeArgs& p, unsigned char* lds, Routes& o) {
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool first = blockIdx.x == 0;
  // The tokens' probabilities fall to the workgroups in turn.
  const auto weighs = [](int t) { return t % gridDim.x == blockIdx.x; };
  const int pairs = p.tokens * p.k, most = max_slots(p.tokens, p.experts, p.k);
  __shared__ int count;
  o.masks = reinterpret_cast<uint64_t*>(lds);
  o.first = reinterpret_cast<int*>(o.masks + p.experts);
  o.slot_words = o.first + p.experts;
  o.slot_pairs = reinterpret_cast<uint32_t*>(o.slot_words + most);
  int* ids = reinterpret_cast<int*>(o.slot_pairs + most * kSlot);
  for (int e = tid; e < p.experts; e += kThreads) o.masks[e] = 0u;
  __syncthreads();
  if (p.chosen) {
    for (int i = tid; i < pairs; i += kThreads) {
      ids[i] = p.ids[i];
      atomicOr(reinterpret_cast<unsigned long long*>(o.masks + ids[i]), 1ull << (i / p.k));
    }
  } else {
    route_tokens(p.logits, p.l_dtype, p.ld_logits, wave, p.tokens, kWaves, p.experts, p.k,
                 [&](int t) { return weighs(t) && !p.renormalize; },
                 [&](int t, const Routed& r) {
                   if (lane < p.k) {
                     ids[t * p.k + lane] = r.id;
                     atomicOr(reinterpret_cast<unsigned long long*>(o.masks + r.id), 1ull << t);
                   }
                   if (weighs(t)) {
                     const float w = route_weight(r, p.k, p.renormalize);
                     if (lane < p.k) p.weights[t * p.k + lane] = w;
                   }
                 });
  }
  __syncthreads();
  if (wave == 0) {
    int before = 0, pairs_before = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
      const int n = e0 + lane < p.experts ? __popcll(o.masks[e0 + lane]) : 0;
      const int own = (n + kSlot - 1) / kSlot;
      int upto = own | n << 16;              // both sums in one number
#pragma unroll
      for (int x = 1; x < 64; x <<= 1) {
        const int v = __shfl_up(upto, x, 64);
        if (lane >= x) upto += v;
      }
      const int at = before + (upto & 0xFFFF) - own, first_pair = pairs_before + (upto >> 16) - n;
      if (own > 0) o.first[e0 + lane] = at;
      for (int i = 0; i < own; ++i)
        o.slot_words[at + i] = slot_word(e0 + lane, min(n - i * kSlot, kSlot), first_pair + i * kSlot);
      upto = __shfl(upto, 63, 64);
      before += upto & 0xFFFF;
      pairs_before += upto >> 16;
    }
    if (lane == 0) count = before;
  }
  __syncthreads();
  for (int i = tid; i < pairs; i += kThreads) {
    const int e = ids[i], t = i / p.k;
    const int at = __popcll(o.masks[e] & (((uint64_t)1 << t) - 1));
    o.slot_pairs[o.first[e] * kSlot + at] = (uint32_t)(i | t << 16);
  }
  __syncthreads();
  if (first) {
    for (int i = tid; i < count; i += kThreads) p.slots[1 + i] = o.slot_words[i];
    for (int i = tid; i < count * kSlot; i += kThreads) p.slot_pairs[i] = o.slot_pairs[i];
    if (tid == 0) p.slots[0] = count;
    for (int i = tid; i < (p.d + kDownRows - 1) / kDownRows; i += kThreads) p.arrived[i] = 0u;
  }
  return __builtin_amdgcn_readfirstlane(count);
}

// Units of X that a wave holds: 4096 columns of a workgroup's eight.
template <int WF> constexpr int kHeld = WF == kMxWeights ? 2 : 4;

// Tiles [lo, hi) of the list: tile n has slot n / tiles, rows 16 (n % tiles) ...
// SPLIT (float16 X, microscaled weights that float16 does not hold): X as the sum of
// two bfloat16 numbers.  Otherwise the result says whether there are such weights.
template <int WF, int XT, bool TAIL, bool SPLIT>
__device__ inline bool up_tiles(const MoeArgs& p, const Routes& routes, int lo, int hi, floatx4* red, u32x4* swap) {
  constexpr int D = kHeld<WF>, kCols = Row<WF>::kCols, kSteps = Row<WF>::kSteps;
  if (lo >= hi) return false;                // there are more workgroups than tiles: no tile to clamp loads to
  const int tid = (int)threadIdx.x, lane = tid & 63, q = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Teams of waves take a tile each; a team's waves share its units or, where there is
  // no whole one, its steps.  A wave of D units at most holds its columns of the slot's
  // X while it goes from tile to tile, and there are as many teams as that allows.
  const int tiles = (p.f + 15) / 16, whole = p.d / kCols, units = TAIL && whole > 0 ? whole + 1 : whole;
  const int members = units > 4 * D || units == 0 ? 8 : units > 2 * D ? 4 : units > D ? 2 : 1, teams = kWaves / members;
  const int team = wave / members, member = wave - team * members;
  const bool held = units <= 8 * D;
  const int u0 = units * member / members, count = units * (member + 1) / members - u0;
  const int steps = (count + D - 1) / D * D;                  // so that a tile starts in the ring's first place
  struct Unit {
    Row<WF> w[2];                            // of G and of U
    u32x4 x[kSteps];
  };
  Unit ring[D];
  floatx4 acc[2];
  uint32_t inexact = 0u;
  // Whether a tile's X is not the one before's.
  auto fresh = [&](int tile, int& slot) {
    const int s = tile / tiles;
    const bool f = !held || s != slot;
    slot = s;
    return f;
  };

  // Where a tile's operands are.
  struct Place {
    const char *codes[2], *scales[2];
    uint32_t w_at[2], s_at[2], x_at;
    int f0;
  };
  auto place = [&](int tile, Place& o) {
    const int slot = tile / tiles, f0 = (tile - slot * tiles) * 16, word = routes.slot_words[slot];
    o.f0 = f0;
    o.x_at = (routes.slot_pairs[slot * kSlot + min(c16, slot_tokens(word) - 1)] >> 16) * (uint32_t)p.ldx *
             2u;
    const int e = __builtin_amdgcn_readfirstlane(slot_expert(word));
    const char *c = matrix_codes<WF>(p.gate_up, e), *s = matrix_scales<WF>(p.gate_up, e);
    const int r = min(c16, p.f - 1 - f0), r_load = min(lane >> 2, p.f - 1 - f0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row0 = f0 + i * p.f, block0 = WF == kMxWeights ? row0 : row0 & ~127;
      o.codes[i] = c + row0 * p.gate_up.ld * (WF == kMxWeights ? 4 : 1);
      o.scales[i] = s + (WF == kMxWeights ? row0 * p.gate_up.lds : (int64_t)(row0 >> 7) * p.gate_up.lds * 4);
      o.w_at[i] = codes_at<WF>(p.gate_up, r_load);
      o.s_at[i] = scales_at<WF>(p.gate_up, row0 - block0 + r);
    }
  };
  // Of the loads.  The loop has no branch around those of the weights, or the compiler
  // would wait for all that are in flight where the branches meet: padded steps load
  // one place of a unit, and past the last tile that tile is loaded again.
  int at_tile = lo + team, at_step = 0, at_slot = -1;
  bool at_fresh = false;
  Place at;
  const char* x = static_cast<const char*>(p.X);
  auto load = [&](Unit& o) {
    if (at_step == 0) {
      const int tile = min(at_tile, hi - 1);
      at_fresh = fresh(tile, at_slot);
      place(tile, at);
    }
    const int u = u0 + min(at_step, count - 1);
    if (at_fresh) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int c = kCols * u + step_col<WF>(s, q);
        o.x[s] = *reinterpret_cast<const u32x4_a2*>(x + (at.x_at + 2u * (TAIL ? min(c, p.d - 8) : c)));
      }
    }
    const bool pad = at_step >= count;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      load_row<TAIL>(o.w[i], at.codes[i], pad ? 0u : at.w_at[i], at.scales[i], pad ? 0u : at.s_at[i], u,
                     pad ? 0 : lane & 3, p.d);
    if (++at_step == steps) {
      at_step = 0;
      at_tile += teams;
    }
  };
  auto multiply = [&](Unit& o, int u, bool fresh_x) {
    if (TAIL && u == whole) {
#pragma unroll
      for (int i = 0; i < 2; ++i) fix_row(o.w[i], u, lane & 3, p.d);
      if (fresh_x) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
          o.x[s] = shift_down(o.x[s], 2 * (kCols * u + step_col<WF>(s, q) - (p.d - 8)));
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) exchange(o.w[i].w, swap, lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      arrange(o.w[i]);
      floatx4 v = WF == kMxWeights ? acc[i] : floatx4{0.f, 0.f, 0.f, 0.f};
      if constexpr (WF == kMxWeights && XT == GPTQ_F16 && !SPLIT)
        inexact |= f16_inexact4(o.w[i].s[0]) | f16_inexact4(o.w[i].s[1]);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if constexpr (SPLIT) {
          u32x4 top, rest;
          split8(o.x[s], top, rest);
          const u32x4 wv = widen<GPTQ_BF16>(o.w[i], s);
          v = mfma16<GPTQ_BF16>(top, wv, v);
          v = mfma16<GPTQ_BF16>(rest, wv, v);
        } else {
          v = mfma16<XT>(o.x[s], widen<XT>(o.w[i], s), v);
        }
      }
      if constexpr (WF == kMxWeights) acc[i] = v;
      else add_scaled(acc[i], o.w[i].s, v);
    }
  };

  if (steps > 0) {
#pragma unroll
    for (int i = 0; i < D; ++i) load(ring[i]);
  }
  for (int n0 = lo, round = 0, slot_now = -1; n0 < hi; n0 += teams, ++round) {
    const bool fresh_x = fresh(min(n0 + team, hi - 1), slot_now);
    acc[0] = acc[1] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < steps; s += D) {
#pragma unroll
      for (int i = 0; i < D; ++i) {
        if (s + i < count) multiply(ring[i], u0 + s + i, fresh_x);
        load(ring[i]);
      }
    }
    for (int step = member; TAIL && whole == 0 && step < kSteps && step_col<WF>(step, 0) < p.d; step += members) {
      Place here;
      place(min(n0 + team, hi - 1), here);
#pragma unroll
      for (int i = 0; i < 2; ++i) here.w_at[i] = codes_at<WF>(p.gate_up, min(c16, p.f - 1 - here.f0));
      const u32x4 xv = load_x8_tail(reinterpret_cast<const uint16_t*>(x + here.x_at),
                                    step_col<WF>(step, q), p.d);
      constexpr int T = SPLIT ? GPTQ_BF16 : XT;
      u32x4 top = xv, rest;
      if constexpr (SPLIT) split8(xv, top, rest);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        Row<WF> o;
        const u32x4 wv =
            load_step<T>(o, here.codes[i], here.w_at[i], here.scales[i], here.s_at[i], 0, step, q, p.d);
        floatx4 v = mfma16<T>(top, wv, WF == kMxWeights ? acc[i] : floatx4{0.f, 0.f, 0.f, 0.f});
        if constexpr (SPLIT) v = mfma16<T>(rest, wv, v);
        if constexpr (WF == kMxWeights && XT == GPTQ_F16 && !SPLIT) inexact |= o.s[0] - kF16Lo < kF16Span ? 0u : 1u;
        if constexpr (WF == kMxWeights) acc[i] = v;
        else add_scaled(acc[i], o.s, v);
      }
    }
    // Two buffers: a round's sums are added while the next round's come in.
    floatx4* to = red + (round & 1) * kWaves * 2 * 64;
    to[(wave * 2) * 64 + lane] = acc[0];
    to[(wave * 2 + 1) * 64 + lane] = acc[1];
    __syncthreads();
    for (int i = tid; i < 256 * teams; i += kThreads) {
      const int n = n0 + (i >> 8), col = (i >> 4) & 15;
      if (n >= hi) break;
      const int slot = n / tiles, r = (n - slot * tiles) * 16 + (i & 15);
      const int word = routes.slot_words[slot];
      if (col >= slot_tokens(word)) continue;
      // Register j of lane l: token 4 (l / 16) + j, row l % 16.
      const float* s = reinterpret_cast<const float*>(to + (i >> 8) * members * 128) +
                       ((col >> 2) * 16 + (i & 15)) * 4 + (col & 3);
      float g = s[0], u = s[256];
      for (int w = 1; w < members; ++w) {
        g += s[w * 512];
        u += s[w * 512 + 256];
      }
      float h = r < p.f ? g / (1.f + expf(-g)) * u : 0.f;
      const int part = col / kPart, columns = h_columns(word, part);
      uint16_t* o = p.h + h_at(word, part, p.f_pad) + 8 * kPlanes * (col - kPart * part);
      uint16_t* to_h = o + 8 * h_chunk<WF>(r) * columns + (r & 7);
#pragma unroll
      for (int j = 0; j < kPlanes; ++j) {
        const uint32_t top = __float_as_uint(h) & 0xFFFF0000u;                 // 8 bits, the rest exact
        to_h[8 * j] = (uint16_t)(top >> 16);
        h = (top & 0x7F800000u) != 0x7F800000u ? h - __uint_as_float(top) : 0.f;
      }
      // Behind the last tile zeros, as the second launch reads whole units.
      if (n - slot * tiles == tiles - 1)
        for (int c = r + 16; c < p.f_pad; c += 16)
#pragma unroll
          for (int j = 0; j < kPlanes; ++j) o[8 * (h_chunk<WF>(c) * columns + j) + (c & 7)] = 0;
    }
  }
  return inexact != 0u;
}

// TAIL: d is no multiple of a unit.  Without it two workgroups fit a CU.
template <int WF, int XT, bool TAIL>
__global__ __launch_bounds__(kThreads, 2) void moe_up_kernel(MoeArgs p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  floatx4* red = reinterpret_cast<floatx4*>(smem);            // [2][wave][gate, up][64]
  u32x4* swap = reinterpret_cast<u32x4*>(smem + kRedBytes + (threadIdx.x >> 6) * kExchange);
  Routes routes;
  const int slots = route_all(p, smem + kRedBytes + kWaves * kExchange, routes);
  const int64_t all = (int64_t)slots * ((p.f + 15) / 16);
  const int lo = (int)(all * blockIdx.x / gridDim.x), hi = (int)(all * (blockIdx.x + 1) / gridDim.x);
  const bool inexact = up_tiles<WF, XT, TAIL, false>(p, routes, lo, hi, red, swap);
  if constexpr (WF == kMxWeights && XT == GPTQ_F16) {
    if (__syncthreads_or(inexact)) up_tiles<WF, XT, TAIL, true>(p, routes, lo, hi, red, swap);
  }
}

// ---------------------------------------------------------------------------
// Down.
// ---------------------------------------------------------------------------
// TAIL: f is no multiple of a unit.
template <int WF, bool TAIL>
__global__ __launch_bounds__(kThreads, 2) void moe_down_kernel(MoeArgs p) {
  constexpr int kCols = Row<WF>::kCols, kSteps = Row<WF>::kSteps;
  constexpr int kParts = kSlot / kPart;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int pairs = p.tokens * p.k, most = max_slots(p.tokens, p.experts, p.k);
  u32x4* swap = reinterpret_cast<u32x4*>(smem + (threadIdx.x >> 6) * kExchange);
  float* sums = reinterpret_cast<float*>(smem + kWaves * kExchange);            // [wave][token][32 rows]
  float* weights = sums + kWaves * p.tokens * kDownRows;
  int* slot_words = reinterpret_cast<int*>(weights + pairs);
  uint32_t* slot_pairs = reinterpret_cast<uint32_t*>(slot_words + most);
  __shared__ int is_last;
  const int tid = (int)threadIdx.x, lane = tid & 63, q = lane >> 4, c16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int groups = (p.d + kDownRows - 1) / kDownRows;
  // The workgroups of an XCD share slots, so its L2 holds their h.
  const int item = (int)xcd_contiguous(blockIdx.x, gridDim.x);
  if (item >= groups * p.splits) return;
  const int group = item % groups, split = item / groups, r0 = group * kDownRows;

  // All that there can be, in one round trip; what lies behind the last slot is not used.
  const int slots = p.slots[0];
  for (int i = tid; i < pairs; i += kThreads) weights[i] = p.weights[i];
  for (int i = tid; i < most; i += kThreads) slot_words[i] = p.slots[1 + i];
  for (int i = tid; i < most * kSlot; i += kThreads) slot_pairs[i] = p.slot_pairs[i];
  for (int i = tid; i < kWaves * p.tokens * kDownRows; i += kThreads) sums[i] = 0.f;
  __syncthreads();

  const int whole = p.f / kCols, per_slot = TAIL && whole > 0 ? whole + 1 : whole;
  const int64_t total = (int64_t)slots * per_slot, shares = (int64_t)p.splits * kWaves, share = split * kWaves + wave;
  const int lo = (int)(total * share / shares), hi = (int)(total * (share + 1) / shares);
  float* mine = sums + wave * p.tokens * kDownRows;
  const int third = c16 / 3;                 // this lane's token of a part

  struct Unit {
    Row<WF> w[kDownTiles];
    u32x4 x[kParts][kSteps];                 // of the slot's parts
  };
  // A part's columns lie at `at` (bytes; lanes without a column repeat another's).
  struct Part {
    uint32_t at;
    int columns;
  };
  auto part_of = [&](int word, int i) {
    Part o;
    o.columns = __builtin_amdgcn_readfirstlane(max(h_columns(word, i), 1));
    o.at = 2u * h_at(word, i, p.f_pad) + 16u * (q * o.columns + min(c16, o.columns - 1));
    return o;
  };
  auto load_h = [&](const Part& o, int u, u32x4 (&x)[kSteps]) {
    const char* h = reinterpret_cast<const char*>(p.h);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      x[s] = *reinterpret_cast<const u32x4*>(h + (o.at + (uint32_t)(kSteps * u + s) * (uint32_t)o.columns * 64u));
  };
  uint32_t w_at[kDownTiles], s_at[kDownTiles];
#pragma unroll
  for (int i = 0; i < kDownTiles; ++i) {
    const int r = min(16 * i + c16, p.d - 1 - r0);
    w_at[i] = codes_at<WF>(p.down, min(16 * i + (lane >> 2), p.d - 1 - r0));
    s_at[i] = WF == kMxWeights ? scales_at<WF>(p.down, r) : 0u;               // 32 rows lie in one block
  }
  auto parts_of = [&](int slot) {
    return __builtin_amdgcn_readfirstlane((slot_tokens(slot_words[slot]) + kPart - 1) / kPart);
  };
  struct Place {
    const char *codes, *scales;
    Part part[kParts];
    int parts;
  };
  auto place = [&](int slot, Place& o) {
    const int word = __builtin_amdgcn_readfirstlane(slot_words[slot]), e = slot_expert(word);
    o.codes = matrix_codes<WF>(p.down, e) + r0 * p.down.ld * (WF == kMxWeights ? 4 : 1);
    o.scales = matrix_scales<WF>(p.down, e) +
               (WF == kMxWeights ? r0 * p.down.lds : (int64_t)(r0 >> 7) * p.down.lds * 4);
#pragma unroll
    for (int j = 0; j < kParts; ++j) o.part[j] = part_of(word, j);
    o.parts = parts_of(slot);
  };
  // Of the loads; past the last unit that unit is loaded again (no branch around the
  // weights' loads, as above).  The parts behind the first go first: one round trip a
  // unit however many parts, where a round trip for each took 44 us for 29.
  int at_slot = 0, at_unit = 0, left = 0;
  Place at;
  auto load = [&](Unit& o) {
#pragma unroll
    for (int j = kParts - 1; j > 0; --j)
      if (j < at.parts) load_h(at.part[j], at_unit, o.x[j]);
#pragma unroll
    for (int i = 0; i < kDownTiles; ++i)
      load_row<TAIL>(o.w[i], at.codes, w_at[i], at.scales, s_at[i], at_unit, lane & 3, p.f);
    load_h(at.part[0], at_unit, o.x[0]);
    if (--left > 0 && ++at_unit == per_slot) {
      at_unit = 0;
      place(++at_slot, at);
    }
  };
  floatx4 acc[kParts][kDownTiles];
  auto clear = [&] {
#pragma unroll
    for (int j = 0; j < kParts; ++j)
#pragma unroll
      for (int i = 0; i < kDownTiles; ++i) acc[j][i] = floatx4{0.f, 0.f, 0.f, 0.f};
  };
  // The weights are widened once for all parts.
  auto multiply_parts = [&](Unit& o, auto parts) {
    constexpr int P = decltype(parts)::value;
#pragma unroll
    for (int i = 0; i < kDownTiles; ++i) {
      floatx4 v[P];
#pragma unroll
      for (int j = 0; j < P; ++j) v[j] = WF == kMxWeights ? acc[j][i] : floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const u32x4 w = widen<GPTQ_BF16>(o.w[i], s);
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = mfma16<GPTQ_BF16>(w, o.x[j][s], v[j]);
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if constexpr (WF == kMxWeights) acc[j][i] = v[j];
        else add_scaled(acc[j][i], o.w[i].s, v[j]);
      }
    }
  };
  static_assert(kParts == 3);
  auto multiply = [&](Unit& o, int u, int parts) {
    if (TAIL && u == whole && whole > 0) {
#pragma unroll
      for (int i = 0; i < kDownTiles; ++i) fix_row(o.w[i], u, lane & 3, p.f);
    }
#pragma unroll
    for (int i = 0; i < kDownTiles; ++i) {
      exchange(o.w[i].w, swap, lane);
      arrange(o.w[i]);
    }
    if (parts == 1) multiply_parts(o, std::integral_constant<int, 1>());
    else if (parts == 2) multiply_parts(o, std::integral_constant<int, 2>());
    else multiply_parts(o, std::integral_constant<int, 3>());
  };
  // Register i of lane l: row 4 (l / 16) + i, column l % 16.  A token's three columns
  // are added; a weight of 0 leaves it without the expert's product, whatever that is.
  auto flush = [&](int slot, int parts) {
    const int n = slot_tokens(slot_words[slot]);
#pragma unroll
    for (int j = 0; j < kParts; ++j) {
      if (j >= parts) break;
      const int token = kPart * j + third;
      const uint32_t pair = slot_pairs[slot * kSlot + min(token, n - 1)];
      const float w = weights[pair & 0xFFFFu];
      const bool there = c16 < 3 * kPart && c16 == 3 * third && token < n && w != 0.f;
      float* to = mine + (pair >> 16) * kDownRows + 4 * q;
#pragma unroll
      for (int i = 0; i < kDownTiles; ++i) {
        floatx4 v = acc[j][i];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += __shfl_down(acc[j][i][r], 1, 64) + __shfl_down(acc[j][i][r], 2, 64);
        if (there) {
          floatx4 s = *reinterpret_cast<floatx4*>(to + 16 * i);
          add_scaled(s, w, v);
          *reinterpret_cast<floatx4*>(to + 16 * i) = s;
        }
      }
    }
  };
  if (lo < hi) {                             // no division by zero units
    int slot = lo / per_slot, u = lo - slot * per_slot, parts = parts_of(slot);
    at_slot = slot, at_unit = u, left = hi - lo;
    place(slot, at);
    Unit next;                               // a second one in flight gained nothing
    load(next);
    clear();
    for (int n = lo; n < hi; ++n) {
      multiply(next, u, parts);
      ++u;
      if (n + 1 == hi || u == per_slot) {
        flush(slot, parts);
        clear();
        u = 0;
        ++slot;
        if (n + 1 < hi) parts = parts_of(slot);
      }
      load(next);
    }
  }
  // Without a whole unit, a slot at a time.
  if (TAIL && whole == 0) {
    const int s0 = (int)(slots * share / shares), s1 = (int)(slots * (share + 1) / shares);
    for (int slot = s0; slot < s1; ++slot) {
      Unit o;
      place(slot, at);
#pragma unroll
      for (int i = 0; i < kDownTiles; ++i)
        load_row_tail(o.w[i], at.codes, w_at[i], at.scales, s_at[i], 0, lane & 3, p.f);
#pragma unroll
      for (int j = 0; j < kParts; ++j)
        if (j == 0 || j < at.parts) load_h(at.part[j], 0, o.x[j]);
      clear();
      multiply(o, 0, at.parts);
      flush(slot, at.parts);
    }
  }
  __syncthreads();
  const int outputs = p.tokens * kDownRows;
  for (int i = tid; i < outputs; i += kThreads) {
    const int t = i / kDownRows, r = r0 + i % kDownRows;
    float v = sums[i];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += sums[w * outputs + i];
    if (r >= p.d) continue;
    if (p.splits == 1) store_y(p, (int64_t)t * p.ldy + r, v);
    // Written through to where every workgroup of the device sees it.
    else __hip_atomic_store(p.part + ((int64_t)split * p.tokens + t) * p.d + r, v, __ATOMIC_RELAXED,
                            __HIP_MEMORY_SCOPE_AGENT);
  }
  if (p.splits == 1) return;
  // The last workgroup of the group adds the parts, in order.  The parts are stored
  // and loaded past the caches of one XCD, and every wave waits for its own stores
  // before its workgroup is counted, so whoever counts last finds all of them; an
  // acquire and release of everything else would write back and drop the whole L2 (6
  // to 9 us of 70 to 130).
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid == 0)
    is_last = __hip_atomic_fetch_add(p.arrived + group, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
              (uint32_t)p.splits - 1u;
  __syncthreads();
  if (!is_last) return;
  // Four outputs and four splits' loads in flight;
  // past the last of either it again, not added.
  constexpr int kOutputs = GPTQ_MOE_MAX_TOKENS * kDownRows / kThreads;
  static_assert(kOutputs == 4);
  if (tid >= outputs) return;
  int64_t from[kOutputs];
  float v[kOutputs];
#pragma unroll
  for (int j = 0; j < kOutputs; ++j) {
    const int i = min(tid + j * kThreads, outputs - 1);
    from[j] = (int64_t)(i / kDownRows) * p.d + min(r0 + i % kDownRows, p.d - 1);
    v[j] = 0.f;
  }
  for (int s = 0; s < p.splits; s += 4) {
    float x[kOutputs][4];
#pragma unroll
    for (int j = 0; j < kOutputs; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[j][i] = __hip_atomic_load(p.part + (int64_t)min(s + i, p.splits - 1) * p.tokens * p.d + from[j],
                                    __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int j = 0; j < kOutputs; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j] += s + i < p.splits ? x[j][i] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < kOutputs; ++j) {
    const int i = tid + j * kThreads, r = r0 + i % kDownRows;
    if (i < outputs && r < p.d) store_y(p, (int64_t)(i / kDownRows) * p.ldy + r, v[j]);
  }
}

// ---------------------------------------------------------------------------
// Host.
// ---------------------------------------------------------------------------
struct Workspace {
  size_t ids, slots, slot_pairs, arrived, h, part, total;          // offsets in bytes
};
constexpr int64_t kMaxSplits = 16;
// Up to here every workgroup of the first launch chooses the experts itself; of more
// tokens that costs it more than a launch before (us, first launch of 61 tokens, 33
// experts 1030 x 2043: 45, against 39 and 5 for the choice; 16 tokens of 64 experts 44,
// against 42 and 5).
constexpr int kRoutedTokens = 16;

int down_splits(int64_t tokens, int64_t experts, int64_t topk, int64_t d, int64_t f) {
  // A workgroup a CU, a unit of 128 columns a wave at least.
  const int64_t groups = ceil_div(d, kDownRows), units = std::min(experts, tokens * topk) * ceil_div(f, 128);
  return (int)std::max<int64_t>(1, std::min({kMaxSplits, 256 / groups, units / kWaves}));
}

Workspace workspace(int64_t tokens, int64_t experts, int64_t topk, int64_t d, int64_t f) {
  const size_t pairs = (size_t)(tokens * topk), f_pad = (size_t)round_up(f, kPadCols);
  const size_t slots = (size_t)max_slots((int)tokens, (int)experts, (int)topk);
  const int splits = down_splits(tokens, experts, topk, d, f);
  Workspace w;                               // the pairs' weights first
  w.ids = align256(pairs * 4);
  w.slots = w.ids + align256(pairs * 4);
  w.slot_pairs = w.slots + align256((slots + 1) * 4);
  w.arrived = w.slot_pairs + align256(slots * kSlot * 4);
  w.h = w.arrived + align256((size_t)ceil_div(d, kDownRows) * 4);
  w.part = w.h + align256(kPlanes * pairs * f_pad * 2);
  w.total = w.part + (splits > 1 ? align256((size_t)splits * (size_t)(tokens * d) * 4) : 0);
  return w;
}

bool sizes_fit(int64_t tokens, int64_t experts, int64_t topk, int64_t d, int64_t f) {
  return tokens <= GPTQ_MOE_MAX_TOKENS && experts <= kMoeMaxExperts && topk <= kMoeMaxTopk && d <= kMxMaxCols &&
         f <= kMxMaxCols / 2;
}

// Rows of a tile, and of X, are addressed with 32 bits.
constexpr int64_t kMaxLd = (int64_t)1 << 23;

// One stack of weights of `rows` x `cols`: words (bytes) and scales to a row, rows of
// scales.
gptq_status check_weights(const Weights& w, int64_t experts, int64_t rows, int64_t words, int64_t scale_rows,
                          int64_t scales) {
  if (w.codes == nullptr || w.scales == nullptr || w.ld < words || w.lds < scales) return GPTQ_ERR_INVALID_ARG;
  if (w.ld > kMaxLd || w.lds > kMaxLd) return GPTQ_ERR_UNSUPPORTED;
  if (experts == 1) return GPTQ_OK;
  if (w.stride < rows * w.ld || w.s_stride < scale_rows * w.lds) return GPTQ_ERR_INVALID_ARG;
  return w.stride > (kMaxLd << 22) || w.s_stride > (kMaxLd << 22) ? GPTQ_ERR_UNSUPPORTED : GPTQ_OK;
}

template <int WF>
gptq_status layer(MoeArgs p, int64_t experts, int64_t d, int64_t f, int x_dtype, int64_t tokens, int topk, void* ws,
                  size_t ws_bytes, void* stream) {
  if (tokens < 0 || experts < 1 || d < 0 || f < 1 || topk < 1 || topk > experts) return GPTQ_ERR_INVALID_ARG;
  if ((x_dtype != GPTQ_F16 && x_dtype != GPTQ_BF16) || !valid_dtype(p.l_dtype) || !valid_dtype(p.y_dtype))
    return GPTQ_ERR_INVALID_ARG;
  if (!sizes_fit(tokens, experts, topk, d, f)) return GPTQ_ERR_UNSUPPORTED;
  if (p.ldx < d || p.ldy < d || p.ld_logits < experts) return GPTQ_ERR_INVALID_ARG;
  if (p.ldx > kMaxLd || p.ldy > (kMaxLd << 17) || p.ld_logits > (kMaxLd << 17)) return GPTQ_ERR_UNSUPPORTED;
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
  p.weights = reinterpret_cast<float*>(base);
  p.ids = reinterpret_cast<int32_t*>(base + w.ids);
  p.slots = reinterpret_cast<int*>(base + w.slots);
  p.slot_pairs = reinterpret_cast<uint32_t*>(base + w.slot_pairs);
  p.arrived = reinterpret_cast<uint32_t*>(base + w.arrived);
  p.h = reinterpret_cast<uint16_t*>(base + w.h);
  p.part = reinterpret_cast<float*>(base + w.part);
  p.tokens = (int)tokens;
  p.experts = (int)experts;
  p.k = topk;
  p.d = (int)d;
  p.f = (int)f;
  p.f_pad = (int)round_up(f, kPadCols);
  p.splits = down_splits(tokens, experts, topk, d, f);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t pairs = tokens * topk, slots = max_slots(p.tokens, p.experts, topk);

  p.chosen = tokens > kRoutedTokens;
  if (p.chosen) {
    rc = moe_choose(p.logits, p.l_dtype, p.ld_logits, p.tokens, p.experts, topk, p.renormalize != 0, p.ids, p.weights,
                    st);
    if (rc != GPTQ_OK) return rc;
  }
  const bool tail = d % Row<WF>::kCols != 0;
  const int up_lds = (int)(kRedBytes + kWaves * kExchange + routes_lds(p.tokens, p.experts, topk));
  const unsigned up_grid = (unsigned)std::min<int64_t>(slots * ceil_div(f, 16), 256);
  const bool f16 = x_dtype == GPTQ_F16;
  const auto up = tail ? (f16 ? moe_up_kernel<WF, GPTQ_F16, true> : moe_up_kernel<WF, GPTQ_BF16, true>)
                       : (f16 ? moe_up_kernel<WF, GPTQ_F16, false> : moe_up_kernel<WF, GPTQ_BF16, false>);
  if (up_lds > 65536)
    GPTQ_TRY_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(up), hipFuncAttributeMaxDynamicSharedMemorySize,
                                     up_lds));
  up<<<up_grid, kThreads, up_lds, st>>>(p);
  GPTQ_TRY_LAUNCH();

  const int down_lds = (int)(kWaves * (kExchange + tokens * kDownRows * 4) + pairs * 4 + slots * 4 * (1 + kSlot));
  const auto k = f % Row<WF>::kCols != 0 ? moe_down_kernel<WF, true> : moe_down_kernel<WF, false>;
  if (down_lds > 65536)
    GPTQ_TRY_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize,
                                     down_lds));
  k<<<(unsigned)round_up(ceil_div(d, kDownRows) * p.splits, kXcds), kThreads, down_lds, st>>>(p);
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
