// Device helpers of the expert router: the k largest of a token's logits and their
// softmax probabilities, one wave a token.
#pragma once

#include "common.h"

namespace gptq {

constexpr int kMoeMaxExperts = GPTQ_MOE_MAX_EXPERTS, kMoeMaxTopk = GPTQ_MOE_MAX_TOPK;

// Logits as unsigned numbers in the same order; both zeros are one number, and a
// NaN counts as -inf.  Experts that do not exist have 0, below every logit.
constexpr uint32_t kRouteLowest = 0x007FFFFFu;              // -inf
__device__ inline uint32_t route_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.f);
  if (l != l) return kRouteLowest;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ inline float route_logit(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// The largest of the 64 lanes' numbers, in every lane: four steps inside rows of
// sixteen lanes, two across them.
__device__ inline uint32_t wave_max(uint32_t x) {
#define GPTQ_MAX_STEP(ctrl) \
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, ctrl, 0xF, 0xF, false))
  GPTQ_MAX_STEP(0x111);                      // row_shr 1, 2, 4, 8
  GPTQ_MAX_STEP(0x112);
  GPTQ_MAX_STEP(0x114);
  GPTQ_MAX_STEP(0x118);
  GPTQ_MAX_STEP(0x142);                      // row_bcast 15, 31
  GPTQ_MAX_STEP(0x143);
#undef GPTQ_MAX_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// What one wave knows of its token: lane i < k has the i-th expert in descending
// order of logits, ties to the lowest index, and its logit's key.
struct Routed {
  int id;
  uint32_t key;
  uint32_t top;                              // the largest key
  float sum;                                 // of exp(logit - largest) over all experts, where asked for
};

// exp(l - m) for logits l <= m; 1 where they are equal, also if infinite.
__device__ inline float route_exp(float l, float m) { return l == m ? 1.f : expf(l - m); }

// A token's keys, expert 64 j + lane in register j.
template <int L> struct RouteKeys {
  uint32_t keys[L];
};
// F32: of float32 logits.  (Chosen at run time, every load stood behind a branch of
// its own, and the compiler waited for each before the next.)
template <int L, bool F32>
__device__ inline void route_load(RouteKeys<L>& o, const void* logits, int64_t row, int experts) {
  const int lane = (int)threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < L; ++j) {
    const int64_t at = row + min(64 * j + lane, experts - 1);
    if constexpr (F32) o.keys[j] = static_cast<const uint32_t*>(logits)[at];
    else o.keys[j] = static_cast<const uint16_t*>(logits)[at];
  }
}

template <int L, bool F32>
__device__ inline Routed route_choose(RouteKeys<L> o, int dtype, int experts, int k, bool want_sum) {
  const int lane = (int)threadIdx.x & 63;
  uint32_t (&keys)[L] = o.keys;
#pragma unroll
  for (int j = 0; j < L; ++j) {
    const float l = F32                 ? __uint_as_float(keys[j])
                    : dtype == GPTQ_F16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)keys[j])
                                        : __uint_as_float(keys[j] << 16);
    keys[j] = 64 * j + lane < experts ? route_key(l) : 0u;
  }
  Routed r{0, 0u, 0u, 0.f};
  for (int i = 0; i < k; ++i) {
    uint32_t best = keys[0];
#pragma unroll
    for (int j = 1; j < L; ++j) best = max(best, keys[j]);
    best = wave_max(best);
    if (i == 0) {
      r.top = best;
      if (want_sum) {
        const float m = route_logit(best);
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < L; ++j) s += keys[j] != 0u ? route_exp(route_logit(keys[j]), m) : 0.f;
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) s += __shfl_xor(s, x, 64);
        r.sum = s;
      }
    }
    // The lowest index: the first register of 64 that has one, its first lane.
    int id = -1;
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const uint64_t hit = __ballot(keys[j] == best);
      const int l = hit != 0 && id < 0 ? __builtin_ctzll(hit) : 64;
      id = l < 64 ? 64 * j + l : id;
      keys[j] = lane == l ? 0u : keys[j];
    }
    r.id = lane == i ? id : r.id;
    r.key = lane == i ? best : r.key;
  }
  return r;
}

// Tokens t, t + step, ... below `tokens`, one after the other; the next one's logits
// are on their way meanwhile.  done(t, Routed); want_sum(t): whether it is to have the
// sum over all experts.
template <int L, bool F32, typename Want, typename Done>
__device__ inline void route_some(const void* logits, int dtype, int64_t ld, int t, int tokens, int step, int experts,
                                  int k, Want want_sum, Done done) {
  if (t >= tokens) return;
  RouteKeys<L> next;
  route_load<L, F32>(next, logits, (int64_t)t * ld, experts);
  for (; t < tokens; t += step) {
    const RouteKeys<L> now = next;
    route_load<L, F32>(next, logits, (int64_t)min(t + step, tokens - 1) * ld, experts);
    done(t, route_choose<L, F32>(now, dtype, experts, k, want_sum(t)));
  }
}
template <bool F32, typename Want, typename Done>
__device__ inline void route_typed(const void* logits, int dtype, int64_t ld, int t, int tokens, int step, int experts,
                                   int k, Want want_sum, Done done) {
  if (experts <= 64) route_some<1, F32>(logits, dtype, ld, t, tokens, step, experts, k, want_sum, done);
  else if (experts <= 256) route_some<4, F32>(logits, dtype, ld, t, tokens, step, experts, k, want_sum, done);
  else route_some<kMoeMaxExperts / 64, F32>(logits, dtype, ld, t, tokens, step, experts, k, want_sum, done);
}
template <typename Want, typename Done>
__device__ inline void route_tokens(const void* logits, int dtype, int64_t ld, int t, int tokens, int step, int experts,
                                    int k, Want want_sum, Done done) {
  if (dtype == GPTQ_F32) route_typed<true>(logits, dtype, ld, t, tokens, step, experts, k, want_sum, done);
  else route_typed<false>(logits, dtype, ld, t, tokens, step, experts, k, want_sum, done);
}

// Lane i's probability of the i-th expert.  A token whose logits are all -inf (or
// NaN) has none.
__device__ inline float route_weight(const Routed& r, int k, bool renormalize) {
  const int lane = (int)threadIdx.x & 63;
  if (r.top <= kRouteLowest) return 0.f;
  float w = lane < k ? route_exp(route_logit(r.key), route_logit(r.top)) : 0.f, sum = r.sum;
  if (renormalize) {
    sum = w;                                 // k <= 16: the first row of lanes
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor(sum, x, 64);
  }
  return w / sum;
}

// Launches the choice alone: ids and weights of tokens >= 1.
gptq_status moe_choose(const void* logits, int dtype, int64_t ld, int tokens, int experts, int k, bool renormalize,
                       int32_t* ids, float* weights, hipStream_t stream);

}  // namespace gptq
