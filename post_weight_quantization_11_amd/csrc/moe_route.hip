// The expert router: each token's k largest logits, their softmax probabilities,
// and the token-expert pairs sorted by expert, as the products grouped by expert
// read them.
//
// Choosing: one wave a token holds the logits in registers (one for every 64
// experts) and takes the maximum k times.  Sorting: one workgroup an expert reads
// all pairs' experts, 4 bytes each, counts those of lower experts (its first
// place) and places its own in their order: nothing but the pairs themselves is
// kept between the launches, and no order depends on timing.  Few tokens take one
// workgroup for all of it: a launch less.
#include "moe.h"
#include "mx.h"

namespace gptq {
namespace {

struct RouteArgs {
  const void* logits;
  int dtype;
  int64_t ld;
  int tokens, experts, k, renormalize;
  int32_t* ids;                              // tokens x k
  float* weights;
  int32_t* offsets;                          // experts + 1
  int32_t* order;                            // tokens * k
};

__device__ inline void put(const RouteArgs& p, int t, const Routed& r) {
  const int lane = (int)threadIdx.x & 63;
  const float w = route_weight(r, p.k, p.renormalize);
  if (lane < p.k) {
    p.ids[(int64_t)t * p.k + lane] = r.id;
    p.weights[(int64_t)t * p.k + lane] = w;
  }
}

__global__ __launch_bounds__(256) void moe_choose_kernel(RouteArgs p) {
  const int t = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
  route_tokens(p.logits, p.dtype, p.ld, t, min(t + 1, p.tokens), 1, p.experts, p.k, [&](int) { return !p.renormalize; },
               [&](int token, const Routed& r) { put(p, token, r); });
}

// Sixteen waves, each with every sixteenth part of the pairs, 1024 at a time: four
// loads in flight, four neighbouring pairs a lane and load.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64, kSortLoads = 4, kSortStep = 256 * kSortLoads;
__global__ __launch_bounds__(kSortThreads) void moe_sort_kernel(RouteArgs p) {
  __shared__ int below[kSortWaves], equal[kSortWaves];
  const int e = (int)blockIdx.x, lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int pairs = p.tokens * p.k;
  const int per = ((pairs + kSortWaves - 1) / kSortWaves + kSortStep - 1) / kSortStep * kSortStep;
  const int lo = min(wave * per, pairs), hi = min(lo + per, pairs);
  u32x4 v[kSortLoads];
  auto load = [&](int b) {
#pragma unroll
    for (int j = 0; j < kSortLoads; ++j) {
      const int at = b + 256 * j + 4 * lane;
      if (b + kSortStep <= hi) {             // the same for all lanes
        v[j] = *reinterpret_cast<const u32x4_a4*>(p.ids + at);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = at + i < hi ? (uint32_t)p.ids[at + i] : 0x7FFFFFFFu;
      }
    }
  };
  int less = 0, same = 0;
  for (int b = lo; b < hi; b += kSortStep) {
    load(b);
#pragma unroll
    for (int j = 0; j < kSortLoads; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        less += (int)v[j][i] < e;
        same += (int)v[j][i] == e;
      }
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    less += __shfl_xor(less, x, 64);
    same += __shfl_xor(same, x, 64);
  }
  if (lane == 0) {
    below[wave] = less;
    equal[wave] = same;
  }
  __syncthreads();
  int first = 0, mine = 0, all = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    first += below[w];
    if (w < wave) mine += equal[w];
    all += equal[w];
  }
  if (threadIdx.x == 0) {
    p.offsets[e] = first;
    if (e == p.experts - 1) p.offsets[p.experts] = first + all;
  }
  if (equal[wave] == 0) return;
  int at = first + mine;
  const uint64_t before = ((uint64_t)1 << lane) - 1;
  for (int b = lo; b < hi; b += kSortStep) {
    load(b);
#pragma unroll
    for (int j = 0; j < kSortLoads; ++j) {
      int mark = at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t hit = __ballot((int)v[j][i] == e);
        mark += __popcll(hit & before);
        at += __popcll(hit);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((int)v[j][i] == e) p.order[mark++] = b + 256 * j + 4 * lane + i;
    }
  }
}

// Both for few tokens: an expert's tokens are the bits of a 64-bit
// number in LDS, whichever wave sets them, and its places a prefix sum, a thread an
// expert.
constexpr int kSmallTokens = 64;
static_assert(kSortThreads >= kMoeMaxExperts && kSortThreads >= kSmallTokens * kMoeMaxTopk);
__global__ __launch_bounds__(kSortThreads) void moe_route_kernel(RouteArgs p) {
  __shared__ int ids[kSmallTokens * kMoeMaxTopk], first[kMoeMaxExperts], sums[kSortWaves];
  __shared__ unsigned long long masks[kMoeMaxExperts];
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  masks[tid] = 0u;
  __syncthreads();
  route_tokens(p.logits, p.dtype, p.ld, wave, p.tokens, kSortWaves, p.experts, p.k, [&](int) { return !p.renormalize; },
               [&](int t, const Routed& r) {
                 put(p, t, r);
                 if (lane < p.k) {
                   ids[t * p.k + lane] = r.id;
                   atomicOr(masks + r.id, 1ull << t);
                 }
               });
  __syncthreads();
  const int own = __popcll(masks[tid]);
  int upto = own;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const int v = __shfl_up(upto, x, 64);
    if (lane >= x) upto += v;
  }
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  for (int w = 0; w < wave; ++w) upto += sums[w];
  first[tid] = upto - own;
  if (tid < p.experts) p.offsets[tid + 1] = upto;
  if (tid == 0) p.offsets[0] = 0;
  __syncthreads();
  if (tid < p.tokens * p.k) {
    const int e = ids[tid], t = tid / p.k;
    p.order[first[e] + __popcll(masks[e] & ((1ull << t) - 1))] = tid;
  }
}

}  // namespace

gptq_status moe_choose(const void* logits, int dtype, int64_t ld, int tokens, int experts, int k, bool renormalize,
                       int32_t* ids, float* weights, hipStream_t stream) {
  const RouteArgs p{logits, dtype, ld, tokens, experts, k, renormalize, ids, weights, nullptr, nullptr};
  moe_choose_kernel<<<(unsigned)ceil_div(tokens, 4), 256, 0, stream>>>(p);
  GPTQ_TRY_LAUNCH();
  return GPTQ_OK;
}

}  // namespace gptq

using namespace gptq;

extern "C" gptq_status gptq_moe_route(const void* logits, int l_dtype, int64_t tokens, int64_t experts,
                                      int64_t ld_logits, int topk, int renormalize, int32_t* ids, float* weights,
                                      int32_t* offsets, int32_t* order, void* stream) {
  if (tokens < 0 || experts < 1 || !valid_dtype(l_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (topk < 1 || topk > experts) return GPTQ_ERR_INVALID_ARG;
  if (experts > kMoeMaxExperts || topk > kMoeMaxTopk || tokens > GPTQ_MX_MAX_ROWS) return GPTQ_ERR_UNSUPPORTED;
  if (ld_logits < experts || (tokens > 0 && (offsets == nullptr) != (order == nullptr))) return GPTQ_ERR_INVALID_ARG;
  if (ld_logits > ((int64_t)1 << 40)) return GPTQ_ERR_UNSUPPORTED;
  if (tokens > 0 && (logits == nullptr || ids == nullptr || weights == nullptr)) return GPTQ_ERR_INVALID_ARG;
  if (tokens == 0 && offsets == nullptr) return GPTQ_OK;
  const RouteArgs p{logits, l_dtype, ld_logits, (int)tokens, (int)experts, topk, renormalize != 0,
                    ids, weights, offsets, order};
  hipStream_t st = static_cast<hipStream_t>(stream);
  // One workgroup up to a token a wave, or few experts (us, one against two launches: 32
  // x 64 6.7 / 7.6, 64 x 8 7.1 / 7.1; 64 x 64 9.8 / 7.8, 32 x 256 11.2 / 8.8).
  if (offsets != nullptr && (tokens <= kSortWaves || (tokens <= kSmallTokens && tokens * experts <= 2048))) {
    moe_route_kernel<<<1, kSortThreads, 0, st>>>(p);
    GPTQ_TRY_LAUNCH();
    return GPTQ_OK;
  }
  const gptq_status rc = moe_choose(logits, l_dtype, ld_logits, (int)tokens, (int)experts, topk, renormalize != 0, ids,
                                    weights, st);
  if (rc != GPTQ_OK) return rc;
  if (offsets != nullptr) {
    moe_sort_kernel<<<(unsigned)experts, kSortThreads, 0, st>>>(p);
    GPTQ_TRY_LAUNCH();
  }
  return GPTQ_OK;
}
