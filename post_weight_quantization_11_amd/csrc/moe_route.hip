// The expert router: each token's k largest logits, their softmax probabilities,
// and the token-expert pairs sorted by expert, as the products grouped by expert
// read them.
//
// Choosing: one wave a token holds the logits in registers (one for every 64
// experts) and takes the maximum k times.  Sorting: one workgroup an expert reads
// all pairs' experts, 4 bytes each, counts those of lower experts (its first
// place) and places its own in their order: nothing but the pairs themselves is
// kept between the launches, and no order depends on timing.  Up to 64 tokens
// take one workgroup for all of it: a launch less.
#include "moe.h"

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

__device__ inline int choose(const RouteArgs& p, int t) {
  const int lane = (int)threadIdx.x & 63;
  const Routed r = route_token(p.logits, p.dtype, (int64_t)t * p.ld, p.experts, p.k, !p.renormalize);
  const float w = route_weight(r, p.k, p.renormalize);
  if (lane < p.k) {
    p.ids[(int64_t)t * p.k + lane] = r.id;
    p.weights[(int64_t)t * p.k + lane] = w;
  }
  return r.id;
}

__global__ __launch_bounds__(256) void moe_choose_kernel(RouteArgs p) {
  const int t = (int)(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (t < p.tokens) choose(p, t);
}

// Sixteen waves, each with every sixteenth part of the pairs, 256 at a time (four
// neighbouring ones a lane).
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
__global__ __launch_bounds__(kSortThreads) void moe_sort_kernel(RouteArgs p) {
  __shared__ int below[kSortWaves], equal[kSortWaves];
  const int e = (int)blockIdx.x, lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int pairs = p.tokens * p.k;
  const int per = ((pairs + kSortWaves - 1) / kSortWaves + 255) / 256 * 256;
  const int lo = min(wave * per, pairs), hi = min(lo + per, pairs);
  auto load4 = [&](int at, int (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = at + i < hi ? p.ids[at + i] : 0x7FFFFFFF;
  };
  int less = 0, same = 0;
  for (int b = lo; b < hi; b += 256) {
    int v[4];
    load4(b + 4 * lane, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      less += v[i] < e;
      same += v[i] == e;
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
  int at = first + mine;
  const uint64_t before = ((uint64_t)1 << lane) - 1;
  for (int b = lo; b < hi; b += 256) {
    int v[4], mark = at;
    load4(b + 4 * lane, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t hit = __ballot(v[i] == e);
      mark += __popcll(hit & before);
      at += __popcll(hit);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (v[i] == e) p.order[mark++] = b + 4 * lane + i;
  }
}

// Both for at most kSmallTokens tokens.
constexpr int kSmallTokens = 64;
__global__ __launch_bounds__(kSortThreads) void moe_route_kernel(RouteArgs p) {
  __shared__ int ids[kSmallTokens * kMoeMaxTopk];
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  for (int t = wave; t < p.tokens; t += kSortWaves) {
    const int id = choose(p, t);
    if (lane < p.k) ids[t * p.k + lane] = id;
  }
  __syncthreads();
  const int pairs = p.tokens * p.k;
  const uint64_t before = ((uint64_t)1 << lane) - 1;
  for (int e = wave; e < p.experts; e += kSortWaves) {
    int at = 0, same = 0;
    for (int b = 0; b < pairs; b += 64) {
      const int v = b + lane < pairs ? ids[b + lane] : 0x7FFFFFFF;
      at += __popcll(__ballot(v < e));
      same += __popcll(__ballot(v == e));
    }
    if (lane == 0) {
      p.offsets[e] = at;
      if (e == p.experts - 1) p.offsets[p.experts] = at + same;
    }
    for (int b = 0; same > 0 && b < pairs; b += 64) {
      const uint64_t hit = __ballot(b + lane < pairs && ids[b + lane] == e);
      if (hit >> lane & 1) p.order[at + __popcll(hit & before)] = b + lane;
      at += __popcll(hit);
    }
  }
}

}  // namespace
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
  if (offsets != nullptr && tokens <= kSmallTokens) {
    moe_route_kernel<<<1, kSortThreads, 0, st>>>(p);
    GPTQ_TRY_LAUNCH();
    return GPTQ_OK;
  }
  moe_choose_kernel<<<(unsigned)ceil_div(tokens, 4), 256, 0, st>>>(p);
  GPTQ_TRY_LAUNCH();
  if (offsets != nullptr) {
    moe_sort_kernel<<<(unsigned)experts, kSortThreads, 0, st>>>(p);
    GPTQ_TRY_LAUNCH();
  }
  return GPTQ_OK;
}
