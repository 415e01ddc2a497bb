// route.cu — the router of a mixture-of-experts layer: logits, scores and
// each token's top_k experts (ttq_moe_route).
//
// One CTA per token: warps take the experts in turn (a lane sums every 32nd
// product in fp32, the lanes' sums are added in fp64), one thread picks.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace ttq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxExperts = 512;

template <typename TX, typename TW>
__global__ void __launch_bounds__(kThreads)
    route_kernel(const TX* __restrict__ X, int64_t K, int64_t ldx,
                 const TW* __restrict__ W, int E, int64_t ldw,
                 const float* __restrict__ bias, int top_k, int score,
                 int renormalize, float scaling, int32_t* __restrict__ ids,
                 float* __restrict__ weights) {
  __shared__ double logit[kMaxExperts], rank[kMaxExperts];
  griddep_enter();
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = warp; e < E; e += kThreads / 32) {
    float acc = 0.f;
    for (int64_t j = lane; j < K; j += 32)
      acc = fmaf(to_f32(X[t * ldx + j]), to_f32(W[e * ldw + j]), acc);
    double sum = acc;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) logit[e] = sum;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  if (score == TTQ_SCORE_SOFTMAX) {
    double mx = -INFINITY, total = 0;
    for (int e = 0; e < E; ++e) mx = fmax(mx, logit[e]);
    for (int e = 0; e < E; ++e) total += exp(logit[e] - mx);
    for (int e = 0; e < E; ++e) {
      const double p = exp(logit[e] - mx) / total;
      rank[e] = bias ? p + (double)bias[e] : logit[e];
      logit[e] = p;
    }
  } else {
    for (int e = 0; e < E; ++e) {
      const double p = 1.0 / (1.0 + exp(-logit[e]));
      rank[e] = bias ? p + (double)bias[e] : p;
      logit[e] = p;
    }
  }
  double sum = 0;
  for (int i = 0; i < top_k; ++i) {
    int best = -1;  // NaN ranks below every number, a taken expert is -2
    for (int e = 0; e < E; ++e) {
      bool taken = false;
      for (int q = 0; q < i; ++q) taken |= ids[t * top_k + q] == e;
      if (taken) continue;
      if (best < 0 || rank[e] > rank[best] ||
          (isnan(rank[best]) && !isnan(rank[e])))
        best = e;
    }
    ids[t * top_k + i] = best;
    sum += logit[best];
  }
  for (int i = 0; i < top_k; ++i) {
    double w = logit[ids[t * top_k + i]];
    if (renormalize) w = sum == 0 ? 0 : w / sum;
    weights[t * top_k + i] = (float)(w * (double)scaling);
  }
}

template <typename TX, typename TW>
ttq_status go(const void* X, int64_t T, int64_t K, int64_t ldx, const void* W,
              int E, int64_t ldw, const float* bias, int top_k, int score,
              int renormalize, float scaling, int32_t* ids, float* weights,
              cudaStream_t st) {
  LaunchShape ls;
  ls.grid = dim3((unsigned)T);
  ls.block = dim3(kThreads);
  return launch(ls, st, route_kernel<TX, TW>, static_cast<const TX*>(X), K,
                ldx, static_cast<const TW*>(W), E, ldw, bias, top_k, score,
                renormalize, scaling, ids, weights);
}

template <typename TX>
ttq_status go_w(ttq_dtype wt, const void* X, int64_t T, int64_t K, int64_t ldx,
                const void* W, int E, int64_t ldw, const float* bias,
                int top_k, int score, int renormalize, float scaling,
                int32_t* ids, float* weights, cudaStream_t st) {
  switch (wt) {
    case TTQ_F32:
      return go<TX, float>(X, T, K, ldx, W, E, ldw, bias, top_k, score,
                           renormalize, scaling, ids, weights, st);
    case TTQ_BF16:
      return go<TX, __nv_bfloat16>(X, T, K, ldx, W, E, ldw, bias, top_k,
                                   score, renormalize, scaling, ids, weights,
                                   st);
    case TTQ_F16:
      return go<TX, __half>(X, T, K, ldx, W, E, ldw, bias, top_k, score,
                            renormalize, scaling, ids, weights, st);
  }
  return TTQ_ERR_INVALID_ARG;
}

}  // namespace

ttq_status launch_moe_route(const void* X, ttq_dtype xt, int64_t T, int64_t K,
                            int64_t ldx, const void* W, ttq_dtype wt,
                            int64_t E, int64_t ldw, const float* bias,
                            int top_k, int score, int renormalize,
                            float scaling, int32_t* ids, float* weights,
                            cudaStream_t st) {
  switch (xt) {
    case TTQ_F32:
      return go_w<float>(wt, X, T, K, ldx, W, (int)E, ldw, bias, top_k, score,
                         renormalize, scaling, ids, weights, st);
    case TTQ_BF16:
      return go_w<__nv_bfloat16>(wt, X, T, K, ldx, W, (int)E, ldw, bias,
                                 top_k, score, renormalize, scaling, ids,
                                 weights, st);
    case TTQ_F16:
      return go_w<__half>(wt, X, T, K, ldx, W, (int)E, ldw, bias, top_k,
                          score, renormalize, scaling, ids, weights, st);
  }
  return TTQ_ERR_INVALID_ARG;
}

}  // namespace ttq
