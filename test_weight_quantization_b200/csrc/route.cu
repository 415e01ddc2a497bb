// route.cu — the router of a mixture-of-experts layer: logits, scores and
// each token's top_k experts (ttq_moe_route).
//
// One launch. A cluster of CTAs takes 8, 16 or 32 tokens; its CTAs split K, a
// CTA's warps split the experts (and K further, where there are few experts).
// The products are mma.sync m16n8k16 with 16 experts as M and 8 tokens as N,
// every value loaded once from global memory into its fragment (a lane takes 8
// consecutive k; mma16.cuh has the types). A part of K is at most 1024 long
// where the cluster allows (K <= 8192): its sum is fp32, the parts are added
// in fp64 through distributed shared memory, so that near neighbours are told
// apart to about 1e-7 of the logits' size.
// Then a warp takes a token: scores in fp64, and top_k rounds that find the
// largest 64-bit key by three warp reductions (high word, low word, lowest
// expert). Measured: 5.8 us for one token (64 experts, K 2048, bf16), 24 us for
// 1000 (128 experts, K 4096, fp32 W; graph replay). Bound by launch and reduction latency for few tokens; for many, by
// reading W from L2, and splitting an fp32 W into terms, once per tile of
// tokens: 32 where 16 would not fit the SMs in one go (1000 tokens, 128
// experts, K 4096, fp32 W: see the launch).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "mma16.cuh"

namespace ttq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t a, uint32_t rank) {
  float v;
  asm volatile(
      "{\n\t.reg .u32 r;\n\t"
      "mapa.shared::cluster.u32 r, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [r];\n\t}"
      : "=f"(v)
      : "r"(a), "r"(rank)
      : "memory");
  return v;
}

struct Pick {
  const float* bias;
  int E, top_k, score, renormalize;
  float scaling;
  int32_t* ids;
  float* weights;
};

// Order-preserving key of a value: 0 is kept for a taken expert, 1 for NaN.
__device__ __forceinline__ unsigned long long key_of(double v) {
  if (isnan(v)) return 1;
  const long long b = __double_as_longlong(v + 0.0);  // -0 becomes +0
  return b < 0 ? ~(unsigned long long)b
               : (unsigned long long)b | 0x8000000000000000ull;
}

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ double warp_add(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Token t's choice by one warp; lane l holds the logits of experts l + 32 i.
template <int NE>
__device__ __forceinline__ void choose(const Pick& a, int64_t t,
                                       double (&p)[NE], int lane) {
  unsigned long long key[NE];
  const bool softmax = a.score == TTQ_SCORE_SOFTMAX;
  if (softmax) {
    double mx = -INFINITY, total = 0;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (lane + 32 * i < a.E) {
        mx = fmax(mx, p[i]);
        nan |= isnan(p[i]);
        if (!a.bias) key[i] = key_of(p[i]);
      }
    mx = warp_max(mx);
    if (__any_sync(0xffffffffu, nan)) mx = NAN;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (lane + 32 * i < a.E) {
        p[i] = exp(p[i] - mx);
        total += p[i];
      }
    total = warp_add(total);
#pragma unroll
    for (int i = 0; i < NE; ++i) p[i] /= total;
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i) p[i] = 1.0 / (1.0 + exp(-p[i]));
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 32 * i;
    if (e >= a.E)
      key[i] = 0;
    else if (a.bias || !softmax)
      key[i] = key_of(a.bias ? p[i] + (double)a.bias[e] : p[i]);
  }
  double sum = 0, mine = 0;  // lane i keeps the score of choice i
  int mine_e = 0;
  for (int r = 0; r < a.top_k; ++r) {
    unsigned long long best = key[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) best = key[i] > best ? key[i] : best;
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
    const uint32_t lo = __reduce_max_sync(
        0xffffffffu, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
    const unsigned long long top = (unsigned long long)hi << 32 | lo;
    uint32_t e = 0xFFFFFFFFu;
#pragma unroll
    for (int i = NE - 1; i >= 0; --i)
      if (key[i] == top && lane + 32 * i < a.E) e = lane + 32 * i;
    e = __reduce_min_sync(0xffffffffu, e);
    double s = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if ((uint32_t)(lane + 32 * i) == e) {
        key[i] = 0;
        s = p[i];
      }
    s = __shfl_sync(0xffffffffu, s, e & 31);
    sum += s;
    if (lane == r) {
      mine = s;
      mine_e = (int)e;
    }
  }
  if (lane < a.top_k) {
    if (a.renormalize) mine = sum == 0 ? 0 : mine / sum;
    a.ids[t * a.top_k + lane] = mine_e;
    a.weights[t * a.top_k + lane] = (float)(mine * (double)a.scaling);
  }
}

// MT: tiles of 16 experts per warp, NT: tiles of 8 tokens. Warps: ew over the
// experts times kWarps / ew over the CTA's part of K.
template <typename TX, typename TW, int MT, int NT>
__global__ void __launch_bounds__(kThreads)
    route_kernel(const TX* __restrict__ X, int T, int K, int64_t ldx,
                 const TW* __restrict__ W, int64_t ldw, int ew, Pick a) {
  using namespace mma16;
  extern __shared__ float part[];  // [K part][token][E]
  constexpr int TT = NT * 8;
  constexpr int XT = mma16::kTerms<TX, TW>, WT = mma16::kTerms<TW, TX>;
  constexpr bool HALF = kHalf<TX, TW>;
  griddep_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.y, ranks = gridDim.y;
  const int we = warp % ew, wk = warp / ew, kp = kWarps / ew;
  const int parts = ranks * kp, pt = rank * kp + wk;
  const int blocks = (K + 31) / 32;
  const int b0 = (int)((int64_t)blocks * pt / parts);
  const int b1 = (int)((int64_t)blocks * (pt + 1) / parts);
  const int64_t t0 = (int64_t)blockIdx.x * TT;
  const TX* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int64_t tok = t0 + n * 8 + g;
    xr[n] = X + (tok < T ? tok : t0) * ldx;
  }
  float acc[MT][NT][4] = {};
  constexpr int UN = MT * 2 + NT <= 6 && sizeof(TX) + sizeof(TW) <= 4 ? 4 : 2;
  for (int bb = b0; bb < b1; bb += UN) {
    Raw<TW, 8> rw[UN][MT][2];
    Raw<TX, 8> rx[UN][NT];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int k = (bb + u) * 32 + 8 * t;
      const bool ok = bb + u < b1 && k < K;
#pragma unroll
      for (int n = 0; n < NT; ++n) load<TX, 8>(xr[n] + k, ok, rx[u][n]);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int e = (we + m * ew) * 16 + h * 8 + g;
          load<TW, 8>(W + (int64_t)e * ldw + k, ok && e < a.E, rw[u][m][h]);
        }
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      uint32_t xt[NT][XT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) terms<TX, TW, 8>(rx[u][n], xt[n]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t wt[2][WT][4];
        terms<TW, TX, 8>(rw[u][m][0], wt[0]);
        terms<TW, TX, 8>(rw[u][m][1], wt[1]);
        // the tensor core cuts its sums instead of rounding them: a block is
        // summed apart and added rounded
        float sum[NT][4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = WT - 1; i >= 0; --i)
#pragma unroll
              for (int j = XT - 1; j >= 0; --j)
                if (i + j <= 2)
                  mma<HALF>(sum[n], wt[0][i][2 * h], wt[1][i][2 * h],
                            wt[0][i][2 * h + 1], wt[1][i][2 * h + 1],
                            xt[n][j][2 * h], xt[n][j][2 * h + 1]);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] += sum[n][i];
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = (we + m * ew) * 16 + g + 8 * (i >> 1);
        const int tok = n * 8 + 2 * t + (i & 1);
        if (e < a.E) part[(wk * TT + tok) * a.E + e] = acc[m][n][i];
      }
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
  const uint32_t at = smem_u32(part);
  // tokens over the cluster's warps
  for (int tok = warp * ranks + rank; tok < TT && t0 + tok < T;
       tok += kWarps * ranks) {
    auto logit = [&](int e) -> double {
      double v = 0;
      for (int k = 0; k < kp; ++k) {
        const int i = (k * TT + tok) * a.E + e;
        if (ranks > 1) {
          for (int r = 0; r < ranks; ++r) v += ld_cluster_f32(at + i * 4, r);
        } else {
          v += part[i];
        }
      }
      return v;
    };
    auto go = [&](auto ne) {
      constexpr int NE = decltype(ne)::value;
      double p[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i)
        p[i] = lane + 32 * i < a.E ? logit(lane + 32 * i) : 0.0;
      choose<NE>(a, t0 + tok, p, lane);
    };
    if (a.E <= 64)
      go(std::integral_constant<int, 2>{});
    else if (a.E <= 128)
      go(std::integral_constant<int, 4>{});
    else if (a.E <= 256)
      go(std::integral_constant<int, 8>{});
    else
      go(std::integral_constant<int, 16>{});
  }
  if (ranks > 1) cluster_sync();  // the parts stay until all have read them
}

template <typename TX, typename TW>
ttq_status go(const void* X, int64_t T, int64_t K, int64_t ldx, const void* W,
              int64_t ldw, const Pick& p, cudaStream_t st) {
  const int et = (p.E + 15) / 16;
  int ew = kWarps;
  while (ew > et) ew /= 2;
  const int mt = (et + ew - 1) / ew;  // at most 4
  // (four CTAs per tile is what K = 4096 takes)
  const int nt = T <= 8 ? 1 : T <= (int64_t)4 * sm_count() ? 2 : 4;
  const int tiles = (int)((T + nt * 8 - 1) / (nt * 8));
  LaunchShape ls;
  // CTAs per tile: enough to fill the SMs, and parts of K of at most 1024
  const int fill = std::min(8, sm_count() / tiles);
  const int exact = (int)std::min<int64_t>(8, (K + 1023) / 1024);
  const int ranks = std::max(1, std::max(fill, exact));
  ls.grid = dim3((unsigned)tiles, (unsigned)ranks);
  ls.block = dim3(kThreads);
  ls.cluster_y = (unsigned)ranks;
  ls.smem = (size_t)(kWarps / ew) * nt * 8 * p.E * sizeof(float);
  auto run = [&](auto m, auto n) -> ttq_status {
    auto kern = route_kernel<TX, TW, decltype(m)::value, decltype(n)::value>;
    if (ls.smem > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)ls.smem) != cudaSuccess)
      return TTQ_ERR_CUDA;
    return launch(ls, st, kern, static_cast<const TX*>(X), (int)T, (int)K, ldx,
                  static_cast<const TW*>(W), ldw, ew, p);
  };
  auto run_m = [&](auto m) -> ttq_status {
    if (nt == 1) return run(m, std::integral_constant<int, 1>{});
    if (nt == 2) return run(m, std::integral_constant<int, 2>{});
    return run(m, std::integral_constant<int, 4>{});
  };
  if (mt == 1) return run_m(std::integral_constant<int, 1>{});
  if (mt == 2) return run_m(std::integral_constant<int, 2>{});
  return run_m(std::integral_constant<int, 4>{});
}

template <typename TX>
ttq_status go_w(ttq_dtype wt, const void* X, int64_t T, int64_t K, int64_t ldx,
                const void* W, int64_t ldw, const Pick& p, cudaStream_t st) {
  switch (wt) {
    case TTQ_F32: return go<TX, float>(X, T, K, ldx, W, ldw, p, st);
    case TTQ_BF16: return go<TX, __nv_bfloat16>(X, T, K, ldx, W, ldw, p, st);
    case TTQ_F16: return go<TX, __half>(X, T, K, ldx, W, ldw, p, st);
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
  Pick p;
  p.bias = bias;
  p.E = (int)E;
  p.top_k = top_k;
  p.score = score;
  p.renormalize = renormalize;
  p.scaling = scaling;
  p.ids = ids;
  p.weights = weights;
  switch (xt) {
    case TTQ_F32: return go_w<float>(wt, X, T, K, ldx, W, ldw, p, st);
    case TTQ_BF16:
      return go_w<__nv_bfloat16>(wt, X, T, K, ldx, W, ldw, p, st);
    case TTQ_F16: return go_w<__half>(wt, X, T, K, ldx, W, ldw, p, st);
  }
  return TTQ_ERR_INVALID_ARG;
}

}  // namespace ttq
