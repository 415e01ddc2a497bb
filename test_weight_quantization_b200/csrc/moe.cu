// moe.cu — a mixture-of-experts layer on packed low-bit experts for a few
// tokens (ttq_moe_lowbit).
//
// Two kernels: a warp per (token, choice, intermediate channel) makes
// h = act(gate) * up * inv_s_mid in fp32, then a warp per (token, output
// channel) sums its experts' D h in the order of the token's choices.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace ttq {
namespace {

constexpr int kThreads = 256;

// (q - z) D of channel j of a packed row.
__device__ __forceinline__ float weight_at(const uint32_t* codes,
                                           const float* delta,
                                           const uint8_t* zero, int j,
                                           int bits, int group) {
  const int bit = j * bits, w = bit >> 5, sh = bit & 31;
  uint32_t v = codes[w] >> sh;
  if (sh + bits > 32) v |= codes[w + 1] << (32 - sh);
  v &= (1u << bits) - 1u;
  return ((float)v - (float)zero[j / group]) * delta[j / group];
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float gated(float g, int act) {
  if (act == TTQ_ACT_SILU) return g / (1.f + expf(-g));
  return 0.5f * g *
         (1.f + tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g)));
}

template <typename TX>
__global__ void __launch_bounds__(kThreads)
    moe_up_kernel(const TX* __restrict__ X, int K, int64_t ldx,
                  const int32_t* __restrict__ ids, int top_k, int E,
                  const float* __restrict__ inv_s,
                  const uint32_t* __restrict__ codes,
                  const float* __restrict__ delta,
                  const uint8_t* __restrict__ zero, int I,
                  const float* __restrict__ inv_s_mid, int bits, int group,
                  int act, float* __restrict__ h, uint32_t* err) {
  griddep_enter();
  const int64_t slot = blockIdx.y, t = slot / top_k;
  const int e = ids[slot];
  if (e >= E && threadIdx.x == 0) flag_error(err, TTQ_DEVERR_INDEX);
  if (e < 0 || e >= E) return;
  const int i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (i >= I) return;
  const int64_t ldc = codes_ld(K, bits), ldg = groups_ld(K, group);
  const int64_t rg = (int64_t)e * 2 * I + i, ru = rg + I;
  float g = 0.f, u = 0.f;
  for (int j = threadIdx.x & 31; j < K; j += 32) {
    const float x = to_f32(X[t * ldx + j]) * inv_s[j];
    g = fmaf(x, weight_at(codes + rg * ldc, delta + rg * ldg, zero + rg * ldg,
                          j, bits, group), g);
    u = fmaf(x, weight_at(codes + ru * ldc, delta + ru * ldg, zero + ru * ldg,
                          j, bits, group), u);
  }
  g = warp_sum(g);
  u = warp_sum(u);
  if ((threadIdx.x & 31) == 0)
    h[slot * I + i] = gated(g, act) * u * inv_s_mid[(int64_t)e * I + i];
}

template <typename TY>
__global__ void __launch_bounds__(kThreads)
    moe_down_kernel(const float* __restrict__ h, int I,
                    const int32_t* __restrict__ ids,
                    const float* __restrict__ weights, int top_k, int E,
                    const uint32_t* __restrict__ codes,
                    const float* __restrict__ delta,
                    const uint8_t* __restrict__ zero, int K, int bits,
                    int group, TY* __restrict__ Y, int64_t ldy) {
  griddep_enter();
  const int64_t t = blockIdx.y;
  const int n = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (n >= K) return;
  const int64_t ldc = codes_ld(I, bits), ldg = groups_ld(I, group);
  float y = 0.f;
  for (int c = 0; c < top_k; ++c) {
    const int64_t slot = t * top_k + c;
    const int e = ids[slot];
    if (e < 0 || e >= E) continue;
    const int64_t r = (int64_t)e * K + n;
    float acc = 0.f;
    for (int j = threadIdx.x & 31; j < I; j += 32)
      acc = fmaf(h[slot * I + j],
                 weight_at(codes + r * ldc, delta + r * ldg, zero + r * ldg,
                           j, bits, group), acc);
    y = fmaf(weights[slot], warp_sum(acc), y);
  }
  if ((threadIdx.x & 31) == 0) Y[t * ldy + n] = from_f32<TY>(y);
}

}  // namespace

size_t moe_workspace_bytes(int64_t T, int64_t K, int64_t I, int top_k) {
  return (size_t)T * top_k * I * sizeof(float);
}

ttq_status launch_moe_lowbit(const MoeArgs& a, cudaStream_t st) {
  float* h = static_cast<float*>(a.workspace);
  LaunchShape up, down;
  up.grid = dim3((unsigned)((a.I + 7) / 8), (unsigned)(a.T * a.top_k));
  down.grid = dim3((unsigned)((a.K + 7) / 8), (unsigned)a.T);
  up.block = down.block = dim3(kThreads);
  auto go_up = [&](auto* x) {
    using TX = std::remove_const_t<std::remove_pointer_t<decltype(x)>>;
    return launch(up, st, moe_up_kernel<TX>, x, (int)a.K, a.ldx, a.ids,
                  a.top_k, (int)a.E, a.inv_s, a.up_codes, a.up_delta,
                  a.up_zero, (int)a.I, a.inv_s_mid, a.bits, a.group,
                  (int)a.act, h, device_error_word());
  };
  auto go_down = [&](auto* y) {
    using TY = std::remove_pointer_t<decltype(y)>;
    return launch(down, st, moe_down_kernel<TY>, h, (int)a.I, a.ids,
                  a.weights, a.top_k, (int)a.E, a.down_codes, a.down_delta,
                  a.down_zero, (int)a.K, a.bits, a.group, y, a.ldy);
  };
  ttq_status s = TTQ_ERR_INVALID_ARG;
  if (a.xt == TTQ_F32) s = go_up(static_cast<const float*>(a.X));
  if (a.xt == TTQ_BF16) s = go_up(static_cast<const __nv_bfloat16*>(a.X));
  if (a.xt == TTQ_F16) s = go_up(static_cast<const __half*>(a.X));
  if (s != TTQ_OK) return s;
  if (a.yt == TTQ_F32) return go_down(static_cast<float*>(a.Y));
  if (a.yt == TTQ_BF16) return go_down(static_cast<__nv_bfloat16*>(a.Y));
  return go_down(static_cast<__half*>(a.Y));
}

}  // namespace ttq
