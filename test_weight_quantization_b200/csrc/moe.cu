// moe.cu — a mixture-of-experts layer on packed low-bit experts for a few
// tokens (ttq_moe_lowbit): the activations' preparation and the launches.
//
// Three launches. prepare_kernel (a CTA per token) scales x = X inv_s by a
// power of two and splits it into fp16 terms; up_kernel makes
// h = act(gate) * up * inv_s_mid, down_kernel sums the experts (moe_tile.cuh).
// All three are launched with programmatic stream serialisation: up_kernel
// and down_kernel build their lists from ids and fetch their first weights
// while the kernel before them is still running.
#include "moe.h"

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace ttq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// xhat[term][t][...] from token t = blockIdx.x. The scale 2^k brings the
// token's largest |x| into [2^13, 2^14): the first term then rounds every
// x above 2^-27 of it by half a unit in 11 bits, the second what is left.
template <typename TX>
__global__ void __launch_bounds__(kThreads)
    prepare_kernel(const TX* __restrict__ X, int64_t ldx,
                   const float* __restrict__ inv_s, int T, int K, int top_k,
                   int terms, bool g16, uint4* xhat, uint32_t* xmax,
                   uint32_t* hmax) {
  __shared__ uint32_t warp_max[kThreads / 32];
  griddep_enter();
  const int t = blockIdx.x, n = K / 8;
  const TX* row = X + t * ldx;
  for (int j = threadIdx.x; j < top_k; j += kThreads) hmax[t * top_k + j] = 0;
  auto load = [&](int i, float (&v)[8]) {
    load8<TX>(row + i * 8, v);
    const float4 a = reinterpret_cast<const float4*>(inv_s)[2 * i];
    const float4 b = reinterpret_cast<const float4*>(inv_s)[2 * i + 1];
    v[0] *= a.x; v[1] *= a.y; v[2] *= a.z; v[3] *= a.w;
    v[4] *= b.x; v[5] *= b.y; v[6] *= b.z; v[7] *= b.w;
  };
  uint32_t mx = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    float v[8];
    load(i, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      mx = max(mx, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) mx = max(mx, warp_max[w]);
  if (threadIdx.x == 0) xmax[t] = mx;
  const int e = (int)(mx >> 23) - 127;
  const float sc =
      __uint_as_float((uint32_t)(127 + min(13 - e, 126)) << 23);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    float v[8];
    load(i, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] *= sc;
    for (int k = 0; k < terms; ++k) {
      uint4* out = xhat + ((int64_t)k * T + t) * n;
      uint32_t r[4];
      if (g16) {
        // channels 4m..4m+3 of a half: lane m's pairs (0, 2), (1, 3)
        r[0] = half2_bits(v[0], v[2]);
        r[1] = half2_bits(v[1], v[3]);
        r[2] = half2_bits(v[4], v[6]);
        r[3] = half2_bits(v[5], v[7]);
        const int blk = i / 4, half = (i >> 1) & 1, m = 2 * (i & 1);
        uint2* o = reinterpret_cast<uint2*>(out + blk * 4);
        o[m * 2 + half] = make_uint2(r[0], r[1]);
        o[(m + 1) * 2 + half] = make_uint2(r[2], r[3]);
        float a[8];
        f16x2_to_f32(r[0], a[0], a[2]);
        f16x2_to_f32(r[1], a[1], a[3]);
        f16x2_to_f32(r[2], a[4], a[6]);
        f16x2_to_f32(r[3], a[5], a[7]);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] -= a[q];
      } else {
        float a[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          r[q] = half2_bits(v[q], v[q + 4]);
          f16x2_to_f32(r[q], a[q], a[q + 4]);
        }
        out[i] = make_uint4(r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] -= a[q];
      }
    }
  }
}

// Workspace: xhat (two terms), h, xmax, hmax; every part a multiple of 16
// bytes.
struct Layout {
  size_t h, xmax, hmax, bytes;
  Layout(int64_t T, int64_t K, int64_t I, int top_k) {
    h = (size_t)2 * T * K * 2;
    xmax = h + (size_t)T * top_k * I * 4;
    hmax = xmax + (size_t)(T + 3) / 4 * 16;
    bytes = hmax + (size_t)(T * top_k + 3) / 4 * 16;
  }
};

}  // namespace

size_t moe_workspace_bytes(int64_t T, int64_t K, int64_t I, int top_k) {
  return Layout(T, K, I, top_k).bytes;
}

ttq_status launch_moe_lowbit(const MoeArgs& a, cudaStream_t st) {
  const Layout w(a.T, a.K, a.I, a.top_k);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  uint32_t* xmax = reinterpret_cast<uint32_t*>(ws + w.xmax);
  uint32_t* hmax = reinterpret_cast<uint32_t*>(ws + w.hmax);
  const int terms = a.yt == TTQ_BF16 ? 1 : 2;
  LaunchShape ls;
  ls.grid = dim3((unsigned)a.T);
  ls.block = dim3(kThreads);
  auto prep = [&](auto* x) {
    using TX = std::remove_const_t<std::remove_pointer_t<decltype(x)>>;
    return launch(ls, st, prepare_kernel<TX>, x, a.ldx, a.inv_s, (int)a.T,
                  (int)a.K, a.top_k, terms, a.group == 16,
                  reinterpret_cast<uint4*>(ws), xmax, hmax);
  };
  const ttq_status s =
      a.xt == TTQ_F32    ? prep(static_cast<const float*>(a.X))
      : a.xt == TTQ_BF16 ? prep(static_cast<const __nv_bfloat16*>(a.X))
                         : prep(static_cast<const __half*>(a.X));
  if (s != TTQ_OK) return s;
  moe::UpArgs u;
  u.xhat = reinterpret_cast<const __half*>(ws);
  u.xmax = xmax;
  u.ids = a.ids;
  u.T = (int)a.T;
  u.K = (int)a.K;
  u.I = (int)a.I;
  u.E = (int)a.E;
  u.top_k = a.top_k;
  u.group = a.group;
  u.act = (int)a.act;
  u.codes = a.up_codes;
  u.delta = a.up_delta;
  u.zero = a.up_zero;
  u.inv_s_mid = a.inv_s_mid;
  u.h = reinterpret_cast<float*>(ws + w.h);
  u.hmax = hmax;
  u.err = device_error_word();
  moe::DownArgs d;
  d.h = u.h;
  d.hmax = hmax;
  d.ids = a.ids;
  d.weights = a.weights;
  d.T = u.T;
  d.K = u.K;
  d.I = u.I;
  d.E = u.E;
  d.top_k = a.top_k;
  d.group = a.group;
  d.codes = a.down_codes;
  d.delta = a.down_delta;
  d.zero = a.down_zero;
  d.Y = a.Y;
  d.yt = a.yt;
  d.ldy = a.ldy;
  switch (a.bits) {
    case 2: return moe::launch_bits<2>(u, d, st);
    case 3: return moe::launch_bits<3>(u, d, st);
    case 4: return moe::launch_bits<4>(u, d, st);
    case 5: return moe::launch_bits<5>(u, d, st);
    case 6: return moe::launch_bits<6>(u, d, st);
    case 7: return moe::launch_bits<7>(u, d, st);
    case 8: return moe::launch_bits<8>(u, d, st);
  }
  return TTQ_ERR_INVALID_ARG;
}

}  // namespace ttq
