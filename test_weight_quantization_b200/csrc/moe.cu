// moe.cu — a mixture-of-experts layer on packed low-bit experts for a few
// tokens (ttq_moe_lowbit): the activations' rows and the launches.
//
// Four launches: rows_kernel brings x = X inv_s into fp16 terms, up_kernel
// makes h = act(gate) * up * inv_s_mid, rows_kernel does the same for h, and
// down_kernel sums the experts (moe_tile.cuh). All are launched with
// programmatic stream serialisation: up_kernel and down_kernel build their
// lists from ids and fetch their first weights while the rows kernel before
// them is still running.
#include "moe.h"

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace ttq {
namespace {

constexpr int kThreads = 256;

// 8 values as fp32 by plain loads (the row may come from the kernel before).
__device__ __forceinline__ void load_row8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0];
  const float4 b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load_row8(const __nv_bfloat16* p,
                                          float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  bf16x2_to_f32(a.x, v[0], v[1]);
  bf16x2_to_f32(a.y, v[2], v[3]);
  bf16x2_to_f32(a.z, v[4], v[5]);
  bf16x2_to_f32(a.w, v[6], v[7]);
}
__device__ __forceinline__ void load_row8(const __half* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  f16x2_to_f32(a.x, v[0], v[1]);
  f16x2_to_f32(a.y, v[2], v[3]);
  f16x2_to_f32(a.z, v[4], v[5]);
  f16x2_to_f32(a.w, v[6], v[7]);
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Row r = blockIdx.x of [rows, n 8-channel vectors], times inv_s unless that
// is NULL, as fp16 terms xhat[term][row]: times 2^k, with k from the row's
// largest value (row_exponent), and 2^(most - at) of the code pair each
// channel meets. sums[row]: the rounded values' sums over each group. The first term rounds every value above 2^-27 of the largest
// to 11 bits, the second what is left.
template <typename TX>
__global__ void __launch_bounds__(kThreads)
    rows_kernel(const TX* X, int64_t ldx, const float* inv_s, int n,
                int terms, bool g16, int4 up, int most, uint4* xhat,
                float* sums, int ldg, int group, uint32_t* xmax,
                const int32_t* ids, int E) {
  __shared__ uint32_t warp_max[kThreads / 32];
  griddep_enter();
  const int r = blockIdx.x;
  // a choice without an expert has no row
  if (ids && (ids[r] < 0 || ids[r] >= E)) return;
  const TX* row = X + r * ldx;
  auto load = [&](int i, float (&v)[8]) {
    load_row8(row + i * 8, v);
    if (inv_s) {
      const float4 a = reinterpret_cast<const float4*>(inv_s)[2 * i];
      const float4 b = reinterpret_cast<const float4*>(inv_s)[2 * i + 1];
      v[0] *= a.x; v[1] *= a.y; v[2] *= a.z; v[3] *= a.w;
      v[4] *= b.x; v[5] *= b.y; v[6] *= b.z; v[7] *= b.w;
    }
  };
  constexpr int kKeep = 2;  // vectors kept in registers between the passes
  float kept[kKeep][8] = {};
  uint32_t mx = 0;
#pragma unroll
  for (int j = 0; j < kKeep; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (i < n) {
      load(i, kept[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        mx = max(mx, __float_as_uint(kept[j][e]) & 0x7FFFFFFFu);
    }
  }
  for (int i = threadIdx.x + kKeep * kThreads; i < n; i += kThreads) {
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
  if (threadIdx.x == 0) xmax[r] = mx;
  const int k2 = moe::row_exponent(mx, most);
  // 2^(k + up): two factors, since their sum may leave the exponent's range
  const float sc = __uint_as_float((uint32_t)(127 + k2) << 23);
  const float s0 = (float)(1 << up.x), s1 = (float)(1 << up.y),
              s2 = (float)(1 << up.z), s3 = (float)(1 << up.w);
  // every lane of a warp calls store together: i < n or not, groups are
  // whole lanes
  auto store = [&](int i, float (&v)[8]) {
    const bool live = i < n;
    float total = 0.f;
    if (g16) {
      // channels 4m..4m+3 of a half: lane m's pairs (0, 2), (1, 3)
      const float f0 = (i >> 1) & 1 ? s2 : s0, f1 = (i >> 1) & 1 ? s3 : s1;
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = v[q] * sc * (q & 1 ? f1 : f0);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        v[q] = v[q] * sc *
               ((q & 3) == 0 ? s0 : (q & 3) == 1 ? s1 : (q & 3) == 2 ? s2
                                                                     : s3);
    }
    for (int k = 0; k < terms; ++k) {
      uint4* out = xhat + ((int64_t)k * gridDim.x + r) * n;
      const bool put = live;
      uint32_t p[4];
      float a[8];
      if (g16) {
        p[0] = half2_bits(v[0], v[2]);
        p[1] = half2_bits(v[1], v[3]);
        p[2] = half2_bits(v[4], v[6]);
        p[3] = half2_bits(v[5], v[7]);
        const int blk = i / 4, half = (i >> 1) & 1, m = 2 * (i & 1);
        uint2* o = reinterpret_cast<uint2*>(out + blk * 4);
        if (put) {
          o[m * 2 + half] = make_uint2(p[0], p[1]);
          o[(m + 1) * 2 + half] = make_uint2(p[2], p[3]);
        }
        f16x2_to_f32(p[0], a[0], a[2]);
        f16x2_to_f32(p[1], a[1], a[3]);
        f16x2_to_f32(p[2], a[4], a[6]);
        f16x2_to_f32(p[3], a[5], a[7]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          p[q] = half2_bits(v[q], v[q + 4]);
          f16x2_to_f32(p[q], a[q], a[q + 4]);
        }
        if (put) out[i] = make_uint4(p[0], p[1], p[2], p[3]);
      }
      // back to the natural size: powers of two, exact
      if (g16) {
        const float f0 = (i >> 1) & 1 ? s2 : s0, f1 = (i >> 1) & 1 ? s3 : s1;
#pragma unroll
        for (int q = 0; q < 8; ++q) total += a[q] / (q & 1 ? f1 : f0);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          total += a[q] / ((q & 3) == 0   ? s0
                           : (q & 3) == 1 ? s1
                           : (q & 3) == 2 ? s2
                                          : s3);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] -= a[q];
    }
    for (int o = group / 16; o > 0; o >>= 1)
      total += __shfl_xor_sync(0xffffffffu, total, o);
    if (live && i % (group / 8) == 0)
      sums[(int64_t)r * ldg + i / (group / 8)] = total;
  };
#pragma unroll
  for (int j = 0; j < kKeep; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (j * kThreads < n) store(i, kept[j]);
  }
  for (int base = kKeep * kThreads; base < n; base += kThreads) {
    const int i = base + threadIdx.x;
    float v[8] = {};
    if (i < n) load(i, v);
    store(i, v);
  }
}

// Workspace: xhat and hhat (two terms each), h, xsum, hsum, xmax, hmax; every
// part a multiple of 16 bytes. The sums are sized for groups of 16.
struct Layout {
  size_t hhat, h, xsum, hsum, xmax, hmax, bytes;
  Layout(int64_t T, int64_t K, int64_t I, int top_k) {
    hhat = (size_t)2 * T * K * 2;
    h = hhat + (size_t)2 * T * top_k * I * 2;
    xsum = h + (size_t)T * top_k * I * 4;
    hsum = xsum + (size_t)T * groups_ld(K, 16) * 4;
    xmax = hsum + (size_t)T * top_k * groups_ld(I, 16) * 4;
    hmax = xmax + (size_t)(T + 3) / 4 * 16;
    bytes = hmax + (size_t)(T * top_k + 3) / 4 * 16;
  }
};

template <typename Args>
ttq_status launch_width(int bits, const Args& a, cudaStream_t st) {
  switch (bits) {
    case 2: return moe::launch_bits<2>(a, st);
    case 3: return moe::launch_bits<3>(a, st);
    case 4: return moe::launch_bits<4>(a, st);
    case 5: return moe::launch_bits<5>(a, st);
    case 6: return moe::launch_bits<6>(a, st);
    case 7: return moe::launch_bits<7>(a, st);
    case 8: return moe::launch_bits<8>(a, st);
  }
  return TTQ_ERR_INVALID_ARG;
}

}  // namespace

size_t moe_workspace_bytes(int64_t T, int64_t K, int64_t I, int top_k) {
  return Layout(T, K, I, top_k).bytes;
}

ttq_status launch_moe_lowbit(const MoeArgs& a, cudaStream_t st) {
  const Layout l(a.T, a.K, a.I, a.top_k);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  uint4* xhat = reinterpret_cast<uint4*>(ws);
  uint4* hhat = reinterpret_cast<uint4*>(ws + l.hhat);
  float* h = reinterpret_cast<float*>(ws + l.h);
  float* xsum = reinterpret_cast<float*>(ws + l.xsum);
  float* hsum = reinterpret_cast<float*>(ws + l.hsum);
  uint32_t* xmax = reinterpret_cast<uint32_t*>(ws + l.xmax);
  uint32_t* hmax = reinterpret_cast<uint32_t*>(ws + l.hmax);
  const bool g16 = a.group == 16;
  // an fp32 Y takes its codes as normal numbers, all in one position
  int4 up = make_int4(0, 0, 0, 0);
  int most = 0;
  if (a.yt != TTQ_F32) {
    const int p[4] = {moe::position(a.bits, g16, 0),
                      moe::position(a.bits, g16, 1),
                      moe::position(a.bits, g16, 2),
                      moe::position(a.bits, g16, 3)};
    most = std::max(std::max(p[0], p[1]), std::max(p[2], p[3]));
    up = make_int4(most - p[0], most - p[1], most - p[2], most - p[3]);
  }
  const int terms = a.yt == TTQ_BF16 ? 1 : 2;
  LaunchShape ls;
  ls.block = dim3(kThreads);
  auto rows = [&](auto* x, int64_t count, int64_t ld, int64_t width,
                  const float* inv_s, uint4* hat, float* sum, uint32_t* max,
                  const int32_t* ids) {
    using TX = std::remove_const_t<std::remove_pointer_t<decltype(x)>>;
    ls.grid = dim3((unsigned)count);
    return launch(ls, st, rows_kernel<TX>, x, ld, inv_s, (int)(width / 8),
                  terms, g16, up, most, hat, sum,
                  (int)groups_ld(width, a.group), a.group, max, ids,
                  (int)a.E);
  };
  auto x_rows = [&](auto* x) {
    return rows(x, a.T, a.ldx, a.K, a.inv_s, xhat, xsum, xmax, nullptr);
  };
  ttq_status s =
      a.xt == TTQ_F32    ? x_rows(static_cast<const float*>(a.X))
      : a.xt == TTQ_BF16 ? x_rows(static_cast<const __nv_bfloat16*>(a.X))
                         : x_rows(static_cast<const __half*>(a.X));
  if (s != TTQ_OK) return s;
  moe::UpArgs u;
  u.xhat = xhat;
  u.xsum = xsum;
  u.xmax = xmax;
  u.ids = a.ids;
  u.T = (int)a.T;
  u.K = (int)a.K;
  u.I = (int)a.I;
  u.E = (int)a.E;
  u.top_k = a.top_k;
  u.group = a.group;
  u.act = (int)a.act;
  u.rs = 1;
  u.codes = a.up_codes;
  u.delta = a.up_delta;
  u.zero = a.up_zero;
  u.inv_s_mid = a.inv_s_mid;
  u.h = h;
  u.yt = a.yt;
  u.err = device_error_word();
  s = launch_width(a.bits, u, st);
  if (s != TTQ_OK) return s;
  s = rows(static_cast<const float*>(h), a.T * a.top_k, a.I, a.I, nullptr,
           hhat, hsum, hmax, a.ids);
  if (s != TTQ_OK) return s;
  moe::DownArgs d;
  d.hhat = hhat;
  d.hsum = hsum;
  d.hmax = hmax;
  d.ids = a.ids;
  d.weights = a.weights;
  d.T = u.T;
  d.K = u.K;
  d.I = u.I;
  d.E = u.E;
  d.top_k = a.top_k;
  d.group = a.group;
  d.rs = 1;
  d.codes = a.down_codes;
  d.delta = a.down_delta;
  d.zero = a.down_zero;
  d.Y = a.Y;
  d.yt = a.yt;
  d.ldy = a.ldy;
  return launch_width(a.bits, d, st);
}

}  // namespace ttq
