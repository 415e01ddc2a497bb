// moe.cu — a mixture-of-experts layer on packed low-bit experts for a few
// tokens (ttq_moe_lowbit): the activations' rows and the launches.
//
// Four launches: rows_kernel brings x = X inv_s into fp16 terms, up_kernel
// makes h = act(gate) * up * inv_s_mid, rows_kernel does the same for h, and
// down_kernel sums the experts (moe_tile.cuh). All are launched with
// programmatic stream serialisation: up_kernel and down_kernel build their
// lists from ids and fetch their first weights while the rows kernel before
// them is still running.
//
// Measured by graph replay, bf16: 20 us for one token on 6 of 64 experts of
// 2048 x 1408 (4 bits, groups of 128; 28 MB), 205 us for 33 tokens on 8 experts
// of 4096 x 11008 (584 MB: 2.9 TB/s), 328 us for 64 tokens on 64 experts of
// 4096 x 1408 (5 bits; 737 MB). The up kernel there issues 52-55 % of the
// time with the ALU pipe 54-65 % busy: unpacking bounds it before HBM does.
#include "moe.h"

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "moe_rows.cuh"

namespace ttq {
namespace {

constexpr int kThreads = 256;

// Row r = blockIdx.x of [rows, n 8-channel vectors] to terms, sums and its
// largest value.
template <typename TX>
__global__ void __launch_bounds__(kThreads)
    rows_kernel(const TX* X, int64_t ldx, const float* inv_s, int n,
                moe::RowFormat f, uint4* xhat, float* sums, int ldg,
                uint32_t* xmax, const int32_t* ids, int E) {
  __shared__ uint32_t warp_max[kThreads / 32];
  griddep_enter();
  const int r = blockIdx.x;
  // a choice without an expert has no row
  if (ids && (ids[r] < 0 || ids[r] >= E)) return;
  const TX* row = X + r * ldx;
  constexpr int kKeep = 2;  // vectors kept in registers between the passes
  float kept[kKeep][8] = {};
  uint32_t mx = 0;
#pragma unroll
  for (int j = 0; j < kKeep; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (i < n) {
      moe::load_scaled(row, inv_s, i, kept[j]);
      mx = max(mx, moe::largest_bits(kept[j]));
    }
  }
  for (int i = threadIdx.x + kKeep * kThreads; i < n; i += kThreads) {
    float v[8];
    moe::load_scaled(row, inv_s, i, v);
    mx = max(mx, moe::largest_bits(v));
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) mx = max(mx, warp_max[w]);
  if (threadIdx.x == 0) xmax[r] = mx;
  uint4* out = xhat + (int64_t)r * n;
  const int64_t term = (int64_t)gridDim.x * n;
  float* sum = sums + (int64_t)r * ldg;
#pragma unroll
  for (int j = 0; j < kKeep; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (j * kThreads < n)
      moe::store_vector(f, i, mx, i < n, kept[j], out, term, sum);
  }
  for (int base = kKeep * kThreads; base < n; base += kThreads) {
    const int i = base + threadIdx.x;
    float v[8] = {};
    if (i < n) moe::load_scaled(row, inv_s, i, v);
    moe::store_vector(f, i, mx, i < n, v, out, term, sum);
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
  moe::RowFormat f;
  f.terms = a.yt == TTQ_BF16 ? 1 : 2;
  f.group = a.group;
  f.most = 0;
  f.up = make_int4(0, 0, 0, 0);
  if (a.yt != TTQ_F32) {
    // (an fp32 Y takes its codes as normal numbers, all in one position)
    const bool g16 = a.group == 16;
    const int p[4] = {moe::position(a.bits, g16, 0),
                      moe::position(a.bits, g16, 1),
                      moe::position(a.bits, g16, 2),
                      moe::position(a.bits, g16, 3)};
    f.most = std::max(std::max(p[0], p[1]), std::max(p[2], p[3]));
    f.up = make_int4(f.most - p[0], f.most - p[1], f.most - p[2],
                     f.most - p[3]);
  }
  LaunchShape ls;
  ls.block = dim3(kThreads);
  auto rows = [&](auto* x, int64_t count, int64_t ld, int64_t width,
                  const float* inv_s, uint4* hat, float* sum, uint32_t* max,
                  const int32_t* ids) {
    using TX = std::remove_const_t<std::remove_pointer_t<decltype(x)>>;
    ls.grid = dim3((unsigned)count);
    return launch(ls, st, rows_kernel<TX>, x, ld, inv_s, (int)(width / 8),
                  f, hat, sum, (int)groups_ld(width, a.group), max, ids,
                  (int)a.E);
  };
  auto x_rows = [&](auto* x) {
    return rows(x, a.T, a.ldx, a.K, a.inv_s, xhat, xsum, xmax, nullptr);
  };
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
  u.codes = a.up_codes;
  u.delta = a.up_delta;
  u.zero = a.up_zero;
  u.inv_s_mid = a.inv_s_mid;
  u.h = h;
  u.yt = a.yt;
  u.err = device_error_word();
  u.X = a.X;
  u.xt = a.xt;
  u.ldx = a.ldx;
  u.inv_s = a.inv_s;
  u.format = f;
  moe::DownArgs d;
  d.h = h;
  d.format = f;
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
  // a few rows: the expert kernels convert their activations themselves
  const bool local = moe::rows_fit(a.T, a.K, a.group, f.terms) &&
                     moe::rows_fit(a.T * a.top_k, a.I, a.group, f.terms);
  u.local = d.local = local;
  ttq_status s = TTQ_OK;
  if (!local) {
    s = a.xt == TTQ_F32    ? x_rows(static_cast<const float*>(a.X))
        : a.xt == TTQ_BF16 ? x_rows(static_cast<const __nv_bfloat16*>(a.X))
                           : x_rows(static_cast<const __half*>(a.X));
    if (s != TTQ_OK) return s;
  }
  s = launch_width(a.bits, u, st);
  if (s != TTQ_OK) return s;
  if (!local) {
    s = rows(static_cast<const float*>(h), a.T * a.top_k, a.I, a.I, nullptr,
             hhat, hsum, hmax, a.ids);
    if (s != TTQ_OK) return s;
  }
  return launch_width(a.bits, d, st);
}

}  // namespace ttq
