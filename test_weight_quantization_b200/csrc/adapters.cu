// adapters.cu — low-rank adapters of many requests beside one shared
// projection: out[t] = Y[t] + scale[a] (X[t] A_a^T) B_a^T, a = index[t].
//
// ttq_adapters_plan sorts a batch's tokens by adapter into tiles of at most
// kTile tokens of one adapter; ttq_adapters_add works tile by tile.
//
// Plan layout (int32): [0] tiles, [1] kTile, [2] T, [3] L, then max_tiles
// entries of 4 (adapter or -1, first position, tokens, 0), then the T tokens
// in sorted order (the order inside an adapter is not fixed; no result
// depends on it, since a token's sums never meet another token's).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace ttq {
namespace {

constexpr int kTile = 32;
constexpr int kPlanThreads = 1024;
constexpr int kHead = 4;

int64_t max_tiles(int64_t T, int64_t L) {
  // every adapter (and "none") ends in at most one partial tile
  return std::min(T, (T + kTile - 1) / kTile + L + 1);
}

// One CTA: counts per adapter, their prefix sums, the tile table, the sorted
// tokens. cnt[key] for key < L an adapter, key = L none.
__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const int32_t* __restrict__ index, int T, int L, int tiles_max,
                int32_t* __restrict__ plan, uint32_t* err) {
  extern __shared__ int cnt[];  // [L + 1] counts, then cursors
  __shared__ int warp_tok[32], warp_til[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i <= L; i += kPlanThreads) cnt[i] = 0;
  griddep_enter();
  __syncthreads();
  const unsigned lt = (1u << lane) - 1u;
  auto key_of = [&](int t) {
    const int a = index[t];
    return a >= 0 && a < L ? a : L;
  };
  const int rounds = (T + kPlanThreads - 1) / kPlanThreads;
  for (int i = 0; i < rounds; ++i) {
    const int t = i * kPlanThreads + tid;
    const int k = t < T ? key_of(t) : -1;
    if (t < T && index[t] >= L) flag_error(err, TTQ_DEVERR_INDEX);
    const unsigned same = __match_any_sync(0xffffffffu, k);
    if (k >= 0 && (same & lt) == 0) atomicAdd(&cnt[k], __popc(same));
  }
  __syncthreads();
  // thread i owns keys [i * per, i * per + per)
  const int per = (L + kPlanThreads) / kPlanThreads;
  int tok = 0, til = 0;
  for (int j = 0; j < per; ++j) {
    const int k = tid * per + j;
    if (k <= L) {
      tok += cnt[k];
      til += (cnt[k] + kTile - 1) / kTile;
    }
  }
  int stok = tok, stil = til;  // inclusive scans
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, stok, o);
    const int b = __shfl_up_sync(0xffffffffu, stil, o);
    if (lane >= o) {
      stok += a;
      stil += b;
    }
  }
  if (lane == 31) {
    warp_tok[warp] = stok;
    warp_til[warp] = stil;
  }
  __syncthreads();
  int btok = 0, btil = 0, all = 0;
  for (int w = 0; w < 32; ++w) {
    if (w < warp) {
      btok += warp_tok[w];
      btil += warp_til[w];
    }
    all += warp_til[w];
  }
  int at = btok + stok - tok, tile = btil + stil - til;
  int4* table = reinterpret_cast<int4*>(plan + kHead);
  for (int j = 0; j < per; ++j) {
    const int k = tid * per + j;
    if (k <= L) {
      const int n = cnt[k];
      for (int i = 0; i < n; i += kTile, ++tile)
        table[tile] = make_int4(k == L ? -1 : k, at + i, min(kTile, n - i), 0);
      cnt[k] = at;  // the cursor of the scatter below
      at += n;
    }
  }
  if (tid == 0) {
    plan[0] = all;
    plan[1] = kTile;
    plan[2] = T;
    plan[3] = L;
  }
  __syncthreads();
  int32_t* order = plan + kHead + 4 * (int64_t)tiles_max;
  for (int i = 0; i < rounds; ++i) {
    const int t = i * kPlanThreads + tid;
    const int k = t < T ? key_of(t) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, k);
    int base = 0;
    if (k >= 0 && (same & lt) == 0) base = atomicAdd(&cnt[k], __popc(same));
    base = __shfl_sync(0xffffffffu, base, __ffs(same) - 1);
    if (k >= 0) order[base + __popc(same & lt)] = t;
  }
}

constexpr int kThreads = 256;

// One CTA per (tile, token of the tile).
template <typename TX, typename TY>
__global__ void __launch_bounds__(kThreads)
    adapters_add_kernel(const TX* __restrict__ X, int T, int K, int64_t ldx,
                        const TX* __restrict__ A, const TX* __restrict__ B,
                        const float* __restrict__ scale, int L, int r, int N,
                        const int32_t* __restrict__ plan, int tiles_max,
                        const TY* Y, int64_t ldy, TY* out, int64_t ldo,
                        uint32_t* err) {
  __shared__ float U[64];
  griddep_enter();
  if (plan[1] != kTile || plan[2] != T || plan[3] != L) {
    if (threadIdx.x == 0) flag_error(err, TTQ_DEVERR_INDEX);
    return;
  }
  if ((int)blockIdx.x >= plan[0]) return;
  const int4 tl = reinterpret_cast<const int4*>(plan + kHead)[blockIdx.x];
  if ((int)blockIdx.y >= tl.z) return;
  const int64_t t =
      plan[kHead + 4 * (int64_t)tiles_max + tl.y + blockIdx.y];
  const TY* y = Y + t * ldy;
  TY* o = out + t * ldo;
  if (tl.x < 0) {
    if (y != o)
      for (int n = threadIdx.x; n < N; n += kThreads) o[n] = y[n];
    return;
  }
  const TX* a = A + (int64_t)tl.x * r * K;
  const TX* b = B + (int64_t)tl.x * N * r;
  for (int q = threadIdx.x >> 5; q < r; q += kThreads / 32) {
    float acc = 0.f;
    for (int j = threadIdx.x & 31; j < K; j += 32)
      acc = fmaf(to_f32(X[t * ldx + j]), to_f32(a[(int64_t)q * K + j]), acc);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
      acc += __shfl_xor_sync(0xffffffffu, acc, s);
    if ((threadIdx.x & 31) == 0) U[q] = acc;
  }
  __syncthreads();
  const float sc = scale ? scale[tl.x] : 1.f;
  for (int n = threadIdx.x; n < N; n += kThreads) {
    float acc = 0.f;
    for (int q = 0; q < r; ++q)
      acc = fmaf(U[q], to_f32(b[(int64_t)n * r + q]), acc);
    o[n] = from_f32<TY>(fmaf(sc, acc, to_f32(y[n])));
  }
}

}  // namespace

int64_t adapters_plan_entries(int64_t T, int64_t L) {
  return kHead + 4 * max_tiles(T, L) + T;
}

ttq_status launch_adapters_plan(const int32_t* index, int64_t T, int64_t L,
                                int32_t* plan, cudaStream_t st) {
  LaunchShape ls;
  ls.grid = dim3(1);
  ls.block = dim3(kPlanThreads);
  ls.smem = (size_t)(L + 1) * sizeof(int);
  return launch(ls, st, plan_kernel, index, (int)T, (int)L,
                (int)max_tiles(T, L), plan, device_error_word());
}

ttq_status launch_adapters_add(const AdapterArgs& a, cudaStream_t st) {
  LaunchShape ls;
  ls.grid = dim3((unsigned)max_tiles(a.T, a.L), kTile);
  ls.block = dim3(kThreads);
  auto go = [&](auto* x, auto* y) {
    using TX = std::remove_const_t<std::remove_pointer_t<decltype(x)>>;
    using TY = std::remove_pointer_t<decltype(y)>;
    return launch(ls, st, adapters_add_kernel<TX, TY>, x, (int)a.T, (int)a.K,
                  a.ldx, static_cast<const TX*>(a.A),
                  static_cast<const TX*>(a.B), a.scale, (int)a.L, a.r,
                  (int)a.N, a.plan, (int)max_tiles(a.T, a.L),
                  static_cast<const TY*>(a.Y), a.ldy, y, a.ldo,
                  device_error_word());
  };
  auto go_y = [&](auto* x) {
    if (a.yt == TTQ_F32) return go(x, static_cast<float*>(a.out));
    if (a.yt == TTQ_BF16) return go(x, static_cast<__nv_bfloat16*>(a.out));
    return go(x, static_cast<__half*>(a.out));
  };
  if (a.xt == TTQ_F32) return go_y(static_cast<const float*>(a.X));
  if (a.xt == TTQ_BF16) return go_y(static_cast<const __nv_bfloat16*>(a.X));
  return go_y(static_cast<const __half*>(a.X));
}

}  // namespace ttq
