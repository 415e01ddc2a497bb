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
#include "mma16.cuh"

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

// ttq_adapters_add, one launch. A cluster of CTAs takes one tile: up to 32
// tokens of one adapter.
//   1. U = X A^T for the tile: A's ranks as M, the tokens as N of mma.sync
//      m16n8k16, K split over the cluster's warps, every value of X and A read
//      once and straight into its fragment (a lane takes 8 consecutive k).
//      Warps add through shared memory, CTAs through distributed shared
//      memory, in order.
//   2. out = Y + scale U B^T: tokens as M, 32 output channels as four tiles of
//      8 whose columns are dealt so that a lane ends with 8 consecutive
//      channels of its tokens: Y is read and written 16 bytes at a time. The
//      cluster's warps split N. With 16-bit types and whole 16-byte rows, B and
//      Y arrive by cp.async in a ring of units of the warp's own, the
//      first of them while U is being added up (loads into registers one unit
//      ahead left the warps waiting 6.7 of 9 cycles per instruction);
//      otherwise straight into registers.
// U stays fp32 until it enters step 2, in two 16-bit terms (fp16 ones with a
// power of two per token, since U may leave fp16's range) or three bf16 terms
// for fp32. Measured (bf16, graph replay): 4096 tokens of 16 adapters, r 32,
// 4096 x 11008, 59 us = 3.9 TB/s of the bytes it cannot do without; 32 tokens
// with an adapter each, r 16, 9.7 us; one token, 4.6 us. Bound by HBM: X once, Y once in and once out, A and B once per
// adapter in use from HBM (once per tile from L2).
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCols = 32;  // output channels of a warp's unit

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

template <typename TX, typename TY>
struct AddArgs {
  const TX *X, *A, *B;
  const float* scale;
  const int32_t* plan;
  const TY* Y;
  TY* out;
  int64_t ldx, ldy, ldo;
  int T, K, L, r, N, tiles_max;
  bool vec;   // rows of Y and out on 16-byte boundaries
  bool ring;  // B and Y through the ring
  uint32_t* err;
};

// The terms U enters the second product in.
template <typename TX>
constexpr int kUTerms = sizeof(TX) == 4 ? 3 : 2;

template <typename TX, int MT>
constexpr int kFrags = MT * 2 * kUTerms<TX>;  // of U: k16 x m-tile x term

template <typename TX, int MT>
constexpr size_t smem_bytes() {
  // warps' sums (reused for U's fragments), the CTA's U, its sum
  const size_t red = (size_t)kWarps * MT * 4 * 128 * 4;
  const size_t frag = (size_t)kFrags<TX, MT> * 32 * 16;
  return (red > frag ? red : frag) + (size_t)MT * 16 * kTile * 4 * 2 +
         kTile * 4;
}

// The ring of step 2: units of up to 32 token rows x 64 bytes of Y and 32 rows
// of B.
template <int MT>
constexpr int kStages = MT == 1 ? 3 : 2;  // two CTAs' worth of shared memory
template <typename TX, typename TY>
constexpr bool kRingTypes = sizeof(TX) == 2 && sizeof(TY) == 2;
template <int MT>
constexpr int kUnitBytes = kTile * 64 + kCols * MT * 32;

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src,
                                            int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(src), "r"(bytes)
               : "memory");
}

// NT: tiles of 8 tokens (1 or 4).
template <typename TX, typename TY, int MT, int NT, bool RING>
__device__ __forceinline__ void add_tile(const AddArgs<TX, TY>& a, int4 tl,
                                         const int32_t* order, int rank,
                                         int ranks, float* sm) {
  using namespace mma16;
  constexpr int TM = NT == 1 ? 1 : 2;  // tiles of 16 tokens in step 2
  constexpr int XT = mma16::kTerms<TX, TX>, UT = kUTerms<TX>;
  constexpr bool HALF = kHalf<TX, TX>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int parts = ranks * kWarps, part = rank * kWarps + warp;
  float* red = sm;                                   // [warp][m][n][128]
  uint4* frag = reinterpret_cast<uint4*>(sm);        // [kk][m][term][lane]
  float* upart = sm + (smem_bytes<TX, MT>() / 4 - MT * 16 * kTile * 2 - kTile);
  float* U = upart + MT * 16 * kTile;                // [token][rank]
  float* down = U + MT * 16 * kTile;                 // per token: 2^-e scale

  // ---- step 1
  const TX* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int i = n * 8 + g;
    xr[n] = a.X + (int64_t)order[i < tl.z ? i : 0] * a.ldx;
  }
  const TX* A = a.A + (int64_t)tl.x * a.r * a.K;
  float acc[MT][NT][4] = {};
  const int blocks = (a.K + 31) / 32;
  const int b0 = (int)((int64_t)blocks * part / parts);
  const int b1 = (int)((int64_t)blocks * (part + 1) / parts);
  // blocks in flight
  constexpr int UN = XT > 1 && MT == 4 ? 1 : MT * 2 + NT <= 6 && XT == 1 ? 4 : 2;
  for (int bb = b0; bb < b1; bb += UN) {
    Raw<TX, 8> ra[UN][MT][2], rx[UN][NT];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int k = (bb + u) * 32 + 8 * t;
      const bool ok = bb + u < b1 && k < a.K;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int q = m * 16 + h * 8 + g;
          load<TX, 8>(A + (int64_t)q * a.K + k, ok && q < a.r, ra[u][m][h]);
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) load<TX, 8>(xr[n] + k, ok, rx[u][n]);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      uint32_t xt[NT][XT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) terms<TX, TX, 8>(rx[u][n], xt[n]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t at[2][XT][4];
        terms<TX, TX, 8>(ra[u][m][0], at[0]);
        terms<TX, TX, 8>(ra[u][m][1], at[1]);
        // The tensor core cuts its sums instead of rounding them. Over a long
        // K that adds up to more than fp32 values should lose (K = 10^4: 1.5e-6
        // against 5e-7), so their blocks are summed apart and added rounded.
        float sum[NT][4] = {};
        float(&to)[NT][4] = XT > 1 ? sum : acc[m];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = XT - 1; i >= 0; --i)
#pragma unroll
              for (int j = XT - 1 - i; j >= 0; --j)
                mma<HALF>(to[n], at[0][i][2 * h], at[1][i][2 * h],
                          at[0][i][2 * h + 1], at[1][i][2 * h + 1],
                          xt[n][j][2 * h], xt[n][j][2 * h + 1]);
        if constexpr (XT > 1) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] += sum[n][i];
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<float4*>(red + ((warp * MT + m) * NT + n) * 128 +
                                 lane * 4) =
          make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);

  // ---- the first unit of step 2: B and Y need not wait for U
  const TX* B = a.B + (int64_t)tl.x * a.N * a.r;
  int64_t yt[TM][2], ot[TM][2];  // rows of the lane's tokens
  bool live[TM][2];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = m * 16 + h * 8 + g;
      live[m][h] = i < tl.z;
      const int64_t tok = order[live[m][h] ? i : 0];
      yt[m][h] = tok * a.ldy;
      ot[m][h] = tok * a.ldo;
    }
  const int units = (a.N + kCols - 1) / kCols;
  struct Unit {
    Raw<TX, 4> b[4][MT];
    Raw<TY, 8> y[TM][2];
  };
  auto fetch = [&](int u, Unit& f) {
    const int n0 = u * kCols;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
      for (int kk = 0; kk < MT; ++kk) {
        const int q = kk * 16 + 4 * t;
        load<TX, 4>(B + (int64_t)n * a.r + q, n < a.N && q < a.r, f.b[j][kk]);
      }
    }
    const int n = n0 + 8 * t;
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const TY* y = a.Y + yt[m][h] + n;
        if (a.vec && n + 8 <= a.N) {
          load<TY, 8>(y, live[m][h], f.y[m][h]);
        } else {
          TY e[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            e[i] = live[m][h] && n + i < a.N ? y[i] : from_f32<TY>(0.f);
          f.y[m][h] = *reinterpret_cast<const Raw<TY, 8>*>(e);
        }
      }
  };
  Unit cur;
  // the ring: the lane's share of a unit's copies
  uint8_t* ring = reinterpret_cast<uint8_t*>(sm) + smem_bytes<TX, MT>() +
                  warp * kStages<MT> * kUnitBytes<MT>;
  const TY* yr[TM * 2];  // its rows of Y, 8 rows per copy, 8 channels per lane
  if constexpr (RING) {
#pragma unroll
    for (int i = 0; i < TM * 2; ++i) {
      const int row = i * 8 + g;
      yr[i] = a.Y + (int64_t)order[row < tl.z ? row : 0] * a.ldy + 8 * t;
    }
  }
  auto issue = [&](int u, int slot) {
    if constexpr (RING) {
      if (u < units) {
        const uint32_t at = smem_u32(ring + slot * kUnitBytes<MT>);
        const int n0 = u * kCols;
        // what a row of Y holds from the lane's channel on
        const int yb = min(16, (a.N - n0 - 8 * t) * 2);
#pragma unroll
        for (int i = 0; i < TM * 2; ++i)
          if (i * 8 + g < tl.z && yb > 0)
            cp_async_16(at + (i * 8 + g) * 64 + t * 16, yr[i] + n0, yb);
        const uint8_t* src =
            reinterpret_cast<const uint8_t*>(B + (int64_t)n0 * a.r);
        const int all = min(kCols, a.N - n0) * a.r * 2;
#pragma unroll
        for (int i = 0; i < MT * 2; ++i) {
          const int p = (lane + 32 * i) * 16;
          if (p < all)
            cp_async_16(at + kTile * 64 + p, src + p, min(16, all - p));
        }
      }
      cp_async_commit();
    }
  };
  if constexpr (RING) {
#pragma unroll
    for (int i = 0; i < kStages<MT>; ++i) issue(part + i * parts, i);
  } else {
    if (part < units) fetch(part, cur);
  }

  // ---- U: the warps', then the cluster's sums
  __syncthreads();
  constexpr int kElems = MT * NT * 128;
  for (int i = tid; i < kElems; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w * kElems + i];
    upart[i] = v;
  }
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
  const float sc = a.scale ? a.scale[tl.x] : 1.f;
  const uint32_t up = smem_u32(upart);
  for (int i = tid; i < kElems; i += kThreads) {
    float v = 0.f;
    if (ranks > 1) {
      for (int q = 0; q < ranks; ++q) v += ld_cluster_f32(up + i * 4, q);
    } else {
      v = upart[i];
    }
    // element: tile (m, n), lane, register -> rank, token
    const int e = i & 127, mn = i >> 7, ln = e >> 2, rg = e & 3;
    const int q = mn / NT * 16 + (ln >> 2) + 8 * (rg >> 1);
    const int tok = mn % NT * 8 + 2 * (ln & 3) + (rg & 1);
    U[tok * (MT * 16) + q] = v * sc;
  }
  if (ranks > 1)
    cluster_sync();  // every CTA has read upart: nothing leaves before that
  else
    __syncthreads();
  // U's fragments: token rows g and g + 8, ranks 4t .. 4t + 3 of each 16
  if constexpr (HALF) {
    // a power of two per token brings its largest U to [2^13, 2^14)
    for (int i = tid; i < 16 * TM; i += kThreads) {
      uint32_t mx = 0;
      if (i < NT * 8)
        for (int q = 0; q < MT * 16; ++q)
          mx = max(mx, __float_as_uint(U[i * (MT * 16) + q]) & 0x7FFFFFFFu);
      const int k = min(13 - ((int)(mx >> 23) - 127), 126);
      down[i] = __uint_as_float((uint32_t)(127 - k) << 23);
    }
    __syncthreads();
  }
  for (int i = tid; i < MT * TM * 32; i += kThreads) {
    const int ln = i & 31, m = (i >> 5) % TM, kk = (i >> 5) / TM;
    const int row = m * 16 + (ln >> 2), q = kk * 16 + 4 * (ln & 3);
    float v[8];  // (row, q), (row, q + 1), (row + 8, ..), (row, q + 2), ..
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int rr = row + ((e >> 1) & 1) * 8, qq = q + (e >> 2) * 2 + (e & 1);
      v[e] = rr < NT * 8 ? U[rr * (MT * 16) + qq] : 0.f;
      if constexpr (HALF)  // exact; a row without values has down = 2^-126
        v[e] = rr < NT * 8 ? v[e] / down[rr] : 0.f;
    }
    uint4* o = frag + (kk * TM + m) * UT * 32 + ln;
    if constexpr (HALF) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < UT; ++k) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          w[p] = f16x2(v[2 * p], v[2 * p + 1]);
          float x, y;
          f16x2_to_f32(w[p], x, y);
          v[2 * p] -= x;
          v[2 * p + 1] -= y;
        }
        o[k * 32] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
      uint32_t w[UT][4];
      split<UT, 4>(v, w);
#pragma unroll
      for (int k = 0; k < UT; ++k)
        o[k * 32] = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
    }
  }
  __syncthreads();

  // ---- step 2
  int slot = 0;
  for (int u = part; u < units; u += parts) {
    const uint8_t* unit = ring + slot * kUnitBytes<MT>;
    if constexpr (RING) {
      cp_async_wait<kStages<MT> - 1>();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
        for (int kk = 0; kk < MT; ++kk) {
          const int q = kk * 16 + 4 * t;
          const uint2 v =
              q < a.r ? *reinterpret_cast<const uint2*>(
                            unit + kTile * 64 + (n * a.r + q) * 2)
                      : make_uint2(0, 0);
          cur.b[j][kk].w[0] = v.x;
          cur.b[j][kk].w[1] = v.y;
        }
      }
    }
    float c[TM][4][4] = {};
#pragma unroll
    for (int kk = 0; kk < MT; ++kk) {
      uint32_t bt[4][XT][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) terms<TX, TX, 4>(cur.b[j][kk], bt[j]);
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int k = 0; k < UT; ++k) {
          const uint4 f = frag[((kk * TM + m) * UT + k) * 32 + lane];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int x = 0; x < XT; ++x)
              if (k + x < UT)
                mma<HALF>(c[m][j], f.x, f.y, f.z, f.w, bt[j][x][0],
                          bt[j][x][1]);
        }
    }
    if constexpr (RING) {
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 v = *reinterpret_cast<const uint4*>(
              unit + (m * 16 + h * 8 + g) * 64 + t * 16);
          cur.y[m][h].w[0] = v.x;
          cur.y[m][h].w[1] = v.y;
          cur.y[m][h].w[2] = v.z;
          cur.y[m][h].w[3] = v.w;
        }
      __syncwarp();  // every lane has read the unit
      issue(u + kStages<MT> * parts, slot);
      slot = slot + 1 == kStages<MT> ? 0 : slot + 1;
    }
    const Unit now = cur;
    if constexpr (!RING)
      if (u + parts < units) fetch(u + parts, cur);
    const int n = u * kCols + 8 * t;
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!live[m][h]) continue;
        const float s = HALF ? down[m * 16 + h * 8 + g] : 1.f;
        TY e[8];
        *reinterpret_cast<Raw<TY, 8>*>(e) = now.y[m][h];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          e[i] = from_f32<TY>(
              fmaf(c[m][i >> 1][2 * h + (i & 1)], s, to_f32(e[i])));
        TY* o = a.out + ot[m][h] + n;
        if ((RING || a.vec) && n + 8 <= a.N) {
          const Raw<TY, 8>& w = *reinterpret_cast<const Raw<TY, 8>*>(e);
#pragma unroll
          for (int i = 0; i < (int)sizeof(TY) / 2; ++i)
            reinterpret_cast<uint4*>(o)[i] =
                make_uint4(w.w[4 * i], w.w[4 * i + 1], w.w[4 * i + 2],
                           w.w[4 * i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n + i < a.N) o[i] = e[i];
        }
      }
  }
}

// CTAs per SM: two where 128 registers hold a unit in flight.
template <typename TX, int MT>
constexpr int kPerSm = sizeof(TX) == 2 && MT <= 2 ? 2 : 1;

template <typename TX, typename TY, int MT>
__global__ void __launch_bounds__(kThreads, kPerSm<TX, MT>)
    adapters_add_kernel(const AddArgs<TX, TY> a) {
  extern __shared__ __align__(16) float sm[];
  griddep_enter();
  // every exit below is the whole cluster's: it has one tile
  if (a.plan[1] != kTile || a.plan[2] != a.T || a.plan[3] != a.L) {
    if (threadIdx.x == 0) flag_error(a.err, TTQ_DEVERR_INDEX);
    return;
  }
  if ((int)blockIdx.x >= a.plan[0]) return;
  const int4 tl = reinterpret_cast<const int4*>(a.plan + kHead)[blockIdx.x];
  const int32_t* order = a.plan + kHead + 4 * (int64_t)a.tiles_max + tl.y;
  const int rank = blockIdx.y, ranks = gridDim.y;
  if (tl.x < 0) {
    if (a.Y == a.out) return;
    for (int i = 0; i < tl.z; ++i) {
      const TY* y = a.Y + (int64_t)order[i] * a.ldy;
      TY* o = a.out + (int64_t)order[i] * a.ldo;
      constexpr int E = 16 / sizeof(TY);
      const int whole = a.vec ? a.N / E : 0;
      for (int n = rank * kThreads + threadIdx.x; n < whole;
           n += ranks * kThreads)
        reinterpret_cast<uint4*>(o)[n] = reinterpret_cast<const uint4*>(y)[n];
      for (int n = whole * E + rank * kThreads + threadIdx.x; n < a.N;
           n += ranks * kThreads)
        o[n] = y[n];
    }
    return;
  }
  if constexpr (kRingTypes<TX, TY>) {
    if (a.ring) {
      if (tl.z <= 8)
        add_tile<TX, TY, MT, 1, true>(a, tl, order, rank, ranks, sm);
      else
        add_tile<TX, TY, MT, 4, true>(a, tl, order, rank, ranks, sm);
      cp_async_wait_all();
      return;
    }
  }
  if (tl.z <= 8)
    add_tile<TX, TY, MT, 1, false>(a, tl, order, rank, ranks, sm);
  else
    add_tile<TX, TY, MT, 4, false>(a, tl, order, rank, ranks, sm);
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
  const int tiles = (int)max_tiles(a.T, a.L);
  ls.block = dim3(kThreads);
  auto go = [&](auto* x, auto* y) -> ttq_status {
    using TX = std::remove_const_t<std::remove_pointer_t<decltype(x)>>;
    using TY = std::remove_pointer_t<decltype(y)>;
    AddArgs<TX, TY> g;
    g.X = x;
    g.A = static_cast<const TX*>(a.A);
    g.B = static_cast<const TX*>(a.B);
    g.scale = a.scale;
    g.plan = a.plan;
    g.Y = static_cast<const TY*>(a.Y);
    g.out = y;
    g.ldx = a.ldx;
    g.ldy = a.ldy;
    g.ldo = a.ldo;
    g.T = (int)a.T;
    g.K = (int)a.K;
    g.L = (int)a.L;
    g.r = a.r;
    g.N = (int)a.N;
    g.tiles_max = tiles;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.Y) |
                         reinterpret_cast<uintptr_t>(a.out) |
                         (uintptr_t)(a.ldy * sizeof(TY)) |
                         (uintptr_t)(a.ldo * sizeof(TY));
    g.vec = at % 16 == 0;
    // every adapter's B and every unit's Y on 16-byte boundaries
    g.ring = kRingTypes<TX, TY> && g.vec && (a.N * a.r) % 8 == 0;
    g.err = device_error_word();
    auto run = [&](auto mt) -> ttq_status {
      constexpr int MT = decltype(mt)::value;
      // up to 8 CTAs share a tile: as many as the SMs hold at once
      const int ranks =
          std::max(1, std::min(8, kPerSm<TX, MT> * sm_count() / tiles));
      ls.grid = dim3((unsigned)tiles, (unsigned)ranks);
      ls.cluster_y = (unsigned)ranks;
      ls.smem = smem_bytes<TX, MT>();
      if (g.ring) ls.smem += (size_t)kWarps * kStages<MT> * kUnitBytes<MT>;
      auto kern = adapters_add_kernel<TX, TY, MT>;
      if (cudaFuncSetAttribute(kern,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)ls.smem) != cudaSuccess)
        return TTQ_ERR_CUDA;
      return launch(ls, st, kern, g);
    };
    if (a.r <= 16) return run(std::integral_constant<int, 1>{});
    if (a.r <= 32) return run(std::integral_constant<int, 2>{});
    return run(std::integral_constant<int, 4>{});
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
