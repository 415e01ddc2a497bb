// moe_tile.cuh — the expert kernels of ttq_moe_lowbit for one code width
// (moe_b2.cu .. moe_b8.cu instantiate them; moe.cu launches).
//
// An expert meets a handful of tokens per step, so its packed weights are
// read once from HBM and used for a few products each: the kernels are bound
// by those bytes, and by the instructions that unpack them. Per warp:
//   - mma.sync m16n8k16 with 16 weight rows as M, up to 32 tokens as N (1, 2
//     or 4 tiles of 8). tcgen05 would want 128 rows per tile and the weights
//     copied to TMEM or shared memory after unpacking; here an unpacked code
//     pair goes from the register it was masked in straight into the MMA.
//   - A code q enters as the fp16 bit pattern q << kAt, the subnormal
//     q 2^(kAt-24): the mask that isolates two codes is all the conversion
//     there is. Per group,
//       acc += D (sum q x - z sum x),
//     with sum x from one more MMA whose A is all ones, in the same
//     accumulator layout. D (fp32) and z are applied in fp32; 2^(24-kAt) and
//     the row's power of two return in the epilogue.
//   - The contraction order inside a 32-code block is free as long as both
//     operands agree: lane t of a quad owns codes 8t..8t+7 (for groups of 16:
//     4t..4t+3 of both halves), which are consecutive bits of one word (4
//     bits) or of two or three, and the activations are stored in that order.
//   - Codes, delta and zero of 32 rows x 128 channels arrive by cp.async in a
//     ring of stages of the warp's own; warps split the contraction and never
//     wait for one another inside it.
#pragma once

#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "moe.h"

namespace ttq {
namespace moe {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 32;      // weight rows of a warp's tile (2 MMA tiles)
constexpr int kChunk = 128;    // channels of one stage

// Bytes between the rows of a stage: 16 b, with 16 more for even b so that 8
// rows start in 8 different groups of 4 banks.
template <int BITS>
constexpr int kPitch = 16 * (BITS | 1);
template <int BITS>
constexpr int kStageCodes = kRows * kPitch<BITS>;
// delta (8 groups of 16 at most) and zero of the stage's rows
constexpr int kStageDelta = kRows * 32;
constexpr int kStageZero = kRows * 8;
template <int BITS, bool G16>
constexpr int kStage =
    kStageCodes<BITS> + (G16 ? kStageDelta + kStageZero
                             : kRows * 16 + kRows * 4);
// Stages per warp: what lets two CTAs of 8 warps share an SM.
template <int BITS>
constexpr int kStages = BITS <= 3 ? 5 : BITS <= 5 ? 3 : 2;

// ------------------------------------------------------------- columns ---

// Which (token, choice) pairs each expert of the batch serves, rebuilt by
// every CTA from ids (at most 64 x 32 of them). A choice given twice for a
// token is one column with the weights added. An entry is an expert with up
// to kMaxCols of its columns.
// The order is by token, so that all CTAs agree on an entry's columns.
struct Lists {
  uint2* tokens;       // [E] bit t: token t has the expert
  int* start;          // [E] the first column of an expert
  float* weight;       // [n] routing weight of a column
  uint16_t* slot;      // [n] the columns' slots, sorted by expert
  int16_t* expert;     // [entries] of an entry: expert, first column, columns
  int16_t* first;
  int16_t* cols;
  int* sums;           // [2 kWarps + 1] of the scans; the last: entries
  int entries;

  static __host__ __device__ int max_entries(int n, int E) {
    return (n < E ? n : E) + n / kMaxCols;
  }
  static __host__ __device__ size_t bytes(int n, int E) {
    const size_t b = (size_t)E * 12 + (size_t)n * 6 +
                     (size_t)max_entries(n, E) * 6 + (2 * kWarps + 1) * 4;
    return (b + 127) / 128 * 128;
  }
  __device__ __forceinline__ Lists(uint8_t* sm, int n, int E) {
    const int m = max_entries(n, E);
    tokens = reinterpret_cast<uint2*>(sm);
    start = reinterpret_cast<int*>(tokens + E);
    weight = reinterpret_cast<float*>(start + E);
    sums = reinterpret_cast<int*>(weight + n);
    slot = reinterpret_cast<uint16_t*>(sums + 2 * kWarps + 1);
    expert = reinterpret_cast<int16_t*>(slot + n);
    first = expert + m;
    cols = first + m;
  }
};

__device__ __forceinline__ void build_lists(Lists& l, const int32_t* ids,
                                            const float* weights, int T,
                                            int top_k, int E, uint32_t* err) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = T * top_k;
  for (int e = tid; e < E; e += kThreads) l.tokens[e] = make_uint2(0, 0);
  __syncthreads();
  for (int p = tid; p < n; p += kThreads) {
    const int e = ids[p], t = p / top_k;
    if (e >= E && err && blockIdx.x == 0) flag_error(err, TTQ_DEVERR_INDEX);
    if (e >= 0 && e < E)
      atomicOr(t < 32 ? &l.tokens[e].x : &l.tokens[e].y, 1u << (t & 31));
  }
  __syncthreads();
  // exclusive sums over the experts, two per thread
  constexpr int kPer = kMaxExperts / kThreads;
  int c[kPer], cols = 0, ents = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    c[i] = e < E ? __popc(l.tokens[e].x) + __popc(l.tokens[e].y) : 0;
    cols += c[i];
    ents += (c[i] + kMaxCols - 1) / kMaxCols;
  }
  int sc = cols, se = ents;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, sc, o);
    const int b = __shfl_up_sync(0xffffffffu, se, o);
    if (lane >= o) {
      sc += a;
      se += b;
    }
  }
  if (lane == 31) {
    l.sums[warp] = sc;
    l.sums[kWarps + warp] = se;
  }
  __syncthreads();
  int bc = sc - cols, be = se - ents, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      bc += l.sums[w];
      be += l.sums[kWarps + w];
    }
    all += l.sums[kWarps + w];
  }
  l.entries = all;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e < E) l.start[e] = bc;
    for (int o = 0; o < c[i]; o += kMaxCols, ++be) {
      l.expert[be] = (int16_t)e;
      l.first[be] = (int16_t)(bc + o);
      l.cols[be] = (int16_t)min(kMaxCols, c[i] - o);
    }
    bc += c[i];
  }
  __syncthreads();
  for (int p = tid; p < n; p += kThreads) {
    const int e = ids[p], t = p / top_k, last = (t + 1) * top_k;
    bool ok = e >= 0 && e < E;  // the first of equal choices stands for all
    for (int q = t * top_k; ok && q < p; ++q) ok = ids[q] != e;
    if (!ok) continue;
    float w = 0.f;
    if (weights) {
      w = weights[p];
      for (int q = p + 1; q < last; ++q)
        if (ids[q] == e) w += weights[q];
    }
    const uint2 m = l.tokens[e];
    const unsigned below = (1u << (t & 31)) - 1u;
    const int at = l.start[e] + (t < 32 ? __popc(m.x & below)
                                        : __popc(m.x) + __popc(m.y & below));
    l.slot[at] = (uint16_t)p;
    l.weight[at] = w;
  }
  __syncthreads();
}

// ------------------------------------------------------------- a stage ---

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
               "l"(src)
               : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async_ca(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst),
               "l"(src), "n"(BYTES)
               : "memory");
}

// The packed matrix of one layer half: stacked rows of `width` channels.
struct Packed {
  const uint32_t* codes;
  const float* delta;
  const uint8_t* zero;
  int64_t ldc, ldg;   // words, entries
  int blocks;         // width / 32
  int group;
};

// Issues the copies of 32 rows (row r of the tile is matrix row base + r for
// r < 16, base2 + r - 16 for the rest) x channels 128 c .. 128 c + 127.
template <int BITS, bool G16>
__device__ __forceinline__ void issue_stage(const Packed& m, uint32_t dst,
                                            int64_t base, int64_t base2, int c,
                                            int lane) {
#pragma unroll
  for (int i = 0; i < BITS; ++i) {
    const int p = lane + 32 * i, r = p / BITS, pc = p % BITS;
    const int64_t row = r < 16 ? base + r : base2 + (r - 16);
    const int word = (c * BITS + pc) * 4;
    if (word < m.ldc)
      cp_async_16(dst + r * kPitch<BITS> + pc * 16,
                  m.codes + row * m.ldc + word);
  }
  const int64_t row = lane < 16 ? base + lane : base2 + (lane - 16);
  const uint32_t dd = dst + kStageCodes<BITS>;
  if constexpr (G16) {
    const float* d = m.delta + row * m.ldg + c * 8;
    cp_async_16(dd + lane * 32, d);
    cp_async_16(dd + lane * 32 + 16, d + 4);
    cp_async_ca<8>(dd + kStageDelta + lane * 8, m.zero + row * m.ldg + c * 8);
  } else {
    const float* d = m.delta + row * m.ldg;
    const uint8_t* z = m.zero + row * m.ldg;
    if (m.group == 32) {
      cp_async_16(dd + lane * 16, d + c * 4);
    } else if (m.group == 64) {
      cp_async_ca<8>(dd + lane * 16, d + c * 2);
    } else {
      cp_async_ca<4>(dd + lane * 16, d + c);
    }
    // the aligned word that holds the stage's zero points
    const int g0 = c * (kChunk / m.group);
    cp_async_ca<4>(dd + kRows * 16 + lane * 4, z + (g0 & ~3));
  }
}

// ----------------------------------------------------------- unpacking ---

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float ldsf(uint32_t a) {
  return __uint_as_float(lds32(a));
}

// How a code pair enters the MMA. NORM: as 1024 + q (the code in the mantissa
// of 1024), from which the caller takes 1024 + z. Otherwise as the subnormal
// q << kAt: the tensor core lines its products up by exponent and does not
// normalise subnormal operands, so a code at bit 0 would lose 10 - b bits of
// the sum (measured: 2-bit codes at bit 0 gave 5e-5 relative error, at bit 6
// 2e-6). The top is 10 - b; up to 3 bits less are taken where that saves a
// shift.
template <int BITS>
constexpr int kAt = BITS <= 3 ? 6 : BITS == 4 ? 4 : BITS == 5 ? 5
                                : BITS == 6 ? 3 : 0;
template <int BITS>
constexpr uint32_t kMask = ((1u << BITS) - 1u) * 0x10001u;

// The code pair whose codes start at bit FROM of both halves of m.
template <int BITS, bool NORM, int FROM>
__device__ __forceinline__ uint32_t pair_at(uint32_t m) {
  if constexpr (NORM) return ((m >> FROM) & kMask<BITS>) | 0x64006400u;
  constexpr int to = kAt<BITS>;
  if constexpr (FROM < to) return (m << (to - FROM)) & (kMask<BITS> << to);
  return (m >> (FROM < to ? 0 : FROM - to)) & (kMask<BITS> << to);
}

// Four registers of code pairs from two fields of four
// codes: (u0, v0), (u1, v1), (u2, v2), (u3, v3).
template <int BITS, bool NORM>
__device__ __forceinline__ void pairs4(uint32_t u, uint32_t v,
                                       uint32_t (&p)[4]) {
  const uint32_t m = __byte_perm(u, v, 0x5410);
  p[0] = pair_at<BITS, NORM, 0>(m);
  p[1] = pair_at<BITS, NORM, BITS>(m);
  if constexpr (BITS <= 4) {
    p[2] = pair_at<BITS, NORM, 2 * BITS>(m);
    p[3] = pair_at<BITS, NORM, 3 * BITS>(m);
  } else {
    const uint32_t n = __byte_perm(u >> (2 * BITS), v >> (2 * BITS), 0x5410);
    p[2] = pair_at<BITS, NORM, 0>(n);
    p[3] = pair_at<BITS, NORM, BITS>(n);
  }
}

// Where a lane (t = lane % 4) finds its codes in a block of BITS words.
template <int BITS, bool G16, bool NORM>
struct Field {
  uint32_t w0, w1, w2, w3;  // byte offsets of words
  uint32_t sh, sh2;         // bit offsets in the first word of each field
  __device__ __forceinline__ explicit Field(int t) {
    const uint32_t last = (BITS - 1) * 4;
    if constexpr (G16) {
      const uint32_t a = 4 * BITS * t, b = 16 * BITS + 4 * BITS * t;
      w0 = a / 32 * 4;
      w1 = min(w0 + 4, last);
      w2 = b / 32 * 4;
      w3 = min(w2 + 4, last);
      sh = a % 32;
      sh2 = b % 32;
    } else {
      const uint32_t a = 8 * BITS * t;
      w0 = a / 32 * 4;
      w1 = min(w0 + 4, last);
      w2 = min(w0 + 8, last);
      w3 = 0;
      sh = a % 32;
      sh2 = 0;
    }
  }
  // p[0], p[1] feed the block's first MMA, p[2], p[3] its second.
  __device__ __forceinline__ void codes(uint32_t at, uint32_t (&p)[4]) const {
    if constexpr (G16) {
      uint32_t u = lds32(at + w0), v = lds32(at + w2);
      if constexpr (BITS == 8) {
      } else {
        u = __funnelshift_r(u, lds32(at + w1), sh);
        v = __funnelshift_r(v, lds32(at + w3), sh2);
      }
      const uint32_t m = __byte_perm(u, u >> (2 * BITS), 0x5410);
      const uint32_t n = __byte_perm(v, v >> (2 * BITS), 0x5410);
      p[0] = pair_at<BITS, NORM, 0>(m);
      p[1] = pair_at<BITS, NORM, BITS>(m);
      p[2] = pair_at<BITS, NORM, 0>(n);
      p[3] = pair_at<BITS, NORM, BITS>(n);
    } else if constexpr (BITS == 4) {
      const uint32_t m = lds32(at + w0);
      p[0] = pair_at<4, NORM, 0>(m);
      p[1] = pair_at<4, NORM, 4>(m);
      p[2] = pair_at<4, NORM, 8>(m);
      p[3] = pair_at<4, NORM, 12>(m);
    } else if constexpr (BITS == 8) {
      pairs4<8, NORM>(lds32(at + w0), lds32(at + w1), p);
    } else if constexpr (BITS == 2) {
      const uint32_t u = lds32(at + w0) >> sh;
      pairs4<2, NORM>(u, u >> 8, p);
    } else if constexpr (BITS == 3) {
      const uint32_t u = __funnelshift_r(lds32(at + w0), lds32(at + w1), sh);
      pairs4<3, NORM>(u, u >> 12, p);
    } else {
      const uint32_t a = lds32(at + w0), b = lds32(at + w1);
      const uint32_t lo = __funnelshift_r(a, b, sh);
      uint32_t hi;
      if constexpr (BITS == 7)
        hi = __funnelshift_r(b, lds32(at + w2), sh);
      else
        hi = b >> sh;
      pairs4<BITS, NORM>(lo, __funnelshift_r(lo, hi, 4 * BITS), p);
    }
  }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0,
                                        uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr uint32_t kOnes = 0x3C003C00u;  // (1, 1)
// what a code's unit is in the accumulators, and its inverse
template <int BITS, int TERMS>
constexpr float kUnit =
    TERMS == 2 ? 1.f : (float)(1 << kAt<BITS>) / 16777216.f;
template <int BITS, int TERMS>
constexpr float kPerUnit = 1.f / kUnit<BITS, TERMS>;

__device__ __forceinline__ void subtract(uint32_t& p, __half2 z) {
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&p), z);
  p = *reinterpret_cast<const uint32_t*>(&d);
}

// One stage's products into acc[row tile][column tile]. x(n, b, v) gives the
// lane's 8 activations of block b for column tile n, a uint4 per term: x, y
// for the block's first MMA, z, w for its second.
template <int BITS, bool G16, int TERMS, int NT, int NTMAX, typename XF>
__device__ __forceinline__ void stage_products(
    uint32_t st, const Field<BITS, G16, TERMS == 2>& f, int group, int c, int nblocks,
    XF&& x, float (&acc)[2][NTMAX][4], int lane) {
  // With two terms the sums are to be good to fp32: z is taken from the codes
  // (exact in fp16), so that sum q x and z sum x never cancel. With one term
  // it is cheaper to take it from the sums.
  constexpr bool kCentre = TERMS == 2;
  const int g = lane >> 2;
  const uint32_t dd = st + kStageCodes<BITS>;
  float cc[2][NT][4], s[NT][4];
  __half2 zc[2][2];
  auto zero_at = [&](int r, int j) -> uint32_t {
    if constexpr (G16) return lds8(dd + kStageDelta + r * 8 + j);
    return lds8(dd + kRows * 16 + r * 4 + ((c * (kChunk / group) + j) & 3));
  };
  auto centre = [&](int j) {
    if constexpr (kCentre) {
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t z =
              (0x6400u | zero_at(rt * 16 + g + 8 * i, j)) * 0x10001u;
          zc[rt][i] = *reinterpret_cast<const __half2*>(&z);
        }
    }
  };
  auto clear = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) cc[0][n][i] = cc[1][n][i] = s[n][i] = 0.f;
  };
  // acc += D (c - z s) for group j of the stage; z0, z1 hold -z in units
  auto flush = [&](int j) {
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      const int r = rt * 16 + g;
      constexpr int pitch = G16 ? 32 : 16;
      const float d0 = ldsf(dd + r * pitch + j * 4);
      const float d1 = ldsf(dd + (r + 8) * pitch + j * 4);
      float z0 = 0.f, z1 = 0.f;
      if constexpr (!kCentre) {
        z0 = zero_at(r, j) * -kUnit<BITS, TERMS>;
        z1 = zero_at(r + 8, j) * -kUnit<BITS, TERMS>;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = kCentre ? cc[rt][n][i]
                         : fmaf(i < 2 ? z0 : z1, s[n][i & 1], cc[rt][n][i]);
        acc[rt][n][0] = fmaf(d0, v[0], acc[rt][n][0]);
        acc[rt][n][1] = fmaf(d0, v[1], acc[rt][n][1]);
        acc[rt][n][2] = fmaf(d1, v[2], acc[rt][n][2]);
        acc[rt][n][3] = fmaf(d1, v[3], acc[rt][n][3]);
      }
    }
  };
  auto products = [&](const uint32_t (&p)[2][2][4], int h, int n, uint32_t b0,
                      uint32_t b1) {
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
      mma_f16(cc[rt][n], p[rt][0][2 * h], p[rt][1][2 * h],
              p[rt][0][2 * h + 1], p[rt][1][2 * h + 1], b0, b1);
    if constexpr (!kCentre)
      mma_f16(s[n], kOnes, kOnes, kOnes, kOnes, b0, b1);
  };
  clear();
  const int bpg = G16 ? 1 : group >> 5;  // blocks per group
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (b < nblocks) {
      uint32_t p[2][2][4];  // [row tile][row g, row g + 8][pair]
      if (!G16 && b % bpg == 0) centre(b / bpg);
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        const uint32_t at =
            st + (rt * 16 + g) * kPitch<BITS> + b * (4 * BITS);
        f.codes(at, p[rt][0]);
        f.codes(at + 8 * kPitch<BITS>, p[rt][1]);
        if constexpr (kCentre && !G16) {
#pragma unroll
          for (int i = 0; i < 8; ++i) subtract(p[rt][i >> 2][i & 3], zc[rt][i >> 2]);
        }
      }
      if constexpr (G16) {
        uint4 xv[NT][TERMS];
#pragma unroll
        for (int n = 0; n < NT; ++n) x(n, b, xv[n]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (kCentre) {
            centre(2 * b + h);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              subtract(p[i >> 2][(i >> 1) & 1][2 * h + (i & 1)],
                       zc[i >> 2][(i >> 1) & 1]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < TERMS; ++k)
              products(p, h, n, h ? xv[n][k].z : xv[n][k].x,
                       h ? xv[n][k].w : xv[n][k].y);
          }
          flush(2 * b + h);
          clear();
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint4 xv[TERMS];
          x(n, b, xv);
#pragma unroll
          for (int k = 0; k < TERMS; ++k) {
            products(p, 0, n, xv[k].x, xv[k].y);
            products(p, 1, n, xv[k].z, xv[k].w);
          }
        }
      }
      if constexpr (!G16) {
        if ((b + 1) % bpg == 0) {
          flush(b / bpg);
          if (b < 3) clear();
        }
      }
    }
  }
}

// 2^k with the row's largest value (its bits) brought into [2^13, 2^14); the
// exponent is kept in the normal range.
__device__ __forceinline__ float row_scale(uint32_t max_bits) {
  const int e = (int)(max_bits >> 23) - 127;
  return __uint_as_float((uint32_t)(127 + min(13 - e, 126)) << 23);
}
__device__ __forceinline__ float row_unscale(uint32_t max_bits) {
  const int e = (int)(max_bits >> 23) - 127;
  return __uint_as_float((uint32_t)(127 - min(13 - e, 126)) << 23);
}

__device__ __forceinline__ float gated(float g, int act) {
  if (act == TTQ_ACT_SILU) return g / (1.f + expf(-g));
  return 0.5f * g *
         (1.f + tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g)));
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The float at this CTA's shared address `a` in CTA `rank` of the cluster.
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

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ------------------------------------------------------------------ up ---

// Units of 16 intermediate channels (16 gate rows and the 16 rows of the
// other factor) of one entry, taken round robin by a persistent grid; the
// warps split K.
template <int BITS, bool G16, int TERMS, int NTMAX>
__global__ void __launch_bounds__(kThreads, 2)
    up_kernel(const UpArgs a) {
  constexpr int S = kStages<BITS>, kSt = kStage<BITS, G16>;
  constexpr int kRedTiles = NTMAX < 2 ? NTMAX : 2;  // column tiles reduced at once
  extern __shared__ __align__(16) uint8_t sm[];
  Lists l(sm, a.T * a.top_k, a.E);
  float* red =
      reinterpret_cast<float*>(sm + Lists::bytes(a.T * a.top_k, a.E));
  // [warp][row tile][column tile][128]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring =
      smem_u32(red) + kWarps * 2 * kRedTiles * 128 * 4 + warp * S * kSt;

  // ids and the packed weights were complete before the kernel that runs
  // before this one started: lists and the first stages need not wait for it
  build_lists(l, a.ids, nullptr, a.T, a.top_k, a.E, a.err);
  const int tiles = a.I / 16, units = l.entries * tiles;
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const int c0 = warp * chunks / kWarps, c1 = (warp + 1) * chunks / kWarps;
  Packed m;
  m.codes = a.codes;
  m.delta = a.delta;
  m.zero = a.zero;
  m.ldc = codes_ld(a.K, BITS);
  m.ldg = groups_ld(a.K, a.group);
  m.blocks = a.K / 32;
  m.group = a.group;
  const Field<BITS, G16, TERMS == 2> f(lane & 3);

  // the warp's stages: its chunks of the CTA's units, one after the other
  int iu = blockIdx.x, ic = c0, ist = 0;
  auto issue = [&]() {
    if (iu < units && c0 < c1) {
      const int en = iu / tiles, tile = iu - en * tiles;
      const int64_t base =
          (int64_t)l.expert[en] * 2 * a.I + tile * 16;
      issue_stage<BITS, G16>(m, ring + ist * kSt, base, base + a.I, ic, lane);
      if (++ic == c1) {
        ic = c0;
        iu += gridDim.x;
      }
    }
    cp_async_commit();
    ist = ist + 1 == S ? 0 : ist + 1;
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue();
  griddep_enter();

  int cst = 0;
  const int t = lane & 3;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int en = u / tiles, tile = u - en * tiles;
    const int cols = l.cols[en], col0 = l.first[en];
    const int nt = (cols + 7) / 8;
    float acc[2][NTMAX][4];
#pragma unroll
    for (int n = 0; n < NTMAX; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[0][n][i] = acc[1][n][i] = 0.f;
    // this lane's column of each tile; columns past the last repeat column
    // 0, whose results are dropped
    const uint4* xr[NTMAX];
#pragma unroll
    for (int n = 0; n < NTMAX; ++n) {
      const int col = n * 8 + (lane >> 2);
      const int tok = l.slot[col0 + (col < cols ? col : 0)] / a.top_k;
      xr[n] = reinterpret_cast<const uint4*>(a.xhat + (int64_t)tok * a.K) + t;
    }
    const int64_t term = (int64_t)a.T * a.K / 8;  // in uint4
    for (int c = c0; c < c1; ++c) {
      cp_async_wait<S - 2>();
      __syncwarp();  // and every lane is done with the stage before
      issue();
      const uint32_t st = ring + cst * kSt;
      const int nb = min(4, m.blocks - 4 * c);
      auto x = [&](int n, int b, uint4 (&v)[TERMS]) {
#pragma unroll
        for (int k = 0; k < TERMS; ++k)
          v[k] = xr[n][k * term + (c * 4 + b) * 4];
      };
      if (NTMAX == 1 || nt == 1)
        stage_products<BITS, G16, TERMS, 1, NTMAX>(st, f, a.group, c, nb, x,
                                                   acc, lane);
      else if (NTMAX == 2 || nt == 2)
        stage_products<BITS, G16, TERMS, (NTMAX < 2 ? NTMAX : 2), NTMAX>(
            st, f, a.group, c, nb, x, acc, lane);
      else
        stage_products<BITS, G16, TERMS, NTMAX, NTMAX>(st, f, a.group, c, nb,
                                                       x, acc, lane);
      cst = cst + 1 == S ? 0 : cst + 1;
    }
    // add the warps' sums, kRedTiles column tiles at a time
#pragma unroll
    for (int n0 = 0; n0 < NTMAX; n0 += kRedTiles) {
      if (n0 >= nt) break;
      __syncthreads();  // the last round's sums have been read
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int n = 0; n < kRedTiles; ++n)
          *reinterpret_cast<float4*>(
              red + ((warp * 2 + rt) * kRedTiles + n) * 128 + lane * 4) =
              make_float4(acc[rt][n0 + n][0], acc[rt][n0 + n][1],
                          acc[rt][n0 + n][2], acc[rt][n0 + n][3]);
      __syncthreads();
      const int n = tid >> 7, i = tid & 127;
      // element i of a tile: lane i / 4, register i % 4
      const int row = (i >> 4) + 8 * ((i >> 1) & 1);
      const int col = (n0 + n) * 8 + 2 * ((i >> 2) & 3) + (i & 1);
      float hv = 0.f;
      int slot = 0;
      const bool live = n < kRedTiles && col < cols;
      if (live) {
        float gs = 0.f, us = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          gs += red[((w * 2 + 0) * kRedTiles + n) * 128 + i];
          us += red[((w * 2 + 1) * kRedTiles + n) * 128 + i];
        }
        slot = l.slot[col0 + col];
        const float un = row_unscale(a.xmax[slot / a.top_k]);
        const int ch = tile * 16 + row;
        hv = gated(gs * kPerUnit<BITS, TERMS> * un, a.act) * (us * kPerUnit<BITS, TERMS> * un) *
             a.inv_s_mid[(int64_t)l.expert[en] * a.I + ch];
        a.h[(int64_t)slot * a.I + ch] = hv;
      }
      // the slot's largest |h|: rows of one column sit in lanes that differ
      // in bits 1 and 4 (all lanes of a warp hold the same n)
      uint32_t mx = __float_as_uint(hv) & 0x7FFFFFFFu;
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      if (live && (lane & 18) == 0) atomicMax(a.hmax + slot, mx);
    }
  }
  cp_async_wait_all();
}

// ---------------------------------------------------------------- down ---

// 32 output channels per cluster; the (entry, 128-channel chunk) pairs of the
// batch are one list, split evenly over the warps of the cluster's CTAs.
// Every warp keeps the sums of all tokens for its share and adds an entry's
// columns to them when it leaves the entry.
template <int BITS, bool G16, int TERMS, int NTMAX>
__global__ void __launch_bounds__(kThreads, 2)
    down_kernel(const DownArgs a) {
  constexpr int S = kStages<BITS>, kSt = kStage<BITS, G16>;
  extern __shared__ __align__(16) uint8_t sm[];
  Lists l(sm, a.T * a.top_k, a.E);
  float* ysum =  // [warp][T][32]
      reinterpret_cast<float*>(sm + Lists::bytes(a.T * a.top_k, a.E));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int region = a.T * kRows;
  const uint32_t ring = smem_u32(ysum + kWarps * region) + warp * S * kSt;
  float* mine = ysum + warp * region;

  // as in up_kernel: nothing before griddep_enter() reads what the kernel
  // before this one writes
  build_lists(l, a.ids, a.weights, a.T, a.top_k, a.E, nullptr);
  for (int i = lane; i < region; i += 32) mine[i] = 0.f;
  const int chunks = (a.I + kChunk - 1) / kChunk;
  const int total = l.entries * chunks;
  const int ranks = gridDim.y, rank = blockIdx.y;
  const int parts = ranks * kWarps, part = rank * kWarps + warp;
  const int s0 = (int)((int64_t)total * part / parts);
  const int s1 = (int)((int64_t)total * (part + 1) / parts);
  const int n0 = blockIdx.x * kRows;
  Packed m;
  m.codes = a.codes;
  m.delta = a.delta;
  m.zero = a.zero;
  m.ldc = codes_ld(a.I, BITS);
  m.ldg = groups_ld(a.I, a.group);
  m.blocks = a.I / 32;
  m.group = a.group;
  const Field<BITS, G16, TERMS == 2> f(lane & 3);
  int is = s0, ien = s0 / chunks, ic = s0 - ien * chunks, ist = 0;
  auto issue = [&]() {
    if (is < s1) {
      const int64_t base = (int64_t)l.expert[ien] * a.K + n0;
      issue_stage<BITS, G16>(m, ring + ist * kSt, base, base + 16, ic, lane);
      ++is;
      if (++ic == chunks) {
        ic = 0;
        ++ien;
      }
    }
    cp_async_commit();
    ist = ist + 1 == S ? 0 : ist + 1;
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue();
  griddep_enter();

  const int t = lane & 3, g = lane >> 2;
  int s = s0, en = s0 / chunks, c = s0 - en * chunks, cst = 0;
  while (s < s1) {
    const int cols = l.cols[en], col0 = l.first[en];
    const int nt = (cols + 7) / 8;
    float acc[2][NTMAX][4];
#pragma unroll
    for (int n = 0; n < NTMAX; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[0][n][i] = acc[1][n][i] = 0.f;
    const float* hr[NTMAX];
    float sc[NTMAX];
#pragma unroll
    for (int n = 0; n < NTMAX; ++n) {
      const int col = n * 8 + g;
      const int slot = l.slot[col0 + (col < cols ? col : 0)];
      hr[n] = a.h + (int64_t)slot * a.I;
      sc[n] = row_scale(a.hmax[slot]);
    }
    const int stop = min(s1, s + chunks - c);
    for (; s < stop; ++s, ++c) {
      cp_async_wait<S - 2>();
      __syncwarp();  // and every lane is done with the stage before
      issue();
      const uint32_t st = ring + cst * kSt;
      const int nb = min(4, m.blocks - 4 * c);
      auto x = [&](int n, int b, uint4 (&v)[TERMS]) {
        const int at = (c * 4 + b) * 32 + (G16 ? 4 : 8) * t;
        const float4 p = *reinterpret_cast<const float4*>(hr[n] + at);
        const float4 q =
            *reinterpret_cast<const float4*>(hr[n] + at + (G16 ? 16 : 4));
        // in the order of the code pairs
        float e[8];
        if constexpr (G16) {
          e[0] = p.x; e[1] = p.z; e[2] = p.y; e[3] = p.w;
          e[4] = q.x; e[5] = q.z; e[6] = q.y; e[7] = q.w;
        } else {
          e[0] = p.x; e[1] = q.x; e[2] = p.y; e[3] = q.y;
          e[4] = p.z; e[5] = q.z; e[6] = p.w; e[7] = q.w;
        }
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[2 * i] *= sc[n];
          e[2 * i + 1] *= sc[n];
          r[i] = half2_bits(e[2 * i], e[2 * i + 1]);
        }
        v[0] = make_uint4(r[0], r[1], r[2], r[3]);
        if constexpr (TERMS == 2) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float h0, h1;
            f16x2_to_f32(r[i], h0, h1);
            r[i] = half2_bits(e[2 * i] - h0, e[2 * i + 1] - h1);
          }
          v[1] = make_uint4(r[0], r[1], r[2], r[3]);
        }
      };
      if (NTMAX == 1 || nt == 1)
        stage_products<BITS, G16, TERMS, 1, NTMAX>(st, f, a.group, c, nb, x,
                                                   acc, lane);
      else if (NTMAX == 2 || nt == 2)
        stage_products<BITS, G16, TERMS, (NTMAX < 2 ? NTMAX : 2), NTMAX>(
            st, f, a.group, c, nb, x, acc, lane);
      else
        stage_products<BITS, G16, TERMS, NTMAX, NTMAX>(st, f, a.group, c, nb,
                                                       x, acc, lane);
      cst = cst + 1 == S ? 0 : cst + 1;
    }
    // leave the entry: its columns are different tokens
#pragma unroll
    for (int n = 0; n < NTMAX; ++n) {
      if (n >= nt) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = n * 8 + 2 * t + i;
        if (col < cols) {
          const int slot = l.slot[col0 + col];
          const float w =
              l.weight[col0 + col] * row_unscale(a.hmax[slot]) * kPerUnit<BITS, TERMS>;
          float* y = mine + slot / a.top_k * kRows + g;
          y[0] = fmaf(w, acc[0][n][i], y[0]);
          y[8] = fmaf(w, acc[0][n][2 + i], y[8]);
          y[16] = fmaf(w, acc[1][n][i], y[16]);
          y[24] = fmaf(w, acc[1][n][2 + i], y[24]);
        }
      }
    }
    __syncwarp();
    ++en;
    c = 0;
  }
  cp_async_wait_all();
  __syncthreads();
  // add the warps' sums, then the CTAs' through distributed shared memory,
  // both in order
  for (int i = tid; i < region; i += kThreads) {
    float v = ysum[i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v += ysum[w * region + i];
    ysum[i] = v;
  }
  if (ranks > 1) cluster_sync(); else __syncthreads();
  const uint32_t ys = smem_u32(ysum);
  for (int i = rank * kThreads + tid; i < region; i += ranks * kThreads) {
    float v = 0.f;
    if (ranks > 1) {
      for (int r = 0; r < ranks; ++r) v += ld_cluster_f32(ys + i * 4, r);
    } else {
      v = ysum[i];
    }
    const int64_t at = (int64_t)(i / kRows) * a.ldy + n0 + i % kRows;
    if constexpr (TERMS == 1) {
      static_cast<__nv_bfloat16*>(a.Y)[at] = __float2bfloat16_rn(v);
    } else {
      if (a.yt == TTQ_F16)
        static_cast<__half*>(a.Y)[at] = __float2half_rn(v);
      else
        static_cast<float*>(a.Y)[at] = v;
    }
  }
  if (ranks > 1) cluster_sync();
}

// -------------------------------------------------------------- launch ---

template <int BITS, bool G16>
size_t up_smem(int ntmax, int n, int E) {
  return Lists::bytes(n, E) + (size_t)kWarps * 2 * std::min(ntmax, 2) * 128 * 4 +
         (size_t)kWarps * kStages<BITS> * kStage<BITS, G16>;
}
template <int BITS, bool G16>
size_t down_smem(int T, int n, int E) {
  return Lists::bytes(n, E) + (size_t)kWarps * T * kRows * 4 +
         (size_t)kWarps * kStages<BITS> * kStage<BITS, G16>;
}

template <typename K>
bool allow_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute(kern,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)bytes) == cudaSuccess;
}

template <int BITS, bool G16, int TERMS, int NTMAX>
ttq_status launch_pair(const UpArgs& u, const DownArgs& d, cudaStream_t st) {
  LaunchShape ls;
  ls.block = dim3(kThreads);
  ls.smem = up_smem<BITS, G16>(NTMAX, u.T * u.top_k, u.E);
  const int64_t per_sm = ls.smem + 1024 <= 114 * 1024 ? 2 : 1;
  const int64_t units =
      (int64_t)Lists::max_entries(u.T * u.top_k, u.E) * (u.I / 16);
  ls.grid = dim3((unsigned)std::min<int64_t>(units, per_sm * sm_count()));
  auto up = up_kernel<BITS, G16, TERMS, NTMAX>;
  if (!allow_smem(up, ls.smem)) return TTQ_ERR_CUDA;
  const ttq_status s = launch(ls, st, up, u);
  if (s != TTQ_OK) return s;
  LaunchShape ld;
  ld.block = dim3(kThreads);
  ld.smem = down_smem<BITS, G16>(d.T, d.T * d.top_k, d.E);
  const int tiles = (int)(d.K / kRows);
  const int slots = (ld.smem + 1024 <= 114 * 1024 ? 2 : 1) * sm_count();
  const int ranks = std::max(1, std::min(8, slots / tiles));
  ld.grid = dim3((unsigned)tiles, (unsigned)ranks);
  ld.cluster_y = (unsigned)ranks;
  auto down = down_kernel<BITS, G16, TERMS, NTMAX>;
  if (!allow_smem(down, ld.smem)) return TTQ_ERR_CUDA;
  return launch(ld, st, down, d);
}

// TERMS: one fp16 term of the activations carries a bf16 output, two an fp16
// or fp32 one. NTMAX: up to 8 tokens fill one column tile; more may put up to
// 32 on one expert, which wants four.
template <int BITS>
ttq_status launch_bits(const UpArgs& u, const DownArgs& d, cudaStream_t st) {
  auto go = [&](auto g16) -> ttq_status {
    constexpr bool G = decltype(g16)::value;
    if (d.yt == TTQ_BF16)
      return u.T <= 8 ? launch_pair<BITS, G, 1, 1>(u, d, st)
                      : launch_pair<BITS, G, 1, 4>(u, d, st);
    return u.T <= 8 ? launch_pair<BITS, G, 2, 1>(u, d, st)
                    : launch_pair<BITS, G, 2, 4>(u, d, st);
  };
  return u.group == 16 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace moe
}  // namespace ttq
