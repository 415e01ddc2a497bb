// moe_tile.cuh — the expert kernels of ttq_moe_lowbit for one code width
// (moe_b2.cu .. moe_b8.cu instantiate them; moe.cu launches).
//
// An expert meets a handful of tokens per step, so its packed weights are
// read once from HBM and used for a few products each: the kernels are bound
// by those bytes, and by the instructions that unpack them. Per warp:
//   - mma.sync m16n8k16 with 16 weight rows as M, up to 16 tokens as N (1 or 2
//     tiles of 8). tcgen05 would want 128 rows per tile and the weights
//     copied to TMEM or shared memory after unpacking; here an unpacked code
//     pair goes from the register it was masked in straight into the MMA.
//   - A code q enters as an fp16 bit pattern, the subnormal q 2^(P-24) for a
//     code at bit P: one AND isolates two codes and is all the conversion
//     there is. Codes are used at several P without a shift; the activations
//     that meet them carry 2^(Pmax-P) (Positions). Per group,
//       acc += D (sum q x) - (D z) (sum x),
//     D in fp32; the second product runs over the groups as a contraction of
//     its own, tf32 MMAs of 4 groups each, with the groups' sums of x made once
//     with the activations. (As fused multiply-adds on the accumulators it
//     took 22 instructions per group, a fifth of all at groups of 32.)
//     2^(24-Pmax) and the row's power of two return in the epilogue.
//   - The contraction order inside a 32-code block is free as long as both
//     operands agree: lane t of a quad owns codes 8t..8t+7 (for groups of 16:
//     4t..4t+3 of both halves), which are consecutive bits of one word (4
//     bits) or of two or three, and the activations are stored in that order.
//   - Codes, delta and zero of 32 rows x 128 channels arrive by cp.async in a
//     ring of stages of the warp's own; warps never wait for one another
//     inside the contraction.
#pragma once

#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "moe.h"
#include "moe_rows.cuh"

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
constexpr int kStage = kRows * kPitch<BITS>;
// delta and zero of the rows for 4 groups (8 of 16 channels): a piece
template <bool G16>
constexpr int kPieceDelta = G16 ? 32 : 16;
template <bool G16>
constexpr int kPiece = kRows * (kPieceDelta<G16> + kPieceDelta<G16> / 4);
// Stages per warp: what lets two CTAs of 8 warps share an SM. As many pieces:
// a stage needs at most one new one.
// Two are enough beside 16 columns (three: 131 against 120 us for 16 tokens,
// 32 experts of 2560 x 1728 at 3 bits), and leave the rest to L1.
template <int BITS, int NTMAX>
constexpr int kStages = BITS <= 3 ? (NTMAX == 1 ? 5 : 3)
                        : BITS <= 5 && NTMAX == 1 ? 3 : 2;
template <int BITS, bool G16, int NTMAX>
constexpr int kRing = kStages<BITS, NTMAX> * (kStage<BITS> + kPiece<G16>);
// Where the rows a CTA converts itself start: after the rings, which start at
// byte `ring`.
template <int BITS, bool G16, int NTMAX>
constexpr int smem_rows(int ring) {
  return ring + 8 * kRing<BITS, G16, NTMAX>;
}

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
  uint8_t* token;      // [n] and their tokens
  int16_t* expert;     // [entries] of an entry: expert, first column, columns
  int16_t* first;
  int16_t* cols;
  int* sums;           // [2 kWarps + 1] of the scans; the last: any choice twice
  int entries;

  static __host__ __device__ int max_entries(int n, int E) {
    return (n < E ? n : E) + n / kMaxCols;
  }
  static __host__ __device__ size_t bytes(int n, int E) {
    const size_t b = (size_t)E * 12 + (size_t)n * 7 +
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
    token = reinterpret_cast<uint8_t*>(cols + m);
  }
};

__device__ __forceinline__ void build_lists(Lists& l, const int32_t* ids,
                                            const float* weights, int T,
                                            int top_k, int E, uint32_t* err) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = T * top_k;
  if (n <= 32) {
    // one choice per lane: every warp finds the groups by matching, the first
    // writes them
    const int e = lane < n ? ids[lane] : -1, t = lane / top_k;
    float w = weights && lane < n ? weights[lane] : 0.f;
    if (e >= E && err && blockIdx.x == 0) flag_error(err, TTQ_DEVERR_INDEX);
    const bool valid = e >= 0 && e < E;
    const unsigned same = __match_any_sync(0xffffffffu, valid ? e : -1);
    const unsigned below = (1u << lane) - 1u;
    const unsigned token =
        (top_k == 32 ? 0xffffffffu : (1u << top_k) - 1u) << (t * top_k);
    // the first of a token's equal choices stands for all of them
    const unsigned mine = same & token;
    const bool first = valid && (mine & below) == 0;
    const float w0 = w;
    if (__any_sync(0xffffffffu, valid && mine != (1u << lane))) {
      w = 0.f;
      for (int q = 0; q < 32; ++q) {
        const float v = __shfl_sync(0xffffffffu, w0, q);
        if (mine >> q & 1) w += v;
      }
    }
    const unsigned firsts = __ballot_sync(0xffffffffu, first);
    const unsigned cols = same & firsts;  // the expert's columns
    const bool leads = first && (cols & below) == 0;
    const unsigned leaders = __ballot_sync(0xffffffffu, leads);
    // columns of the experts led by lower lanes
    int at = leads ? __popc(cols) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += v;
    }
    const int start = at - __popc(cols);  // of the leader's own
    const int lead = cols ? __ffs(cols) - 1 : 0;
    const int from = __shfl_sync(0xffffffffu, start, lead);
    l.entries = __popc(leaders);
    if (warp == 0) {
      if (first) {
        const int c = from + __popc(cols & below);
        l.slot[c] = (uint16_t)lane;
        l.token[c] = (uint8_t)t;
        l.weight[c] = w;
      }
      if (leads) {
        const int i = __popc(leaders & below);
        l.expert[i] = (int16_t)e;
        l.first[i] = (int16_t)start;
        l.cols[i] = (int16_t)__popc(cols);
      }
    }
    __syncthreads();
    return;
  }
  for (int e = tid; e < E; e += kThreads) l.tokens[e] = make_uint2(0, 0);
  if (tid == 0) l.sums[2 * kWarps] = 0;
  __syncthreads();
  for (int p = tid; p < n; p += kThreads) {
    const int e = ids[p], t = p / top_k;
    if (e >= E && err && blockIdx.x == 0) flag_error(err, TTQ_DEVERR_INDEX);
    if (e >= 0 && e < E) {
      const unsigned bit = 1u << (t & 31);
      if (atomicOr(t < 32 ? &l.tokens[e].x : &l.tokens[e].y, bit) & bit)
        l.sums[2 * kWarps] = 1;
    }
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
    bool ok = e >= 0 && e < E;
    float w = weights ? weights[p] : 0.f;
    if (l.sums[2 * kWarps]) {  // the first of equal choices stands for all
      for (int q = t * top_k; ok && q < p; ++q) ok = ids[q] != e;
      if (ok && weights)
        for (int q = p + 1; q < last; ++q)
          if (ids[q] == e) w += weights[q];
    }
    if (!ok) continue;
    const uint2 m = l.tokens[e];
    const unsigned below = (1u << (t & 31)) - 1u;
    const int at = l.start[e] + (t < 32 ? __popc(m.x & below)
                                        : __popc(m.x) + __popc(m.y & below));
    l.slot[at] = (uint16_t)p;
    l.weight[at] = w;
    l.token[at] = (uint8_t)t;
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

// The packed matrices of one side of the experts, rows of 32 `blocks`
// channels.
struct Packed {
  const uint32_t* codes;
  const float* delta;
  const uint8_t* zero;
  int ldc, ldg;   // words, entries
  int blocks;
  int lg;         // blocks per group = 1 << lg (groups of 32, 64, 128)

  __device__ __forceinline__ Packed(const uint32_t* codes_,
                                    const float* delta_, const uint8_t* zero_,
                                    int K, int bits, int group)
      : codes(codes_), delta(delta_), zero(zero_),
        ldc((int)codes_ld(K, bits)), ldg((int)groups_ld(K, group)),
        blocks(K / 32), lg(group == 128 ? 2 : group == 64 ? 1 : 0) {}
  // Whether chunk c starts a piece of 4 groups (for groups of 16, 8: always).
  __device__ __forceinline__ bool new_piece(int c) const {
    return (c & ((1 << lg) - 1)) == 0;
  }
};

// A lane's share of the copies of 32 rows: the tile's rows 0..15 are
// consecutive matrix rows, 16..31 start `skip` rows after the first. Offsets
// are bytes from the tile's first row; an expert's matrix is below 2^31 bytes.
template <int BITS, bool G16, int S>
struct Stream {
  uint32_t code_off[BITS];  // the lane's 16-byte pieces of the codes
  uint32_t row_off;         // entries from the first row to the lane's row
  const uint8_t* codes;     // of the tile's first row, at the next chunk
  const float* delta;       // of the lane's row
  const uint8_t* zero;
  int c;                    // the next chunk
  int stage, piece;         // ring positions of the next copies
  bool fresh;               // the next chunk is the tile's first

  __device__ __forceinline__ Stream(const Packed& m, int skip, int lane)
      : stage(0), piece(0), fresh(true) {
#pragma unroll
    for (int i = 0; i < BITS; ++i) {
      const int p = lane + 32 * i, r = p / BITS;
      code_off[i] =
          (uint32_t)(r < 16 ? r : skip + r - 16) * (uint32_t)m.ldc * 4u +
          (uint32_t)(p % BITS) * 16u;
    }
    row_off = (uint32_t)(lane < 16 ? lane : skip + lane - 16) *
              (uint32_t)m.ldg;
  }
  // To chunk c0 of the tile whose first matrix row is `row`.
  __device__ __forceinline__ void seek(const Packed& m, int64_t row, int c0) {
    codes = reinterpret_cast<const uint8_t*>(m.codes + row * m.ldc) +
            (int64_t)c0 * (16 * BITS);
    delta = m.delta + row * m.ldg + row_off;
    zero = m.zero + row * m.ldg + row_off;
    c = c0;
    fresh = true;
  }
  // Issues the copies of the next chunk and moves on.
  __device__ __forceinline__ void copy(const Packed& m, uint32_t ring,
                                       int lane) {
    const uint32_t dst = ring + stage * kStage<BITS>;
    const int left = m.ldc - c * (4 * BITS);  // words of the row from here
    if (left >= 4 * BITS) {
#pragma unroll
      for (int i = 0; i < BITS; ++i) {
        const int p = lane + 32 * i;
        cp_async_16(dst + p / BITS * kPitch<BITS> + p % BITS * 16,
                    codes + code_off[i]);
      }
    } else {  // the row ends inside the chunk
#pragma unroll
      for (int i = 0; i < BITS; ++i) {
        const int p = lane + 32 * i;
        if (p % BITS * 4 < left)
          cp_async_16(dst + p / BITS * kPitch<BITS> + p % BITS * 16,
                      codes + code_off[i]);
      }
    }
    // The pitch of delta and zero is a multiple of 16 entries: a piece is
    // always there.
    if (fresh || m.new_piece(c)) {
      constexpr int kD = kPieceDelta<G16>;
      const uint32_t dd = ring + S * kStage<BITS> + piece * kPiece<G16>;
      if constexpr (G16) {
        cp_async_16(dd + lane * kD, delta + c * 8);
        cp_async_16(dd + lane * kD + 16, delta + c * 8 + 4);
        cp_async_ca<8>(dd + kRows * kD + lane * 8, zero + c * 8);
      } else {
        const int q = (c >> m.lg) * 4;
        cp_async_16(dd + lane * kD, delta + q);
        cp_async_ca<4>(dd + kRows * kD + lane * 4, zero + q);
      }
      piece = piece + 1 == S ? 0 : piece + 1;
      fresh = false;
    }
    codes += 16 * BITS;
    ++c;
  }
  __device__ __forceinline__ void advance() {
    stage = stage + 1 == S ? 0 : stage + 1;
  }
};

// ----------------------------------------------------------- unpacking ---

__device__ __forceinline__ uint32_t word(const uint8_t* p) {
  return *reinterpret_cast<const uint32_t*>(p);
}

template <int BITS>
constexpr uint32_t kMask = ((1u << BITS) - 1u) * 0x10001u;

// The code pair I of a lane's block, from `m` whose halves hold the fields'
// codes from bit FROM on. NORM: as 1024 + q, from which the caller takes
// 1024 + z. Otherwise the subnormal at Positions' bit.
template <int BITS, bool G16, bool NORM, int I, int FROM>
__device__ __forceinline__ uint32_t pair_at(uint32_t m) {
  if constexpr (NORM) return ((m >> FROM) & kMask<BITS>) | 0x64006400u;
  constexpr int to = Positions<BITS, G16>::at(I);
  static_assert(to <= FROM, "codes move down");
  return (m >> (FROM - to)) & (kMask<BITS> << to);
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
  template <int I, int FROM>
  static __device__ __forceinline__ uint32_t pair(uint32_t m) {
    return pair_at<BITS, G16, NORM, I, FROM>(m);
  }
  // p[0], p[1] feed the block's first MMA, p[2], p[3] its second.
  __device__ __forceinline__ void codes(const uint8_t* at,
                                        uint32_t (&p)[4]) const {
    if constexpr (G16) {
      // pairs (0, 2), (1, 3) of each half's four codes
      uint32_t u = word(at + w0), v = word(at + w2);
      if constexpr (BITS != 8) {
        u = __funnelshift_r(u, word(at + w1), sh);
        v = __funnelshift_r(v, word(at + w3), sh2);
      }
      const uint32_t m = __byte_perm(u, u >> (2 * BITS), 0x5410);
      const uint32_t n = __byte_perm(v, v >> (2 * BITS), 0x5410);
      p[0] = pair<0, 0>(m);
      p[1] = pair<1, BITS>(m);
      p[2] = pair<2, 0>(n);
      p[3] = pair<3, BITS>(n);
    } else {
      // u: codes 0..3, v: codes 4..7 from bit 0 on; pairs (i, i + 4)
      uint32_t u, v;
      if constexpr (BITS == 2) {
        u = word(at + w0) >> sh;
        v = u >> 8;
      } else if constexpr (BITS == 3) {
        u = __funnelshift_r(word(at + w0), word(at + w1), sh);
        v = u >> 12;
      } else if constexpr (BITS == 4) {
        u = word(at + w0);
        v = u >> 16;
      } else if constexpr (BITS == 8) {
        u = word(at + w0);
        v = word(at + w1);
      } else {
        const uint32_t a = word(at + w0), b = word(at + w1);
        u = __funnelshift_r(a, b, sh);
        const uint32_t hi = BITS == 7 ? __funnelshift_r(b, word(at + w2), sh)
                                      : b >> sh;
        v = __funnelshift_r(u, hi, 4 * BITS);
      }
      const uint32_t m = BITS == 4 ? u : __byte_perm(u, v, 0x5410);
      p[0] = pair<0, 0>(m);
      p[1] = pair<1, BITS>(m);
      if constexpr (BITS <= 4) {
        p[2] = pair<2, 2 * BITS>(m);
        p[3] = pair<3, 3 * BITS>(m);
      } else {
        const uint32_t n =
            BITS == 8 ? __byte_perm(u, v, 0x7632)
                      : __byte_perm(u >> (2 * BITS), v >> (2 * BITS), 0x5410);
        p[2] = pair<2, 0>(n);
        p[3] = pair<3, BITS>(n);
      }
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

// The same from a zero accumulator: no registers to clear first.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0,
                                              uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Two tf32 contractions over 4 positions each: a0, a1 (rows g, g + 8) with b0
// and a2, a3 with b1.
__device__ __forceinline__ void mma_tf32(float (&c)[4], float a0, float a1,
                                         float a2, float a3, float b0,
                                         float b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)),
        "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
        "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}
// The first 11 bits of v, which tf32 holds; the MMA cuts the rest of what it
// is given in the same way.
__device__ __forceinline__ float tf32_head(float v) {
  return __uint_as_float(__float_as_uint(v) & 0xFFFFE000u);
}

// What the kernels do with the activations' precision.
//   kOne: one fp16 term (11 bits), for a bf16 Y (8 bits).
//   kTwo: two fp16 terms (22 bits), for an fp16 Y.
//   kExact: two terms, and z taken from the codes before the MMA, with the
//     codes as normal numbers, for an fp32 Y: subnormal operands are not
//     normalised before the tensor core lines its products up, which costs up
//     to 10 - b bits of the sum (measured: 5e-5 relative error for 2-bit codes
//     at bit 0), and sum q x and z sum x cancel by a few bits more.
enum Mode { kOne = 1, kTwo = 2, kExact = 3 };

template <int MODE>
constexpr int kTerms = MODE == kOne ? 1 : 2;

// what a code's unit is in the accumulators
template <int BITS, bool G16, int MODE>
constexpr float kUnit =
    MODE == kExact
        ? 1.f
        : (float)(1 << Positions<BITS, G16>::kMost) / 16777216.f;

__device__ __forceinline__ void subtract(uint32_t& p, __half2 z) {
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&p), z);
  p = *reinterpret_cast<const uint32_t*>(&d);
}

// One stage's products into acc[row tile][column tile]. st: the stage's codes,
// dd: its piece of delta and zero, j0: the stage's first group in it. LG: as
// Packed::lg. FULL: the stage has 4 blocks (no branch then keeps the blocks'
// instructions apart), otherwise nblocks. xp[n] (and xp[n] + term for the
// second term) points at the lane's activations of the stage: 16 bytes per
// 32-channel block, 64 bytes apart, .x and .y for the block's first MMA, .z
// and .w for its second. x holds those of the next DEPTH blocks and is refilled
// as it is used, across stages, while there are blocks (`more` from the
// stage's first on): they come from L1 or L2, further away than a block of
// instructions.
template <int BITS, bool G16, int LG, bool FULL, int MODE, int NT, int NTMAX,
          int DEPTH>
__device__ __forceinline__ void stage_products(
    const uint8_t* st, const uint8_t* dd, int j0,
    const Field<BITS, G16, MODE == kExact>& f, int nblocks,
    const uint4* const (&xp)[NTMAX], int64_t term,
    int more, uint4 (&x)[DEPTH][NT][kTerms<MODE>],
    float (&acc)[2][NTMAX][4], int lane) {
  constexpr int TERMS = kTerms<MODE>;
  constexpr bool kCentre = MODE == kExact;
  constexpr int kD = kPieceDelta<G16>;
  const int g = lane >> 2;
  st += g * kPitch<BITS>;
  const uint8_t* dp = dd + g * kD + j0 * 4;
  const uint8_t* zp = dd + kRows * kD + g * (kD / 4) + j0;
  float cc[2][NT][4];
  __half2 zc[2][2];
  // row i * 8 + g of the tile, group j of the stage
  auto zero_at = [&](int i, int j) -> uint32_t {
    return zp[i * 8 * (kD / 4) + j];
  };
  auto delta_at = [&](int i, int j) -> float {
    return __uint_as_float(word(dp + i * 8 * kD + j * 4));
  };
  auto centre = [&](int j) {
    if constexpr (kCentre) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t z = (0x6400u | zero_at(i, j)) * 0x10001u;
        zc[i >> 1][i & 1] = *reinterpret_cast<const __half2*>(&z);
      }
    }
  };
  // acc += D c for group j of the stage
  auto flush = [&](int j) {
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      const float d0 = delta_at(2 * rt, j), d1 = delta_at(2 * rt + 1, j);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[rt][n][0] = fmaf(d0, cc[rt][n][0], acc[rt][n][0]);
        acc[rt][n][1] = fmaf(d0, cc[rt][n][1], acc[rt][n][1]);
        acc[rt][n][2] = fmaf(d1, cc[rt][n][2], acc[rt][n][2]);
        acc[rt][n][3] = fmaf(d1, cc[rt][n][3], acc[rt][n][3]);
      }
    }
  };
  // first: the group's first MMA
  auto products = [&](const uint32_t (&p)[2][2][4], int h, int n, uint32_t b0,
                      uint32_t b1, bool first) {
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      if (first)
        mma_f16_first(cc[rt][n], p[rt][0][2 * h], p[rt][1][2 * h],
                      p[rt][0][2 * h + 1], p[rt][1][2 * h + 1], b0, b1);
      else
        mma_f16(cc[rt][n], p[rt][0][2 * h], p[rt][1][2 * h],
                p[rt][0][2 * h + 1], p[rt][1][2 * h + 1], b0, b1);
    }
  };
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (FULL || b < nblocks) {
      uint4(&xv)[NT][TERMS] = x[b % DEPTH];
      uint32_t p[2][2][4];  // [row tile][row g, row g + 8][pair]
      if (!G16 && (b & ((1 << LG) - 1)) == 0) centre(b >> LG);
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        const uint8_t* at = st + rt * 16 * kPitch<BITS> + b * (4 * BITS);
        f.codes(at, p[rt][0]);
        f.codes(at + 8 * kPitch<BITS>, p[rt][1]);
        if constexpr (kCentre && !G16) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            subtract(p[rt][i >> 2][i & 3], zc[rt][i >> 2]);
        }
      }
      if constexpr (G16) {
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
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < TERMS; ++k)
              products(p, h, n, h ? xv[n][k].z : xv[n][k].x,
                       h ? xv[n][k].w : xv[n][k].y, k == 0);
          flush(2 * b + h);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < TERMS; ++k)
              products(p, h, n, h ? xv[n][k].z : xv[n][k].x,
                       h ? xv[n][k].w : xv[n][k].y,
                       h == 0 && k == 0 && (b & ((1 << LG) - 1)) == 0);
        if (((b + 1) & ((1 << LG) - 1)) == 0) flush(b >> LG);
      }
      if (b + DEPTH < more) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < TERMS; ++k)
            xv[n][k] = xp[n][k * term + (b + DEPTH) * 4];
      }
    }
  }
}

// acc -= (D z) (sum x), both factors in two tf32 terms (z is several times the
// spread of the codes around it: one term of 11 bits cost a bf16 Y 5e-3), for
// the groups of a piece (dd) that the warp contracts:
// group g0 + t (for groups of 16: g0 + 2t and g0 + 2t + 1) of lane (g, t) if
// it is in [lo, hi); g0 + j1 is one that is. sp[n]: column g's sums.
template <int BITS, bool G16, int MODE, int NT, int NTMAX>
__device__ __forceinline__ void zero_products(const uint8_t* dd, int g0,
                                              int j1, int lo, int hi,
                                              const float* const (&sp)[NTMAX],
                                              float (&acc)[2][NTMAX][4],
                                              int lane) {
  constexpr int kD = kPieceDelta<G16>, kPer = G16 ? 2 : 1;
  constexpr float u = kUnit<BITS, G16, MODE>;
  const int g = lane >> 2;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = (lane & 3) * kPer + i;
    const bool mine = g0 + at >= lo && g0 + at < hi;
    const int j = mine ? at : j1;  // what lies outside may not be a number
    const uint8_t* dp = dd + g * kD + j * 4;
    const uint8_t* zp = dd + kRows * kD + g * (kD / 4) + j;
    float a[4], b[4];  // -D z in units of rows g, g + 8, ..: head, tail
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      // -z in units: 2^23 + z by one OR, and one exact fused multiply-add
      const float z =
          fmaf(__uint_as_float(0x4B000000u | zp[r * 8 * (kD / 4)]), -u,
               8388608.f * u);
      const float v = __uint_as_float(word(dp + r * 8 * kD)) * z;
      a[r] = tf32_head(v);
      b[r] = v - a[r];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float s = mine ? sp[n][g0 + j] : 0.f;
      const float s0 = tf32_head(s), s1 = s - s0;
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        mma_tf32(acc[rt][n], a[2 * rt], a[2 * rt + 1], b[2 * rt],
                 b[2 * rt + 1], s0, s0);
        mma_tf32(acc[rt][n], a[2 * rt], a[2 * rt + 1], b[2 * rt],
                 b[2 * rt + 1], s1, s1);
      }
    }
  }
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

// 2^-k of the scale the rows carry (rows_kernel in moe.cu).
__device__ __forceinline__ float row_unscale(uint32_t max_bits, int most) {
  return __uint_as_float((uint32_t)(127 - row_exponent(max_bits, most)) << 23);
}

// One warp's walk through its stages: activation rows, products.
template <int BITS, bool G16, int MODE, int NTMAX>
struct Tile {
  static constexpr int TERMS = kTerms<MODE>;
  static constexpr int S = kStages<BITS, NTMAX>;
  const Field<BITS, G16, MODE == kExact> f;
  const uint8_t* ring;
  int lane, nt;
  int stage, piece;        // ring positions of the next ones
  bool fresh;
  const uint8_t* dd;       // the last piece
  const uint4* xp[NTMAX];  // the lane's activations at the next stage
  const float* sp[NTMAX];  // its column's group sums
  int64_t term;
  float acc[2][NTMAX][4];

  __device__ __forceinline__ Tile(const uint8_t* ring_, int lane_,
                                  int64_t term_)
      : f(lane_ & 3), ring(ring_), lane(lane_), stage(0), piece(0),
        term(term_) {}

  // Starts a tile with `cols` columns at chunk c; row(col) gives a column's
  // row of the activations x and their group sums (columns past the last
  // repeat column 0: their results are dropped).
  template <typename RF>
  __device__ __forceinline__ void start(const Packed& m, const uint4* x,
                                        const float* sum, int cols, int c,
                                        RF&& row) {
    nt = (cols + 7) / 8;
    fresh = true;
#pragma unroll
    for (int n = 0; n < NTMAX; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[0][n][i] = acc[1][n][i] = 0.f;
      const int col = n * 8 + (lane >> 2);
      const int64_t r = row(col < cols ? col : 0);
      xp[n] = x + r * (m.blocks * 4) + c * 16 + (lane & 3);
      sp[n] = sum + r * m.ldg;
    }
  }
  // Chunks c .. c_end - 1; next() issues the copies that refill the ring.
  template <int LG, int NT, typename NF>
  __device__ __forceinline__ void run_nt(const Packed& m, int c, int c_end,
                                         NF&& next) {
    constexpr int kPer = G16 ? 8 : 4 >> LG;  // groups per chunk
    const int lo = c * kPer;
    const int hi = min(c_end * kPer, G16 ? m.blocks * 2 : m.blocks >> LG);
    // blocks of activations in flight: what the registers hold
    constexpr int DEPTH = NT * TERMS <= 2 ? 2 : 1;
    const int last = min(c_end * 4, m.blocks);
    uint4 x[DEPTH][NT][TERMS];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < TERMS; ++k)
          x[d][n][k] = 4 * c + d < last ? xp[n][k * term + d * 4]
                                        : make_uint4(0, 0, 0, 0);
    for (; c < c_end; ++c) {
      cp_async_wait<S - 1>();
      __syncwarp();  // every lane's part of the stage is there
      if (fresh || m.new_piece(c)) {
        dd = ring + S * kStage<BITS> + piece * kPiece<G16>;
        piece = piece + 1 == S ? 0 : piece + 1;
        fresh = false;
        if constexpr (MODE != kExact)
          zero_products<BITS, G16, MODE, NT, NTMAX>(
              dd, G16 ? c * 8 : (c >> LG) * 4, G16 ? 0 : (c * (4 >> LG)) & 3,
              lo, hi, sp, acc, lane);
      }
      const uint8_t* st = ring + stage * kStage<BITS>;
      const int j0 = G16 ? 0 : (c * (4 >> LG)) & 3;
      const int nb = m.blocks - 4 * c;
      if (nb >= 4)
        stage_products<BITS, G16, LG, true, MODE, NT, NTMAX, DEPTH>(
            st, dd, j0, f, 4, xp, term, last - 4 * c, x, acc, lane);
      else
        stage_products<BITS, G16, LG, false, MODE, NT, NTMAX, DEPTH>(
            st, dd, j0, f, nb, xp, term, last - 4 * c, x, acc, lane);
#pragma unroll
      for (int n = 0; n < NT; ++n) xp[n] += 16;
      stage = stage + 1 == S ? 0 : stage + 1;
      __syncwarp();  // every lane has left the stage
      next();
    }
  }
  template <int LG, typename NF>
  __device__ __forceinline__ void run(const Packed& m, int c, int c_end,
                                      NF&& next) {
    if (NTMAX == 1 || nt == 1)
      run_nt<LG, 1>(m, c, c_end, next);
    else
      run_nt<LG, NTMAX>(m, c, c_end, next);
  }
};

// ------------------------------------------------------------------ up ---

// A tile is 16 intermediate channels of an entry: their 16 gate rows and the
// 16 rows of the other factor, which end in the same lanes and registers. A CTA
// of the persistent grid takes an even share of consecutive tiles. Rounds of 8
// tiles, one per warp, come first: the warps are then at about the same
// channels of the same tokens and share their activations through L1. What is
// left (fewer than 8 tiles) is cut into 8 even runs of chunks: a warp that
// starts a tile and does not end it adds what the warps after it contracted
// (through shared memory, in order). So all warps do the same number of steps
// whatever the number of tiles, and one barrier joins them.
template <int BITS, bool G16, int LG, int MODE, int NTMAX, bool LOCAL>
__global__ void __launch_bounds__(kThreads, 2)
    up_kernel(const UpArgs a) {
  using TileT = Tile<BITS, G16, MODE, NTMAX>;
  constexpr int S = TileT::S;
  extern __shared__ __align__(16) uint8_t sm[];
  Lists l(sm, a.T * a.top_k, a.E);
  float* red =  // [warp][row tile][column tile][128]: what ends a tile
      reinterpret_cast<float*>(sm + Lists::bytes(a.T * a.top_k, a.E));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint8_t* ring = reinterpret_cast<const uint8_t*>(
                            red + kWarps * 2 * NTMAX * 128) +
                        warp * kRing<BITS, G16, NTMAX>;
  const uint32_t ring_at = smem_u32(ring);

  // Behind rows_kernel, ids and the packed weights were complete before that
  // kernel let this one start: lists and the first stages need not wait for
  // it. With LOCAL this is the call's first kernel, and whatever runs before it
  // (the router, the quantizer) may still be writing them.
  if constexpr (LOCAL) griddep_enter();
  build_lists(l, a.ids, nullptr, a.T, a.top_k, a.E, a.err);
  const int tiles = a.I / 16;  // of an entry
  const int chunks = (a.K + kChunk - 1) / kChunk;
  // the CTA's tiles t0 .. (the first `rest` CTAs take one more) and steps
  const unsigned all = (unsigned)l.entries * tiles;
  const unsigned each = all / gridDim.x, rest = all - each * gridDim.x;
  const unsigned t0 = each * blockIdx.x + min(blockIdx.x, rest);
  const int mine = each + (blockIdx.x < rest ? 1 : 0);
  const int rounds = mine / kWarps;
  // the runs: steps of the tiles from t1 on
  const unsigned t1 = t0 + rounds * kWarps;
  const unsigned steps = (mine - rounds * kWarps) * chunks;
  auto share = [&](int w) { return (int)(steps * w / kWarps); };
  const int s0 = share(warp), s1 = share(warp + 1);
  const Packed m(a.codes, a.delta, a.zero, a.K, BITS, a.group);
  Stream<BITS, G16, S> w(m, a.I, lane);

  int iround = 0, left = s1 - s0;
  unsigned itile = 0;  // of the whole list
  auto seek = [&](int c) {
    const unsigned en = itile / (unsigned)tiles;
    w.seek(m, (int64_t)l.expert[en] * 2 * a.I + (itile - en * tiles) * 16, c);
  };
  auto seek_first = [&]() {  // of a round, or of the run
    if (iround < rounds) {
      itile = t0 + iround * kWarps + warp;
      seek(0);
    } else if (left > 0) {
      const unsigned q = s0 / chunks;
      itile = t1 + q;
      seek(s0 - q * chunks);
    }
  };
  seek_first();
  auto issue = [&]() {
    if (iround < rounds) {
      w.copy(m, ring_at, lane);
      if (w.c == chunks) {
        ++iround;
        seek_first();
      }
    } else if (left > 0) {
      w.copy(m, ring_at, lane);
      if (--left > 0 && w.c == chunks) {
        ++itile;
        seek(0);
      }
    }
    cp_async_commit();
    w.advance();
  };
#pragma unroll
  for (int i = 0; i < S; ++i) issue();
  if constexpr (!LOCAL) griddep_enter();

  const uint4* xhat = a.xhat;
  const float* xsum = a.xsum;
  const uint32_t* xmax = a.xmax;
  if constexpr (LOCAL) {
    uint4* x = reinterpret_cast<uint4*>(sm + smem_rows<BITS, G16, NTMAX>(
        (int)(reinterpret_cast<const uint8_t*>(red) - sm) +
        kWarps * 2 * NTMAX * 128 * 4));
    float* sum = reinterpret_cast<float*>(
        x + (int64_t)a.T * a.K / 8 * a.format.terms);
    uint32_t* mx = reinterpret_cast<uint32_t*>(sum + a.T * m.ldg);
    auto convert = [&](auto* rows) {
      convert_rows<kThreads>(a.format, a.T, a.K / 8, a.inv_s, x,
                             a.T * (a.K / 8), sum, m.ldg, mx,
                             [&](int r) { return rows + r * a.ldx; });
    };
    if (a.xt == TTQ_F32)
      convert(static_cast<const float*>(a.X));
    else if (a.xt == TTQ_BF16)
      convert(static_cast<const __nv_bfloat16*>(a.X));
    else
      convert(static_cast<const __half*>(a.X));
    xhat = x;
    xsum = sum;
    xmax = mx;
  }
  TileT tl(ring, lane, (int64_t)a.T * a.K / 8);
  // h of a finished tile
  auto finish = [&](int en, int tile) {
    constexpr float per_unit = 1.f / kUnit<BITS, G16, MODE>;
    constexpr int most = MODE == kExact ? 0 : Positions<BITS, G16>::kMost;
    const int cols = l.cols[en], col0 = l.first[en];
    const int ch = tile * 16 + (lane >> 2);
    const float* mid = a.inv_s_mid + (int64_t)l.expert[en] * a.I + ch;
    const float mid0 = mid[0], mid1 = mid[8];
#pragma unroll
    for (int n = 0; n < NTMAX; ++n) {
      if (n >= tl.nt) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = n * 8 + 2 * (lane & 3) + i;
        if (col < cols) {
          const int slot = l.slot[col0 + col];
          const float un = row_unscale(xmax[l.token[col0 + col]], most);
          float* h = a.h + (int64_t)slot * a.I + ch;
          h[0] = gated(tl.acc[0][n][i] * per_unit * un, a.act) *
                 (tl.acc[1][n][i] * per_unit * un) * mid0;
          h[8] = gated(tl.acc[0][n][2 + i] * per_unit * un, a.act) *
                 (tl.acc[1][n][2 + i] * per_unit * un) * mid1;
        }
      }
    }
  };
  unsigned en = 0, tile = 0;
  bool open = false;  // the last tile goes on in the next warp
  for (int r = 0, s = s0; r < rounds || s < s1;) {
    // chunks c .. c_end - 1 of tile `at` of the list
    unsigned at;
    int c = 0, c_end = chunks;
    if (r < rounds) {
      at = t0 + r * kWarps + warp;
      ++r;
    } else {
      const int q = s / chunks;
      at = t1 + q;
      c = s - q * chunks;
      c_end = min(chunks, c + s1 - s);
      s += c_end - c;
    }
    en = at / (unsigned)tiles;
    tile = at - en * tiles;
    const int col0 = l.first[en];
    tl.start(m, xhat, xsum, l.cols[en], c,
             [&](int col) { return (int64_t)l.token[col0 + col]; });
    tl.template run<LG>(m, c, c_end, issue);
    if (c > 0) {  // the warp before started it
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int n = 0; n < NTMAX; ++n)
          *reinterpret_cast<float4*>(
              red + ((warp * 2 + rt) * NTMAX + n) * 128 + lane * 4) =
              make_float4(tl.acc[rt][n][0], tl.acc[rt][n][1],
                          tl.acc[rt][n][2], tl.acc[rt][n][3]);
    } else if (c_end == chunks) {
      finish(en, tile);
    } else {
      open = true;
    }
  }
  cp_async_wait_all();
  __syncthreads();
  if (open) {
    // the tile ends chunks - (steps the warp did) after s1
    const int start = s1 / chunks * chunks;  // the tile's first step
    for (int k = warp + 1; k < kWarps; ++k) {
      if (share(k) >= start + chunks) break;
      if (share(k) == share(k + 1)) continue;
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int n = 0; n < NTMAX; ++n) {
          const float4 v = *reinterpret_cast<const float4*>(
              red + ((k * 2 + rt) * NTMAX + n) * 128 + lane * 4);
          tl.acc[rt][n][0] += v.x;
          tl.acc[rt][n][1] += v.y;
          tl.acc[rt][n][2] += v.z;
          tl.acc[rt][n][3] += v.w;
        }
    }
    finish(en, tile);
  }
}

// ---------------------------------------------------------------- down ---

// A warp's tile is 32 output channels; a CTA's 8 warps are `rs` neighbouring
// tiles times 8 / rs parts. The (entry, 128-channel chunk) pairs of the batch
// are one list, split evenly over the parts of all CTAs of a cluster. Every
// warp keeps the sums of all tokens for its share and adds an entry's columns
// to them when it leaves the entry; parts are added at the end, in order.
template <int BITS, bool G16, int LG, int MODE, int NTMAX, bool LOCAL>
__global__ void __launch_bounds__(kThreads, 2)
    down_kernel(const DownArgs a) {
  using TileT = Tile<BITS, G16, MODE, NTMAX>;
  constexpr int S = TileT::S;
  extern __shared__ __align__(16) uint8_t sm[];
  Lists l(sm, a.T * a.top_k, a.E);
  float* ysum =  // [warp][T][32]
      reinterpret_cast<float*>(sm + Lists::bytes(a.T * a.top_k, a.E));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int region = a.T * kRows;
  const uint8_t* ring =
      reinterpret_cast<const uint8_t*>(ysum + kWarps * region) +
      warp * kRing<BITS, G16, NTMAX>;
  const uint32_t ring_at = smem_u32(ring);
  float* mine = ysum + warp * region;

  // nothing before griddep_enter() reads what the kernel before this one
  // writes, and that kernel let this one start only after its own wait
  build_lists(l, a.ids, a.weights, a.T, a.top_k, a.E, nullptr);
  for (int i = lane; i < region; i += 32) mine[i] = 0.f;
  const int rs = a.rs, ks = kWarps / rs;
  const int wr = warp % rs, wk = warp / rs;
  const int tile = blockIdx.x * rs + wr;
  const int chunks = (a.I + kChunk - 1) / kChunk;
  const int whole = l.entries * chunks;
  const int total = tile * kRows < a.K ? whole : 0;
  const int ranks = gridDim.y, rank = blockIdx.y;
  const int parts = ranks * ks, part = rank * ks + wk;
  const int s0 = (int)((unsigned)total * part / parts);
  const int s1 = (int)((unsigned)total * (part + 1) / parts);
  const Packed m(a.codes, a.delta, a.zero, a.I, BITS, a.group);
  Stream<BITS, G16, S> w(m, 16, lane);
  int is = s0, ien = s0 / chunks;
  auto seek = [&](int c) {
    w.seek(m, (int64_t)l.expert[ien] * a.K + tile * kRows, c);
  };
  if (s0 < s1) seek(s0 - ien * chunks);
  auto issue = [&]() {
    if (is < s1) {
      w.copy(m, ring_at, lane);
      if (++is < s1 && w.c == chunks) {
        ++ien;
        seek(0);
      }
    }
    cp_async_commit();
    w.advance();
  };
#pragma unroll
  for (int i = 0; i < S; ++i) issue();
  griddep_enter();

  const uint4* hhat = a.hhat;
  const float* hsum = a.hsum;
  const uint32_t* hmax = a.hmax;
  const int slots = a.T * a.top_k;
  int row0 = 0;  // LOCAL: rows are columns from here on, otherwise slots
  if constexpr (LOCAL) {
    uint4* x = reinterpret_cast<uint4*>(sm + smem_rows<BITS, G16, NTMAX>(
        (int)(reinterpret_cast<const uint8_t*>(ysum) - sm) +
        kWarps * region * 4));
    float* sum =
        reinterpret_cast<float*>(x + (int64_t)slots * a.I / 8 * a.format.terms);
    uint32_t* mx = reinterpret_cast<uint32_t*>(sum + slots * m.ldg);
    // the columns of the entries that the CTA's parts meet
    const int from = (int)((unsigned)whole * (rank * ks) / parts);
    const int to = (int)((unsigned)whole * (rank * ks + ks) / parts);
    if (from < to) {
      const int e0 = from / chunks, e1 = (to - 1) / chunks;
      row0 = l.first[e0];
      convert_rows<kThreads>(
          a.format, l.first[e1] + l.cols[e1] - row0, a.I / 8, nullptr, x,
          slots * (a.I / 8), sum, m.ldg, mx,
          [&](int r) { return a.h + (int64_t)l.slot[row0 + r] * a.I; });
    }
    hhat = x;
    hsum = sum;
    hmax = mx;
  }
  const int t = lane & 3, g = lane >> 2;
  TileT tl(ring, lane, (int64_t)slots * a.I / 8);
  int s = s0, en = s0 / chunks, c = s0 - en * chunks;
  while (s < s1) {
    const int cols = l.cols[en], col0 = l.first[en];
    tl.start(m, hhat, hsum, cols, c,
             [&](int col) {
               return (int64_t)(LOCAL ? col0 + col - row0
                                      : l.slot[col0 + col]);
             });
    const int stop = min(s1, s + chunks - c);
    tl.template run<LG>(m, c, c + stop - s, issue);
    s = stop;
    // leave the entry: its columns are different tokens
    constexpr float per_unit = 1.f / kUnit<BITS, G16, MODE>;
    constexpr int most = MODE == kExact ? 0 : Positions<BITS, G16>::kMost;
#pragma unroll
    for (int n = 0; n < NTMAX; ++n) {
      if (n >= tl.nt) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = n * 8 + 2 * t + i;
        if (col < cols) {
          const int r = LOCAL ? col0 + col - row0 : l.slot[col0 + col];
          const float wt =
              l.weight[col0 + col] * row_unscale(hmax[r], most) *
              per_unit;
          float* y = mine + l.token[col0 + col] * kRows + g;
          y[0] = fmaf(wt, tl.acc[0][n][i], y[0]);
          y[8] = fmaf(wt, tl.acc[0][n][2 + i], y[8]);
          y[16] = fmaf(wt, tl.acc[1][n][i], y[16]);
          y[24] = fmaf(wt, tl.acc[1][n][2 + i], y[24]);
        }
      }
    }
    __syncwarp();
    ++en;
    c = 0;
  }
  cp_async_wait_all();
  __syncthreads();
  // add the CTA's parts, then the cluster's through distributed shared
  // memory, both in order
  for (int i = tid; i < rs * region; i += kThreads) {
    float v = ysum[i];
    for (int k = 1; k < ks; ++k) v += ysum[k * rs * region + i];
    ysum[i] = v;
  }
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
  const uint32_t ys = smem_u32(ysum);
  for (int i = rank * kThreads + tid; i < rs * region; i += ranks * kThreads) {
    float v = 0.f;
    if (ranks > 1) {
      for (int r = 0; r < ranks; ++r) v += ld_cluster_f32(ys + i * 4, r);
    } else {
      v = ysum[i];
    }
    const int q = i / region, e = i - q * region;
    const int row = (blockIdx.x * rs + q) * kRows + e % kRows;
    if (row < a.K) {
      const int64_t at = (int64_t)(e / kRows) * a.ldy + row;
      if constexpr (MODE == kOne)
        static_cast<__nv_bfloat16*>(a.Y)[at] = __float2bfloat16_rn(v);
      else if constexpr (MODE == kTwo)
        static_cast<__half*>(a.Y)[at] = __float2half_rn(v);
      else
        static_cast<float*>(a.Y)[at] = v;
    }
  }
  if (ranks > 1) cluster_sync();
}

// -------------------------------------------------------------- launch ---

template <int BITS, bool G16, int NTMAX>
size_t up_smem(int n, int E) {
  return Lists::bytes(n, E) + (size_t)kWarps * 2 * NTMAX * 128 * 4 +
         (size_t)kWarps * kRing<BITS, G16, NTMAX>;
}
template <int BITS, bool G16, int NTMAX>
size_t down_smem(int T, int n, int E) {
  return Lists::bytes(n, E) + (size_t)kWarps * T * kRows * 4 +
         (size_t)kWarps * kRing<BITS, G16, NTMAX>;
}

// Lets a kernel use all of an SM's shared memory, once per device.
template <auto KERN>
bool allow_smem() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
  const uint64_t bit = (uint64_t)1 << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return true;
  if (cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           227 * 1024) != cudaSuccess)
    return false;
  if (dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

inline int ctas_per_sm(size_t smem) { return smem + 1024 <= 114 * 1024 ? 2 : 1; }

template <int BITS, bool G16, int LG, int MODE, int NTMAX, bool LOCAL>
ttq_status launch_up(UpArgs u, cudaStream_t st) {
  LaunchShape ls;
  ls.block = dim3(kThreads);
  ls.smem = up_smem<BITS, G16, NTMAX>(u.T * u.top_k, u.E);
  if (LOCAL) ls.smem += rows_bytes(u.T, u.K, u.group, u.format.terms) + 32;
  const int64_t slots = ctas_per_sm(ls.smem) * sm_count();
  const int64_t tiles =
      (int64_t)Lists::max_entries(u.T * u.top_k, u.E) * (u.I / 16);
  ls.grid = dim3((unsigned)std::min<int64_t>(tiles, slots));
  constexpr auto kern = up_kernel<BITS, G16, LG, MODE, NTMAX, LOCAL>;
  if (!allow_smem<kern>()) return TTQ_ERR_CUDA;
  return launch(ls, st, kern, u);
}

template <int BITS, bool G16, int LG, int MODE, int NTMAX, bool LOCAL>
ttq_status launch_down(DownArgs d, cudaStream_t st) {
  LaunchShape ls;
  ls.block = dim3(kThreads);
  ls.smem = down_smem<BITS, G16, NTMAX>(d.T, d.T * d.top_k, d.E);
  if (LOCAL)
    ls.smem += rows_bytes(d.T * d.top_k, d.I, d.group, d.format.terms) + 32;
  const int slots = ctas_per_sm(ls.smem) * sm_count();
  const int tiles = d.K / kRows;
  // as many neighbouring tiles as still leave a cluster of up to 8 per SM slot
  d.rs = kWarps;
  while (d.rs > 1 && (tiles + d.rs - 1) / d.rs * 8 < slots) d.rs /= 2;
  const int grid = (tiles + d.rs - 1) / d.rs;
  const int ranks = std::max(1, std::min(8, slots / grid));
  ls.grid = dim3((unsigned)grid, (unsigned)ranks);
  ls.cluster_y = (unsigned)ranks;
  constexpr auto kern = down_kernel<BITS, G16, LG, MODE, NTMAX, LOCAL>;
  if (!allow_smem<kern>()) return TTQ_ERR_CUDA;
  return launch(ls, st, kern, d);
}

// NTMAX: up to 8 tokens fill one column tile; more may put up to 16 on one
// entry. (Four tiles did not fit the registers of two CTAs per SM: an expert
// with more than 16 tokens becomes two entries, the second read from L2.)
template <int BITS, bool G16, int LG, int MODE>
ttq_status launch_mode(const UpArgs& u, cudaStream_t st) {
  if (u.T > 8) return launch_up<BITS, G16, LG, MODE, 2, false>(u, st);
  return u.local ? launch_up<BITS, G16, LG, MODE, 1, true>(u, st)
                 : launch_up<BITS, G16, LG, MODE, 1, false>(u, st);
}
template <int BITS, bool G16, int LG, int MODE>
ttq_status launch_mode(const DownArgs& d, cudaStream_t st) {
  if (d.T > 8) return launch_down<BITS, G16, LG, MODE, 2, false>(d, st);
  return d.local ? launch_down<BITS, G16, LG, MODE, 1, true>(d, st)
                 : launch_down<BITS, G16, LG, MODE, 1, false>(d, st);
}

template <int BITS, bool G16, int LG, typename Args>
ttq_status launch_group(const Args& a, cudaStream_t st) {
  switch (a.yt) {
    case TTQ_BF16: return launch_mode<BITS, G16, LG, kOne>(a, st);
    case TTQ_F16: return launch_mode<BITS, G16, LG, kTwo>(a, st);
    case TTQ_F32: return launch_mode<BITS, G16, LG, kExact>(a, st);
  }
  return TTQ_ERR_INVALID_ARG;
}

template <int BITS, typename Args>
ttq_status launch_bits(const Args& a, cudaStream_t st) {
  switch (a.group) {
    case 16: return launch_group<BITS, true, 0>(a, st);
    case 32: return launch_group<BITS, false, 0>(a, st);
    case 64: return launch_group<BITS, false, 1>(a, st);
    case 128: return launch_group<BITS, false, 2>(a, st);
  }
  return TTQ_ERR_INVALID_ARG;
}

}  // namespace moe
}  // namespace ttq
