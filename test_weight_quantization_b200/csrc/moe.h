// moe.h — what the expert kernels of ttq_moe_lowbit share with their
// launcher (moe.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ttq.h"

namespace ttq {
namespace moe {

constexpr int kMaxExperts = 512;
constexpr int kMaxCols = 16;  // columns of an entry: 2 MMA tiles of 8

// The bit of an fp16 at which the code pairs of a lane's block enter the MMA
// (pair i), and the largest of them. A pair is used where the unpacking finds
// it if it ends below bit 10 there, otherwise it is shifted down; the
// activations that meet pair i are stored with 2^(kMost - at(i)).
template <int BITS, bool G16>
struct Positions {
  static constexpr int kMost = BITS == 2 ? (G16 ? 2 : 6)
                               : BITS == 3 ? (G16 ? 3 : 6)
                               : BITS <= 5 ? BITS
                                           : 0;
  static __host__ __device__ constexpr int at(int i) {
    if (BITS >= 6) return 0;
    if (G16 || BITS == 5) return i & 1 ? BITS : 0;
    if (BITS == 2) return 2 * i;
    if (BITS == 3) return i < 3 ? 3 * i : 6;
    return i & 1 ? 4 : 0;
  }
};
inline int position(int bits, bool g16, int i) {
  switch (bits) {
    case 2: return g16 ? Positions<2, true>::at(i) : Positions<2, false>::at(i);
    case 3: return g16 ? Positions<3, true>::at(i) : Positions<3, false>::at(i);
    case 4: return g16 ? Positions<4, true>::at(i) : Positions<4, false>::at(i);
    case 5: return g16 ? Positions<5, true>::at(i) : Positions<5, false>::at(i);
  }
  return 0;
}

// k of the power of two that a row of activations carries: its largest value
// (its bits) times 2^k 2^most lies in [2^13, 2^14).
__host__ __device__ inline int row_exponent(uint32_t max_bits, int most) {
  const int e = (int)(max_bits >> 23) - 127;
  const int k = 13 - most - e;
  return k < 126 ? k : 126;
}

// Bytes of `rows` rows of `width` channels in fp16 terms with their sums, and
// whether the expert kernels hold them in shared memory: what is left beside
// the largest rings when two CTAs share an SM.
inline size_t rows_bytes(int64_t rows, int64_t width, int group, int terms) {
  const int64_t sums = (width / group + 15) / 16 * 16;  // groups_ld
  return (size_t)(rows * width * 2 * terms + rows * sums * 4 + 16);
}
inline bool rows_fit(int64_t rows, int64_t width, int group, int terms) {
  return rows <= 8 && rows_bytes(rows, width, group, terms) <= 18 * 1024;
}

// What every row of activations is converted by (moe_rows.cuh).
struct RowFormat {
  int terms;  // fp16 terms
  int group;  // channels per sum
  int most;   // Positions::kMost
  int4 up;    // kMost - at(i) of code pair i
};

// xhat: fp16 terms of the rows, [term][T][K], in the order the code pairs
// want; xsum [T][groups_ld]: the rows' sums over every group (times 2^k);
// xmax: bits of a token's largest |x|. h [T top_k][I] fp32, and
// hhat, hsum, hmax for its rows.
struct UpArgs {
  const uint4* xhat;
  const float* xsum;
  const uint32_t* xmax;
  const int32_t* ids;
  int T, K, I, E, top_k, group, act;
  const uint32_t* codes;
  const float* delta;
  const uint8_t* zero;
  const float* inv_s_mid;
  float* h;
  ttq_dtype yt;
  uint32_t* err;
  // local: the rows are converted from X by every CTA
  bool local;
  const void* X;
  ttq_dtype xt;
  int64_t ldx;
  const float* inv_s;
  RowFormat format;
};
struct DownArgs {
  const uint4* hhat;
  const float* hsum;
  const uint32_t* hmax;
  const int32_t* ids;
  const float* weights;
  int T, K, I, E, top_k, group, rs;
  const uint32_t* codes;
  const float* delta;
  const uint8_t* zero;
  void* Y;
  ttq_dtype yt;
  int64_t ldy;
  bool local;  // the rows are converted from h by every CTA
  const float* h;
  RowFormat format;
};

template <int BITS, typename Args>
ttq_status launch_bits(const Args& a, cudaStream_t st);

}  // namespace moe
}  // namespace ttq
