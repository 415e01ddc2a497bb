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
constexpr int kMaxCols = 32;  // columns of an entry: 4 MMA tiles of 8

// xhat: fp16 terms of x 2^k, [term][T][K], in the order the code pairs want;
// xmax: bits of a token's largest |x|; h [T top_k][I] fp32 and hmax likewise.
struct UpArgs {
  const __half* xhat;
  const uint32_t* xmax;
  const int32_t* ids;
  int T, K, I, E, top_k, group, act;
  const uint32_t* codes;
  const float* delta;
  const uint8_t* zero;
  const float* inv_s_mid;
  float* h;
  uint32_t* hmax;
  uint32_t* err;
};
struct DownArgs {
  const float* h;
  const uint32_t* hmax;
  const int32_t* ids;
  const float* weights;
  int T, K, I, E, top_k, group;
  const uint32_t* codes;
  const float* delta;
  const uint8_t* zero;
  void* Y;
  ttq_dtype yt;
  int64_t ldy;
};

template <int BITS>
ttq_status launch_bits(const UpArgs& u, const DownArgs& d, cudaStream_t st);

}  // namespace moe
}  // namespace ttq
