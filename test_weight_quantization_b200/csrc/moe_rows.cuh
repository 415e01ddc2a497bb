// moe_rows.cuh — the activations of the expert kernels: rows of fp32 or
// 16-bit values to fp16 terms in the order of the code pairs.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "moe.h"

namespace ttq {
namespace moe {

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

// 8 channels (vector i of the row) times inv_s (NULL for none).
template <typename TX>
__device__ __forceinline__ void load_scaled(const TX* row, const float* inv_s,
                                            int i, float (&v)[8]) {
  load_row8(row + (int64_t)i * 8, v);
  if (inv_s) {
    const float4 a = reinterpret_cast<const float4*>(inv_s)[2 * i];
    const float4 b = reinterpret_cast<const float4*>(inv_s)[2 * i + 1];
    v[0] *= a.x; v[1] *= a.y; v[2] *= a.z; v[3] *= a.w;
    v[4] *= b.x; v[5] *= b.y; v[6] *= b.z; v[7] *= b.w;
  }
}

__device__ __forceinline__ uint32_t largest_bits(const float (&v)[8]) {
  uint32_t mx = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) mx = max(mx, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  return mx;
}

// Stores vector i of a row whose largest value has the bits mx, as fp16 terms
// out[k * term] (term in vectors), and the sum of its group. The values carry
// 2^k (row_exponent) times 2^(most - at) of the code pair each channel meets:
// the first term rounds every value above 2^-27 of the largest to 11 bits, the
// second what is left. The sums are of the rounded values without the 2^(most
// - at). All lanes of a warp call together; the lanes of a group are
// neighbours. `live`: the vector exists.
__device__ __forceinline__ void store_vector(const RowFormat& f, int i,
                                             uint32_t mx, bool live,
                                             float (&v)[8], uint4* out,
                                             int64_t term, float* sums) {
  const float sc =
      __uint_as_float((uint32_t)(127 + row_exponent(mx, f.most)) << 23);
  // two factors, since the sum of the exponents may leave the range
  const float s0 = (float)(1 << f.up.x), s1 = (float)(1 << f.up.y),
              s2 = (float)(1 << f.up.z), s3 = (float)(1 << f.up.w);
  const bool g16 = f.group == 16;
  // factors of channels q and q + 4: pair q & 3, or for groups of 16 the pair
  // of the channel's half and parity
  const bool second = (i >> 1) & 1;
  float fac[4];
  fac[0] = g16 ? (second ? s2 : s0) : s0;
  fac[1] = g16 ? (second ? s3 : s1) : s1;
  fac[2] = g16 ? fac[0] : s2;
  fac[3] = g16 ? fac[1] : s3;
  float inv[4];  // of powers of two
#pragma unroll
  for (int q = 0; q < 4; ++q)
    inv[q] = __uint_as_float(0x7F000000u - __float_as_uint(fac[q]));
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = v[q] * sc * fac[q & 3];
  float total = 0.f;
  for (int k = 0; k < f.terms; ++k) {
    uint32_t p[4];
    float a[8];
    if (g16) {
      // channels 4m..4m+3 of a half: lane m's pairs (0, 2), (1, 3)
      p[0] = half2_bits(v[0], v[2]);
      p[1] = half2_bits(v[1], v[3]);
      p[2] = half2_bits(v[4], v[6]);
      p[3] = half2_bits(v[5], v[7]);
      if (live) {
        const int m = 2 * (i & 1), half = second;
        uint2* o = reinterpret_cast<uint2*>(out + k * term + i / 4 * 4);
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
      if (live) out[k * term + i] = make_uint4(p[0], p[1], p[2], p[3]);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      total += a[q] * inv[q & 3];
      v[q] -= a[q];
    }
  }
  const int lanes = f.group / 8;
  for (int o = lanes / 2; o > 0; o >>= 1)
    total += __shfl_xor_sync(0xffffffffu, total, o);
  if (live && i % lanes == 0) sums[i / lanes] = total;
}

// rows rows (row j read at src(j)) to shared memory, by the whole CTA; `term`
// vectors between the terms. mx: shared, a word per row. Ends with a
// __syncthreads().
template <int THREADS, typename SF>
__device__ __forceinline__ void convert_rows(const RowFormat& f, int rows,
                                             int n, const float* inv_s,
                                             uint4* out, int term,
                                             float* sums, int ldg,
                                             uint32_t* mx, SF&& src) {
  const int tid = threadIdx.x, all = rows * n;
  if (tid < rows) mx[tid] = 0;
  __syncthreads();
  for (int i = tid; i < all; i += THREADS) {
    const int r = i / n;
    float v[8];
    load_scaled(src(r), inv_s, i - r * n, v);
    atomicMax(mx + r, largest_bits(v));
  }
  __syncthreads();
  for (int base = 0; base < all; base += THREADS) {
    const int i = base + tid;
    const bool live = i < all;
    const int r = live ? i / n : 0, j = live ? i - r * n : 0;
    float v[8] = {};
    if (live) load_scaled(src(r), inv_s, j, v);
    store_vector(f, j, mx[r], live, v, out + r * n, term, sums + r * ldg);
  }
  __syncthreads();
}

}  // namespace moe
}  // namespace ttq
