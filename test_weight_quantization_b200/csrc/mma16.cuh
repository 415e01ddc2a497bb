// mma16.cuh — 16-bit operands of any activation type for mma.sync m16n8k16.
//
// A value enters as one 16-bit number where its type is 16 bits wide, and as
// three bf16 terms where it is fp32 (8 + 8 + 8 bits, each the rounding of what
// the terms before leave): x = x0 + x1 + x2 to 2^-24. A product of two values
// is the sum of the term products i + j <= 2; what is left out is below
// 2^-24 of |x y|. fp16 beside another type becomes two bf16 terms, exactly.
#pragma once

#include "common.cuh"

namespace ttq {
namespace mma16 {

template <typename T>
struct Native {
  static constexpr bool half = false;
};
template <>
struct Native<__half> {
  static constexpr bool half = true;
};

// Terms of a T when its partner is a P.
template <typename T, typename P>
constexpr int kTerms = sizeof(T) == 4 ? 3
                       : Native<T>::half && !Native<P>::half ? 2
                                                             : 1;
// Whether the MMA of T and P takes fp16 operands (bf16 otherwise).
template <typename T, typename P>
constexpr bool kHalf = Native<T>::half && Native<P>::half;

template <bool HALF>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1,
                                    uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (HALF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// TERMS bf16 terms of N pairs of floats, v overwritten by what is left.
template <int TERMS, int N>
__device__ __forceinline__ void split(float (&v)[2 * N],
                                      uint32_t (&out)[TERMS][N]) {
#pragma unroll
  for (int k = 0; k < TERMS; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      out[k][i] = bf16x2(v[2 * i], v[2 * i + 1]);
      float a, b;
      bf16x2_to_f32(out[k][i], a, b);
      v[2 * i] -= a;
      v[2 * i + 1] -= b;
    }
}

// As it was loaded: 8 (or 4) consecutive values.
template <typename T, int N>
struct Raw {
  uint32_t w[N * sizeof(T) / 4];
};

template <typename T, int N>
__device__ __forceinline__ void load(const T* p, bool ok, Raw<T, N>& r) {
  constexpr int words = N * sizeof(T) / 4;
  static_assert(words == 2 || words == 4 || words == 8, "whole vectors");
  if constexpr (words == 2) {
    const uint2 v =
        ok ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
    r.w[0] = v.x;
    r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < words / 4; ++i) {
      const uint4 v = ok ? reinterpret_cast<const uint4*>(p)[i]
                         : make_uint4(0, 0, 0, 0);
      r.w[4 * i] = v.x;
      r.w[4 * i + 1] = v.y;
      r.w[4 * i + 2] = v.z;
      r.w[4 * i + 3] = v.w;
    }
  }
}

// The N / 2 operand registers of each term.
template <typename T, typename P, int N>
__device__ __forceinline__ void terms(
    const Raw<T, N>& r, uint32_t (&out)[kTerms<T, P>][N / 2]) {
  if constexpr (kTerms<T, P> == 1) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) out[0][i] = r.w[i];
  } else {
    float v[N];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r.w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        f16x2_to_f32(r.w[i], v[2 * i], v[2 * i + 1]);
    }
    split<kTerms<T, P>, N / 2>(v, out);
  }
}

}  // namespace mma16
}  // namespace ttq
