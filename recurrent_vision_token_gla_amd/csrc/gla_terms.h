// Floats as sums of bf16 terms, x = t0 + t1 [+ t2], each the rounding of what is
// left: two terms hold 16 bits, three 24, in float's range. Products of terms add
// up in the matrix cores' float accumulators.
#pragma once

#include "gla_tile.h"

namespace gla {
namespace terms {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ floatx4 mma(bf8 a, bf8 b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Eight or four floats as NT bf16 terms.
template <int NT> struct Split8 { bf8 t[NT]; };
template <int NT> struct Split4 { bf4 t[NT]; };
// Two floats' leading bf16 terms in one register, and what they leave: pairs,
// written out, take one conversion and two subtractions per term (whole
// vectors were converted element by element).
__device__ __forceinline__ unsigned term2(float& a, float& b, bool rest) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  const unsigned u = __builtin_bit_cast(unsigned, __builtin_convertvector(f2{a, b}, bf2));
  if (rest) {
    a -= __uint_as_float(u << 16);
    b -= __uint_as_float(u & 0xffff0000u);
  }
  return u;
}
template <int NT>
__device__ __forceinline__ Split8<NT> split8(const float* x) {
  Split8<NT> s;
  float r[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) r[c] = x[c];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    tile::u32x4 u;
#pragma unroll
    for (int c = 0; c < 4; ++c) u[c] = term2(r[2 * c], r[2 * c + 1], t + 1 < NT);
    s.t[t] = __builtin_bit_cast(bf8, u);
  }
  return s;
}
template <int NT>
__device__ __forceinline__ Split4<NT> split4(floatx4 x) {
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  Split4<NT> s;
  float r[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const u32x2 u = {term2(r[0], r[1], t + 1 < NT), term2(r[2], r[3], t + 1 < NT)};
    s.t[t] = __builtin_bit_cast(bf4, u);
  }
  return s;
}

// c += a b over 32 contracted elements: the products of terms i + j < NT, and
// with three terms the middle ones' product.
template <int NT>
__device__ __forceinline__ floatx4 mm(const Split8<NT>& a, const Split8<NT>& b, floatx4 c) {
  if constexpr (NT == 3) {
    c = mma(a.t[2], b.t[0], c);
    c = mma(a.t[0], b.t[2], c);
    c = mma(a.t[1], b.t[1], c);
  }
  c = mma(a.t[1], b.t[0], c);
  c = mma(a.t[0], b.t[1], c);
  return mma(a.t[0], b.t[0], c);
}

}  // namespace terms
}  // namespace gla
