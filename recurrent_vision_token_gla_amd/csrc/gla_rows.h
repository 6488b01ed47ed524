// What the kernels over rows share: sums over the threads of a row and
// rounding to the stream's type.
#pragma once

#include "gla_device.h"

namespace gla {
namespace norm {

// Sum or largest value over the TPR threads of a row (64: one wave; 256: the
// workgroup, through LDS).
template <int TPR, bool kMax>
__device__ __forceinline__ float row_reduce(float x, float* lds) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const float y = __shfl_xor(x, m);
    x = kMax ? fmaxf(x, y) : x + y;
  }
  if constexpr (TPR > 64) {
    __syncthreads();  // earlier readers of lds are done
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = lds[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) x = kMax ? fmaxf(x, lds[w]) : x + lds[w];
  }
  return x;
}

// s rounded to the stream's type (what is stored, and what the norm is of)
__device__ __forceinline__ float round_to(float x, half_t) { return (float)(half_t)x; }
__device__ __forceinline__ float round_to(float x, float) { return x; }

}  // namespace norm
}  // namespace gla
