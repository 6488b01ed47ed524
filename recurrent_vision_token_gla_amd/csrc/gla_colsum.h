// Column sums of partial rows, the last step of the weights' gradients.
#pragma once

#include "gla_device.h"

namespace gla {
namespace norm {

// out[col] = sum over the P partial rows: 16 columns and 64 groups of rows per
// workgroup, each thread with 16 loads in flight, the groups joined in LDS in
// a fixed order. 915 rows of 768: 4.7 us, a launch's latency and one round of
// loads. (With 16 groups and one load at a time it took 20 us, two thirds of
// the gradient it finishes.)
static __global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ part,
                                                          float* __restrict__ out, int P, int F) {
  constexpr int W = 16;
  __shared__ float s[64][17];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  float y = 0.f;
  if (col < F) {
    for (int p = g; p < P; p += 64 * W) {
      float x[W];
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = p + 64 * i < P ? part[(long)(p + 64 * i) * F + col] : 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) y += x[i];
    }
  }
  s[g][c] = y;
  __syncthreads();
  if (g < 8) {
    y = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) y += s[g + 8 * i][c];
    s[g][c] = y;  // no other thread reads row g
  }
  __syncthreads();
  if (g == 0 && col < F) {
    y = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) y += s[i][c];
    out[col] = y;
  }
}

}  // namespace norm
}  // namespace gla
