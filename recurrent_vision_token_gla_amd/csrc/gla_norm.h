// Host-side launch interface of the norm kernels (gla_norm.hip): the residual
// sum with its root-mean-square norm and their gradient, and the gradient of
// the output gate.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "gla_device.h"

namespace gla {

constexpr int kNormMaxF = 16384;  // widest row the norm kernels take

struct NormArgs {
  long rows;
  int F, dtype;
  const void *x, *residual;  // residual may be nullptr
  const float* weight;
  float eps;
  void *sum, *y;  // sum may be nullptr
  void* y8;       // 8-bit output instead of y
  float* scales;
};
hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s);

struct NormBwdArgs {
  long rows;
  int F, dtype;
  const void *sum, *gy, *gsum;  // gsum may be nullptr
  const float* weight;
  float eps;
  void* gx;
  float* gweight;
};
size_t norm_bwd_workspace(long rows, int F);
hipError_t launch_norm_bwd(const NormBwdArgs& a, float* ws, hipStream_t s);

struct GateBwdArgs {
  long rows;  // (batch, token, head) rows of dv values
  int dv, dtype;
  const void *o, *gate, *gy;
  const float* weight;
  float eps;
  void *go, *ggate;
  float* gweight;
};
size_t gate_bwd_workspace(long rows, int dv);
hipError_t launch_gate_bwd(const GateBwdArgs& a, float* ws, hipStream_t s);

}  // namespace gla
