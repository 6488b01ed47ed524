// Host-side launch interface of the norms after and before a block
// (gla_gated_norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "gla_norm.h"

namespace gla {

// sum = residual + scale * gate[row / (rows / groups)] * p, p = RMSNorm(x) * post
// (x itself without post), y = RMSNorm(sum) * weight
struct GatedNormArgs {
  long rows, groups;
  int F, dtype;
  const void *x, *residual;
  const float* post;   // or nullptr
  const void* gate;    // [groups][F], or nullptr
  const float* scale;  // or nullptr
  const float* weight;
  float eps;
  void *sum, *y;  // sum may be nullptr
};
hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t s);

struct GatedNormBwdArgs {
  long rows, groups;
  int F, dtype;
  const void *x, *sum, *gy, *gsum;  // gsum may be nullptr
  const float* post;
  const void* gate;
  const float *scale, *weight;
  float eps;
  void *gx, *gresidual, *ggate;  // ggate, gpost, gscale where gate, post, scale are
  float *gpost, *gscale, *gweight;
};
size_t gated_norm_bwd_workspace(long rows, long groups, int F);
hipError_t launch_gated_norm_bwd(const GatedNormBwdArgs& a, float* ws, hipStream_t s);

}  // namespace gla
