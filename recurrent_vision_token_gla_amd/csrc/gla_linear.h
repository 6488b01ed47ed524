// Host-side launch interface of the linear and gated products (gla_linear.hip)
// and of their gradients (gla_linear_bwd.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace gla {

constexpr int kLinearMaxWidth = 65536;  // widest x, y and h

// y = alpha act(x W^T + bias) + residual, x [rows][K], W [N][K], y [rows][N]
struct LinearArgs {
  long rows;
  int K, N, act, dtype;
  float alpha;
  const void *x, *weight;
  const float* bias;     // or nullptr
  const void* residual;  // or nullptr
  void* pre;             // x W^T + bias, or nullptr
  void* y;
};
hipError_t launch_linear(const LinearArgs& a, hipStream_t s);

// h = act(x Wg^T) * (x Wu^T)
struct GatedArgs {
  long rows;
  int K, F, act, dtype;
  const void *x, *gate_weight, *up_weight;
  void *gate_out, *up_out;  // the two products, or nullptr
  void* h;
};
hipError_t launch_gated(const GatedArgs& a, hipStream_t s);

// The workspace of a gradient, by byte offsets, and how its products are cut up:
// the tiles of both, the splits of the rows that the weights' sums over, and
// whether one launch takes both (on tiles of one kind).
struct LinearBwdLayout {
  size_t g[2];     // gradients behind the activation, [rows][N] each
  size_t colsum;   // float [parts][N]
  size_t partial;  // float [splits][parts of the weights][N][K]
  size_t total;
  int tile_x, tile_w, splits;
  long steps, each;
  bool pair;
};

struct LinearBwdArgs {
  long rows;
  int K, N, act, dtype;
  float alpha;
  const void *x, *weight, *pre, *gy;
  void *gx, *gweight;  // each may be nullptr
  float* gbias;        // or nullptr
};
LinearBwdLayout linear_bwd_layout(long rows, int K, int N, int act, int dtype);
hipError_t launch_linear_bwd(const LinearBwdArgs& a, const LinearBwdLayout& l, char* ws, hipStream_t s);

struct GatedBwdArgs {
  long rows;
  int K, F, act, dtype;
  const void *x, *gate_weight, *up_weight, *gate, *up, *gh;
  void *gx, *ggate_weight, *gup_weight;
};
LinearBwdLayout gated_bwd_layout(long rows, int K, int F, int dtype);
hipError_t launch_gated_bwd(const GatedBwdArgs& a, const LinearBwdLayout& l, char* ws, hipStream_t s);

}  // namespace gla
