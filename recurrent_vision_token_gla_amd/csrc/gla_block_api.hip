// C ABI of the products and norms between a block's mixers and of their
// gradients (declared in include/gla.h). As in gla_api.hip, every entry point
// checks its arguments on the host before any HIP call and then only enqueues
// kernels on the caller's stream.
#include "gla.h"
#include "gla_check.h"
#include "gla_gated_norm.h"
#include "gla_linear.h"

using namespace gla::api;

namespace {

// Rows, widths and codes of a product with `in` values in and `out` values out
// a row; `in` may be 0 where there are no rows or no outputs.
int check_product(int64_t rows, int in, int out, int act, int dtype, bool* empty) {
  if (rows < 0 || in < 0 || out < 0) return GLA_E_ARG;
  if (dtype != GLA_F16 && dtype != GLA_F32) return GLA_E_ARG;
  if (act < GLA_ACT_NONE || act > GLA_ACT_LOGSIGMOID) return GLA_E_ARG;
  if (in % 8 != 0 || out % 8 != 0 || in > gla::kLinearMaxWidth || out > gla::kLinearMaxWidth ||
      rows > (1LL << 31))
    return GLA_E_UNSUPPORTED;
  *empty = rows == 0 || out == 0;
  return !*empty && in == 0 ? GLA_E_UNSUPPORTED : GLA_OK;
}

int check_float_weight(const float* w) { return w && aligned(w, 16) ? GLA_OK : GLA_E_ARG; }

// Groups of a gate's rows: as many rows in each. No rows may have no groups.
int check_groups(int64_t rows, const void* gate, int64_t* groups) {
  if (!gate || (rows == 0 && *groups == 0)) *groups = 1;
  return *groups >= 1 && rows % *groups == 0 ? GLA_OK : GLA_E_ARG;
}

}  // namespace

extern "C" {

int gla_linear(const void* x, const void* weight, const float* bias, const void* residual, void* pre,
               void* y, int64_t rows, int K, int N, int act, float alpha, int dtype, void* stream) {
  bool empty;
  GLA_TRY(check_product(rows, K, N, act, dtype, &empty));
  if (empty) return GLA_OK;
  for (const void* t : {x, weight, (const void*)y}) GLA_TRY(check_tensor(t));
  for (const void* t : {(const void*)bias, residual, (const void*)pre}) GLA_TRY(check_optional(t));
  const size_t es = elem(dtype), nx = (size_t)rows * K * es, nw = (size_t)N * K * es;
  const size_t ny = (size_t)rows * N * es;
  // y may be residual itself: a value is read before it is written there
  GLA_TRY(check_disjoint<2, 4>({{y, ny}, {pre, ny}},
                               {{x, nx}, {weight, nw}, {bias, N * sizeof(float)},
                                {residual == y ? nullptr : residual, ny}}));
  gla::LinearArgs a{(long)rows, K, N, act, dtype, alpha, x, weight, bias, residual, pre, y};
  const hipError_t e = gla::launch_linear(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail_hip(e, "linear launch");
  return GLA_OK;
}

size_t gla_linear_bwd_workspace_bytes(int64_t rows, int K, int N, int act, int dtype) {
  bool empty;
  if (check_product(rows, K, N, act, dtype, &empty) != GLA_OK || empty) return 0;
  return gla::linear_bwd_layout((long)rows, K, N, act, dtype).total;
}

int gla_linear_bwd(const void* x, const void* weight, const void* pre, const void* gy, void* gx,
                   void* gweight, float* gbias, int64_t rows, int K, int N, int act, float alpha,
                   int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  bool empty;
  GLA_TRY(check_product(rows, K, N, act, dtype, &empty));
  if (empty || (!gx && !gweight && !gbias)) return GLA_OK;
  GLA_TRY(check_tensor(gy));
  if (gweight) GLA_TRY(check_tensor(x));
  if (gx) GLA_TRY(check_tensor(weight));
  if (act != GLA_ACT_NONE) GLA_TRY(check_tensor(pre));
  for (const void* t : {(const void*)gx, (const void*)gweight, (const void*)gbias})
    GLA_TRY(check_optional(t));
  const gla::LinearBwdLayout layout = gla::linear_bwd_layout((long)rows, K, N, act, dtype);
  const size_t need = layout.total;
  GLA_TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t es = elem(dtype), nx = (size_t)rows * K * es, nw = (size_t)N * K * es;
  const size_t ny = (size_t)rows * N * es;
  GLA_TRY(check_disjoint<4, 4>(
      {{gx, nx}, {gweight, nw}, {gbias, N * sizeof(float)}, {workspace, need}},
      {{gweight ? x : nullptr, nx}, {gx ? weight : nullptr, nw},
       {act != GLA_ACT_NONE ? pre : nullptr, ny}, {gy, ny}}));
  gla::LinearBwdArgs a{(long)rows, K, N, act, dtype, alpha, x, weight, pre, gy, gx, gweight, gbias};
  const hipError_t e =
      gla::launch_linear_bwd(a, layout, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail_hip(e, "linear backward launch");
  return GLA_OK;
}

int gla_gated_ff(const void* x, const void* gate_weight, const void* up_weight, void* gate, void* up,
                 void* h, int64_t rows, int K, int F, int act, int dtype, void* stream) {
  bool empty;
  GLA_TRY(check_product(rows, K, F, act, dtype, &empty));
  if (empty) return GLA_OK;
  for (const void* t : {x, gate_weight, up_weight, (const void*)h}) GLA_TRY(check_tensor(t));
  GLA_TRY(check_optional(gate));
  GLA_TRY(check_optional(up));
  const size_t es = elem(dtype), nx = (size_t)rows * K * es, nw = (size_t)F * K * es;
  const size_t nh = (size_t)rows * F * es;
  GLA_TRY(check_disjoint<3, 3>({{h, nh}, {gate, nh}, {up, nh}}, {{x, nx}, {gate_weight, nw}, {up_weight, nw}}));
  gla::GatedArgs a{(long)rows, K, F, act, dtype, x, gate_weight, up_weight, gate, up, h};
  const hipError_t e = gla::launch_gated(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail_hip(e, "gated feed-forward launch");
  return GLA_OK;
}

size_t gla_gated_ff_bwd_workspace_bytes(int64_t rows, int K, int F, int dtype) {
  bool empty;
  if (check_product(rows, K, F, GLA_ACT_SILU, dtype, &empty) != GLA_OK || empty) return 0;
  return gla::gated_bwd_layout((long)rows, K, F, dtype).total;
}

int gla_gated_ff_bwd(const void* x, const void* gate_weight, const void* up_weight, const void* gate,
                     const void* up, const void* gh, void* gx, void* ggate_weight, void* gup_weight,
                     int64_t rows, int K, int F, int act, int dtype, void* workspace,
                     size_t workspace_bytes, void* stream) {
  bool empty;
  GLA_TRY(check_product(rows, K, F, act, dtype, &empty));
  if (!ggate_weight != !gup_weight) return GLA_E_ARG;
  if (empty || (!gx && !ggate_weight)) return GLA_OK;
  for (const void* t : {gate, up, gh}) GLA_TRY(check_tensor(t));
  if (ggate_weight) GLA_TRY(check_tensor(x));
  if (gx) {
    GLA_TRY(check_tensor(gate_weight));
    GLA_TRY(check_tensor(up_weight));
  }
  for (const void* t : {(const void*)gx, (const void*)ggate_weight, (const void*)gup_weight})
    GLA_TRY(check_optional(t));
  const gla::LinearBwdLayout layout = gla::gated_bwd_layout((long)rows, K, F, dtype);
  const size_t need = layout.total;
  GLA_TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t es = elem(dtype), nx = (size_t)rows * K * es, nw = (size_t)F * K * es;
  const size_t nh = (size_t)rows * F * es;
  GLA_TRY(check_disjoint<4, 6>(
      {{gx, nx}, {ggate_weight, nw}, {gup_weight, nw}, {workspace, need}},
      {{ggate_weight ? x : nullptr, nx}, {gx ? gate_weight : nullptr, nw}, {gx ? up_weight : nullptr, nw},
       {gate, nh}, {up, nh}, {gh, nh}}));
  gla::GatedBwdArgs a{(long)rows, K, F, act, dtype, x, gate_weight, up_weight, gate, up, gh,
                      gx, ggate_weight, gup_weight};
  const hipError_t e =
      gla::launch_gated_bwd(a, layout, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail_hip(e, "gated feed-forward backward launch");
  return GLA_OK;
}

int gla_gated_add_rmsnorm(const void* x, const void* residual, const float* post_weight, const void* gate,
                          int64_t groups, const float* scale, const float* weight, float eps, void* sum,
                          void* y, int64_t rows, int F, int dtype, void* stream) {
  GLA_TRY(check_rows(rows, F, dtype));
  GLA_TRY(check_groups(rows, gate, &groups));
  if (rows == 0 || F == 0) return GLA_OK;
  for (const void* t : {x, residual, (const void*)y}) GLA_TRY(check_tensor(t));
  for (const void* t : {(const void*)post_weight, gate, (const void*)scale, (const void*)sum})
    GLA_TRY(check_optional(t));
  GLA_TRY(check_float_weight(weight));
  if (!(eps >= 0.f)) return GLA_E_ARG;
  const size_t nb = (size_t)rows * F * elem(dtype), ng = (size_t)groups * F * elem(dtype);
  const size_t nw = (size_t)F * sizeof(float);
  GLA_TRY(check_disjoint<2, 4>({{sum, nb}, {y, nb}},
                               {{post_weight, nw}, {gate, ng}, {scale, nw}, {weight, nw}}));
  // a row is read whole before it is written, so sum and y may be x or
  // residual themselves; nothing else may overlap
  for (const void* in : {x, residual})
    for (const void* out : {sum, y})
      if (out && out != in && overlaps(out, nb, in, nb)) return GLA_E_ARG;
  gla::GatedNormArgs a{(long)rows, (long)groups, F, dtype, x, residual, post_weight, gate, scale, weight,
                       eps, sum, y};
  const hipError_t e = gla::launch_gated_norm(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail_hip(e, "gated add rmsnorm launch");
  return GLA_OK;
}

size_t gla_gated_add_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t groups, int F) {
  if (check_rows(rows, F, GLA_F16) != GLA_OK || rows == 0 || F == 0) return 0;
  if (groups < 1 || rows % groups != 0) return 0;
  return gla::gated_norm_bwd_workspace((long)rows, (long)groups, F);
}

int gla_gated_add_rmsnorm_bwd(const void* x, const void* sum, const float* post_weight, const void* gate,
                              int64_t groups, const float* scale, const float* weight, float eps,
                              const void* gy, const void* gsum, void* gx, void* gresidual,
                              float* gpost_weight, void* ggate, float* gscale, float* gweight,
                              int64_t rows, int F, int dtype, void* workspace, size_t workspace_bytes,
                              void* stream) {
  GLA_TRY(check_rows(rows, F, dtype));
  GLA_TRY(check_groups(rows, gate, &groups));
  if ((gpost_weight && !post_weight) || (ggate && !gate) || (gscale && !scale)) return GLA_E_ARG;
  if (rows == 0 || F == 0) return GLA_OK;
  for (const void* t : {x, sum, gy, (const void*)gx, (const void*)gresidual}) GLA_TRY(check_tensor(t));
  for (const void* t : {(const void*)post_weight, gate, (const void*)scale, gsum, (const void*)gpost_weight,
                        (const void*)ggate, (const void*)gscale})
    GLA_TRY(check_optional(t));
  GLA_TRY(check_float_weight(weight));
  GLA_TRY(check_float_weight(gweight));
  if (!(eps >= 0.f)) return GLA_E_ARG;
  const size_t need = gla::gated_norm_bwd_workspace((long)rows, (long)groups, F);
  GLA_TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t nb = (size_t)rows * F * elem(dtype), ng = (size_t)groups * F * elem(dtype);
  const size_t nw = (size_t)F * sizeof(float);
  const Range weights[4] = {{post_weight, nw}, {gate, ng}, {scale, nw}, {weight, nw}};
  const Range small[5] = {{gpost_weight, nw}, {ggate, ng}, {gscale, nw}, {gweight, nw}, {workspace, need}};
  const Range streams[4] = {{x, nb}, {sum, nb}, {gy, nb}, {gsum, nb}};
  const Range grads[2] = {{gx, nb}, {gresidual, nb}};
  GLA_TRY(check_disjoint(small, weights));
  GLA_TRY(check_disjoint(small, streams));
  GLA_TRY(check_disjoint(small, grads));
  GLA_TRY(check_disjoint(grads, weights));
  // gx and gresidual may each be an input row for row
  for (const Range& g : grads)
    for (const Range& in : streams)
      if (in.p && g.p != in.p && overlaps(g.p, nb, in.p, nb)) return GLA_E_ARG;
  gla::GatedNormBwdArgs a{(long)rows, (long)groups, F, dtype, x, sum, gy, gsum, post_weight, gate, scale,
                          weight, eps, gx, gresidual, ggate, gpost_weight, gscale, gweight};
  const hipError_t e =
      gla::launch_gated_norm_bwd(a, static_cast<float*>(workspace), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail_hip(e, "gated add rmsnorm backward launch");
  return GLA_OK;
}

}  // extern "C"
