// C ABI of the gradients, the single-token recurrence and the residual norm
// (declared in include/gla.h). As in gla_api.hip, every entry point checks its
// arguments on the host before any HIP call and then only enqueues kernels on
// the caller's stream.
#include "gla.h"
#include "gla_bwd.h"
#include "gla_check.h"
#include "gla_norm.h"
#include "gla_step.h"

using namespace gla::api;

namespace {

int add_rmsnorm_impl(const void* x, const void* residual, const float* weight, float eps, void* sum,
                     void* y, void* y8, float* scales, int64_t rows, int F, int dtype, void* stream) {
  GLA_TRY(check_rows(rows, F, dtype));
  if (rows == 0 || F == 0) return GLA_OK;
  GLA_TRY(check_tensor(x));
  GLA_TRY(check_optional(residual));
  GLA_TRY(check_optional(sum));
  GLA_TRY(check_tensor(y8 ? y8 : y));
  if (!weight || !aligned(weight, 16) || !(eps >= 0.f)) return GLA_E_ARG;
  if (y8 && (!scales || !aligned(scales, 4))) return GLA_E_ARG;
  const size_t n = (size_t)rows * F, nb = n * elem(dtype);
  const void* out = y8 ? y8 : y;
  const size_t on = y8 ? n : nb;
  const Range w{weight, (size_t)F * sizeof(float)}, sc{scales, (size_t)rows * sizeof(float)};
  GLA_TRY(check_disjoint<4, 1>({{sum, nb}, {out, on}, y8 ? sc : Range{nullptr, 0}, {nullptr, 0}}, {w}));
  // a row is read whole before it is written, so sum and y may be x or
  // residual themselves (the 8-bit output may not); nothing else may overlap
  for (const void* in : {x, residual}) {
    if (!in) continue;
    if (sum && sum != in && overlaps(sum, nb, in, nb)) return GLA_E_ARG;
    if ((y8 || out != in) && overlaps(out, on, in, nb)) return GLA_E_ARG;
    if (y8 && overlaps(scales, sc.n, in, nb)) return GLA_E_ARG;
  }
  gla::NormArgs a{(long)rows, F, dtype, x, residual, weight, eps, sum, y, y8, scales};
  const hipError_t e = gla::launch_add_rmsnorm(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail_hip(e, "add rmsnorm launch");
  return GLA_OK;
}

int step_impl(const void* q, const void* k, const void* v, const void* gk, const void* gate,
              const float* norm_weight, float eps, bool gated, void* o, int B, int H, int dk, int dv,
              int dtype, float* state, int64_t n_slots, const int32_t* slots, void* stream) {
  if (B < 0 || H < 0 || n_slots < 0) return GLA_E_ARG;
  if (dtype != GLA_F16 && dtype != GLA_F32) return GLA_E_ARG;
  if ((dk != 32 && dk != 64) || (dv != 32 && dv != 64)) return GLA_E_UNSUPPORTED;
  if (B > 65535 || H > 65535 || n_slots > (1LL << 31)) return GLA_E_UNSUPPORTED;
  if (B == 0 || H == 0) return GLA_OK;
  GLA_TRY(check_tensor(q));
  GLA_TRY(check_tensor(k));
  GLA_TRY(check_tensor(v));
  GLA_TRY(check_tensor(gk));
  GLA_TRY(check_tensor(o));
  GLA_TRY(check_tensor(state));
  if (slots ? !aligned(slots, 4) : n_slots < B) return GLA_E_ARG;
  if (gated) {
    GLA_TRY(check_tensor(gate));
    if (!norm_weight || !aligned(norm_weight, 16) || !(eps >= 0.f)) return GLA_E_ARG;
  }
  const size_t es = elem(dtype), nk = (size_t)B * H * dk * es, nv = (size_t)B * H * dv * es;
  const size_t ns = (size_t)n_slots * H * dk * dv * sizeof(float);
  GLA_TRY(check_disjoint<2, 7>(
      {{o, nv}, {state, ns}},
      {{q, nk}, {k, nk}, {v, nv}, {gk, nk}, {slots, (size_t)B * sizeof(int32_t)},
       {gated ? gate : nullptr, nv}, {gated ? norm_weight : nullptr, dv * sizeof(float)}}));
  gla::StepArgs a{B, H, dk, dv, dtype, q, k, v, gk, o, state, (long)n_slots, slots, gla::Epilogue()};
  if (gated) a.epi.gate = gate, a.epi.weight = norm_weight, a.epi.eps = eps;
  const hipError_t e = gla::launch_step(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail_hip(e, "step launch");
  return GLA_OK;
}

}  // namespace

extern "C" {

size_t gla_bwd_workspace_bytes(int B, int H, int grid_h, int grid_w, int dk, int dv) {
  gla::Problem p;
  bool empty;
  if (make_problem(B, H, grid_h, grid_w, dk, dv, gla::kBwdChunk, GLA_F16, &p, &empty) != GLA_OK)
    return 0;
  return empty ? 0 : gla::bwd_layout(p).total;
}

int gla_bwd(const void* q, const void* k, const void* v, const void* gk, const void* go, void* gq,
            void* gkey, void* gv, void* ggk, int B, int H, int grid_h, int grid_w, int dk, int dv,
            const int32_t* dir, int dtype, const float* s0, const float* gs_final, float* gs0,
            void* workspace, size_t workspace_bytes, void* stream) {
  gla::Problem p;
  bool empty;
  GLA_TRY(make_problem(B, H, grid_h, grid_w, dk, dv, gla::kBwdChunk, dtype, &p, &empty));
  if (empty) return GLA_OK;
  if (p.T > 0x7fffffff - gla::kBwdChunk) return GLA_E_UNSUPPORTED;
  for (const void* t : {q, k, v, gk, go}) GLA_TRY(check_tensor(t));
  for (const void* t : {gq, gkey, gv, ggk}) GLA_TRY(check_tensor(t));
  GLA_TRY(check_optional(s0));
  GLA_TRY(check_optional(gs_final));
  GLA_TRY(check_optional(gs0));
  GLA_TRY(check_dirs(dir, B));
  const size_t need = gla::bwd_layout(p).total;
  GLA_TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t rows = (size_t)B * p.T * H, nk = rows * dk * elem(dtype), nv = rows * dv * elem(dtype);
  const size_t ns = (size_t)B * H * dk * dv * sizeof(float);
  // gs0 may be gs_final itself (each element is read before it is written)
  GLA_TRY(check_disjoint<6, 7>(
      {{gq, nk}, {gkey, nk}, {gv, nv}, {ggk, nk}, {gs0, ns}, {workspace, need}},
      {{q, nk}, {k, nk}, {v, nv}, {gk, nk}, {go, nv}, {s0, ns},
       {(const void*)gs_final == (const void*)gs0 ? nullptr : gs_final, ns}}));
  const gla::BwdArgs a{q, k, v, gk, go, gq, gkey, gv, ggk, s0, gs_final, gs0};
  // at most 2^21 chains (batch elements x heads) per launch: the scans take a
  // thread per four state elements
  int most = (1 << 21) / H;
  if (most > gla::kMaxBatchPerLaunch) most = gla::kMaxBatchPerLaunch;
  for (int b0 = 0; b0 < B; b0 += most) {
    const int nb = B - b0 < most ? B - b0 : most;
    const hipError_t e = gla::launch_bwd(p, b0, nb, pack_dirs(dir, b0, nb), a,
                                         static_cast<char*>(workspace),
                                         static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail_hip(e, "backward launch");
  }
  return GLA_OK;
}

int gla_step(const void* q, const void* k, const void* v, const void* gk, void* o, int B, int H,
             int dk, int dv, int dtype, float* state, int64_t n_slots, const int32_t* slots,
             void* stream) {
  return step_impl(q, k, v, gk, nullptr, nullptr, 0.f, false, o, B, H, dk, dv, dtype, state, n_slots,
                   slots, stream);
}

int gla_step_gated(const void* q, const void* k, const void* v, const void* gk, const void* gate,
                   const float* norm_weight, float eps, void* y, int B, int H, int dk, int dv,
                   int dtype, float* state, int64_t n_slots, const int32_t* slots, void* stream) {
  return step_impl(q, k, v, gk, gate, norm_weight, eps, true, y, B, H, dk, dv, dtype, state, n_slots,
                   slots, stream);
}

int gla_add_rmsnorm(const void* x, const void* residual, const float* weight, float eps, void* sum,
                    void* y, int64_t rows, int F, int dtype, void* stream) {
  return add_rmsnorm_impl(x, residual, weight, eps, sum, y, nullptr, nullptr, rows, F, dtype, stream);
}

int gla_add_rmsnorm_q8(const void* x, const void* residual, const float* weight, float eps, void* sum,
                       void* y8, float* scales, int64_t rows, int F, int dtype, void* stream) {
  GLA_TRY(check_rows(rows, F, dtype));
  if (rows > 0 && F > 0 && !y8) return GLA_E_ARG;
  return add_rmsnorm_impl(x, residual, weight, eps, sum, nullptr, y8, scales, rows, F, dtype, stream);
}

size_t gla_add_rmsnorm_bwd_workspace_bytes(int64_t rows, int F) {
  if (check_rows(rows, F, GLA_F16) != GLA_OK || rows == 0 || F == 0) return 0;
  return gla::norm_bwd_workspace((long)rows, F);
}

int gla_add_rmsnorm_bwd(const void* sum, const float* weight, float eps, const void* gy,
                        const void* gsum, void* gx, float* gweight, int64_t rows, int F, int dtype,
                        void* workspace, size_t workspace_bytes, void* stream) {
  GLA_TRY(check_rows(rows, F, dtype));
  if (rows == 0 || F == 0) return GLA_OK;
  GLA_TRY(check_tensor(sum));
  GLA_TRY(check_tensor(gy));
  GLA_TRY(check_optional(gsum));
  GLA_TRY(check_tensor(gx));
  GLA_TRY(check_tensor(gweight));
  if (!weight || !aligned(weight, 16) || !(eps >= 0.f)) return GLA_E_ARG;
  const size_t need = gla::norm_bwd_workspace((long)rows, F);
  GLA_TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t nb = (size_t)rows * F * elem(dtype), nw = (size_t)F * sizeof(float);
  GLA_TRY(check_disjoint<2, 4>({{gweight, nw}, {workspace, need}},
                               {{weight, nw}, {sum, nb}, {gy, nb}, {gsum, nb}}));
  GLA_TRY(check_disjoint<3, 1>({{gweight, nw}, {workspace, need}, {gx, nb}}, {{weight, nw}}));
  for (const void* in : {sum, gy, gsum})  // gx may be one of them, row for row
    if (in && gx != in && overlaps(gx, nb, in, nb)) return GLA_E_ARG;
  gla::NormBwdArgs a{(long)rows, F, dtype, sum, gy, gsum, weight, eps, gx, gweight};
  const hipError_t e =
      gla::launch_norm_bwd(a, static_cast<float*>(workspace), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail_hip(e, "rmsnorm backward launch");
  return GLA_OK;
}

size_t gla_gate_bwd_workspace_bytes(int64_t rows, int dv) {
  if (rows <= 0 || rows > (1LL << 40) || (dv != 32 && dv != 64)) return 0;
  return gla::gate_bwd_workspace((long)rows, dv);
}

int gla_gate_bwd(const void* o, const void* gate, const float* norm_weight, float eps, const void* gy,
                 void* go, void* ggate, float* gnorm_weight, int64_t rows, int dv, int dtype,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if (rows < 0) return GLA_E_ARG;
  if (dtype != GLA_F16 && dtype != GLA_F32) return GLA_E_ARG;
  if ((dv != 32 && dv != 64) || rows > (1LL << 40)) return GLA_E_UNSUPPORTED;
  if (rows == 0) return GLA_OK;
  for (const void* t : {o, gate, gy}) GLA_TRY(check_tensor(t));
  GLA_TRY(check_tensor(go));
  GLA_TRY(check_tensor(ggate));
  GLA_TRY(check_tensor(gnorm_weight));
  if (!norm_weight || !aligned(norm_weight, 16) || !(eps >= 0.f)) return GLA_E_ARG;
  const size_t need = gla::gate_bwd_workspace((long)rows, dv);
  GLA_TRY(check_workspace(workspace, workspace_bytes, need));
  const size_t nb = (size_t)rows * dv * elem(dtype), nw = dv * sizeof(float);
  GLA_TRY(check_disjoint<4, 4>({{go, nb}, {ggate, nb}, {gnorm_weight, nw}, {workspace, need}},
                               {{o, nb}, {gate, nb}, {gy, nb}, {norm_weight, nw}}));
  gla::GateBwdArgs a{(long)rows, dv, dtype, o, gate, gy, norm_weight, eps, go, ggate, gnorm_weight};
  const hipError_t e =
      gla::launch_gate_bwd(a, static_cast<float*>(workspace), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail_hip(e, "gate backward launch");
  return GLA_OK;
}

}  // extern "C"
