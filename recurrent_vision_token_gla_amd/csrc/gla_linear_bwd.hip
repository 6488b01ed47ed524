// Gradients of the products in gla_linear.hip. With gp the gradient behind the
// activation, gp = gy act'(pre) (gated: ga = gh u act'(a), gu = gh act(a)),
//   gx = alpha gp W,   gW = alpha gp^T x,   gbias = alpha sum over rows of gp:
// one pass forms gp (and the column sums) and two products follow, whose
// operands lie down the columns where the forward's lie along the contraction.
// gp is kept in the input type between them, as gy itself is; sums are float.
#include "gla_linear.h"

#include "gla_colsum.h"
#include "gla_gemm.h"

namespace gla {
namespace gemm {

// gp = gy act'(pre) and/or alpha times its column sums over the rows of this
// workgroup (part[blockIdx.y][N]). 2^shift threads side by side take eight
// columns each, the others further rows.
template <typename T>
__global__ __launch_bounds__(256) void slope_kernel(const T* __restrict__ pre, const T* __restrict__ gy,
                                                    T* __restrict__ gp, float* __restrict__ part,
                                                    float alpha, int act, long rows, int N, int shift) {
  __shared__ float s[256][9];
  const int tx = threadIdx.x & ((1 << shift) - 1), ty = threadIdx.x >> shift, per = 256 >> shift;
  const long n = 8L * (((long)blockIdx.x << shift) + tx);
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (n < N) {
    for (long r = (long)blockIdx.y * per + ty; r < rows; r += (long)gridDim.y * per) {
      float g[8];
      load8(gy + r * N + n, g);
      if (pre) {
        float z[8];
        load8(pre + r * N + n, z);
#pragma unroll
        for (int c = 0; c < 8; ++c) g[c] *= slope(z[c], act);
      }
      if (gp) store8(gp + r * N + n, g);
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[c] += g[c];
    }
  }
  if (!part) return;
#pragma unroll
  for (int c = 0; c < 8; ++c) s[threadIdx.x][c] = sum[c];
  __syncthreads();
  if (ty == 0 && n < N) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      float y = 0.f;
      for (int t = 0; t < per; ++t) y += s[tx + (t << shift)][c];
      sum[c] = alpha * y;
    }
    tile::store_f8(part + (long)blockIdx.y * N + n, sum);
  }
}

// ga = gh u act'(a), gu = gh act(a), eight values a thread.
template <typename T>
__global__ __launch_bounds__(256) void gated_slope_kernel(const T* __restrict__ ap, const T* __restrict__ up,
                                                          const T* __restrict__ ghp, T* __restrict__ gap,
                                                          T* __restrict__ gup, int act, long groups) {
  for (long t = 256L * blockIdx.x + threadIdx.x; t < groups; t += 256L * gridDim.x) {
    float a[8], u[8], g[8];
    load8(ap + 8 * t, a);
    load8(up + 8 * t, u);
    load8(ghp + 8 * t, g);
#pragma unroll
    for (int c = 0; c < 8; ++c) u[c] *= g[c] * slope(a[c], act);
    activate(a, act);
#pragma unroll
    for (int c = 0; c < 8; ++c) a[c] *= g[c];
    store8(gap + 8 * t, u);
    store8(gup + 8 * t, a);
  }
}

// out = alpha times the sum over the splits, for both parts of the weights.
template <typename T>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ partial, T* out0, T* out1,
                                                   float alpha, int splits, long groups, long per_part) {
  for (long t = 256L * blockIdx.x + threadIdx.x; t < groups; t += 256L * gridDim.x) {
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s) {
      float x[8];
      load8(partial + 8 * (s * groups + t), x);
#pragma unroll
      for (int c = 0; c < 8; ++c) y[c] += x[c];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) y[c] *= alpha;
    store8(t < per_part ? out0 + 8 * t : out1 + 8 * (t - per_part), y);
  }
}

// Workgroups that a grid-stride pass over `n` units takes.
unsigned spread(long n) { return (unsigned)(n < 4096 ? n : 4096); }

// The weights' gradient: its tiles, and the splits of its long contraction, by
// the tiles' cost and that of the partial sums' way through memory (4 TB/s and
// a launch).
template <typename T>
void weight_plan(long rows, int K, int N, int mparts, LinearBwdLayout* l) {
  const long step = Num<T>::kStep, steps = (rows + step - 1) / step;
  float least = 0.f;
  for (long s : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32}) {
    if (s > 1 && steps < 4 * s) break;
    const long each = (steps + s - 1) / s, splits = (steps + each - 1) / each;
    const float join = splits > 1 ? 4.f + 2e-6f * splits * mparts * N * K : 0.f;
    float c;
    const int t = best_tile<T, true, kPartial>(N, K, mparts * splits, each, &c);
    c += join;
    if (least == 0.f || c < least) least = c, l->tile_w = t, l->splits = (int)splits, l->each = each;
  }
  l->steps = steps;
}

// gx = alpha (a[0] b[0] + a[1] b[1]), a [rows][C], b [C][N]
template <typename T>
hipError_t input_gradient(Args g, long rows, int C, int N, int parts, float alpha, T* gx, int tile,
                          hipStream_t s) {
  constexpr long most = 1L << 22, step = Num<T>::kStep;
  g.K = g.lda = C, g.ldb = g.N = N, g.alpha = alpha, g.parts = parts, g.mparts = g.splits = 1;
  const T* a[2] = {static_cast<const T*>(g.a[0]), static_cast<const T*>(g.a[1])};
  g.steps = g.each = parts * ((C + step - 1) / step);
  for (long r = 0; r < rows; r += most) {
    g.M = rows - r < most ? rows - r : most;
    for (int p = 0; p < parts; ++p) g.a[p] = a[p] + r * C;
    g.out[0] = gx + r * N;
    const hipError_t e = launch_product<T, false, true, kLinear>(g, tile, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// out[p] = alpha a[p]^T x, a[p] [rows][N], x [rows][K]
template <typename T>
hipError_t weight_gradient(Args g, long rows, int K, int N, int mparts, float alpha, const LinearBwdLayout& l,
                           float* partial, hipStream_t s) {
  g.lda = N, g.ldb = K, g.M = N, g.N = K, g.K = rows, g.alpha = alpha;
  g.parts = 1, g.mparts = mparts, g.splits = l.splits, g.steps = l.steps, g.each = l.each;
  g.partial = partial;
  if (l.splits == 1) return launch_product<T, true, true, kLinear>(g, l.tile_w, s);
  const hipError_t e = launch_product<T, true, true, kPartial>(g, l.tile_w, s);
  if (e != hipSuccess) return e;
  const long per_part = (long)N * K / 8, groups = mparts * per_part;
  hipLaunchKernelGGL((join_kernel<T>), dim3(spread((groups + 255) / 256)), dim3(256), 0, s, partial,
                     static_cast<T*>(g.out[0]), static_cast<T*>(g.out[1]), alpha, l.splits, groups, per_part);
  return hipGetLastError();
}

// Threads side by side and row parts of slope_kernel.
struct SlopePlan {
  int shift, blocks, parts;
};
SlopePlan slope_plan(long rows, int N) {
  SlopePlan p;
  p.shift = 0;
  while (p.shift < 5 && (8 << p.shift) < N) ++p.shift;
  p.blocks = (N / 8 + (1 << p.shift) - 1) >> p.shift;
  const long per = 256 >> p.shift, steps = (rows + per - 1) / per;
  long most = 2048 / p.blocks;
  if (most < 1) most = 1;
  const long each = (steps + most - 1) / most;
  p.parts = (int)((steps + each - 1) / each);
  return p;
}

size_t pad(size_t n) { return (n + 255) & ~(size_t)255; }

template <typename T>
void input_plan(long rows, int K, int N, int parts, LinearBwdLayout* l) {
  const long step = Num<T>::kStep;
  l->tile_x = best_tile<T, false, kLinear>(rows < 1L << 22 ? rows : 1L << 22, K, 1, parts * ((N + step - 1) / step));
}

LinearBwdLayout layout(long rows, int K, int N, int dtype, int sides, bool sums, int mparts) {
  LinearBwdLayout l = {};
  const size_t es = dtype == 0 ? 2 : 4;
  size_t at = 0;
  for (int p = 0; p < 2; ++p) {
    l.g[p] = at;
    if (p < sides) at += pad((size_t)rows * N * es);
  }
  l.colsum = at;
  if (sums) at += pad((size_t)slope_plan(rows, N).parts * N * sizeof(float));
  l.partial = at;
  if (dtype == 0) weight_plan<half_t>(rows, K, N, mparts, &l), input_plan<half_t>(rows, K, N, mparts, &l);
  else weight_plan<float>(rows, K, N, mparts, &l), input_plan<float>(rows, K, N, mparts, &l);
  if (l.splits > 1) at += pad((size_t)l.splits * mparts * N * K * sizeof(float));
  l.total = at ? at : 256;
  return l;
}

template <typename T>
hipError_t linear_bwd_t(const LinearBwdArgs& a, const LinearBwdLayout& l, char* ws, hipStream_t s) {
  T* gp = reinterpret_cast<T*>(ws + l.g[0]);
  float* sums = reinterpret_cast<float*>(ws + l.colsum);
  const bool own = a.act != 0;
  const bool wanted = a.gx || a.gweight;
  if ((own && wanted) || a.gbias) {
    const SlopePlan p = slope_plan(a.rows, a.N);
    hipLaunchKernelGGL((slope_kernel<T>), dim3(p.blocks, p.parts), dim3(256), 0, s,
                       own ? static_cast<const T*>(a.pre) : nullptr, static_cast<const T*>(a.gy),
                       own && wanted ? gp : nullptr, a.gbias ? sums : nullptr, a.alpha, a.act, a.rows, a.N,
                       p.shift);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.gbias) {
      hipLaunchKernelGGL(norm::column_sum_kernel, dim3((a.N + 15) / 16), dim3(1024), 0, s, sums, a.gbias,
                         p.parts, a.N);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  const void* g = own ? gp : a.gy;
  Args args = {};
  args.a[0] = g;
  if (a.gx) {
    args.b[0] = args.b[1] = a.weight;
    const hipError_t e = input_gradient<T>(args, a.rows, a.N, a.K, 1, a.alpha, static_cast<T*>(a.gx),
                                             l.tile_x, s);
    if (e != hipSuccess) return e;
  }
  if (!a.gweight) return hipSuccess;
  args.b[0] = args.b[1] = a.x;
  args.out[0] = args.out[1] = a.gweight;
  return weight_gradient<T>(args, a.rows, a.K, a.N, 1, a.alpha, l, reinterpret_cast<float*>(ws + l.partial), s);
}

template <typename T>
hipError_t gated_bwd_t(const GatedBwdArgs& a, const LinearBwdLayout& l, char* ws, hipStream_t s) {
  T *ga = reinterpret_cast<T*>(ws + l.g[0]), *gu = reinterpret_cast<T*>(ws + l.g[1]);
  const long groups = a.rows * a.F / 8;
  hipLaunchKernelGGL((gated_slope_kernel<T>), dim3(spread((groups + 255) / 256)), dim3(256), 0, s,
                     static_cast<const T*>(a.gate), static_cast<const T*>(a.up),
                     static_cast<const T*>(a.gh), ga, gu, a.act, groups);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  Args args = {};
  args.a[0] = ga, args.a[1] = gu, args.b[0] = a.gate_weight, args.b[1] = a.up_weight;
  if (a.gx) {
    e = input_gradient<T>(args, a.rows, a.F, a.K, 2, 1.f, static_cast<T*>(a.gx), l.tile_x, s);
    if (e != hipSuccess) return e;
  }
  if (!a.ggate_weight) return hipSuccess;
  args.b[0] = args.b[1] = a.x;
  args.out[0] = a.ggate_weight, args.out[1] = a.gup_weight;
  return weight_gradient<T>(args, a.rows, a.K, a.F, 2, 1.f, l, reinterpret_cast<float*>(ws + l.partial), s);
}

}  // namespace gemm

LinearBwdLayout linear_bwd_layout(long rows, int K, int N, int act, int dtype) {
  return gemm::layout(rows, K, N, dtype, act != 0 ? 1 : 0, true, 1);
}
LinearBwdLayout gated_bwd_layout(long rows, int K, int F, int dtype) {
  return gemm::layout(rows, K, F, dtype, 2, false, 2);
}

hipError_t launch_linear_bwd(const LinearBwdArgs& a, const LinearBwdLayout& l, char* ws, hipStream_t s) {
  return a.dtype == 0 ? gemm::linear_bwd_t<half_t>(a, l, ws, s) : gemm::linear_bwd_t<float>(a, l, ws, s);
}
hipError_t launch_gated_bwd(const GatedBwdArgs& a, const LinearBwdLayout& l, char* ws, hipStream_t s) {
  return a.dtype == 0 ? gemm::gated_bwd_t<half_t>(a, l, ws, s) : gemm::gated_bwd_t<float>(a, l, ws, s);
}

}  // namespace gla
