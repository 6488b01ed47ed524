// Gradients of the products in gla_linear.hip. With gp the gradient behind the
// activation, gp = gy act'(pre) (gated: ga = gh u act'(a), gu = gh act(a)),
//   gx = alpha gp W,   gW = alpha gp^T x,   gbias = alpha sum over rows of gp:
// one pass forms gp (and the column sums) and two products follow, whose
// operands lie down the columns where the forward's lie along the contraction.
// gp is kept in the input type between them, as gy itself is; sums are float. Half, the
// rounding of every gp by up to 2^-11 adds to that of the outputs: 2.9e-4 of the largest
// value against 64 bits, 2.1e-4 without. A second term for what it leaves would double
// both products (25,600 x 768 x 2,048 gated: 323 of 390 us), and dividing values beyond
// half's range by a power of two takes either a launch more for every call (17.3 -> 19.9
// us for 421 x 384 x 1,032) and digits of all other rows, or a look at every step of the
// products (5 to 20% more).
#include "gla_linear.h"

#include "gla_colsum.h"
#include "gla_gemm.h"

namespace gla {
namespace gemm {

// Half gradients behind silu and gelu are kept times 7/8: slopes reach 1.0998 and
// 1.1290 (0.988 times 8/7), so that a gradient of up to 65504 stays one. (A half of
// them would lose a bit of those below 2^-14.)
template <typename T>
float kept_factor(int act) {
  return sizeof(T) == 2 && (act == 1 || act == 2) ? 0.875f : 1.f;
}

// gp = gy act'(pre), `keep` times, and/or alpha times its column sums over the rows
// of this workgroup (part[blockIdx.y][N]). 2^shift threads side by side take eight
// columns each, the others further rows. 1,600 x 768 half 6.0 us (7.4 MB): a load's,
// the exchange's and a launch's latency.
template <typename T>
__global__ __launch_bounds__(256) void slope_kernel(const T* __restrict__ pre, const T* __restrict__ gy,
                                                    T* __restrict__ gp, float* __restrict__ part,
                                                    float alpha, float keep, int act, long rows, int N, int shift) {
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
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[c] += g[c], g[c] *= keep;
      if (gp) store8(gp + r * N + n, g);
    }
  }
  if (!part) return;
#pragma unroll
  for (int c = 0; c < 8; ++c) s[threadIdx.x][c] = sum[c];
  __syncthreads();
  const long col = ((8L * blockIdx.x) << shift) + threadIdx.x;  // one column a thread
  if (threadIdx.x >= 8 << shift || col >= N) return;
  float y = 0.f;
  for (int t = 0; t < per; ++t) y += s[(threadIdx.x >> 3) + (t << shift)][threadIdx.x & 7];
  part[(long)blockIdx.y * N + col] = alpha * y;
}

// ga = gh u act'(a), gu = gh act(a), eight values a thread. Bound by memory: 25,600 x
// 2,048 half 92 us, 525 MB at 5.7 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void gated_slope_kernel(const T* __restrict__ ap, const T* __restrict__ up,
                                                          const T* __restrict__ ghp, T* __restrict__ gap,
                                                          T* __restrict__ gup, int act, long groups) {
  for (long t = 256L * blockIdx.x + threadIdx.x; t < groups; t += 256L * gridDim.x) {
    float a[8], u[8], g[8];
    load8(ap + 8 * t, a);
    load8(up + 8 * t, u);
    load8(ghp + 8 * t, g);
    if (act == 1 || act == 2) {  // zero at -Inf, as a kept product below half's range is stored
#pragma unroll
      for (int c = 0; c < 8; ++c) a[c] = a[c] == -__builtin_inff() ? -65504.f : a[c];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) u[c] *= g[c] * slope(a[c], act);
    activate(a, act);
#pragma unroll
    for (int c = 0; c < 8; ++c) a[c] *= g[c];
    store8(gap + 8 * t, u);
    store8(gup + 8 * t, a);
  }
}

// out = alpha times the sum over the splits, for both parts of the weights. Five
// splits of 2 x 2,048 x 768 11 us (69 MB), three of 520 x 1,000 4.8: a launch.
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

// The sums over a gradient's partial rows, in the launch of its products.
struct Sums {
  const float* part;  // [parts][N], or nullptr
  float* out;
  int parts, N;
};

// Both products of a gradient and its column sums in one launch, for those that
// leave CUs idle or cost little more than a launch: workgroups 0 .. nw - 1 take
// the weights' tiles, the next nx the input's, the others 16 columns each. 1,600 x
// 768 x 768 half: the whole gradient 19 us instead of 28; what is left is the 25
// steps of a weights' tile.
template <typename T, int kTile>
__global__ __launch_bounds__((kTileThreads<T, kTile, false>)) void pair_kernel(const Args x, const Args w, const Sums sums,
                                                                          int nx, int nw) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) char shared[kTileBytes<T, kTile, false>];
  const int id = blockIdx.x;
  if (id < nw) {
    gemm_tile<T, kTile, true, true, kLinear>(w, id, nw, shared);
  } else if (id < nw + nx) {
    gemm_tile<T, kTile, false, true, kLinear>(x, id - nw, nx, shared);
  } else {
    constexpr int G = kTileThreads<T, kTile, false> / 16, W = 8;
    float(*s)[17] = reinterpret_cast<float(*)[17]>(shared);
    const int c = threadIdx.x & 15, g = threadIdx.x >> 4, col = (id - nw - nx) * 16 + c;
    float y = 0.f;
    if (col < sums.N) {
      for (int p = g; p < sums.parts; p += G * W) {
        float v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = p + G * i < sums.parts ? sums.part[(long)(p + G * i) * sums.N + col] : 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) y += v[i];
      }
    }
    s[g][c] = y;
    __syncthreads();
    if (g == 0 && col < sums.N) {
      for (int i = 1; i < G; ++i) y += s[i][c];
      sums.out[col] = y;
    }
  }
#endif
}

template <typename T, int kTile = k128x128>
hipError_t launch_pair(Args x, Args w, const Sums& sums, int tile, hipStream_t s) {
  if constexpr (kTile == kTiles) {
    return hipErrorInvalidValue;
  } else {
    if (tile != kTile) return launch_pair<T, kTile + 1>(x, w, sums, tile, s);
    constexpr TileShape S = tile_shape(kTile, sizeof(T) == 4, false);
    for (Args* g : {&x, &w}) g->tiles_m = (int)((g->M + S.m - 1) / S.m), g->tiles_n = (int)((g->N + S.n - 1) / S.n);
    const int nx = x.tiles_m * x.tiles_n, nw = w.tiles_m * w.mparts * w.tiles_n * w.splits;
    const int ns = sums.part ? (sums.N + 15) / 16 : 0;
    hipLaunchKernelGGL((pair_kernel<T, kTile>), dim3((unsigned)(nx + nw + ns)), dim3(kTileThreads<T, kTile, false>), 0, s,
                       x, w, sums, nx, nw);
    return hipGetLastError();
  }
}

// Tiles of both products and splits of the weights' long contraction, by the
// tiles' cost, that of the partial sums' way through memory (4 TB/s and a
// launch), and whether one launch for both is less (a launch costs 3 us, and
// half of the longer tile is left at its end).
template <typename T>
void plan(long rows, int K, int N, int mparts, LinearBwdLayout* l) {
  const long step = Num<T>::kStep, steps = (rows + step - 1) / step, steps_x = mparts * ((N + step - 1) / step);
  float x, least = 0.f;
  l->tile_x = best_tile<T, false>(rows < 1L << 22 ? rows : 1L << 22, K, 1, steps_x, &x);
  l->steps = steps;
  for (long s : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32}) {
    if (s > 1 && steps < 4 * s) break;
    const long each = (steps + s - 1) / s, splits = (steps + each - 1) / each;
    const float join = splits > 1 ? 4.f + 2e-6f * splits * mparts * N * K : 0.f;
    float w;
    const int t = best_tile<T, true>(N, K, mparts * splits, each, &w);
    float c = w + join + x + 3.f;
    if (least == 0.f || c < least) least = c, l->tile_w = t, l->splits = (int)splits, l->each = each, l->pair = false;
    for (int p = k128x128; rows <= 1L << 20 && p < kTiles; ++p) {
      const TileShape a = tile_shape(p, sizeof(T) == 4, false);
      const long nx = tile_count(a, rows, K), nw = tile_count(a, N, K) * mparts * splits;
      const long slots = (long)kCus * a.per_cu, per = (nx + nw + kCus - 1) / kCus;
      const long on = per < a.per_cu ? per : a.per_cu;
      const float rx = round_cost<T>(a, steps_x, on, false), rw = round_cost<T>(a, each, on, true);
      const float longer = rx > rw ? rx : rw;
      c = join + (nx + nw <= slots ? longer : (nx * rx + nw * rw) / slots + 0.5f * longer);
      if (c < least) least = c, l->tile_w = l->tile_x = p, l->splits = (int)splits, l->each = each, l->pair = true;
    }
    if (!l->pair) l->tile_x = best_tile<T, false>(rows < 1L << 22 ? rows : 1L << 22, K, 1, steps_x);
  }
}

// gx = alpha (a[0] b[0] + a[1] b[1]), a [rows][C], b [C][N]
template <typename T>
Args input_gradient(const void* a0, const void* a1, const void* b0, const void* b1, long rows, int C, int N, int parts,
                    float alpha, void* gx) {
  Args g = {};
  g.a[0] = a0, g.a[1] = a1, g.b[0] = b0, g.b[1] = b1, g.out[0] = gx, g.alpha = alpha;
  g.M = rows, g.K = g.lda = C, g.ldb = g.N = N, g.parts = parts, g.mparts = g.splits = 1;
  g.steps = g.each = parts * ((C + Num<T>::kStep - 1) / Num<T>::kStep);
  return g;
}
// out[p] = alpha a[p]^T x, a[p] [rows][N], x [rows][K]
template <typename T>
Args weight_gradient(const void* a0, const void* a1, const void* x, long rows, int K, int N, int mparts, float alpha,
                     void* out0, void* out1, const LinearBwdLayout& l, char* ws) {
  Args g = {};
  g.a[0] = a0, g.a[1] = a1, g.b[0] = g.b[1] = x, g.out[0] = out0, g.out[1] = out1, g.alpha = alpha;
  g.M = g.lda = N, g.N = g.ldb = K, g.K = rows, g.parts = 1, g.mparts = mparts;
  g.splits = l.splits, g.steps = l.steps, g.each = l.each;
  g.partial = reinterpret_cast<float*>(ws + l.partial);
  return g;
}

template <typename T>
hipError_t launch_input(Args g, int tile, hipStream_t s) {
  constexpr long most = 1L << 22;  // rows per launch, so that the grid's numbers fit 32 bits
  const Args all = g;
  for (long r = 0; r < all.M; r += most) {
    g.M = all.M - r < most ? all.M - r : most;
    for (int p = 0; p < g.parts; ++p) g.a[p] = static_cast<const T*>(all.a[p]) + r * g.lda;
    g.out[0] = static_cast<T*>(all.out[0]) + r * g.N;
    const hipError_t e = launch_product<T, false, true, kLinear>(g, tile, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The products of a gradient, each wanted where its output is, and its column
// sums where they are.
template <typename T>
hipError_t launch_products(const Args& x, const Args& w, const Sums& sums, const LinearBwdLayout& l, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (l.pair && x.out[0] && w.out[0]) {
    e = launch_pair<T>(x, w, sums, l.tile_x, s);
  } else {
    if (sums.part) {
      hipLaunchKernelGGL(norm::column_sum_kernel, dim3((sums.N + 15) / 16), dim3(1024), 0, s, sums.part, sums.out,
                         sums.parts, sums.N);
      e = hipGetLastError();
    }
    if (e == hipSuccess && x.out[0]) e = launch_input<T>(x, l.tile_x, s);
    if (e == hipSuccess && w.out[0]) e = launch_product<T, true, true, kLinear>(w, l.tile_w, s);
  }
  if (e != hipSuccess || !w.out[0] || w.splits == 1) return e;
  const long per_part = w.M * w.N / 8, groups = w.mparts * per_part;
  hipLaunchKernelGGL((join_kernel<T>), dim3(spread((groups + 255) / 256)), dim3(256), 0, s, w.partial,
                     static_cast<T*>(w.out[0]), static_cast<T*>(w.out[1]), w.alpha, w.splits, groups, per_part);
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
  if (dtype == 0) plan<half_t>(rows, K, N, mparts, &l);
  else plan<float>(rows, K, N, mparts, &l);
  if (l.splits > 1) at += pad((size_t)l.splits * mparts * N * K * sizeof(float));
  l.total = at ? at : 256;
  return l;
}

template <typename T>
hipError_t linear_bwd_t(const LinearBwdArgs& a, const LinearBwdLayout& l, char* ws, hipStream_t s) {
  T* gp = reinterpret_cast<T*>(ws + l.g[0]);
  Sums sums = {};
  const bool own = a.act != 0, products = a.gx || a.gweight;
  if ((own && products) || a.gbias) {
    const SlopePlan p = slope_plan(a.rows, a.N);
    if (a.gbias) sums = Sums{reinterpret_cast<float*>(ws + l.colsum), a.gbias, p.parts, a.N};
    hipLaunchKernelGGL((slope_kernel<T>), dim3(p.blocks, p.parts), dim3(256), 0, s,
                       own ? static_cast<const T*>(a.pre) : nullptr, static_cast<const T*>(a.gy),
                       own && products ? gp : nullptr, const_cast<float*>(sums.part), a.alpha, kept_factor<T>(a.act),
                       a.act, a.rows, a.N, p.shift);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const void* g = own ? gp : a.gy;
  const float alpha = a.alpha / kept_factor<T>(a.act);
  return launch_products<T>(
      input_gradient<T>(g, nullptr, a.weight, nullptr, a.rows, a.N, a.K, 1, alpha, a.gx),
      weight_gradient<T>(g, nullptr, a.x, a.rows, a.K, a.N, 1, alpha, a.gweight, a.gweight, l, ws), sums, l, s);
}

template <typename T>
hipError_t gated_bwd_t(const GatedBwdArgs& a, const LinearBwdLayout& l, char* ws, hipStream_t s) {
  T *ga = reinterpret_cast<T*>(ws + l.g[0]), *gu = reinterpret_cast<T*>(ws + l.g[1]);
  const long groups = a.rows * a.F / 8;
  hipLaunchKernelGGL((gated_slope_kernel<T>), dim3(spread((groups + 255) / 256)), dim3(256), 0, s,
                     static_cast<const T*>(a.gate), static_cast<const T*>(a.up),
                     static_cast<const T*>(a.gh), ga, gu, a.act, groups);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_products<T>(
      input_gradient<T>(ga, gu, a.gate_weight, a.up_weight, a.rows, a.F, a.K, 2, 1.f, a.gx),
      weight_gradient<T>(ga, gu, a.x, a.rows, a.K, a.F, 2, 1.f, a.ggate_weight, a.gup_weight, l, ws), Sums{}, l, s);
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
