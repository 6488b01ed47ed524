// The products around a block's mixers: y = alpha act(x W^T + b) + residual, and
// the gated h = act(x Wg^T) * (x Wu^T) from one reading of x, with everything
// behind the sums in the kernel that forms them.
#include "gla_linear.h"

#include "gla_gemm.h"

namespace gla {
namespace gemm {

// Up to 16 MI rows. A workgroup takes 16 columns (gated: 16 of both weights);
// its eight waves take steps of the contraction in turn, straight from memory
// into the operands of the matrix cores: lane i, q holds row i and the 32 bytes
// 32 q .. of the step's 128, whole lines of a weight row by four lanes. The
// waves' sums meet in LDS.
constexpr int kSkinnyWaves = 8;

template <typename T, int MI, bool kDual>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_kernel(const Args g) {
  constexpr int kUnit = Num<T>::kUnit, kStep = Num<T>::kStep, ND = kDual ? 2 : 1;
  using Frag = typename std::conditional<sizeof(T) == 2, half8, floatx4>::type;
  __shared__ __attribute__((aligned(16))) float red[kSkinnyWaves][ND][16 * MI][16];
  const int i = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3, w = wave();
  const long n0 = 16L * blockIdx.x, n = min(n0 + i, g.N - 1);
  const T* pw[2] = {static_cast<const T*>(g.b[0]) + n * g.ldb, static_cast<const T*>(g.b[ND - 1]) + n * g.ldb};
  const T* px[MI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) px[mi] = static_cast<const T*>(g.a[0]) + min(16L * mi + i, g.M - 1) * g.lda;
  floatx4 acc[ND][MI];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) acc[d][mi] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int steps = (int)g.steps;
  // two steps a round, all of their loads in flight; beyond the contraction's
  // end they read its last elements, which then count as zero
  for (int s = w; s < steps; s += 2 * kSkinnyWaves) {
    Frag fw[ND][4], fx[MI][4];
    bool in[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long k = (long)(s + (u >> 1) * kSkinnyWaves) * kStep + (2 * q + (u & 1)) * kUnit;
      const long at = min(k, g.K - kUnit);
      in[u] = k < g.K;
#pragma unroll
      for (int d = 0; d < ND; ++d) fw[d][u] = *reinterpret_cast<const Frag*>(pw[d] + at);
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) fx[mi][u] = *reinterpret_cast<const Frag*>(px[mi] + at);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        const Frag x = in[u] ? fx[mi][u] : Frag{};
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[d][mi] = product(in[u] ? fw[d][u] : Frag{}, x, acc[d][mi]);
      }
  }
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) *reinterpret_cast<floatx4*>(&red[w][d][16 * mi + i][4 * q]) = acc[d][mi];
  __syncthreads();
  for (int t = threadIdx.x; t < 64 * MI; t += 64 * kSkinnyWaves) {
    const int r = t >> 2, c = 4 * (t & 3);
    const long nn = n0 + c;
    if (r >= g.M || nn >= g.N) continue;
    float x[ND][4];
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      floatx4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < kSkinnyWaves; ++v) y += *reinterpret_cast<const floatx4*>(&red[v][d][r][c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[d][e] = y[e];
    }
    if constexpr (kDual) finish_gated<T>(g, r, nn, x[0], x[1]);
    else finish<T>(g, 0, r, nn, x[0]);
  }
}

template <typename T, bool kDual>
hipError_t skinny(const Args& g, hipStream_t s) {
  const dim3 grid((unsigned)((g.N + 15) / 16)), block(64 * kSkinnyWaves);
  if (g.M <= 16) hipLaunchKernelGGL((skinny_kernel<T, 1, kDual>), grid, block, 0, s, g);
  else if (g.M <= 32) hipLaunchKernelGGL((skinny_kernel<T, 2, kDual>), grid, block, 0, s, g);
  else hipLaunchKernelGGL((skinny_kernel<T, 4, kDual>), grid, block, 0, s, g);
  return hipGetLastError();
}

template <typename T, int kEpi>
hipError_t forward(const Args& g, hipStream_t s) {
  constexpr bool kDual = kEpi == kGated;
  if (g.M <= 64) return skinny<T, kDual>(g, s);
  return launch_product<T, false, false, kEpi>(g, best_tile<T, false, kEpi>(g.M, kDual ? 2 * g.N : g.N, 1, g.steps), s);
}

// Any number of rows: at most 2^22 per launch, so that the grid's numbers fit 32
// bits.
template <int kEpi>
hipError_t products(const Args& all, int dtype, hipStream_t s) {
  constexpr long most = 1L << 22;
  const long es = dtype == 0 ? 2 : 4;
  auto on = [&](auto* p, long rows, long width) {
    return p ? (decltype(p))((uintptr_t)p + (size_t)(rows * width * es)) : p;
  };
  Args g = all;
  g.parts = g.mparts = g.splits = 1;
  g.steps = g.each = (g.K * es + 127) / 128;
  for (long r = 0; r < all.M; r += most) {
    g.M = all.M - r < most ? all.M - r : most;
    g.a[0] = on(all.a[0], r, g.lda);
    g.out[0] = on(all.out[0], r, g.N);
    g.pre = on(all.pre, r, g.N);
    g.residual = on(all.residual, r, g.N);
    g.gate_out = on(all.gate_out, r, g.N);
    g.up_out = on(all.up_out, r, g.N);
    const hipError_t e = dtype == 0 ? forward<half_t, kEpi>(g, s) : forward<float, kEpi>(g, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gemm

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  gemm::Args g = {};
  g.a[0] = a.x, g.b[0] = a.weight, g.out[0] = a.y;
  g.M = a.rows, g.N = a.N, g.K = g.lda = g.ldb = a.K;
  g.pre = a.pre, g.bias = a.bias, g.residual = a.residual, g.alpha = a.alpha, g.act = a.act;
  return gemm::products<gemm::kLinear>(g, a.dtype, s);
}

hipError_t launch_gated(const GatedArgs& a, hipStream_t s) {
  gemm::Args g = {};
  g.a[0] = a.x, g.b[0] = a.gate_weight, g.b[1] = a.up_weight, g.out[0] = a.h;
  g.M = a.rows, g.N = a.F, g.K = g.lda = g.ldb = a.K;
  g.gate_out = a.gate_out, g.up_out = a.up_out, g.act = a.act;
  return gemm::products<gemm::kGated>(g, a.dtype, s);
}

}  // namespace gla
