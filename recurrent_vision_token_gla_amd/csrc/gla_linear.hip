// The products around a block's mixers: y = alpha act(x W^T + b) + residual, and
// the gated h = act(x Wg^T) * (x Wu^T) from one reading of x, with everything
// behind the sums in the kernel that forms them.
#include "gla_linear.h"

#include "gla_gemm.h"

namespace gla {
namespace gemm {

// Up to 16 rows. A workgroup takes the 16 columns of the matrix cores' tile (gated:
// eight of either weight, so that a small F still occupies the CUs: 16 rows x 768 x
// 2,048 with 16 of both 5.1 us, with eight 4.3); its eight waves take steps of the
// contraction in turn, straight from memory into the operands of the matrix cores:
// lane i, q holds row i and the 32 bytes 32 q .. of the step's 128, whole lines of a
// weight row by four lanes. The waves' sums meet in LDS. Bound by the latency of
// one load, the exchange and the launch (one row x 768 x 3,840: 4.0 us; four rows x
// 8,192 x 1,024: 13.1, 1.3 TB/s, where the tiles take 21.2).
constexpr int kSkinnyWaves = 8;

template <typename T, bool kDual>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_kernel(const Args g) {
  constexpr int kUnit = Num<T>::kUnit, kStep = Num<T>::kStep, kCols = kFewCols<kDual>;
  using Frag = typename std::conditional<sizeof(T) == 2, half8, floatx4>::type;
  __shared__ __attribute__((aligned(16))) float red[kSkinnyWaves][kFewRows][16];
  const int i = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3, w = wave();
  const long n0 = (long)kCols * blockIdx.x, n = min(n0 + i % kCols, g.N - 1);
  const T* pw = static_cast<const T*>(g.b[kDual ? i >> 3 : 0]) + n * g.ldb;
  const T* px = static_cast<const T*>(g.a[0]) + min((long)i, g.M - 1) * g.lda;
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  const int steps = (int)g.steps;
  // two steps a round, all of their loads in flight; beyond the contraction's
  // end they read its last elements, which then count as zero
  for (int s = w; s < steps; s += 2 * kSkinnyWaves) {
    Frag fw[4], fx[4];
    bool in[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long k = (long)(s + (u >> 1) * kSkinnyWaves) * kStep + (2 * q + (u & 1)) * kUnit;
      const long at = min(k, g.K - kUnit);
      in[u] = k < g.K;
      fw[u] = *reinterpret_cast<const Frag*>(pw + at);
      fx[u] = *reinterpret_cast<const Frag*>(px + at);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) acc = product(in[u] ? fw[u] : Frag{}, in[u] ? fx[u] : Frag{}, acc);
  }
  *reinterpret_cast<floatx4*>(&red[w][i][4 * q]) = acc;
  __syncthreads();
  const int r = threadIdx.x / (kCols / 4), c = 4 * (threadIdx.x % (kCols / 4));
  const long nn = n0 + c;
  if (r >= g.M || nn >= g.N) return;
  float x[kDual ? 2 : 1][4];
#pragma unroll
  for (int d = 0; d < (kDual ? 2 : 1); ++d) {
    floatx4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kSkinnyWaves; ++v) y += *reinterpret_cast<const floatx4*>(&red[v][r][8 * d + c]);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[d][e] = y[e];
  }
  if constexpr (kDual) finish_gated<T>(g, r, nn, x[0], x[1]);
  else finish<T>(g, 0, r, nn, x[0]);
}

// The form for few rows, or the tiles.
template <typename T, int kEpi>
hipError_t forward(const Args& g, hipStream_t s) {
  constexpr bool kDual = kEpi == kGated;
  const int tile = forward_tile<T, kEpi>(g.M, g.N, g.steps);
  if (tile == kTiles) {
    hipLaunchKernelGGL((skinny_kernel<T, kDual>), dim3((unsigned)((g.N + kFewCols<kDual> - 1) / kFewCols<kDual>)),
                       dim3(64 * kSkinnyWaves), 0, s, g);
    return hipGetLastError();
  }
  return launch_product<T, false, false, kEpi>(g, tile, s);
}

// Any number of rows, rows_at_once of them per launch.
template <int kEpi>
hipError_t products(const Args& all, int dtype, hipStream_t s) {
  const long most = rows_at_once(all.N);
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
