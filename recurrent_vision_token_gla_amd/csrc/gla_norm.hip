// The norm that stands before each mixer of a block, with the residual's
// addition, s = x + r, y = s / sqrt(mean(s^2) + eps) * w, in the input type or
// in 8 bits; its gradient; and the gradient of the output gate
// y = o / sqrt(mean(o^2) + eps) * w * silu(z).
//
// All of them read each input once and write each output once, a few flops per
// byte: memory bounds them. A row stays in registers from its load to its
// store. Statistics and weight gradients are float; a weight gradient sums
// over rows in a fixed order (per workgroup, then over the workgroups'
// partial sums in a second kernel), so it does not change from run to run.
// Measured, half: norm of 6,400 x 768 9.0 us (4.4 TB/s), with the 8-bit output
// of 25,600 x 768 26.1 us (5.3 TB/s); gradients of 25,600 x 768 30.6 us (5.1
// TB/s) and of 409,600 gate rows of 64 43 us (6.1 TB/s), with 4.0 and 4.7 us of
// column sums. (A copy of 256 MB runs at 5.4 TB/s.) Rows of less than 512 columns
// leave lanes of their wave idle: the norm of 409,600 x 64 takes 83 us (2.5
// TB/s), of 409,600 x 128 127 us (3.3 TB/s).
#include "gla_colsum.h"
#include "gla_norm.h"
#include "gla_rows.h"
#include "gla_tile.h"

namespace gla {
namespace norm {

using tile::fexp2;

__device__ __forceinline__ void load_w(const float* p, float (&x)[8]) { tile::load_f8(p, x); }

// TPR threads per row, each with up to VPT groups of eight columns. sum and y
// may be x or residual: a thread has read its columns when it writes them.
template <int TPR, int VPT, typename InT, bool kQ8>
__global__ __launch_bounds__(256) void add_rmsnorm_kernel(
    const InT* xp, const InT* rp, const float* __restrict__ wp, float eps, InT* sp, InT* yp,
    unsigned char* __restrict__ y8, float* __restrict__ scales, long rows, int F) {
  __shared__ float lds[4];
  const int t = threadIdx.x % TPR, nv = F / 8;
  const long row = (long)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  if (row >= rows) return;  // whole waves (TPR 64) or never (TPR 256)
  float s[VPT][8], ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int u = t + TPR * i;
    const long at = row * F + 8 * u;
#pragma unroll
    for (int c = 0; c < 8; ++c) s[i][c] = 0.f;
    if (u < nv) {
      load8(xp + at, s[i]);
      if (rp) {
        float r[8];
        load8(rp + at, r);
#pragma unroll
        for (int c = 0; c < 8; ++c) s[i][c] = round_to(s[i][c] + r[c], InT());
      }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) ss = fmaf(s[i][c], s[i][c], ss);
  }
  ss = row_reduce<TPR, false>(ss, lds);
  const float rstd = __builtin_amdgcn_rsqf(ss / (float)F + eps);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int u = t + TPR * i;
    const long at = row * F + 8 * u;
    if (u < nv) {
      float w[8];
      load_w(wp + 8 * u, w);
      if (sp) store8(sp + at, s[i]);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        s[i][c] *= rstd * w[c];
        top = fmaxf(top, fabsf(s[i][c]));
      }
      if constexpr (!kQ8) store8(yp + at, s[i]);
    }
  }
  if constexpr (kQ8) {
    top = row_reduce<TPR, true>(top, lds);
    // the row's largest value becomes e4m3's largest, 448; a row of zeros
    // keeps scale 1, and a scale is never below the smallest normal float
    const float scale = top > 0.f ? fmaxf(top * (1.f / 448.f), 0x1p-126f) : 1.f;
    const float inv = 1.f / scale;
    if (t == 0) scales[row] = scale;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = t + TPR * i;
      if (u < nv) {
        int lo = 0, hi = 0;
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[i][0] * inv, s[i][1] * inv, lo, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[i][2] * inv, s[i][3] * inv, lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[i][4] * inv, s[i][5] * inv, hi, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[i][6] * inv, s[i][7] * inv, hi, true);
        *reinterpret_cast<int2*>(y8 + row * F + 8 * u) = int2{lo, hi};
      }
    }
  }
}

// Gradient of the norm, with n = s rstd:
//   gx = rstd (gy w - n mean(gy w n)) + gsum,   gweight = sum over rows of gy n.
// A workgroup walks rows with a stride and keeps its columns' weight sums in
// registers; part[workgroup][F] takes them at the end. gx may be s, gy or
// gsum: a thread has read its columns of a row when it writes them.
template <int TPR, int VPT, typename InT>
__global__ __launch_bounds__(256) void norm_bwd_kernel(
    const InT* sp, const InT* gyp, const InT* gsp, const float* __restrict__ wp, float eps, InT* gxp,
    float* __restrict__ part, long rows, int F) {
  constexpr int RPB = 256 / TPR;  // rows per workgroup and step
  // gsum is loaded with the others (25,600 x 768 half: 31 us, or 35 where it
  // waits for the sums), but not where its registers would not be left
  constexpr bool kEarly = VPT <= 4;
  __shared__ float lds[4];
  __shared__ float sW[RPB > 1 ? RPB * TPR * VPT * 8 : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR, nv = F / 8;
  float gw[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) gw[i][c] = 0.f;
  for (long row = (long)blockIdx.x * RPB + sub; row < rows; row += (long)gridDim.x * RPB) {
    float s[VPT][8], g[VPT][8], x[kEarly ? VPT : 1][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = t + TPR * i;
      const long at = row * F + 8 * u;
#pragma unroll
      for (int c = 0; c < 8; ++c) s[i][c] = g[i][c] = x[kEarly ? i : 0][c] = 0.f;
      if (u < nv) {
        load8(sp + at, s[i]);
        load8(gyp + at, g[i]);
        if (kEarly && gsp) load8(gsp + at, x[kEarly ? i : 0]);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) ss = fmaf(s[i][c], s[i][c], ss);
    }
    ss = row_reduce<TPR, false>(ss, lds);
    const float rstd = __builtin_amdgcn_rsqf(ss / (float)F + eps);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = t + TPR * i;
      float w[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (u < nv) load_w(wp + 8 * u, w);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        s[i][c] *= rstd;  // n
        gw[i][c] = fmaf(g[i][c], s[i][c], gw[i][c]);
        g[i][c] *= w[c];
        dot = fmaf(g[i][c], s[i][c], dot);
      }
    }
    dot = row_reduce<TPR, false>(dot, lds) / (float)F;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = t + TPR * i;
      const long at = row * F + 8 * u;
      if (u < nv) {
        float(&y)[8] = x[kEarly ? i : 0];
        if (!kEarly) {
#pragma unroll
          for (int c = 0; c < 8; ++c) y[c] = 0.f;
          if (gsp) load8(gsp + at, y);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) y[c] = fmaf(rstd, g[i][c] - s[i][c] * dot, y[c]);
        store8(gxp + at, y);
      }
    }
  }
  float* out = part + (long)blockIdx.x * F;
  if constexpr (RPB > 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) sW[(sub * VPT + i) * (TPR * 8) + 8 * t + c] = gw[i][c];
    __syncthreads();
    for (int col = threadIdx.x; col < F; col += 256) {
      float x = 0.f;
#pragma unroll
      for (int r = 0; r < RPB; ++r) x += sW[(r * VPT + col / (TPR * 8)) * (TPR * 8) + col % (TPR * 8)];
      out[col] = x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (t + TPR * i < nv) tile::store_f8(out + 8 * (t + TPR * i), gw[i]);
  }
}

// Gradient of the output gate, rows of DV values, with n = o rstd and
// sig = 1 / (1 + exp(-z)):
//   gn = gy w z sig,  go = rstd (gn - n mean(gn n)),
//   gz = gy n w sig (1 + z (1 - sig)),  gweight = sum over rows of gy n z sig.
// DV/8 neighbouring lanes hold a row, so its sums are lane permutations.
template <int DV, typename InT>
__global__ __launch_bounds__(256) void gate_bwd_kernel(
    const InT* __restrict__ op, const InT* __restrict__ zp, const InT* __restrict__ gyp,
    const float* __restrict__ wp, float eps, InT* __restrict__ gop, InT* __restrict__ gzp,
    float* __restrict__ part, long rows) {
  constexpr int LPR = DV / 8, RPB = 256 / LPR;
  __shared__ float sW[4][DV];
  const int c8 = 8 * (threadIdx.x % LPR);
  float w[8], gw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  load_w(wp + c8, w);
  for (long r0 = (long)blockIdx.x * RPB; r0 < rows; r0 += (long)gridDim.x * RPB) {
    const long row = r0 + threadIdx.x / LPR;
    const bool in = row < rows;
    const long at = (in ? row : rows - 1) * DV + c8;
    float o[8], z[8], gy[8], gn[8], ss = 0.f, dot = 0.f;
    load8(op + at, o);
    load8(zp + at, z);
    load8(gyp + at, gy);
#pragma unroll
    for (int c = 0; c < 8; ++c) ss = fmaf(o[c], o[c], ss);
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor(ss, m);
    const float rstd = __builtin_amdgcn_rsqf(ss * (1.f / DV) + eps);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float sig = __builtin_amdgcn_rcpf(1.f + fexp2(-z[c] * kLog2e));
      const float act = z[c] * sig;
      o[c] *= rstd;  // n
      gn[c] = gy[c] * w[c] * act;
      dot = fmaf(gn[c], o[c], dot);
      gw[c] += in ? gy[c] * o[c] * act : 0.f;
      z[c] = gy[c] * o[c] * w[c] * (sig * fmaf(z[c], 1.f - sig, 1.f));
    }
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) dot += __shfl_xor(dot, m);
    dot *= 1.f / DV;
#pragma unroll
    for (int c = 0; c < 8; ++c) gn[c] = rstd * (gn[c] - o[c] * dot);
    if (in) {
      store8(gop + at, gn);
      store8(gzp + at, z);
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
#pragma unroll
    for (int m = LPR; m < 64; m <<= 1) gw[c] += __shfl_xor(gw[c], m);
  }
  if ((threadIdx.x & 63) < LPR) {
#pragma unroll
    for (int c = 0; c < 8; ++c) sW[threadIdx.x >> 6][c8 + c] = gw[c];
  }
  __syncthreads();
  if (threadIdx.x < DV)
    part[(long)blockIdx.x * DV + threadIdx.x] =
        (sW[0][threadIdx.x] + sW[1][threadIdx.x]) + (sW[2][threadIdx.x] + sW[3][threadIdx.x]);
}

// Workgroups of the two gradient kernels: enough to fill the GPU, and few enough
// that the partial sums stay small beside many rows. At most 512, 1024 or 2048
// of them: the norm's gradient of 25,600 x 768 half rows 42, 37 or 41 us, the
// gate's of 409,600 rows of 64 the same within 1 us. Few wide rows are not
// many: up to 1,024 rows of more than 1,024 columns each have a partial sum of
// their own, more bytes than half rows (1,024 x 4,096 19.7 us, 4,096 x 4,096
// 27.9).
constexpr long kMaxParts = 1024;
// every workgroup takes the same number of steps of `per` rows, but the last
int even_parts(long rows, long per) {
  const long steps = (rows + per - 1) / per;
  const long each = (steps + kMaxParts - 1) / kMaxParts;
  return (int)((steps + each - 1) / each);
}
int norm_parts(long rows, int F) { return even_parts(rows, F <= 1024 ? 4 : 1); }
int gate_parts(long rows, int dv) { return even_parts(rows, 256 / (dv / 8)); }

template <int TPR, int VPT, typename InT>
hipError_t norm_t(const NormArgs& a, hipStream_t s) {
  // at most 2^22 workgroups (2^30 threads) per launch
  constexpr long rpb = 256 / TPR, most = rpb << 22;
  auto kernel = a.y8 ? add_rmsnorm_kernel<TPR, VPT, InT, true> : add_rmsnorm_kernel<TPR, VPT, InT, false>;
  auto at = [](auto* p, long off) { return p ? p + off : p; };
  for (long r0 = 0; r0 < a.rows; r0 += most) {
    const long rows = a.rows - r0 < most ? a.rows - r0 : most, off = r0 * a.F;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((rows + rpb - 1) / rpb)), dim3(256), 0, s,
                       static_cast<const InT*>(a.x) + off, at(static_cast<const InT*>(a.residual), off),
                       a.weight, a.eps, at(static_cast<InT*>(a.sum), off), at(static_cast<InT*>(a.y), off),
                       at(static_cast<unsigned char*>(a.y8), off), at(a.scales, r0), rows, a.F);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int TPR, int VPT, typename InT>
hipError_t norm_bwd_t(const NormBwdArgs& a, float* ws, hipStream_t s) {
  const int P = norm_parts(a.rows, a.F);
  hipLaunchKernelGGL((norm_bwd_kernel<TPR, VPT, InT>), dim3(P), dim3(256), 0, s,
                     static_cast<const InT*>(a.sum), static_cast<const InT*>(a.gy),
                     static_cast<const InT*>(a.gsum), a.weight, a.eps, static_cast<InT*>(a.gx), ws,
                     a.rows, a.F);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(column_sum_kernel, dim3((a.F + 15) / 16), dim3(1024), 0, s, ws, a.gweight, P, a.F);
  return hipGetLastError();
}

// One wave per row up to 1024 columns, else one workgroup. 12,800 half rows
// take, with a wave or a workgroup per row, 29.7 or 26.2 us for 1536 columns
// and 40.5 or 35.9 for 2048, their gradient 38.9 or 36.5 and 50.0 or 43.3 (but
// of 1024 rows of 2048 13.2 or 14.3).
#define GLA_NORM_DISPATCH(FN, InT, ...)                                    \
  do {                                                                     \
    const int F_ = a.F;                                                    \
    if (F_ <= 512) return FN<64, 1, InT>(__VA_ARGS__);                     \
    if (F_ <= 1024) return FN<64, 2, InT>(__VA_ARGS__);                    \
    if (F_ <= 2048) return FN<256, 1, InT>(__VA_ARGS__);                   \
    if (F_ <= 4096) return FN<256, 2, InT>(__VA_ARGS__);                   \
    if (F_ <= 8192) return FN<256, 4, InT>(__VA_ARGS__);                   \
    return FN<256, 8, InT>(__VA_ARGS__);                                   \
  } while (0)

template <int DV, typename InT>
hipError_t gate_bwd_t(const GateBwdArgs& a, float* ws, hipStream_t s) {
  const int P = gate_parts(a.rows, a.dv);
  hipLaunchKernelGGL((gate_bwd_kernel<DV, InT>), dim3(P), dim3(256), 0, s,
                     static_cast<const InT*>(a.o), static_cast<const InT*>(a.gate),
                     static_cast<const InT*>(a.gy), a.weight, a.eps, static_cast<InT*>(a.go),
                     static_cast<InT*>(a.ggate), ws, a.rows);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(column_sum_kernel, dim3((DV + 15) / 16), dim3(1024), 0, s, ws, a.gweight, P, DV);
  return hipGetLastError();
}

}  // namespace norm

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s) {
  if (a.dtype == 0) GLA_NORM_DISPATCH(norm::norm_t, half_t, a, s);
  GLA_NORM_DISPATCH(norm::norm_t, float, a, s);
}

size_t norm_bwd_workspace(long rows, int F) {
  return (size_t)norm::norm_parts(rows, F) * F * sizeof(float);
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, float* ws, hipStream_t s) {
  if (a.dtype == 0) GLA_NORM_DISPATCH(norm::norm_bwd_t, half_t, a, ws, s);
  GLA_NORM_DISPATCH(norm::norm_bwd_t, float, a, ws, s);
}

size_t gate_bwd_workspace(long rows, int dv) {
  return (size_t)norm::gate_parts(rows, dv) * dv * sizeof(float);
}

hipError_t launch_gate_bwd(const GateBwdArgs& a, float* ws, hipStream_t s) {
  if (a.dtype == 0)
    return a.dv == 64 ? norm::gate_bwd_t<64, half_t>(a, ws, s) : norm::gate_bwd_t<32, half_t>(a, ws, s);
  return a.dv == 64 ? norm::gate_bwd_t<64, float>(a, ws, s) : norm::gate_bwd_t<32, float>(a, ws, s);
}

}  // namespace gla
