// Norms after and before a block with its gate and residual scale,
//   p = x / sqrt(mean(x^2) + eps) * post,  s = residual + scale gate p,
//   y = s / sqrt(mean(s^2) + eps) * w,
// and their gradient. A few flops per byte: memory bounds them (4 x 6,400 x 768 half
// with gates: 27.4 us, 5.7 TB/s; the gradient 44.0, 5.4 TB/s, and 5.7 for the join of
// its sums; 1,600 x 768 5.5 us, a launch's and two loads' latency). A team of TPR
// threads holds a row in registers, VPT groups of eight columns a thread, from
// its loads to its stores, and walks rows, so that the weights are read once.
// Statistics, weight gradients and the gate's gradient are summed in float in a
// fixed order.
#include "gla_gated_norm.h"

#include "gla_rows.h"
#include "gla_tile.h"

namespace gla {
namespace norm {

// Sums of N values over the TPR threads of a team (TPR > 64: the workgroup).
template <int TPR, int N>
__device__ __forceinline__ void team_sums(float (&x)[N], float* lds) {
  constexpr int kIn = TPR < 64 ? TPR : 64;
#pragma unroll
  for (int m = kIn / 2; m >= 1; m >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] += __shfl_xor(x[n], m);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    __syncthreads();  // earlier readers of lds are done
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) lds[n * W + (threadIdx.x >> 6)] = x[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      x[n] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) x[n] += lds[n * W + w];
    }
  }
}

// scale * post of a thread's columns (1 where neither is)
__device__ __forceinline__ void factor8(const float* post, const float* scale, int col, float (&f)[8]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) f[c] = 1.f;
  if (post) tile::load_f8(post + col, f);
  if (scale) {
    float x[8];
    tile::load_f8(scale + col, x);
#pragma unroll
    for (int c = 0; c < 8; ++c) f[c] *= x[c];
  }
}

// Eight columns as loaded, converted where they are used.
template <typename T>
struct Raw8;
template <>
struct Raw8<half_t> {
  half8 v;
  __device__ __forceinline__ void load(const half_t* p) { v = *reinterpret_cast<const half8*>(p); }
  __device__ __forceinline__ float operator[](int c) const { return (float)v[c]; }
};
template <>
struct Raw8<float> {
  floatx4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = *reinterpret_cast<const floatx4*>(p);
    v[1] = *reinterpret_cast<const floatx4*>(p + 4);
  }
  __device__ __forceinline__ float operator[](int c) const { return v[c / 4][c % 4]; }
};

template <int TPR>
constexpr int kTeamThreads = TPR > 256 ? TPR : 256;

// A uniform pointer that the compiler takes for another: what is loaded through it is
// loaded there, not kept from an earlier load of the same.
template <typename T>
__device__ __forceinline__ const T* again(const T* p) {
  asm volatile("" : "+s"(p));
  return p;
}

// sum and y may be x or residual: a thread has read its columns when it writes them.
template <int TPR, int VPT, typename T>
__global__ __launch_bounds__(kTeamThreads<TPR>) void gated_norm_kernel(
    const T* xp, const T* rp, const float* __restrict__ post, const T* __restrict__ gate,
    const float* __restrict__ scale, const float* __restrict__ wp, float eps, T* sp, T* yp, long rows,
    long per, int F) {
  constexpr int RPB = kTeamThreads<TPR> / TPR;
  // float rows of more than 8,192 columns: the 128 registers of 1,024 threads hold the row and the next one, and
  // factors and gate are read where they are used, from L2 (2,368 rows of 8,200: 72 us; kept, with 64 registers
  // spilled, 127)
  constexpr bool kAgain = TPR == 1024 && sizeof(T) == 4;
  constexpr int K = kAgain ? 1 : VPT;
  __shared__ float lds[TPR > 64 ? TPR / 64 : 1];
  const int t = threadIdx.x % TPR, nv = F / 8;
  const float over = 1.f / (float)F;
  float f[K][8], w[K][8];
#pragma unroll
  for (int i = 0; i < (kAgain ? 0 : VPT); ++i) {
    const int u = t + TPR * i;
#pragma unroll
    for (int c = 0; c < 8; ++c) f[i][c] = w[i][c] = 0.f;
    if (u < nv) {
      factor8(post, scale, 8 * u, f[i]);
      tile::load_f8(wp + 8 * u, w[i]);
    }
  }
  const long stride = (long)gridDim.x * RPB;
  long row = (long)blockIdx.x * RPB + threadIdx.x / TPR;
  Raw8<T> nx[VPT], nr[VPT], ng[K];  // the next row
  auto fetch = [&](long at) {
    const long grow = gate ? at / per : 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = t + TPR * i;
      if (u < nv) {
        nx[i].load(xp + at * F + 8 * u);
        nr[i].load(rp + at * F + 8 * u);
        if (!kAgain && gate) ng[i % K].load(gate + grow * F + 8 * u);
      }
    }
  };
  if (row < rows) fetch(row);
  for (; row < rows; row += stride) {
    float x[VPT][8], r[VPT][8], g[K][8], ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = t + TPR * i;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        x[i][c] = u < nv ? nx[i][c] : 0.f, r[i][c] = u < nv ? nr[i][c] : 0.f;
        if (!kAgain) g[i % K][c] = u < nv && gate ? ng[i % K][c] : 1.f;
        ss[0] = fmaf(x[i][c], x[i][c], ss[0]);
      }
    }
    if (row + stride < rows) fetch(row + stride);
    float rx = 1.f;
    if (post) {
      team_sums<TPR>(ss, lds);
      rx = __builtin_amdgcn_rsqf(fmaf(ss[0], over, eps));
    }
    ss[0] = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if constexpr (kAgain) {
        const int u = t + TPR * i;
        if (u >= nv) break;
        factor8(again(post), again(scale), 8 * u, f[0]);
#pragma unroll
        for (int c = 0; c < 8; ++c) g[0][c] = 1.f;
        if (gate) load8(again(gate) + row / per * F + 8 * u, g[0]);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        x[i][c] = round_to(fmaf(x[i][c] * rx, f[i % K][c] * g[i % K][c], r[i][c]), T());
        ss[0] = fmaf(x[i][c], x[i][c], ss[0]);
      }
    }
    team_sums<TPR>(ss, lds);
    const float rs = __builtin_amdgcn_rsqf(fmaf(ss[0], over, eps));
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = t + TPR * i;
      if (u < nv) {
        const long at = row * F + 8 * u;
        if (sp) store8(sp + at, x[i]);
        if constexpr (kAgain) tile::load_f8(again(wp) + 8 * u, w[0]);
#pragma unroll
        for (int c = 0; c < 8; ++c) x[i][c] *= rs * w[i % K][c];
        store8(yp + at, x[i]);
      }
    }
  }
}

// Gradient. With n = x rx and m = s rs (rx, rs the reciprocal roots; n = x without
// post), f = scale post gate:
//   gS = gsum + rs (gy w - m mean(gy w m)),     gresidual = gS,
//   gx = rx (gS f - n mean(gS f n))             (gS f without post),
//   gw = sum gy m,   Q = sum over a group's rows of gS n:
//   ggate = scale post Q,  gpost = scale sum gate Q,  gscale = post sum gate Q.
// mean(gS f n) is put together from sums that do not wait for gS,
//   sum gS f n = sum gsum f n + rs (sum gy w f n - mean(gy w m) sum f n m),
// and half rows, whose values are far from float's ends, take them of x and s and
// put rx and rs in front, so that all six sums of a row go over the team at once.
// Float rows would leave float's range there (x, s of 1e18 and f of 1e3 have a
// product of 1e39): their two squares go first.
// kOwn: a team takes whole groups and writes ggate itself; part[workgroup] holds
// gw and sum gate Q. Else a workgroup takes rows of one chunk of a group;
// part[group][chunk] holds gw and Q.
template <int TPR, int VPT, typename T, bool kOwn>
__global__ __launch_bounds__(kTeamThreads<TPR>) void gated_norm_bwd_kernel(
    const T* xp, const T* sp, const T* gyp, const T* gsp, const float* __restrict__ post,
    const T* __restrict__ gate, const float* __restrict__ scale, const float* __restrict__ wp, float eps,
    T* gxp, T* grp, T* __restrict__ ggp, float* __restrict__ part, long groups, long per, int chunks, int F) {
  constexpr int RPB = kTeamThreads<TPR> / TPR, NS = 6;
  constexpr bool kFirst = sizeof(T) == 4;  // m and n before the other sums
  __shared__ float lds[TPR > 64 ? NS * TPR / 64 : 1];
  __shared__ float join[RPB > 1 ? kTeamThreads<TPR> * VPT * 8 : 1];
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR, nv = F / 8;
  const float over = 1.f / (float)F;
  // 512 threads have 256 registers each: sum gate Q waits in LDS where it would be spilled (2,368 half rows of
  // 8,192 columns with a gate each 91 us instead of 100, float ones, of which 8 registers still are, 153 and 160)
  constexpr bool kPark = kOwn && TPR == 512;
  __shared__ floatx4 park[kPark ? 2 * VPT * TPR : 1];
  constexpr int P = kOwn && !kPark ? VPT : 1;
  float f[VPT][8], w[VPT][8], gw[VPT][8], q[VPT][8], p[P][8], g[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int u = t + TPR * i;
#pragma unroll
    for (int c = 0; c < 8; ++c) f[i][c] = w[i][c] = gw[i][c] = q[i][c] = p[i % P][c] = 0.f, g[i][c] = 1.f;
    if constexpr (kPark) park[t + TPR * 2 * i] = park[t + TPR * (2 * i + 1)] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (u < nv) {
      factor8(post, scale, 8 * u, f[i]);
      tile::load_f8(wp + 8 * u, w[i]);
    }
  }
  auto load_gate = [&](long group) {
    if (!gate) return;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (t + TPR * i < nv) load8(gate + group * F + 8 * (t + TPR * i), g[i]);
  };
  auto do_row = [&](long row) {
    float x[VPT][8], s[VPT][8], gy[VPT][8], gs[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = t + TPR * i;
      const long at = row * F + 8 * u;
#pragma unroll
      for (int c = 0; c < 8; ++c) x[i][c] = s[i][c] = gy[i][c] = gs[i][c] = 0.f;
      if (u < nv) {
        load8(xp + at, x[i]);
        load8(sp + at, s[i]);
        load8(gyp + at, gy[i]);
        if (gsp) load8(gsp + at, gs[i]);
      }
    }
    float squares[2] = {0.f, 0.f}, rs = 1.f, rx = 1.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        squares[0] = fmaf(s[i][c], s[i][c], squares[0]);
        squares[1] = fmaf(x[i][c], x[i][c], squares[1]);
      }
    auto roots = [&](float ss, float xx) {
      rs = __builtin_amdgcn_rsqf(fmaf(ss, over, eps));
      rx = post ? __builtin_amdgcn_rsqf(fmaf(xx, over, eps)) : 1.f;
    };
    if constexpr (kFirst) {
      team_sums<TPR>(squares, lds);
      roots(squares[0], squares[1]);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) s[i][c] *= rs, x[i][c] *= rx;
    }
    float z[kFirst ? 4 : 6] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float fx = f[i][c] * g[i][c] * x[i][c], gm = gy[i][c] * w[i][c];
        z[0] = fmaf(gm, s[i][c], z[0]);
        z[1] = fmaf(gs[i][c], fx, z[1]);
        z[2] = fmaf(gm, fx, z[2]);
        z[3] = fmaf(fx, s[i][c], z[3]);
      }
    if constexpr (!kFirst) z[4] = squares[0], z[5] = squares[1];
    team_sums<TPR>(z, lds);
    if constexpr (!kFirst) {
      roots(z[4], z[5]);
      z[0] *= rs, z[1] *= rx, z[2] *= rx, z[3] *= rx * rs;
    }
    const float dot = z[0] * over;  // mean(gy w m)
    const float mean = post ? over * fmaf(rs, fmaf(-dot, z[3], z[2]), z[1]) : 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = t + TPR * i;
      const long at = row * F + 8 * u;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float m = kFirst ? s[i][c] : s[i][c] * rs, n = kFirst ? x[i][c] : x[i][c] * rx;
        gw[i][c] = fmaf(gy[i][c], m, gw[i][c]);
        gs[i][c] = fmaf(rs, fmaf(gy[i][c], w[i][c], -m * dot), gs[i][c]);
        q[i][c] = fmaf(gs[i][c], n, q[i][c]);
        x[i][c] = rx * fmaf(gs[i][c], f[i][c] * g[i][c], -n * mean);
      }
      if (u < nv) {
        store8(grp + at, gs[i]);
        store8(gxp + at, x[i]);
      }
    }
  };
  if constexpr (kOwn) {
    // every team of the workgroup takes as many steps (their sums meet at barriers)
    for (long g0 = (long)blockIdx.x * RPB; g0 < groups; g0 += (long)gridDim.x * RPB) {
      const long group = g0 + team;
      if (group >= groups) break;  // whole teams; with more than a wave a team there is one
      load_gate(group);
      for (long r = 0; r < per; ++r) do_row(group * per + r);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float y[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          y[c] = f[i][c] * q[i][c];
          if constexpr (!kPark) p[i][c] = fmaf(g[i][c], q[i][c], p[i][c]);
        }
        if constexpr (kPark) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            floatx4 z = park[t + TPR * (2 * i + h)];
#pragma unroll
            for (int c = 0; c < 4; ++c) z[c] = fmaf(g[i][4 * h + c], q[i][4 * h + c], z[c]);
            park[t + TPR * (2 * i + h)] = z;
          }
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) q[i][c] = 0.f;
        if (ggp && t + TPR * i < nv) store8(ggp + group * F + 8 * (t + TPR * i), y);
      }
    }
  } else {
    const long group = blockIdx.x / chunks;
    const int chunk = blockIdx.x % chunks;
    load_gate(group);
    for (long r = (long)chunk * RPB + team; r < per; r += (long)chunks * RPB) do_row(group * per + r);
  }
  float* out = part + 2L * blockIdx.x * F;
  auto write = [&](float* to, float (&a)[VPT][8]) {
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) join[(team * VPT + i) * (TPR * 8) + 8 * t + c] = a[i][c];
      __syncthreads();
      for (int col = threadIdx.x; col < F; col += kTeamThreads<TPR>) {
        float y = 0.f;
        for (int r = 0; r < RPB; ++r) y += join[(r * VPT + col / (TPR * 8)) * (TPR * 8) + col % (TPR * 8)];
        to[col] = y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (t + TPR * i < nv) tile::store_f8(to + 8 * (t + TPR * i), a[i]);
    }
  };
  write(out, gw);
  if constexpr (kPark) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) q[i][c] = park[t + TPR * (2 * i + c / 4)][c % 4];
  }
  if constexpr (kOwn && !kPark) write(out + F, p);
  else write(out + F, q);
}

// The same for rows of more than 8,192 columns, a workgroup of 1,024 threads to a
// row: their 128 registers do not hold what the kernel above keeps of a column (it
// spilled 34 to 195 of them: 2,368 half rows of 8,200 columns 230 us, with a gate of
// every row's own 425; here 97 and 119, 2.4 and 2.6 TB/s, as a CU has one row in
// flight and two exchanges in it). Up to 8,192 columns the kernel above is faster
// (2,368 x 8,192 62 us against 92). The weights' sums wait in LDS, where a thread comes
// back to its own columns, and the factors are read again, from L2, where they are
// used; the row is kept as it was loaded. kRows: every row is a group, or a workgroup
// takes whole groups of rows, or rows of one chunk of a group.
enum WideRows { kEachAGroup, kGroups, kChunks };
template <typename T, WideRows kRows>
__global__ __launch_bounds__(1024) void gated_norm_bwd_wide_kernel(
    const T* xp, const T* sp, const T* gyp, const T* gsp, const float* __restrict__ post,
    const T* __restrict__ gate, const float* __restrict__ scale, const float* __restrict__ wp, float eps,
    T* gxp, T* grp, T* __restrict__ ggp, float* __restrict__ part, long groups, long per, int chunks, int F) {
  constexpr int TPR = 1024, VPT = 2;
  __shared__ float lds[4 * TPR / 64];
  // gw, and sum gate Q (kChunks: Q): the first four columns of every eight, then the others
  __shared__ floatx4 sums[2][2 * VPT * TPR];
  const int t = threadIdx.x, nv = F / 8;
  const float over = 1.f / (float)F;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 2 * VPT; ++i) sums[h][t + TPR * i] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto add = [&](int h, int u, const float (&y)[8]) {
    sums[h][u] += floatx4{y[0], y[1], y[2], y[3]};
    sums[h][VPT * TPR + u] += floatx4{y[4], y[5], y[6], y[7]};
  };
  auto factors = [&](long group, int u, float (&f)[8], float (&g)[8]) {
    factor8(again(post), again(scale), 8 * u, f);
#pragma unroll
    for (int c = 0; c < 8; ++c) g[c] = 1.f;
    if (gate) load8(again(gate) + group * F + 8 * u, g);
  };
  // the group's sums take the registers of float rows' gsum, which is read again as the factors are
  constexpr bool kTwice = kRows == kGroups && sizeof(T) == 4;
  float q[kRows == kGroups ? VPT : 1][8];
  auto do_row = [&](long group, long row) {
    Raw8<T> x[VPT], s[VPT], gy[VPT], kept[kTwice ? 1 : VPT];
    float squares[2] = {0.f, 0.f}, z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = t + TPR * i;
      const long at = row * F + 8 * u;
      x[i] = s[i] = gy[i] = kept[kTwice ? 0 : i] = Raw8<T>{};
      if (u < nv) {
        x[i].load(xp + at);
        s[i].load(sp + at);
        gy[i].load(gyp + at);
        if (!kTwice && gsp) kept[kTwice ? 0 : i].load(gsp + at);
      }
    }
    auto carried = [&](int i, long at) {
      Raw8<T> gs = {};
      if constexpr (!kTwice) gs = kept[i];
      else if (gsp) gs.load(again(gsp) + at);
      return gs;
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        squares[0] = fmaf(s[i][c], s[i][c], squares[0]);
        squares[1] = fmaf(x[i][c], x[i][c], squares[1]);
      }
    team_sums<TPR>(squares, lds);
    const float rs = __builtin_amdgcn_rsqf(fmaf(squares[0], over, eps));
    const float rx = post ? __builtin_amdgcn_rsqf(fmaf(squares[1], over, eps)) : 1.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = t + TPR * i;
      if (u < nv) {
        float f[8], g[8], w[8];
        factors(group, u, f, g);
        tile::load_f8(again(wp) + 8 * u, w);
        const Raw8<T> gs = carried(i, row * F + 8 * u);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float m = s[i][c] * rs, fn = f[c] * g[c] * (x[i][c] * rx), gm = gy[i][c] * w[c];
          z[0] = fmaf(gm, m, z[0]);
          z[1] = fmaf(gs[c], fn, z[1]);
          z[2] = fmaf(gm, fn, z[2]);
          z[3] = fmaf(fn, m, z[3]);
        }
      }
    }
    team_sums<TPR>(z, lds);
    const float dot = z[0] * over;  // mean(gy w m)
    const float mean = post ? over * fmaf(rs, fmaf(-dot, z[3], z[2]), z[1]) : 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int u = t + TPR * i;
      if (u < nv) {
        const long at = row * F + 8 * u;
        float y[8], r[8], f[8], g[8];
        tile::load_f8(again(wp) + 8 * u, r);
        const Raw8<T> gs = carried(i, at);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float m = s[i][c] * rs;
          y[c] = gy[i][c] * m;
          r[c] = fmaf(rs, fmaf(gy[i][c], r[c], -m * dot), gs[c]);
        }
        add(0, u, y);
        store8(grp + at, r);
        factors(group, u, f, g);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float n = x[i][c] * rx;
          y[c] = rx * fmaf(r[c], f[c] * g[c], -n * mean);
          r[c] *= n;
          if constexpr (kRows == kGroups) q[i][c] += r[c];
        }
        store8(gxp + at, y);
        if constexpr (kRows == kEachAGroup) {
#pragma unroll
          for (int c = 0; c < 8; ++c) f[c] *= r[c], r[c] *= g[c];
          if (ggp) store8(ggp + at, f);
        }
        if constexpr (kRows != kGroups) add(1, u, r);
      }
    }
  };
  if constexpr (kRows == kEachAGroup) {
    for (long row = blockIdx.x; row < groups; row += gridDim.x) do_row(row, row);
  } else if constexpr (kRows == kGroups) {
    for (long group = blockIdx.x; group < groups; group += gridDim.x) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) q[i][c] = 0.f;
      for (long r = 0; r < per; ++r) do_row(group, group * per + r);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int u = t + TPR * i;
        if (u < nv) {
          float f[8], g[8];
          factors(group, u, f, g);
#pragma unroll
          for (int c = 0; c < 8; ++c) f[c] *= q[i][c], g[c] *= q[i][c];
          if (ggp) store8(ggp + group * F + 8 * u, f);
          add(1, u, g);
        }
      }
    }
  } else {
    const long group = blockIdx.x / chunks;
    for (long r = blockIdx.x % chunks; r < per; r += chunks) do_row(group, group * per + r);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int u = t + TPR * i;
    if (u >= nv) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      floatx4* to = reinterpret_cast<floatx4*>(part + (2L * blockIdx.x + h) * F + 8 * u);
      to[0] = sums[h][u], to[1] = sums[h][VPT * TPR + u];
    }
  }
}

// Sums of the pairs of rows of part, gw and Q (or sum gate Q), `count` of them in
// each of `groups` groups (kLast; else in group blockIdx.y): 16 columns and 64
// rows of threads per workgroup. gate: the sums are Q, of which ggate (if wanted)
// and gate Q are made; kEach: as many groups as pairs, each pair one group's whole
// sum. kLast: into the weights' gradients. Else into pair blockIdx.y of `next`.
template <typename T, bool kLast, bool kEach>
__global__ __launch_bounds__(1024) void gated_norm_join_kernel(
    const float* __restrict__ part, float* __restrict__ next, int count, int groups, int F,
    const float* __restrict__ post, const T* __restrict__ gate, const float* __restrict__ scale,
    T* __restrict__ ggp, float* __restrict__ gpost, float* __restrict__ gscale, float* __restrict__ gweight) {
  constexpr int W = 8;
  __shared__ float s[2][64][17];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  // `each` rows of threads to a group, a power of two and at least eight
  const int each = groups == 1 ? 64 : groups == 2 ? 32 : groups <= 4 ? 16 : 8, o = g / each, r = g % each;
  const long group = kLast ? o : blockIdx.y;
  const float a = post && col < F ? post[col] : 1.f, b = scale && col < F ? scale[col] : 1.f;
  float y[2] = {0.f, 0.f};
  if (col < F && o < groups) {
    const float* from = part + 2 * group * count * F + col;
    for (int p = r; p < count; p += each * W) {
      float x[2][W];
#pragma unroll
      for (int i = 0; i < W; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) x[h][i] = p + each * i < count ? from[(2L * (p + each * i) + h) * F] : 0.f;
      if constexpr (kEach) {
        float gates[W];
#pragma unroll
        for (int i = 0; i < W; ++i) gates[i] = p + each * i < count ? (float)gate[(long)(p + each * i) * F + col] : 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          if (ggp && p + each * i < count) ggp[(long)(p + each * i) * F + col] = (T)(a * b * x[1][i]);
          x[1][i] *= gates[i];
        }
      }
#pragma unroll
      for (int i = 0; i < W; ++i) y[0] += x[0][i], y[1] += x[1][i];
    }
  }
  s[0][g][c] = y[0], s[1][g][c] = y[1];
  __syncthreads();
  if (g % 8 == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      y[h] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[h] += s[h][g + i][c];
      s[h][g][c] = y[h];  // no other thread reads rows g .. g + 7
    }
  }
  __syncthreads();
  if (r == 0 && o < groups && col < F) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      for (int i = 8; i < each; i += 8) y[h] += s[h][g + i][c];
    if (!kEach && gate) {
      if (ggp) ggp[group * F + col] = (T)(a * b * y[1]);
      y[1] *= (float)gate[group * F + col];
    }
    if constexpr (!kLast) {
      next[2 * group * F + col] = y[0];
      next[(2 * group + 1) * F + col] = y[1];
    } else {
      s[0][g][c] = y[0], s[1][g][c] = y[1];
    }
  }
  if constexpr (kLast) {
    __syncthreads();
    if (g == 0 && col < F) {
      for (int i = 1; i < groups; ++i) y[0] += s[0][i * each][c], y[1] += s[1][i * each][c];
      gweight[col] = y[0];
      if (gpost) gpost[col] = b * y[1];
      if (gscale) gscale[col] = a * y[1];
    }
  }
}

// How the gradient's rows are shared out: teams that own groups where these are many
// and short, else chunks of each group's rows, in as many workgroups as the CUs hold
// at once (25,600 x 768 half: 58.6 us with 512, 70.7 with 1,024) and at least one a
// group. Up to eight groups the last launch takes side by side (four of 6,400 rows
// of 768: 5.4 us instead of 9.1 for two launches), and one-chunk groups row by row.
// A team needs 1.2 to 2.3 us for a row of its group, the last launch 7 for 512
// groups of chunks. Teams against chunks, half: 600 groups of 1,000 rows of 64
// 1,140 and 95 us, 512 of 392 of 768 924 and 337, 512 of 8 24.8 and 21.4, of 5 17.1
// and 19.6; 6,000 of 24 254 and 320, 6,000 of 100 of 64 147 and 139, 9,000 164 and 211.
constexpr long kMaxParts2 = 512, kMaxAtOnce = 8;
int teams(int F) { return F <= 64 ? 32 : F <= 256 ? 16 : F <= 512 ? 8 : F <= 1024 ? 4 : 1; }
struct GroupPlan {
  bool own;
  int chunks;   // of each group
  long blocks;  // workgroups of the first kernel
};
GroupPlan group_plan(long rows, long groups, int F) {
  GroupPlan p;
  const long rpb = teams(F), per = rows / groups;
  p.own = groups >= kMaxParts2 && per <= groups / 85;
  p.chunks = 1;
  if (p.own) {
    const long steps = (groups + rpb - 1) / rpb, each = (steps + kMaxParts2 - 1) / kMaxParts2;
    p.blocks = (steps + each - 1) / each;
  } else {
    const long steps = (per + rpb - 1) / rpb;
    long most = kMaxParts2 / groups;
    if (most < 1) most = 1;
    const long each = (steps + most - 1) / most;
    p.chunks = (int)((steps + each - 1) / each);
    p.blocks = groups * p.chunks;
  }
  return p;
}

// Each workgroup's sums are a whole group's, and there are more groups than the last
// launch takes side by side.
bool each_a_group(const GroupPlan& p, long groups) { return !p.own && p.chunks == 1 && groups > kMaxAtOnce; }

template <int TPR, int VPT, typename T>
hipError_t gated_norm_t(const GatedNormArgs& a, hipStream_t s) {
  constexpr long rpb = kTeamThreads<TPR> / TPR;
  // as many workgroups as the CUs hold at once, each with its next row in flight
  // (25,600 x 768 half, inputs from memory: 768 workgroups 30.0 us, 512 and 1,024
  // 30.6 and 36.3; 4,096 without the row in flight 38.4)
  constexpr long most = VPT == 1 ? 1536 : 768;
  const long steps = (a.rows + rpb - 1) / rpb, blocks = steps < most ? steps : most;
  hipLaunchKernelGGL((gated_norm_kernel<TPR, VPT, T>), dim3((unsigned)blocks), dim3(kTeamThreads<TPR>), 0, s,
                     static_cast<const T*>(a.x), static_cast<const T*>(a.residual), a.post,
                     static_cast<const T*>(a.gate), a.scale, a.weight, a.eps, static_cast<T*>(a.sum),
                     static_cast<T*>(a.y), a.rows, a.rows / a.groups, a.F);
  return hipGetLastError();
}

template <int TPR, int VPT, typename T>
hipError_t gated_norm_bwd_t(const GatedNormBwdArgs& a, float* ws, hipStream_t s) {
  const GroupPlan p = group_plan(a.rows, a.groups, a.F);
  const long per = a.rows / a.groups;
  auto kernel = [&] {
    if constexpr (TPR * VPT > 1024)
      return !p.own     ? gated_norm_bwd_wide_kernel<T, kChunks>
             : per == 1 ? gated_norm_bwd_wide_kernel<T, kEachAGroup>
                        : gated_norm_bwd_wide_kernel<T, kGroups>;
    else return p.own ? gated_norm_bwd_kernel<TPR, VPT, T, true> : gated_norm_bwd_kernel<TPR, VPT, T, false>;
  }();
  const T* gate = static_cast<const T*>(a.gate);
  T* ggate = static_cast<T*>(a.ggate);
  hipLaunchKernelGGL(kernel, dim3((unsigned)p.blocks), dim3(kTeamThreads<TPR>), 0, s,
                     static_cast<const T*>(a.x), static_cast<const T*>(a.sum), static_cast<const T*>(a.gy),
                     static_cast<const T*>(a.gsum), a.post, gate, a.scale, a.weight, a.eps,
                     static_cast<T*>(a.gx), static_cast<T*>(a.gresidual), p.own ? ggate : nullptr, ws,
                     a.groups, per, p.chunks, a.F);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned cols = (unsigned)((a.F + 15) / 16);
  const float* part = ws;
  // the sums of teams that own groups have the gate in them
  int count = p.own ? (int)p.blocks : p.chunks, groups = p.own ? 1 : (int)a.groups;
  bool gated = p.own;
  if (each_a_group(p, groups)) {
    hipLaunchKernelGGL((gated_norm_join_kernel<T, true, true>), dim3(cols), dim3(1024), 0, s, part, nullptr, groups, 1,
                       a.F, a.post, gate, a.scale, ggate, a.gpost, a.gscale, a.gweight);
    return hipGetLastError();
  }
  if (groups > kMaxAtOnce) {
    float* next = ws + 2 * p.blocks * a.F;
    hipLaunchKernelGGL((gated_norm_join_kernel<T, false, false>), dim3(cols, (unsigned)groups), dim3(1024), 0, s, ws,
                       next, count, 1, a.F, a.post, gate, a.scale, ggate, nullptr, nullptr, nullptr);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    part = next, count = groups, groups = 1, gated = true;
  }
  hipLaunchKernelGGL((gated_norm_join_kernel<T, true, false>), dim3(cols), dim3(1024), 0, s, part, nullptr, count,
                     groups, a.F, a.post, gated ? nullptr : gate, a.scale, ggate, a.gpost, a.gscale, a.gweight);
  return hipGetLastError();
}

#define GLA_TEAM_DISPATCH(FN, T, ...)                    \
  do {                                                   \
    const int F_ = a.F;                                  \
    if (F_ <= 64) return FN<8, 1, T>(__VA_ARGS__);       \
    if (F_ <= 128) return FN<16, 1, T>(__VA_ARGS__);     \
    if (F_ <= 256) return FN<16, 2, T>(__VA_ARGS__);     \
    if (F_ <= 512) return FN<32, 2, T>(__VA_ARGS__);     \
    if (F_ <= 1024) return FN<64, 2, T>(__VA_ARGS__);    \
    if (F_ <= 4096) return FN<256, 2, T>(__VA_ARGS__);   \
    if (F_ <= 8192) return FN<512, 2, T>(__VA_ARGS__);   \
    return FN<1024, 2, T>(__VA_ARGS__);                  \
  } while (0)

}  // namespace norm

hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t s) {
  if (a.dtype == 0) GLA_TEAM_DISPATCH(norm::gated_norm_t, half_t, a, s);
  GLA_TEAM_DISPATCH(norm::gated_norm_t, float, a, s);
}

size_t gated_norm_bwd_workspace(long rows, long groups, int F) {
  const norm::GroupPlan p = norm::group_plan(rows, groups, F);
  const long joined = !p.own && p.chunks > 1 && groups > norm::kMaxAtOnce ? groups : 0;
  return (size_t)2 * (p.blocks + joined) * F * sizeof(float);
}

hipError_t launch_gated_norm_bwd(const GatedNormBwdArgs& a, float* ws, hipStream_t s) {
  if (a.dtype == 0) GLA_TEAM_DISPATCH(norm::gated_norm_bwd_t, half_t, a, ws, s);
  GLA_TEAM_DISPATCH(norm::gated_norm_bwd_t, float, a, ws, s);
}

}  // namespace gla
