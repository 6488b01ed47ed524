// One new token per sequence: S <- diag(exp(gk)) S + k^T v, o = q S, on states
// held in a pool (float [slot][H][dk][dv]), optionally with the block's output
// gate on o. The serving form of the recurrence: the state is read and written
// once, 8 dk dv bytes per (row, head) against 5 dk dv flops, so the memory
// bounds it (and the launch, for a few rows).
//
// One workgroup per (row, head). A thread holds four neighbouring value
// columns of every (256 / (dv/4))-th key dim, so a wave's accesses are
// contiguous, and all of them are in flight before the first is used. The sum
// over key dims goes through lane permutations and then LDS, in a fixed order.
// 256 rows of 16 heads of 64/64 (134 MB): 23.5 us, 5.7 TB/s; 37 rows of 12
// heads of 32/64: 3.8 us, one row of 6 heads: 3.3 us, both a launch's latency.
//
// Rows of one call that name the same slot are consecutive tokens of one
// sequence: the workgroup of the first such row applies all of them in row
// order with the state in registers, and those of the others leave. Every wave
// finds them by comparing the call's slots, 256 per round of loads; the first
// round's go out before the state's, which would be waited for with them (29.5
// us instead of 23.5 for the 256 rows). Beyond them every round is waited for:
// 1,024 ungated rows take 100 us, or 81 without slots (6.8 TB/s), 4,096 rows 594
// or 401.
#include "gla_step.h"
#include "gla_tile.h"

namespace gla {
namespace step {

// Which of the rows j0 .. j0 + 255 name a slot: four loads, then four ballots
// (apart, so that a caller's loads can go out in between).
struct Slots {
  static constexpr int kRows = 256;
  int32_t s[4];
  unsigned long long hit[4];
  __device__ __forceinline__ void load(const int32_t* __restrict__ slots, int j0, int B) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = 0;
      if (j0 + 64 * i < B) s[i] = slots[min(j0 + 64 * i + (int)(threadIdx.x & 63), B - 1)];
    }
  }
  __device__ __forceinline__ void compare(int slot, int j0, int B) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      hit[i] = __ballot(j0 + 64 * i + (int)(threadIdx.x & 63) < B && s[i] == slot);
  }
  // first hit of rows >= lo (of j0 ..), or B
  __device__ __forceinline__ int first(int lo, int j0, int B) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int base = j0 + 64 * i;
      const unsigned long long m =
          lo <= base ? hit[i] : lo - base < 64 ? hit[i] & (~0ull << (lo - base)) : 0ull;
      if (m) return base + __builtin_ctzll(m);
    }
    return B;
  }
};

template <int DK, int DV, typename InT, bool kGate>
__global__ __launch_bounds__(kThreads) void step_kernel(
    const InT* __restrict__ qp, const InT* __restrict__ kp, const InT* __restrict__ vp,
    const InT* __restrict__ gp, const InT* __restrict__ zp, const float* __restrict__ nw, float eps,
    InT* __restrict__ op, float* __restrict__ state, long n_slots, const int32_t* __restrict__ slots,
    int B, int H) {
  constexpr int LPR = DV / 4, RPP = kThreads / LPR, NG = DK / RPP;
  static_assert(DK % RPP == 0, "whole passes over the key dims");
  __shared__ float sPart[kThreads / 64][DV];
  const int h = blockIdx.x, b = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e4 = 4 * (tid % LPR), d0 = tid / LPR;
  const long slot = slots ? (long)slots[b] : (long)b;
  if (slot < 0 || slot >= n_slots) return;  // a padding row
  Slots rows0;
  if (slots) rows0.load(slots, 0, B);
  float* S = state + (slot * H + h) * (long)(DK * DV) + d0 * DV + e4;
  floatx4 s[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) s[i] = *reinterpret_cast<const floatx4*>(S + i * RPP * DV);
  // first row >= lo of this slot, or B
  auto find = [&](int lo) {
    int r = lo < Slots::kRows ? rows0.first(lo, 0, B) : B;
    for (int j0 = lo < Slots::kRows ? Slots::kRows : lo & -Slots::kRows; r >= B && j0 < B; j0 += Slots::kRows) {
      Slots more;
      more.load(slots, j0, B);
      more.compare((int)slot, j0, B);
      r = more.first(lo, j0, B);
    }
    return r;
  };
  if (slots) {
    rows0.compare((int)slot, 0, B);
    if (find(0) < b) return;  // that row's workgroup does this one too
  }
  for (int r = b;;) {
    const long row = (long)r * H + h;
    float x[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = (float)vp[row * DV + e4 + c];
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const long at = row * DK + d0 + i * RPP;
      const float a = tile::fexp2((float)gp[at] * kLog2e), kd = (float)kp[at], qd = (float)qp[at];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[i][c] = fmaf(a, s[i][c], kd * x[c]);
        o[c] = fmaf(qd, s[i][c], o[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int m = LPR; m < 64; m <<= 1) o[c] += __shfl_xor(o[c], m);
    }
    if (lane < LPR) *reinterpret_cast<floatx4*>(&sPart[wave][e4]) = floatx4{o[0], o[1], o[2], o[3]};
    __syncthreads();
    if (tid < DV) {
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) y += sPart[w][tid];
      if constexpr (kGate) {
        const float z = (float)zp[row * DV + tid];
        float ss = y * y;
#pragma unroll
        for (int m = 1; m < DV; m <<= 1) ss += __shfl_xor(ss, m);
        const float sig = __builtin_amdgcn_rcpf(1.f + tile::fexp2(-z * kLog2e));
        y *= __builtin_amdgcn_rsqf(ss * (1.f / DV) + eps) * nw[tid] * z * sig;
      }
      op[row * DV + tid] = (InT)y;
    }
    // the next row of the same sequence
    const int next = slots ? find(r + 1) : B;
    if (next >= B) break;
    r = next;
    __syncthreads();  // sPart is read
  }
#pragma unroll
  for (int i = 0; i < NG; ++i) *reinterpret_cast<floatx4*>(S + i * RPP * DV) = s[i];
}

template <int DK, int DV, typename InT>
hipError_t step_t(const StepArgs& a, hipStream_t s) {
  auto kernel = a.epi.gate ? step_kernel<DK, DV, InT, true> : step_kernel<DK, DV, InT, false>;
  hipLaunchKernelGGL(kernel, dim3(a.H, a.B), dim3(kThreads), 0, s, static_cast<const InT*>(a.q),
                     static_cast<const InT*>(a.k), static_cast<const InT*>(a.v),
                     static_cast<const InT*>(a.gk), static_cast<const InT*>(a.epi.gate),
                     a.epi.weight, a.epi.eps, static_cast<InT*>(a.out), a.state, a.n_slots, a.slots,
                     a.B, a.H);
  return hipGetLastError();
}

}  // namespace step

hipError_t launch_step(const StepArgs& a, hipStream_t s) {
  const bool f16 = a.dtype == 0;
#define GLA_STEP_CASE(DK, DV)              \
  if (a.dk == DK && a.dv == DV)            \
    return f16 ? step::step_t<DK, DV, half_t>(a, s) : step::step_t<DK, DV, float>(a, s);
  GLA_STEP_CASE(32, 32)
  GLA_STEP_CASE(32, 64)
  GLA_STEP_CASE(64, 32)
  GLA_STEP_CASE(64, 64)
#undef GLA_STEP_CASE
  return hipErrorInvalidValue;
}

}  // namespace gla
