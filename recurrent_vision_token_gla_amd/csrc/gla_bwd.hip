// Backward pass of the chunkwise key-only gated linear recurrence.
//
// Forward: S_t = diag(2^g_t) S_{t-1} + k_t^T v_t, o_t = q_t S_t (g the decay in
// log2). With go_t = dL/do_t and the gradient of the state after the last
// token, the gradient of the state runs the same recurrence from the end:
//   E_t = D_t + q_t^T go_t,   D_{t-1} = diag(2^g_t) E_t,
//   gq_t = S_t go_t,  gk_t = E_t v_t,  gv_t = E_t^T k_t,
//   gg_t[d] = sum_e 2^g_t[d] S_{t-1}[d][e] E_t[d][e].
// In chunks of 64 tokens, with b the in-chunk inclusive cumulative decay (log2)
// and B its last value:
//   U_n = sum_j (k_j 2^(B-b_j))^T v_j,   S_{n+1} = 2^B S_n + U_n   (forward)
//   R_n = sum_i (q_i 2^b_i)^T go_i,      D_{n-1} = 2^B D_n + R_n   (from the end)
//   P_ij = go_i . v_j,  A_ij = sum_d q_i k_j 2^(b_i-b_j)           (j <= i)
//   gq_i = 2^b_i S_n go_i + sum_{j<=i} P_ij k_j 2^(b_i-b_j)
//   gk_j = 2^(B-b_j) D_n v_j + sum_{i>=j} P_ij q_i 2^(b_i-b_j)
//   gv_j = D_n^T (k_j 2^(B-b_j)) + sum_{i>=j} A_ij go_i
// The decay's gradient at token t collects every path that crosses t: from the
// state before the chunk to the state behind it, from that state to the
// outputs at t and later, from the inputs before t to the state behind the
// chunk, and the pairs i >= t > j inside the chunk:
//   gg_t = 2^B <S_n, D_n> + sum_{i>=t} q_i gq_i^state + sum_{j<t} k_j gk_j^state
//          + sum_{i>=t} (q_i gq_i^pairs - k_i gk_i^pairs),
// rows of the inner product over e. In the last sum a token's pair with itself
// (no decay) is left out of both terms, where it would only cancel, so that
// what is left of a strongly decaying channel is not lost in its rounding.
//
// Products run on the matrix cores over operands split into bf16 terms
// (x = t0 + t1 [+ t2], each the rounding of what is left): bf16 has float's
// range, so no operand needs a scale, two terms hold 16 bits (half inputs are
// exact in them) and three hold float's 24. The products of two operands'
// terms are added in float, the smallest ones left out. The scans carry states
// from chunk to chunk in float; what the gradients read of each is float too,
// or for half inputs its two bf16 terms.
#include "gla_bwd.h"
#include "gla_tile.h"

namespace gla {
namespace bwd {

using tile::fexp2;
using tile::row_scan16;
using tile::token_row;

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf4 __attribute__((ext_vector_type(4)));

constexpr int C = kBwdChunk, NB = C / 16;
// A token's decay is taken as at least 2^-160: float rounds anything beyond
// 2^-149 to zero. A token that forgets everything puts that much into a
// cumulative sum, whose last bits are then coarse (2^-17 at 160, 2^-13 at
// 2048), so no decay between two tokens is a difference of sums that hold more
// than the decay of a sub-block with a reference: sums run from the token to
// where they are needed, or the tokens' decays are multiplied.
constexpr float kMinLog2 = -160.f;
__device__ __forceinline__ float log2_decay(float gk) {
  const float x = gk * kLog2e;
  return x < kMinLog2 ? kMinLog2 : x;  // NaN stays
}

__device__ __forceinline__ floatx4 mma(bf8 a, bf8 b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Eight or four floats as NT bf16 terms.
template <int NT> struct Split8 { bf8 t[NT]; };
template <int NT> struct Split4 { bf4 t[NT]; };
// Two floats' leading bf16 terms in one register, and what they leave: pairs,
// written out, take one conversion and two subtractions per term (whole
// vectors were converted element by element).
__device__ __forceinline__ unsigned term2(float& a, float& b, bool rest) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  const unsigned u = __builtin_bit_cast(unsigned, __builtin_convertvector(f2{a, b}, bf2));
  if (rest) {
    a -= __uint_as_float(u << 16);
    b -= __uint_as_float(u & 0xffff0000u);
  }
  return u;
}
template <int NT>
__device__ __forceinline__ Split8<NT> split8(const float* x) {
  Split8<NT> s;
  float r[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) r[c] = x[c];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    tile::u32x4 u;
#pragma unroll
    for (int c = 0; c < 4; ++c) u[c] = term2(r[2 * c], r[2 * c + 1], t + 1 < NT);
    s.t[t] = __builtin_bit_cast(bf8, u);
  }
  return s;
}
template <int NT>
__device__ __forceinline__ Split4<NT> split4(floatx4 x) {
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  Split4<NT> s;
  float r[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const u32x2 u = {term2(r[0], r[1], t + 1 < NT), term2(r[2], r[3], t + 1 < NT)};
    s.t[t] = __builtin_bit_cast(bf4, u);
  }
  return s;
}

// c += a b over 32 contracted elements: the products of terms i + j < NT, and
// with three terms the middle ones' product.
template <int NT>
__device__ __forceinline__ floatx4 mm(const Split8<NT>& a, const Split8<NT>& b, floatx4 c) {
  if constexpr (NT == 3) {
    c = mma(a.t[2], b.t[0], c);
    c = mma(a.t[0], b.t[2], c);
    c = mma(a.t[1], b.t[1], c);
  }
  c = mma(a.t[1], b.t[0], c);
  c = mma(a.t[0], b.t[1], c);
  return mma(a.t[0], b.t[0], c);
}

__device__ __forceinline__ bf8 join(bf4 a, bf4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
// c += x p over 16 contracted elements, four per lane: the 32 places of one
// matrix product hold two terms of x against the same term of p.
template <int NT>
__device__ __forceinline__ floatx4 mm16(const Split4<NT>& x, const Split4<NT>& p, floatx4 c) {
  const bf8 x01 = join(x.t[0], x.t[1]);
  if constexpr (NT == 3) c = mma(join(x.t[2], x.t[0]), join(p.t[0], p.t[2]), c);
  c = mma(x01, join(p.t[1], p.t[1]), c);
  return mma(x01, join(p.t[0], p.t[0]), c);
}

// Orders a wave's LDS writes before its own later LDS reads (the LDS unit
// keeps a wave's accesses in order; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A lane's values of a token row as loaded, eight neighbours per ks (half
// inputs stay packed, and are converted where a product uses them).
template <typename InT, int NEL> struct Raw {
  typedef InT V8 __attribute__((ext_vector_type(8)));
  V8 v[NEL / 8];
  __device__ __forceinline__ void load(const InT* p) {  // dims 32 ks + 0..7 from p
#pragma unroll
    for (int ks = 0; ks < NEL / 8; ++ks) v[ks] = *reinterpret_cast<const V8*>(p + 32 * ks);
  }
  __device__ __forceinline__ void zero_if(bool pad) {
#pragma unroll
    for (int ks = 0; ks < NEL / 8; ++ks) v[ks] = pad ? V8{} : v[ks];
  }
  __device__ __forceinline__ float operator[](int e) const { return (float)v[e / 8][e % 8]; }
  template <int NT> __device__ __forceinline__ Split8<NT> terms(int ks) const {
    float x[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = (*this)[8 * ks + c];
    return split8<NT>(x);
  }
};

// Inclusive suffix sum over the 16 lanes of a DPP row; neighbours' values.
__device__ __forceinline__ float row_suffix16(float x) {
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x101, 0xf, 0xf, true));
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x102, 0xf, 0xf, true));
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x104, 0xf, 0xf, true));
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x108, 0xf, 0xf, true));
  return x;
}
__device__ __forceinline__ float row_before16(float x) {  // the lane before's, or zero
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x111, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_after16(float x) {  // the next lane's, or zero
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x101, 0xf, 0xf, true));
}

template <int CTRL>
__device__ __forceinline__ float row_add(float x) {  // x plus the lane's that CTRL shifts in
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
// For values x of 16 tokens, s = the sum over tokens 8..i, or less the sum over
// i+1..7; and, on lane 0, lo = the sum over 0..7. (Step by step over all values:
// a lane permutation waits for the instruction before it.)
template <int N>
__device__ __forceinline__ void from_middle16(const float (&x)[N], float (&s)[N], float (&lo)[N]) {
  const bool low = (threadIdx.x & 8) == 0;
#pragma unroll
  for (int e = 0; e < N; ++e) lo[e] = low ? x[e] : 0.f, s[e] = low ? 0.f : x[e];
#pragma unroll
  for (int e = 0; e < N; ++e) lo[e] = row_add<0x101>(lo[e]), s[e] = row_add<0x111>(s[e]);
#pragma unroll
  for (int e = 0; e < N; ++e) lo[e] = row_add<0x102>(lo[e]), s[e] = row_add<0x112>(s[e]);
#pragma unroll
  for (int e = 0; e < N; ++e) lo[e] = row_add<0x104>(lo[e]), s[e] = row_add<0x114>(s[e]);
#pragma unroll
  for (int e = 0; e < N; ++e) s[e] -= row_after16(lo[e]);
}

// LDS tiles have rows of W 16-bit values without padding; the 16-byte chunk c
// of a row lies at chunk c ^ swz(row). The equal chunks of the eight rows that
// an operand read along rows touches together, and the four rows' 8-byte
// pieces of a transposed read, then fall on different banks. Rows of a tile
// are tokens or, with kDims, the dims of a state.
template <int W, bool kDims>
__device__ __forceinline__ int swz(int row) {
  const int far = row >> (kDims ? 3 : 2);
  return W == 64 ? ((row & 2) << 1) | ((far & 1) << 1) | (row & 1) : far & 3;
}
template <int W, bool kDims>
__device__ __forceinline__ int at_chunk(int row, int c) {
  return row * W + 8 * (c ^ swz<W, kDims>(row));
}
// A lane works on eight neighbouring dims 32 ks + 8 lq + 0..7 (lq = lane / 16),
// so the blocks D = 2 ks + h of 16 dims that a product takes are 32 ks + 8 (m /
// 4) + 4 h + m % 4, m = 0..15: the dim of block D that is row (or column) m.
__device__ __forceinline__ int dim_row(int D, int lr) {
  return 32 * (D / 2) + 8 * (lr >> 2) + 4 * (D % 2) + (lr & 3);
}
// A lane's places in a tile of tokens, relative to a row that is a multiple of
// 16: its eight contracted values of row lr, chunk 4 ks + lq; and its part of
// the transposed read of column block D along rows 4 lq + 0..3. In a state:
// the same of block D's rows (`row` and 4 (D % 2) W further: the swizzle does
// not look at that bit), and of column block E along rows 8 lq + 0..3.
// Chunk 4 ks + c is chunk c with bit 2 of the place flipped (W = 64), so ks may
// be a variable.
template <int W, bool kDims>
struct Lane {
  int row, col;
  __device__ __forceinline__ Lane() {
    const int lr = threadIdx.x & 15, lq = (threadIdx.x >> 4) & 3;
    row = at_chunk<W, kDims>(kDims ? dim_row(0, lr) : lr, lq);
    col = at_chunk<W, kDims>((kDims ? 8 : 4) * lq + (lr >> 2), lr & 3);
  }
  __device__ __forceinline__ bf8 rows(const __bf16* tl, int ks) const {
    return *reinterpret_cast<const bf8*>(tl + (row ^ 32 * ks));
  }
  __device__ __forceinline__ void put(__bf16* tl, int ks, bf8 x) const {
    *reinterpret_cast<bf8*>(tl + (row ^ 32 * ks)) = x;
  }
  __device__ __forceinline__ bf4 cols(const __bf16* tl, int D) const {
    return __builtin_bit_cast(bf4, __builtin_amdgcn_ds_read_tr16_b64_v4f16(
                                       (tile::lds_fp16x4_t*)(tl + (col ^ 32 * (D / 2)) + 4 * (D % 2))));
  }
};

// ===========================================================================
// Chunk summaries: one workgroup per (chunk, head, batch) and direction of
// time: U_n and the decay a_n from (k, v), or R_n from (q, go). A wave scales
// the 16 tokens of its sub-block by their decay to the sub-block's end (k) or
// from its start (q), and stages them as token rows; both operands of the
// contraction over tokens come back through the transposing read. The sub-
// blocks are added farthest from the chunk's end (k) or start (q) first, and
// what is accumulated decays through each of them: a lane's column of the
// transposed product is one key dim, so that is one factor per sub-block.
// The scaled operand has NX bf16 terms: three for half inputs too (the other
// is exact in two) where the initial state's gradient is returned, in float:
// it is then off by 2e-7 of its size instead of 4e-6, for 4 us more at the
// sizes below, while the other gradients, rounded to half, do not change.
//
// The memory bounds it: 25,600 half tokens x 16 heads of 64/64 (6,400 chunks,
// 307 MB read and 206 written by the counters) take 87 us, 5.9 TB/s; the 150
// chunks of 1,600 tokens x 6 heads 8.2 us, where a workgroup's own 9,000 cycles
// of loads, factors and products in turn are what is left to wait for. Three
// workgroups per CU: LDS holds four, and more registers per lane (up to 128),
// or all sub-blocks' products before the first decay, changed nothing.
// ===========================================================================
template <int DK, int DV, typename InT, int NT, int NX>
__global__ __launch_bounds__(kThreads, 3) void bwd_summary_kernel(
    const InT* __restrict__ kp, const InT* __restrict__ vp, const InT* __restrict__ qp,
    const InT* __restrict__ dop, const InT* __restrict__ gp, float* __restrict__ Uws,
    float* __restrict__ Rws, float* __restrict__ Aws, int T, int H, int N, int gh, int gw,
    DirPack dirs) {
  constexpr int NKS = DK / 32, NEL = 8 * NKS, NES = DV / 32, ND = DK / 16;
  constexpr int KB = 16 * DK, VB = 16 * DV;  // 16 rows of a tile
  __shared__ __attribute__((aligned(16))) __bf16 sX[NX][C * DK];
  __shared__ __attribute__((aligned(16))) __bf16 sY[NT][C * DV];
  __shared__ __attribute__((aligned(16))) float sE[NB][DK];  // decay of a sub-block
  const bool rev = blockIdx.z & 1;
  const int n = blockIdx.x, h = blockIdx.y, b = blockIdx.z >> 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lq = lane >> 4;
  const int rr = token_row(n * C + 16 * wave + lr, T, gh, gw, dirs.get(b));
  const bool pad = rr < 0;
  const long row = ((long)b * T + (pad ? 0 : rr)) * H + h;
  const Lane<DK, false> lk;
  const Lane<DV, false> lv;
  Raw<InT, NEL> x, g;
  Raw<InT, 8 * NES> y;
  g.load(gp + row * DK + 8 * lq);
  x.load((rev ? qp : kp) + row * DK + 8 * lq);
  y.load((rev ? dop : vp) + row * DV + 8 * lq);
  if ((n + 1) * C > T) {  // the chain's last chunk: padding rows are zeros without decay
    g.zero_if(pad);
    x.zero_if(pad);
    y.zero_if(pad);
  }
  // cumulative decay from the sub-block's start to each token (q), or from
  // behind it to the end (k): sums of just the tokens between
  float s[NEL];
  if (rev) {
#pragma unroll
    for (int e = 0; e < NEL; ++e) s[e] = row_scan16(log2_decay(g[e]));
  } else {
#pragma unroll
    for (int e = 0; e < NEL; ++e) s[e] = row_suffix16(log2_decay(g[e]));
  }
  if (lr == (rev ? 15 : 0)) {
#pragma unroll
    for (int e = 0; e < NEL; e += 4)
      *reinterpret_cast<floatx4*>(&sE[wave][32 * (e / 8) + 8 * lq + e % 8]) =
          floatx4{s[e], s[e + 1], s[e + 2], s[e + 3]};
  }
  wave_sync();
  for (int d = lane; d < DK; d += 64) sE[wave][d] = fexp2(sE[wave][d]);
  if (!rev) {
#pragma unroll
    for (int e = 0; e < NEL; ++e) s[e] = row_after16(s[e]);
  }
#pragma unroll
  for (int ks = 0; ks < NKS; ++ks) {
    float o[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] = tile::mulw(x[8 * ks + c], fexp2(s[8 * ks + c]));
    const Split8<NX> t = split8<NX>(o);
#pragma unroll
    for (int i = 0; i < NX; ++i) lk.put(&sX[i][wave * KB], ks, t.t[i]);
  }
#pragma unroll
  for (int ks = 0; ks < NES; ++ks) {
    const Split8<NT> t = y.template terms<NT>(ks);
#pragma unroll
    for (int i = 0; i < NT; ++i) lv.put(&sY[i][wave * VB], ks, t.t[i]);
  }
  __syncthreads();

  const long bhn = ((long)b * H + h) * N + n;
  if (!rev && tid < DK) {
    float a = sE[0][tid];
#pragma unroll
    for (int J = 1; J < NB; ++J) a *= sE[J][tid];
    Aws[bhn * DK + tid] = a;
  }
  // Y^T X for pairs of value blocks (32 columns): a lane ends up with eight
  // neighbouring value columns of one key dim
  float* out = (rev ? Rws : Uws) + bhn * (long)(DK * DV);
  constexpr int NPAIR = ND * NES, PPW = NPAIR / 4 > 0 ? NPAIR / 4 : 1;
#pragma unroll
  for (int i = 0; i < PPW; ++i) {
    const int pr = wave * PPW + i, D = pr / NES, ks = pr % NES;
    if (pr >= NPAIR) break;
    floatx4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    const int d = dim_row(D, lr);
#pragma unroll
    for (int step = 0; step < NB; ++step) {
      const int J = rev ? NB - 1 - step : step;
      Split4<NX> xs;
#pragma unroll
      for (int m = 0; m < NX; ++m) xs.t[m] = lk.cols(&sX[m][J * KB], D);
      const bf8 x01 = join(xs.t[0], xs.t[1]), x22 = join(xs.t[NX - 1], xs.t[NT == 3 ? 0 : NX - 1]);
      const float e = sE[J][d];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        Split4<NT> ys;
#pragma unroll
        for (int m = 0; m < NT; ++m) ys.t[m] = lv.cols(&sY[m][J * VB], 2 * ks + hh);
        if (step) acc[hh] *= e;
        if (NX == 3) acc[hh] = mma(join(ys.t[0], ys.t[NT - 1]), x22, acc[hh]);
        acc[hh] = mma(join(ys.t[1], ys.t[1]), x01, acc[hh]);
        acc[hh] = mma(join(ys.t[0], ys.t[0]), x01, acc[hh]);
      }
    }
    float* o = out + d * DV + 32 * ks + 8 * lq;
    *reinterpret_cast<floatx4*>(o) = acc[0];
    *reinterpret_cast<floatx4*>(o + 4) = acc[1];
  }
}

// ===========================================================================
// State scans, in place: S_n over U_n in forward order, D_n over R_n from the
// end; every state element is its own first-order recurrence over the chunks,
//   x_0 given or 0,  x_{i+1} = a_i x_i + u_i,
// held in float. What the gradients read back (x_i) is stored as float, or
// for half inputs as the two bf16 terms their products take: 16 bytes per
// four elements either way, {t0 of the four, t1 of the four}.
// ===========================================================================
template <bool kTerms>
__device__ __forceinline__ void put_state4(float* p, floatx4 s) {
  if constexpr (kTerms) {
    const Split4<2> t = split4<2>(s);
    *reinterpret_cast<bf8*>(p) = join(t.t[0], t.t[1]);
  } else {
    *reinterpret_cast<floatx4*>(p) = s;
  }
}
__device__ __forceinline__ floatx4 step4(float a, floatx4 s, floatx4 u) {
#pragma unroll
  for (int c = 0; c < 4; ++c) s[c] = fmaf(a, s[c], u[c]);
  return s;
}

// Many chains: one thread walks four elements of a chain in order, the next
// W/2 to W chunks' loads in flight (the window is refilled half by half, and
// whole windows run without a condition, which would wait for every load).
// The memory bounds it: 64 chains of 100 chunks (211 MB read, 205 written)
// take 67 us, 6.2 TB/s, part of it from the last-level cache.
template <int W, bool kTerms>
__global__ __launch_bounds__(kThreads) void bwd_scan_serial_kernel(
    float* Uws, float* Rws, const float* __restrict__ Aws, const float* s0, const float* gsf,
    float* gs0, int N, int DK, int DV, long groups) {
  const long gid = (long)blockIdx.x * kThreads + threadIdx.x;
  if (gid >= groups) return;
  const bool rev = blockIdx.y;
  const long DKDV = (long)DK * DV, per = DKDV / 4;
  const long bh = gid / per;
  const int x4 = 4 * (int)(gid - bh * per), d = x4 / DV;
  // chunk i of the walk is chunk i, or N-1-i
  const long first = rev ? N - 1 : 0, sx = rev ? -DKDV : DKDV, sa = rev ? -DK : DK;
  float* X = (rev ? Rws : Uws) + (bh * N + first) * DKDV + x4;
  const float* A = Aws + (bh * N + first) * DK + d;
  const float* init = rev ? gsf : s0;
  floatx4 s = {0.f, 0.f, 0.f, 0.f};
  if (init) s = *reinterpret_cast<const floatx4*>(init + bh * DKDV + x4);
  floatx4 u[W];
  float a[W];
  constexpr int HW = W / 2;
  auto refill = [&](int h, int i0) {  // half h of the window: chunks i0.. (clamped)
#pragma unroll
    for (int j = 0; j < HW; ++j) {
      const long m = i0 + j < N ? i0 + j : N - 1;
      u[h * HW + j] = *reinterpret_cast<const floatx4*>(X + m * sx);
      a[h * HW + j] = A[m * sa];
    }
  };
  auto step = [&](int w, int i) {
    put_state4<kTerms>(X + i * sx, s);
    s = step4(a[w], s, u[w]);
  };
  refill(0, 0);
  refill(1, HW);
  int n0 = 0;
  for (; n0 + W <= N; n0 += W) {
#pragma unroll
    for (int j = 0; j < HW; ++j) step(j, n0 + j);
    __builtin_amdgcn_sched_barrier(0);
    refill(0, n0 + W);
#pragma unroll
    for (int j = 0; j < HW; ++j) step(HW + j, n0 + HW + j);
    __builtin_amdgcn_sched_barrier(0);
    refill(1, n0 + W + HW);
  }
#pragma unroll
  for (int w = 0; w < W - 1; ++w)
    if (n0 + w < N) step(w, n0 + w);
  if (rev && gs0) *reinterpret_cast<floatx4*>(gs0 + bh * DKDV + x4) = s;
}

// Few chains: a workgroup takes 64 groups of four elements (1 KB of a state, a
// load or store of a wave) and windows of 16 segments of up to R chunks, a wave
// each. A wave folds its segment into (a, u), the 16 are composed from LDS, and
// the wave replays its segment, still in registers, from the state entering it.
// 6 chains of 25 or 100 chunks: 4.8 or 9.6 us. (With the segments on the lanes of
// a row, composed by lane permutations, accesses were 64 bytes wide: 12 us.)
template <int R, bool kTerms>
__global__ __launch_bounds__(1024) void bwd_scan_kernel(
    float* Uws, float* Rws, const float* __restrict__ Aws, const float* s0, const float* gsf,
    float* gs0, int N, int DK, int DV, int L) {
  __shared__ floatx4 sU[16][64];
  __shared__ float sA[16][64];
  const int seg = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const bool rev = blockIdx.y;
  const int DKDV = DK * DV, per = DKDV / 256;  // workgroups per chain
  const long bh = blockIdx.x / per;
  const int x4 = 4 * ((int)(blockIdx.x % per) * 64 + lane), d = x4 / DV;
  // chunk i of the walk is chunk i, or N-1-i
  const long first = rev ? N - 1 : 0, sx = rev ? -DKDV : DKDV, sa = rev ? -DK : DK;
  float* X = (rev ? Rws : Uws) + (bh * N + first) * DKDV + x4;
  const float* A = Aws + (bh * N + first) * DK + d;
  const float* init = rev ? gsf : s0;
  floatx4 s = {0.f, 0.f, 0.f, 0.f};
  if (init) s = *reinterpret_cast<const floatx4*>(init + bh * DKDV + x4);
  for (int base = 0; base < N; base += 16 * L) {
    const int n0 = base + seg * L, m = min(L, N - n0);  // this wave's chunks, maybe none
    floatx4 u[R], ug = {0.f, 0.f, 0.f, 0.f};
    float a[R], ag = 1.f;
    if (m > 0) {
#pragma unroll
      for (int i = 0; i < R; ++i) {  // clamped, all in flight together
        const long c = n0 + min(i, m - 1);
        u[i] = *reinterpret_cast<const floatx4*>(X + c * sx);
        a[i] = A[c * sa];
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (i < m) {
          ug = step4(a[i], ug, u[i]);
          ag *= a[i];
        }
      }
    }
    if (base) __syncthreads();  // the last window's sums are read
    sU[seg][lane] = ug;
    sA[seg][lane] = ag;
    __syncthreads();
    floatx4 x = s;  // the state that enters the segment
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      x = j == seg ? s : x;
      s = step4(sA[j][lane], s, sU[j][lane]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i < m) {
        put_state4<kTerms>(X + (n0 + i) * sx, x);
        x = step4(a[i], x, u[i]);
      }
    }
  }
  if (rev && gs0 && seg == 0) *reinterpret_cast<floatx4*>(gs0 + bh * DKDV + x4) = s;
}

// ===========================================================================
// Gradients: one workgroup per (chunk, head, batch), four waves; wave w owns
// the 16 tokens of sub-block w as queries (gq) and as keys (gk, gv). A lane
// holds token lr = lane % 16 of it and the dims d = 32 ks + 8 lq + c (lq = lane
// / 16): as an operand these are eight contracted places per ks, and a product
// written transposed (rows = dims, columns = tokens) in blocks D = 2 ks + h of
// the dims 32 ks + 8 (m / 4) + 4 h + m % 4, m = 0..15, leaves exactly the same
// token and dims in the lane, so inputs, factors and results meet in registers
// and a lane loads and stores 16 contiguous bytes of a row.
//
// With s the cumulative decay inside a sub-block (log2), tot its last value
// and ref its value at the 8th token, the rows kept in LDS are
//   qx = q 2^(s-ref),  kx = k 2^(ref-s),
// so the pairs inside the sub-block need no other factor, and pairs of two
// sub-blocks I > J only factors by dim, all <= 1 (tables in LDS):
//   2^(b_i-b_j) = 2^(s_i-ref_I) [2^ref_I prod_{J<M<I} 2^tot_M] [2^(tot_J-ref_J) 2^(ref_J-s_j)].
// s - ref is summed from the 8th token outwards, so it holds the decays between
// the two tokens only (a first token that forgets everything is in ref alone).
// Where none exceeds 66 in magnitude, values up to 65504 keep qx and kx below
// 2^82 and every product finite (P is at most 64 products of two such values).
// The factors are applied so that no intermediate underflows unless the pair's
// whole factor is below 2^-60: gq's sums take 2^(tot_J-ref_J) and then 2^ref_I,
// which is a normal float unless the first token alone decays by 2^-60; a key's
// last bracket is multiplied first, to 2^(tot_J-s_j) <= 1. A sub-block that
// decays more keeps q 2^s and k 2^(tot-s) instead (2^ref and 2^(tot-ref) are
// then 1) and takes its own pairs from products of the tokens' decays.
//
// A workgroup's own chain of steps bounds it: alone on a CU it takes 22,100
// cycles, with a second one 24,400, in which each SIMD issues vector
// instructions for 15,800 (1,979 per wave, half of them factors, splits and
// scans; 172 matrix products). 25,600 half tokens x 16 heads of 64/64: 166 us
// (461 MB read, 205 written: 4.0 TB/s); 1,600 tokens x 6 heads, less than a
// workgroup per CU: 12 us. Pairs taken from products of decays cost a wave that
// does so 15 steps of a permutation and five products per dim: the whole pass of
// those 25,600 tokens takes 321 us without, 332 with a token that forgets
// everything in every 1,000 and 426 with one in every 23. Eight waves with
// queries and keys apart have 128 registers a lane and spilled (1.2 times the
// time); so did all gradients stored at the end, or D_n's rows read again for
// <S_n, D_n>.
// ===========================================================================
constexpr float kMaxSpan = 66.f;

// Two workgroups per CU where their LDS fits (at most 80 KB; a half input's
// largest takes 79, a float's 80 with 32 key dims): one alone leaves the SIMDs
// waiting more than half of the time (2 x 4,099 float tokens x 4 heads of 32/64
// with one or two: 31 or 23 us). A float's 64/64 takes 119 KB and has one: a
// pass of 2 x 3,600 tokens x 8 heads 92 us, of half inputs 53.
template <int DK, int DV, typename InT, int NT>
__global__ __launch_bounds__(kThreads, sizeof(InT) == 2 || DK == 32 ? 2 : 1) void bwd_grad_kernel(
    const InT* __restrict__ qp, const InT* __restrict__ kp, const InT* __restrict__ vp,
    const InT* __restrict__ gp, const InT* __restrict__ dop, const float* __restrict__ Sws,
    const float* __restrict__ Dws, InT* __restrict__ gqp, InT* __restrict__ gkp,
    InT* __restrict__ gvp, InT* __restrict__ ggp, int T, int H, int N, int gh, int gw,
    DirPack dirs) {
  constexpr bool kHalf = sizeof(InT) == 2;
  constexpr int NKS = DK / 32, NES = DV / 32, ND = DK / 16, NE = DV / 16;
  constexpr int NEL = 4 * ND, NVL = 4 * NE;  // a lane's dims of q/k/g and of v/go
  constexpr int NP = NB * (NB - 1) / 2;      // pairs of sub-blocks
  constexpr int KB = 16 * DK, VB = 16 * DV;  // 16 rows of a tile
  __shared__ __attribute__((aligned(16))) __bf16 sQ[NT][C * DK];             // qx
  __shared__ __attribute__((aligned(16))) __bf16 sK[NT][C * DK];             // kx
  __shared__ __attribute__((aligned(16))) __bf16 sO[NT][C * DV];             // go
  __shared__ __attribute__((aligned(16))) __bf16 sV[kHalf ? 1 : 2][C * DV];  // v as it is (float: upper and lower halves)
  __shared__ __attribute__((aligned(16))) __bf16 sX[NT][DK * DV];            // S_n, then D_n
  __shared__ __attribute__((aligned(16))) float sF[NP][DK];   // factors between two sub-blocks
  __shared__ __attribute__((aligned(16))) float sA[NB][DK];   // tot; factors to the chunk's end; sums
  __shared__ __attribute__((aligned(16))) float sB[NB][DK];   // ref; sums of k gk^state
  __shared__ __attribute__((aligned(16))) float sE[NB][DK];   // 2^tot
  __shared__ __attribute__((aligned(16))) float sEQ[NB][DK];  // 2^ref (1 in a direct sub-block)
  __shared__ __attribute__((aligned(16))) float sEK[NB][DK];  // 2^(tot-ref) (likewise)
  __shared__ __attribute__((aligned(16))) float sAD[DK];      // 2^B <S_n, D_n> by rows
  __shared__ float sSelf[C];                                  // P_tt
  __shared__ int sDirect[NB];
  const int n = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lq = lane >> 4;
  const int dir = dirs.get(b), t = 16 * wave + lr;
  const long bhn = ((long)b * H + h) * N + n;
  auto dim = [&](int D) { return 32 * (D / 2) + 8 * lq + 4 * (D % 2); };  // the first of a lane's four in block D
  const Lane<DK, false> lk;
  const Lane<DV, false> lv;
  const Lane<DV, true> lx;

  // -- this lane's token row
  const int rr = token_row(n * C + t, T, gh, gw, dir);
  const bool pad = rr < 0;
  const long row = ((long)b * T + (pad ? 0 : rr)) * H + h;
  Raw<InT, NEL> q, k, g;
  Raw<InT, NVL> v, go;
  g.load(gp + row * DK + dim(0));
  q.load(qp + row * DK + dim(0));
  k.load(kp + row * DK + dim(0));
  v.load(vp + row * DV + dim(0));
  go.load(dop + row * DV + dim(0));
  // -- a state of the chunk's ends: 16 bytes of it per thread and step
  constexpr int NG = DK * DV / 4 / kThreads, LPR = DV / 4;
  floatx4 st[NG];
  auto load_state = [&](const float* p) {
#pragma unroll
    for (int i = 0; i < NG; ++i)
      st[i] = *reinterpret_cast<const floatx4*>(p + bhn * (DK * DV) + 4 * (tid + kThreads * i));
  };
  auto put_state = [&]() {
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int u = tid + kThreads * i, d = u / LPR, e = 4 * (u % LPR);
      const int p = at_chunk<DV, true>(d, e / 8) + e % 8;
      if constexpr (kHalf) {
        const bf8 x = __builtin_bit_cast(bf8, st[i]);
        *reinterpret_cast<bf4*>(&sX[0][p]) = __builtin_shufflevector(x, x, 0, 1, 2, 3);
        *reinterpret_cast<bf4*>(&sX[1][p]) = __builtin_shufflevector(x, x, 4, 5, 6, 7);
      } else {
        const Split4<NT> sp = split4<NT>(st[i]);
#pragma unroll
        for (int j = 0; j < NT; ++j) *reinterpret_cast<bf4*>(&sX[j][p]) = sp.t[j];
      }
    }
  };
  load_state(Sws);
  if ((n + 1) * C > T) {  // the chain's last chunk: padding rows are zeros without decay
    g.zero_if(pad);
    q.zero_if(pad);
    k.zero_if(pad);
    v.zero_if(pad);
    go.zero_if(pad);
  }
  // -- decay between each token and the sub-block's 8th: s - ref, a sum over
  // tokens 8..i, or less one over i+1..7; the first token's own is in ref alone
  float s[NEL], lo[NEL];
  {
    float x[NEL];
#pragma unroll
    for (int e = 0; e < NEL; ++e) x[e] = log2_decay(g[e]);
    from_middle16(x, s, lo);
  }
  auto row4 = [&](const float* x, int D) { return floatx4{x[4 * D], x[4 * D + 1], x[4 * D + 2], x[4 * D + 3]}; };
  if (lr == 15) {
#pragma unroll
    for (int D = 0; D < ND; ++D) *reinterpret_cast<floatx4*>(&sA[wave][dim(D)]) = row4(s, D);
  }
  if (lr == 0) {
#pragma unroll
    for (int D = 0; D < ND; ++D) *reinterpret_cast<floatx4*>(&sB[wave][dim(D)]) = row4(lo, D);
  }
  // -- the factors, which the gradients take too
  float cq[NEL], ck[NEL], span = 0.f;
#pragma unroll
  for (int e = 0; e < NEL; ++e) span = fmaxf(span, fabsf(s[e]));
  const bool direct = !__all(span <= kMaxSpan);
  if (!direct) {
#pragma unroll
    for (int e = 0; e < NEL; ++e) {
      ck[e] = fexp2(-s[e]);
      cq[e] = fexp2(s[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < NEL; ++e) {
      const float x = log2_decay(g[e]);
      ck[e] = fexp2(row_after16(row_suffix16(x)));
      cq[e] = fexp2(row_scan16(x));
      s[e] = fexp2(x);  // the token's own decay is what the pairs below take
    }
  }
  wave_sync();  // tot - ref and ref
  for (int d = lane; d < DK; d += 64) {
    const float td = sA[wave][d], rd = sB[wave][d];
    sE[wave][d] = fexp2(td + rd);
    sEQ[wave][d] = direct ? 1.f : fexp2(rd);
    sEK[wave][d] = direct ? 1.f : fexp2(td);
  }
  if (lane == 0) sDirect[wave] = direct;
  const floatx4 zero4 = {0.f, 0.f, 0.f, 0.f};
  floatx4 an = zero4;  // A inside the sub-block, rows i
#pragma unroll
  for (int ks = 0; ks < NKS; ++ks) {
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = tile::mulw(q[8 * ks + i], cq[8 * ks + i]);
      y[i] = tile::mulw(k[8 * ks + i], ck[8 * ks + i]);
    }
    const Split8<NT> xs = split8<NT>(x), ys = split8<NT>(y);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      lk.put(&sQ[i][wave * KB], ks, xs.t[i]);
      lk.put(&sK[i][wave * KB], ks, ys.t[i]);
    }
    an = mm<NT>(xs, ys, an);
  }
  // -- v and go to LDS; P inside the sub-block: transposed (rows j) for gq,
  // and rows i for gk
  floatx4 pt = zero4, pn = zero4;
#pragma unroll
  for (int ks = 0; ks < NES; ++ks) {
    const Split8<NT> os = go.template terms<NT>(ks);
#pragma unroll
    for (int i = 0; i < NT; ++i) lv.put(&sO[i][wave * VB], ks, os.t[i]);
    if constexpr (kHalf) {
      lv.put(&sV[0][wave * VB], ks, __builtin_bit_cast(bf8, v.v[ks]));
      pt = mfma16x16x32(v.v[ks], go.v[ks], pt);
      pn = mfma16x16x32(go.v[ks], v.v[ks], pn);
    } else {
      const Split8<NT> vs = v.template terms<NT>(ks);
      tile::u32x4 hi, lo;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const unsigned a = __float_as_uint(v.v[ks][2 * c]), b = __float_as_uint(v.v[ks][2 * c + 1]);
        hi[c] = __builtin_amdgcn_perm(b, a, 0x07060302);
        lo[c] = __builtin_amdgcn_perm(b, a, 0x05040100);
      }
      lv.put(&sV[0][wave * VB], ks, __builtin_bit_cast(bf8, hi));
      lv.put(&sV[1][wave * VB], ks, __builtin_bit_cast(bf8, lo));
      pt = mm<NT>(vs, os, pt);
      pn = mm<NT>(os, vs, pn);
    }
  }
  put_state();  // S_n
  // operands from LDS: 16 rows of a tile (from element `at` of its planes)
  // contracted along the row; 16 columns (block D) contracted along 16 rows
  auto rows8 = [&](const auto& ln, const auto& tl, int at, int ks) {
    Split8<NT> sp;
#pragma unroll
    for (int i = 0; i < NT; ++i) sp.t[i] = ln.rows(&tl[i][at], ks);
    return sp;
  };
  auto state_at = [&](int D) { return 2 * (D / 2) * VB + 4 * (D % 2) * DV; };  // block D of a state's rows
  auto cols4 = [&](const auto& ln, const auto& tl, int at, int D) {
    Split4<NT> sp;
#pragma unroll
    for (int i = 0; i < NT; ++i) sp.t[i] = ln.cols(&tl[i][at], D);
    return sp;
  };
  // P of block J's keys with this wave's queries, transposed; and of block I's
  // queries with this wave's keys (half inputs: exact, four products of terms)
  auto p_keys = [&](int J) {
    floatx4 p = zero4;
#pragma unroll
    for (int ks = 0; ks < NES; ++ks) {
      if constexpr (kHalf) {
        p = mfma16x16x32(__builtin_bit_cast(half8, lv.rows(&sV[0][J * VB], ks)), go.v[ks], p);
      } else {
        const tile::u32x4 hi = __builtin_bit_cast(tile::u32x4, lv.rows(&sV[0][J * VB], ks));
        const tile::u32x4 lo = __builtin_bit_cast(tile::u32x4, lv.rows(&sV[1][J * VB], ks));
        float x[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[2 * c] = __uint_as_float(__builtin_amdgcn_perm(hi[c], lo[c], 0x05040100));
          x[2 * c + 1] = __uint_as_float(__builtin_amdgcn_perm(hi[c], lo[c], 0x07060302));
        }
        p = mm<NT>(split8<NT>(x), go.template terms<NT>(ks), p);
      }
    }
    return p;
  };
  Split8<NT> vs[NES];
  auto p_queries = [&](int I) {
    floatx4 p = zero4;
#pragma unroll
    for (int ks = 0; ks < NES; ++ks) {
      const Split8<NT> o = rows8(lv, sO, I * VB, ks);
      if constexpr (kHalf) p = mma(o.t[1], vs[ks].t[1], p);
      p = mm<NT>(o, vs[ks], p);
    }
    return p;
  };
  // -- pairs inside the sub-block, a token's pair with itself left out of gq
  // and gk (added at the end); the rows are this wave's own
  floatx4 gq[ND], gk[ND], gv[NE];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (4 * lq + r == lr) sSelf[t] = pn[r];
  wave_sync();
  if (!direct) {
    floatx4 ps;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int x = 4 * lq + r;
      pt[r] = x < lr ? pt[r] : 0.f;
      ps[r] = x > lr ? pn[r] : 0.f;
    }
    const Split4<NT> pts = split4<NT>(pt), pns = split4<NT>(ps);
#pragma unroll
    for (int D = 0; D < ND; ++D) {
      gq[D] = mm16<NT>(cols4(lk, sK, wave * KB, D), pts, zero4);
      gk[D] = mm16<NT>(cols4(lk, sQ, wave * KB, D), pns, zero4);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        gq[D][r] *= cq[4 * D + r];
        gk[D][r] *= ck[4 * D + r];
      }
    }
  } else {
    // every pair on its own, at distance x = i - j from 0 to 15: with a_t the
    // tokens' decays, k_{i-x} a_{i-x+1} .. a_i is the lane before's of x - 1
    // times a_i, and q_{j+x} a_{j+1} .. a_{j+x} the next lane's times its a; a
    // lane without one reads zero. Component y of the 16 that P and A spread
    // over the four lanes of a token:
    auto component = [&](const floatx4& p, int y) {
      const float a = (y & 1) ? p[1] : p[0], c = (y & 1) ? p[3] : p[2];
      return __shfl((y & 2) ? c : a, 16 * ((y & 15) / 4) + lr);
    };
    an = zero4;
#pragma unroll
    for (int D = 0; D < ND; ++D) gq[D] = gk[D] = zero4;
#pragma unroll
    for (int ks = 0; ks < NKS; ++ks) {  // eight dims at a time: more do not fit the registers
      float m[8], w[8], aij = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        m[c] = k[8 * ks + c], w[c] = q[8 * ks + c];
        aij = fmaf(w[c], m[c], aij);
      }
#pragma unroll 1
      for (int x = 0;;) {
        aij += __shfl_xor(aij, 16);
        aij += __shfl_xor(aij, 32);
#pragma unroll
        for (int r = 0; r < 4; ++r) an[r] += 4 * lq + r == lr + x ? aij : 0.f;
        if (++x == 16) break;
        float pij = component(pt, lr - x), pji = component(pn, lr + x);  // P[lr][lr-x], P[lr+x][lr]
        pij = x <= lr ? pij : 0.f;
        pji = x < 16 - lr ? pji : 0.f;
        aij = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int e = 8 * ks + c;
          m[c] = row_before16(m[c]) * s[e];
          w[c] = row_after16(w[c] * s[e]);
          gq[e / 4][e % 4] = fmaf(pij, m[c], gq[e / 4][e % 4]);
          gk[e / 4][e % 4] = fmaf(pji, w[c], gk[e / 4][e % 4]);
          aij = fmaf(w[c], k[e], aij);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) an[r] = 4 * lq + r >= lr ? an[r] : 0.f;
  {
    const Split4<NT> as = split4<NT>(an);
#pragma unroll
    for (int E = 0; E < NE; ++E) gv[E] = mm16<NT>(cols4(lv, sO, wave * VB, E), as, zero4);
  }
  __syncthreads();
  load_state(Dws);
  // -- gq from the entering state, S_n go; the rows of S_n of column block
  // `wave` are kept for <S_n, D_n>
  floatx4 acc[ND];
  Split8<NT> keep[NES];
#pragma unroll
  for (int D = 0; D < ND; ++D) acc[D] = zero4;
#pragma unroll
  for (int ks = 0; ks < NES; ++ks) {
    const Split8<NT> o = rows8(lv, sO, wave * VB, ks);
#pragma unroll
    for (int D = 0; D < ND; ++D) acc[D] = mm<NT>(rows8(lx, sX, state_at(D), ks), o, acc[D]);
    keep[ks] = rows8(lx, sX, state_at(wave % ND), ks);
  }
  // -- the first brackets of the pairs of sub-blocks, and prod 2^tot_M over all
  // later sub-blocks M
  if (tid < NB * DK) {
    const int J = tid / DK, d = tid % DK;
    float o = 1.f, e[NB], eq[NB];
#pragma unroll
    for (int M = 1; M < NB; ++M) e[M] = sE[M][d], eq[M] = sEQ[M][d];
#pragma unroll
    for (int M = 1; M < NB; ++M) {
      if (M > J) {
        sF[M * (M - 1) / 2 + J][d] = o * eq[M];
        o *= e[M];
      }
    }
    sA[J][d] = o;
  }
  __syncthreads();  // S_n is read, the factors are written
  put_state();      // D_n
  // -- gq from the earlier sub-blocks, farthest first: what is accumulated is
  // decayed from one sub-block's reference to the next one's
  auto decay = [&](int J, const float(*tab)[DK]) {  // from block J-1's end to tab's point in block J
#pragma unroll
    for (int D = 0; D < ND; ++D) {
      // one factor after the other: their product alone may be too small
      if (J > 0) acc[D] *= *reinterpret_cast<const floatx4*>(&sEK[J - 1][dim(D)]);
      acc[D] *= *reinterpret_cast<const floatx4*>(&tab[J][dim(D)]);
    }
  };
  for (int J = 0; J < wave; ++J) {
    const Split4<NT> ps = split4<NT>(p_keys(J));
    decay(J, sDirect[J] ? sE : sEQ);
#pragma unroll
    for (int D = 0; D < ND; ++D) acc[D] = mm16<NT>(cols4(lk, sK, J * KB, D), ps, acc[D]);
  }
  decay(wave, sEQ);
#pragma unroll
  for (int D = 0; D < ND; ++D)
#pragma unroll
    for (int r = 0; r < 4; ++r) gq[D][r] = fmaf(acc[D][r], cq[4 * D + r], gq[D][r]);
  // (a store's wait would be the next one's: each goes out as it is ready)
  const float self = sSelf[t];
  if (!pad) {
#pragma unroll
    for (int ks = 0; ks < NKS; ++ks) {
      float x[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) x[c] = fmaf(self, k[8 * ks + c], gq[2 * ks + c / 4][c % 4]);
      store8(gqp + row * DK + dim(2 * ks), x);
    }
  }
#pragma unroll
  for (int e = 0; e < NEL; ++e) gq[e / 4][e % 4] = tile::mulw(q[e], gq[e / 4][e % 4]);  // all that is left to use
  // -- gk and gv from the later sub-blocks
#pragma unroll
  for (int ks = 0; ks < NES; ++ks) vs[ks] = v.template terms<NT>(ks);
#pragma unroll
  for (int D = 0; D < ND; ++D) {
    acc[D] = zero4;
    const floatx4 f = *reinterpret_cast<const floatx4*>(&sEK[wave][dim(D)]);
#pragma unroll
    for (int r = 0; r < 4; ++r) ck[4 * D + r] *= f[r];  // 2^(tot - s)
  }
#pragma unroll
  for (int I = 1; I < NB; ++I) {
    if (I <= wave) continue;
    const float* f = &sF[I * (I - 1) / 2 + wave][8 * lq];
    floatx4 a = zero4;
#pragma unroll
    for (int ks = 0; ks < NKS; ++ks) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = tile::mulw(k[8 * ks + i], ck[8 * ks + i] * f[32 * ks + i]);
      a = mm<NT>(rows8(lk, sQ, I * KB, ks), split8<NT>(x), a);
    }
    const Split4<NT> ps = split4<NT>(p_queries(I)), as = split4<NT>(a);
#pragma unroll
    for (int D = 0; D < ND; ++D) {
      const floatx4 o = mm16<NT>(cols4(lk, sQ, I * KB, D), ps, zero4);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[D][r] = fmaf(o[r], f[32 * (D / 2) + 4 * (D % 2) + r], acc[D][r]);
    }
#pragma unroll
    for (int E = 0; E < NE; ++E) gv[E] = mm16<NT>(cols4(lv, sO, I * VB, E), as, gv[E]);
  }
#pragma unroll
  for (int D = 0; D < ND; ++D) {
    const floatx4 f = *reinterpret_cast<const floatx4*>(&sA[wave][dim(D)]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      gk[D][r] = fmaf(acc[D][r], ck[4 * D + r], gk[D][r]);
      ck[4 * D + r] *= f[r];  // 2^(B - b)
    }
  }
  __syncthreads();  // D_n is written
  // -- gk and gv from the state behind the chunk
#pragma unroll
  for (int ks = 0; ks < NKS; ++ks) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = tile::mulw(k[8 * ks + i], ck[8 * ks + i]);
    const Split8<NT> xs = split8<NT>(x);
#pragma unroll
    for (int E = 0; E < NE; ++E) {
      Split8<NT> dt;
#pragma unroll
      for (int i = 0; i < NT; ++i)
        dt.t[i] = join(lx.cols(&sX[i][2 * ks * VB], E), lx.cols(&sX[i][2 * ks * VB + 4 * DV], E));
      gv[E] = mm<NT>(dt, xs, gv[E]);
    }
  }
  auto store_row = [&](InT* p, const floatx4* x, int ks) {
    const float y[8] = {x[2 * ks][0], x[2 * ks][1], x[2 * ks][2], x[2 * ks][3],
                        x[2 * ks + 1][0], x[2 * ks + 1][1], x[2 * ks + 1][2], x[2 * ks + 1][3]};
    store8(p + dim(2 * ks), y);
  };
  if (!pad) {
#pragma unroll
    for (int ks = 0; ks < NES; ++ks) store_row(gvp + row * DV, gv, ks);
  }
#pragma unroll
  for (int D = 0; D < ND; ++D) acc[D] = zero4;
  floatx4 sd = zero4;
#pragma unroll
  for (int ks = 0; ks < NES; ++ks) {
#pragma unroll
    for (int D = 0; D < ND; ++D) acc[D] = mm<NT>(rows8(lx, sX, state_at(D), ks), vs[ks], acc[D]);
    sd = mm<NT>(keep[ks], rows8(lx, sX, state_at(wave % ND), ks), sd);
  }
  // -- 2^B <S_n, D_n>: the diagonals of the blocks of S_n D_n^T
  if (wave < ND) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (4 * lq + r == lr) {
        const int d = dim_row(wave, lr);
        float o = sd[r];
#pragma unroll
        for (int J = 0; J < NB; ++J) o *= sE[J][d];
        sAD[d] = o;
      }
    }
  }
  // -- the decay's gradient: suffix sums of q gq - k gk^pairs, and sums of
  // k gk^state over the tokens before
  float z[NEL], w[NEL];
#pragma unroll
  for (int e = 0; e < NEL; ++e) {  // no branch in between: the scans' steps interleave
    acc[e / 4][e % 4] *= ck[e];
    z[e] = row_suffix16(fmaf(-k[e], gk[e / 4][e % 4], gq[e / 4][e % 4]));
    w[e] = row_scan16(tile::mulw(k[e], acc[e / 4][e % 4]));
    gk[e / 4][e % 4] = fmaf(self, q[e], gk[e / 4][e % 4] + acc[e / 4][e % 4]);
  }
  if (!pad) {
#pragma unroll
    for (int ks = 0; ks < NKS; ++ks) store_row(gkp + row * DK, gk, ks);
  }
  if (lr == 0) {
#pragma unroll
    for (int D = 0; D < ND; ++D) *reinterpret_cast<floatx4*>(&sB[wave][dim(D)]) = row4(z, D);
  }
  if (lr == 15) {
#pragma unroll
    for (int D = 0; D < ND; ++D) *reinterpret_cast<floatx4*>(&sEQ[wave][dim(D)]) = row4(w, D);
  }
  __syncthreads();
#pragma unroll
  for (int D = 0; D < ND; ++D) {
    floatx4 o = *reinterpret_cast<const floatx4*>(&sAD[dim(D)]);
#pragma unroll
    for (int J = 0; J < NB; ++J)  // the sums of the tokens behind, and of those before
      if (J != wave) o += *reinterpret_cast<const floatx4*>(J < wave ? &sEQ[J][dim(D)] : &sB[J][dim(D)]);
#pragma unroll
    for (int r = 0; r < 4; ++r) gk[D][r] = o[r] + z[4 * D + r] + row_before16(w[4 * D + r]);
  }
  if (!pad) {
#pragma unroll
    for (int ks = 0; ks < NKS; ++ks) store_row(ggp + row * DK, gk, ks);
  }
}

// The serial scan replaces the segmented one from this many groups of four
// state elements per launch and direction. Serial and segmented, in us, for
// chains of 64/64 states (1024 groups each):
//              25 chunks      100 chunks     256 chunks
//    6 chains   6.2   4.8     15.7   9.9     34.4  19.8
//   16 chains   8.2   7.4     18.7  20.5     72.2  48.2
//   24 chains   8.6  11.5     24.7  29.8     81.4  76.7
//   64 chains  16.9  23.6     66.2  76.2
// Few chains leave the serial one waiting for its loads; many fill the card
// either way, and the segments' exchange then costs more.
constexpr long kSerialGroups = 24576;

template <int DK, int DV, typename InT>
hipError_t bwd_t(const Problem& p, int b0, int nb, const DirPack& dirs, const BwdArgs& a, char* ws,
                 hipStream_t s) {
  constexpr int NT = sizeof(InT) == 2 ? 2 : 3;
  const BwdLayout w = bwd_layout(p);
  const long rows = (long)b0 * p.T * p.H, bh0 = (long)b0 * p.H, bhn = bh0 * p.N;
  const InT* q = static_cast<const InT*>(a.q) + rows * DK;
  const InT* k = static_cast<const InT*>(a.k) + rows * DK;
  const InT* v = static_cast<const InT*>(a.v) + rows * DV;
  const InT* g = static_cast<const InT*>(a.gk) + rows * DK;
  const InT* go = static_cast<const InT*>(a.go) + rows * DV;
  float* S = reinterpret_cast<float*>(ws + w.off_S) + bhn * DK * DV;
  float* D = reinterpret_cast<float*>(ws + w.off_D) + bhn * DK * DV;
  float* A = reinterpret_cast<float*>(ws + w.off_a) + bhn * DK;
  auto summary = a.gs0 ? bwd_summary_kernel<DK, DV, InT, NT, 3> : bwd_summary_kernel<DK, DV, InT, NT, NT>;
  hipLaunchKernelGGL(summary, dim3(p.N, p.H, 2 * nb), dim3(kThreads), 0, s, k, v, q, go, g, S, D, A,
                     p.T, p.H, p.N, p.gh, p.gw, dirs);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr bool kTerms = NT == 2;
  const float* s0 = a.s0 ? a.s0 + bh0 * DK * DV : nullptr;
  const float* gsf = a.gs_final ? a.gs_final + bh0 * DK * DV : nullptr;
  float* gs0 = a.gs0 ? a.gs0 + bh0 * DK * DV : nullptr;
  const long groups = (long)nb * p.H * (DK * DV / 4);
  if (groups >= kSerialGroups) {
    const dim3 grid((unsigned)((groups + kThreads - 1) / kThreads), 2);
    hipLaunchKernelGGL((bwd_scan_serial_kernel<8, kTerms>), grid, dim3(kThreads), 0, s, S, D, A, s0,
                       gsf, gs0, p.N, DK, DV, groups);
  } else {
    // windows of 64 chunks where one holds the chain (16 chains of 64 chunks
    // 12.2 us, in room for 128 15.3), else of 128 (1 chain of 256 12.1, in
    // windows of 64 14.5; with more chains the two are within 15%)
    const int L = p.N > 16 * 8 ? 8 : (p.N + 15) / 16;
    auto scan = L <= 4 ? bwd_scan_kernel<4, kTerms> : bwd_scan_kernel<8, kTerms>;
    hipLaunchKernelGGL(scan, dim3((unsigned)(groups / 64), 2), dim3(1024), 0, s, S, D, A, s0, gsf, gs0,
                       p.N, DK, DV, L);
  }
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((bwd_grad_kernel<DK, DV, InT, NT>), dim3(p.N, p.H, nb), dim3(kThreads), 0, s,
                     q, k, v, g, go, S, D, static_cast<InT*>(a.gq) + rows * DK,
                     static_cast<InT*>(a.gkey) + rows * DK, static_cast<InT*>(a.gv) + rows * DV,
                     static_cast<InT*>(a.ggk) + rows * DK, p.T, p.H, p.N, p.gh, p.gw, dirs);
  return hipGetLastError();
}

}  // namespace bwd

BwdLayout bwd_layout(const Problem& p) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t units = (size_t)p.B * p.H * p.N;
  BwdLayout w;
  w.off_S = 0;
  w.off_D = up(units * p.dk * p.dv * sizeof(float));
  w.off_a = 2 * w.off_D;
  w.total = w.off_a + up(units * p.dk * sizeof(float));
  return w;
}

hipError_t launch_bwd(const Problem& p, int b0, int nb, const DirPack& dirs, const BwdArgs& a,
                      char* ws, hipStream_t s) {
  const bool f16 = p.dtype == 0;
#define GLA_BWD_CASE(DK, DV)                                                                   \
  if (p.dk == DK && p.dv == DV)                                                                \
    return f16 ? bwd::bwd_t<DK, DV, half_t>(p, b0, nb, dirs, a, ws, s)                         \
               : bwd::bwd_t<DK, DV, float>(p, b0, nb, dirs, a, ws, s);
  GLA_BWD_CASE(32, 32)
  GLA_BWD_CASE(32, 64)
  GLA_BWD_CASE(64, 32)
  GLA_BWD_CASE(64, 64)
#undef GLA_BWD_CASE
  return hipErrorInvalidValue;
}

}  // namespace gla
