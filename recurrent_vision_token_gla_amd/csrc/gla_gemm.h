// Tiles of a matrix product D[m][n] = sum_k A(m, k) B(n, k) on the matrix
// cores, for the linear products and their gradients: either operand is stored
// with the contraction along its rows ([m][k]) or down its columns ([k][m]).
//
// A workgroup takes BM x BN outputs. Each step of the contraction brings 128
// bytes of every row (64 halves, 32 floats) into LDS by buffer loads that write
// LDS directly; a load past the operand's end gives zero. While a step is
// multiplied the next ones are in flight (kStages buffers, one barrier a step).
// Large half products run at 1.0 to 1.05 PFLOP/s (25,600 x 2,048 x 768 78 us; a
// library's 8192^3 1.36): the matrix cores are busy 51 to 65% of the time, the rest
// goes to the barriers, where sixteen waves meet, and to a tile's start and end.
// Half operands go through the 16x16x32 product as they are, float ones as three
// bf16 terms (24 bits), of whose products six are kept (the rest is below 2^-24
// of the largest): 96 cycles of the matrix cores for what the float instruction
// needs 256 for. Splitting them on every read costs about as many cycles of the
// vector units again: 20,000 x 768 x 768 190 -> 143 us, 12,000 x 520 x 1,000 125 ->
// 97, the error against 64 bits halved. Sums are float.
#pragma once

#include <type_traits>

#include "gla_terms.h"
#include "gla_tile.h"

namespace gla {
namespace gemm {

constexpr unsigned kOut = 0x80000000u;  // an offset past every buffer's end
constexpr int kXcds = 8;

template <typename T>
struct Num {
  static constexpr int kUnit = 16 / (int)sizeof(T);   // elements of 16 bytes
  static constexpr int kStep = 128 / (int)sizeof(T);  // elements of the contraction per step
};

__device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

template <int N>
__device__ __forceinline__ void wait_loads() {  // all but the last N loads, and all LDS reads
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ void barrier() {  // no LDS read or load moves across it
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The transposing read of a tile's rows (tile::ld_tr), told apart from the loads
// that write LDS: `restrict` gives it a scope of its own, without which the
// compiler waits for every load in flight before each such read. The waits that
// it needs stand at the barriers.
__device__ __forceinline__ half4 read_turned(tile::lds_fp16x4_t* __restrict__ p) {
  return __builtin_bit_cast(half4, __builtin_amdgcn_ds_read_tr16_b64_v4f16(p));
}

// One operand's R rows (or columns) of a step in LDS, R * 128 bytes, in 16-byte
// units. Stored along the contraction: R rows of 8 units, unit u of row r in
// slot u ^ (r mod 8), so that the 16 rows a fragment reads lie in distinct
// banks. Stored down the columns: kStep rows of R elements, as they are in
// memory, with unit u of row r in slot u ^ g(r), for the transposing read (half)
// or plain reads (float) of 16 neighbouring columns.
template <typename T, int R, bool kCol>
struct Operand {
  static constexpr int kUnit = Num<T>::kUnit, kStep = Num<T>::kStep;
  static constexpr int kPerRow = kCol ? R / kUnit : 8;  // units per stored row
  static constexpr int kBytes = R * 128;

  static __device__ __forceinline__ int twist(int row) {
    if (!kCol) return row & 7;
    if (sizeof(T) == 2) return (2 * (row & 3) | (row & 8)) & (kPerRow - 1);
    return (row >> 1) & 4 & (kPerRow - 1);
  }

  // Eight elements of the contraction for row r0 + lane % 16: 32 ks + 8 q + 0..7
  // with q = lane / 16.
  static __device__ __forceinline__ void read(const char* lds, int r0, int ks, half8& x) {
    const int i = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3;
    if constexpr (!kCol) {
      const int row = r0 + i;
      x = *reinterpret_cast<const half8*>(lds + row * 128 + 16 * ((4 * ks + q) ^ twist(row)));
    } else {
      half4 h[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int row = 32 * ks + 8 * q + 4 * p + (i >> 2), col = r0 + 4 * (i & 3);
        const char* at = lds + row * (2 * R) + 16 * ((col >> 3) ^ twist(row)) + 2 * (col & 7);
        h[p] = read_turned((tile::lds_fp16x4_t*)at);
      }
      x = half8{h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
    }
  }
  static __device__ __forceinline__ void read(const char* lds, int r0, int, terms::Split8<3>& x) {
    const int i = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3;
    float y[8];
    if constexpr (!kCol) {
      const int row = r0 + i;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const floatx4 v = *reinterpret_cast<const floatx4*>(lds + row * 128 + 16 * ((2 * q + h) ^ twist(row)));
#pragma unroll
        for (int c = 0; c < 4; ++c) y[4 * h + c] = v[c];
      }
    } else {
      const int col = r0 + i;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = 8 * q + j;
        y[j] = *reinterpret_cast<const float*>(lds + row * (4 * R) + 16 * ((col >> 2) ^ twist(row)) + 4 * (col & 3));
      }
    }
    x = terms::split8<3>(y);
  }

  // How thread `tid` of NT, of wave w, loads its units of a step.
  template <int NT>
  struct Loader {
    static constexpr int kUnits = R * 8, kLoads = (kUnits + NT - 1) / NT;
    static_assert(kUnits % 64 == 0, "whole waves load");
    // bytes from a whole step's first element, and from the last one's, of which
    // `tail` elements of the contraction exist
    unsigned off[kLoads], last[kLoads];
    // left: rows (columns) of the tile that exist; wrap: rows that lie
    // one behind the other in memory (a tile of two operands has two such runs)
    __device__ __forceinline__ void init(long left, long ld, int tail, int tid, int wrap = R) {
#pragma unroll
      for (int it = 0; it < kLoads; ++it) {
        const int j = tid + NT * it, row = j / kPerRow, unit = (j % kPerRow) ^ twist(row);
        const int at = kCol ? row : row % wrap;
        const bool in = kCol ? unit * kUnit < left : at < left;
        off[it] = in ? (unsigned)((at * ld + unit * kUnit) * (long)sizeof(T)) : kOut;
        last[it] = (kCol ? row : unit * kUnit) < tail ? off[it] : kOut;
      }
    }
    __device__ __forceinline__ void one(const char* base, bool ends, char* lds, int it, int w) const {
      if (NT * it + 64 * w >= kUnits) return;  // the last round may be some waves'
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, 0x7fffffff, 0x00020000),
          (__attribute__((address_space(3))) void*)(lds + 16 * (NT * it + 64 * w)), 16, ends ? last[it] : off[it],
          0, 0, 0);
    }
  };
};

__device__ __forceinline__ floatx4 product(half8 a, half8 b, floatx4 c) { return mfma16x16x32(a, b, c); }
__device__ __forceinline__ floatx4 product(const terms::Split8<3>& a, const terms::Split8<3>& b, floatx4 c) {
  return terms::mm<3>(a, b, c);
}
__device__ __forceinline__ floatx4 product(floatx4 a, floatx4 b, floatx4 c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}

// A neighbouring pair of 16-column blocks, of which each lane holds four
// columns 4q.. of both: afterwards x holds the eight columns
// 16 (q mod 2) + 8 (q / 2) .. of the pair (rows of 16 lanes swapped).
__device__ __forceinline__ void pair8(floatx4 lo, floatx4 hi, float (&x)[8]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const auto y = __builtin_amdgcn_permlane16_swap(__float_as_uint(lo[r]), __float_as_uint(hi[r]), false, false);
    x[r] = __uint_as_float(y[0]);
    x[4 + r] = __uint_as_float(y[1]);
  }
}

// Values of the activations and of their derivatives (codes of gla.h), in float, on
// the reciprocal and exp2 units (the rounding of exp2's argument grows with it): the
// values within (8 + |z| + z^2) 2^-22 of themselves, the derivatives within as much
// of the magnitudes of the two terms that they are sums of (s and z s (1 - s), Phi(z)
// and z phi(z); they cancel where silu' and gelu' cross zero). What a sigmoid or a
// bell below 2^-126 makes counts as zero.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + tile::fexp2(-z * kLog2e));
}
// exp(-z^2 / 2)
__device__ __forceinline__ float bell(float z) { return tile::fexp2(z * z * (-0.5f * kLog2e)); }
// The normal distribution's integral up to z, erfc(-z / sqrt 2) / 2: for x >= 0
// erfc(x) exp(x^2) (1 + x / 2) is smooth in t = 1 / (1 + x / 2), and this
// polynomial in t, a least-squares fit weighted to even out its relative error,
// is within 5.5e-8 of it on 0.14 <= t <= 1 (beyond, x > 12, exp(-x^2) is zero in
// float). The lower tail keeps its digits.
__device__ __forceinline__ float normal_below(float z) {
  const float x = fabsf(z) * 0.70710678118654752f, t = __builtin_amdgcn_rcpf(fmaf(0.5f, x, 1.f));
  float p = -0.059374962002038956f;
  p = fmaf(p, t, 0.2860681116580963f);
  p = fmaf(p, t, -0.49029138684272766f);
  p = fmaf(p, t, 0.2816026210784912f);
  p = fmaf(p, t, -0.029059266671538353f);
  p = fmaf(p, t, 0.20371514558792114f);
  p = fmaf(p, t, 0.24284444749355316f);
  p = fmaf(p, t, 0.2824108302593231f);
  p = fmaf(p, t, 0.2820844054222107f);
  const float tail = 0.5f * p * t * bell(z);
  return z < 0.f ? tail : 1.f - tail;
}
// log(1 + e) for 0 <= e <= 1, as 2 artanh(s) with s = e / (2 + e) <= 1/3: the
// series' first terms left out are below 2^-25 of it
__device__ __forceinline__ float log_1p(float e) {
  const float s = e * __builtin_amdgcn_rcpf(2.f + e), y = s * s;
  float p = 1.f / 15.f;
  p = fmaf(p, y, 1.f / 13.f);
  p = fmaf(p, y, 1.f / 11.f);
  p = fmaf(p, y, 1.f / 9.f);
  p = fmaf(p, y, 1.f / 7.f);
  p = fmaf(p, y, 1.f / 5.f);
  p = fmaf(p, y, 1.f / 3.f);
  p = fmaf(p, y, 1.f);
  return 2.f * s * p;
}
template <int W>
__device__ __forceinline__ void activate(float (&z)[W], int act) {
  if (act == 1) {  // silu
#pragma unroll
    for (int c = 0; c < W; ++c) z[c] *= sigmoid(z[c]);
  } else if (act == 2) {  // gelu
#pragma unroll
    for (int c = 0; c < W; ++c) z[c] *= normal_below(z[c]);
  } else if (act == 3) {  // log sigmoid
#pragma unroll
    for (int c = 0; c < W; ++c) z[c] = fminf(z[c], 0.f) - log_1p(tile::fexp2(-fabsf(z[c]) * kLog2e));
  }
}
// At +-Inf, as a kept sum beyond half's range is stored, the limits 1 and 0.
__device__ __forceinline__ float slope(float z, int act) {
  z = fabsf(z) == __builtin_inff() ? copysignf(65504.f, z) : z;
  if (act == 1) {
    const float s = sigmoid(z);
    return s * fmaf(z, 1.f - s, 1.f);
  }
  if (act == 2) return fmaf(z * 0.39894228040143268f, bell(z), normal_below(z));
  if (act == 3) return sigmoid(-z);
  return 1.f;
}

struct Args {
  const void *a[2], *b[2];
  long lda, ldb;  // elements between stored rows
  long M, N, K;   // outputs of one part of the rows, and contraction of one part
  int parts;      // parts of the contraction, one behind the other (a[p], b[p])
  int mparts;     // parts of the rows (a[p], out[p])
  int tiles_m, tiles_n;  // of one part of the rows
  int splits;            // of the contraction
  long steps, each;      // steps of the contraction, and of one split
  void* out[2];
  float* partial;  // [split][mparts * M][N] float instead of out, where there are splits
  void* pre;       // x W^T + bias, or nullptr
  const float* bias;
  const void* residual;
  float alpha;
  int act;
  void *gate_out, *up_out;  // the gated product's two sides, or nullptr
};

enum { kLinear, kGated };

template <typename T>
__device__ __forceinline__ void load_to(const T* p, float (&x)[8]) { load8(p, x); }
template <typename T>
__device__ __forceinline__ void store_from(T* p, const float (&x)[8]) { store8(p, x); }
template <typename T>
__device__ __forceinline__ void load_to(const T* p, float (&x)[4]) {
  typedef T vec __attribute__((ext_vector_type(4)));
  const vec v = *reinterpret_cast<const vec*>(p);
#pragma unroll
  for (int c = 0; c < 4; ++c) x[c] = (float)v[c];
}
template <typename T>
__device__ __forceinline__ void store_from(T* p, const float (&x)[4]) {
  typedef T vec __attribute__((ext_vector_type(4)));
  *reinterpret_cast<vec*>(p) = vec{(T)x[0], (T)x[1], (T)x[2], (T)x[3]};
}

// W neighbouring outputs from their sums: y = alpha act(sum + bias) + residual.
template <typename T, int W>
__device__ __forceinline__ void finish(const Args& g, int part, long m, long n, float (&x)[W]) {
  const long o = m * g.N + n;
  if (g.bias) {
    float b[W];
    load_to(g.bias + n, b);
#pragma unroll
    for (int c = 0; c < W; ++c) x[c] += b[c];
  }
  if (g.pre) store_from(static_cast<T*>(g.pre) + o, x);
  activate(x, g.act);
#pragma unroll
  for (int c = 0; c < W; ++c) x[c] *= g.alpha;
  if (g.residual) {
    float r[W];
    load_to(static_cast<const T*>(g.residual) + o, r);
#pragma unroll
    for (int c = 0; c < W; ++c) x[c] += r[c];
  }
  store_from(static_cast<T*>(g.out[part]) + o, x);
}

// and of the gated product: h = act(x) u.
template <typename T, int W>
__device__ __forceinline__ void finish_gated(const Args& g, long m, long n, float (&x)[W], const float (&u)[W]) {
  const long o = m * g.N + n;
  if (g.gate_out) store_from(static_cast<T*>(g.gate_out) + o, x);
  if (g.up_out) store_from(static_cast<T*>(g.up_out) + o, u);
  activate(x, g.act);
#pragma unroll
  for (int c = 0; c < W; ++c) x[c] *= u[c];
  store_from(static_cast<T*>(g.out[0]) + o, x);
}

// The tile a workgroup takes: the numbers of one XCD's workgroups are brought
// together, so that they share rows of both operands in its L2, in groups of
// eight row tiles by all column tiles.
struct Place {
  int split, part;
  long m0, n0;  // of the part's rows, and of the columns
  __device__ __forceinline__ Place(const Args& g, int id, int count, int BM, int BN) {
    const int x = id % kXcds, q = count / kXcds, r = count % kXcds;
    const int lin = x * q + min(x, r) + id / kXcds;
    const int tm = g.tiles_m * g.mparts, tiles = tm * g.tiles_n;
    split = lin / tiles;
    const int t = lin % tiles, band = 8 * g.tiles_n, f = t / band * 8, in = min(8, tm - f);
    const int m = f + t % band % in;
    part = m / g.tiles_m;
    m0 = (long)(m % g.tiles_m) * BM;
    n0 = (long)(t % band / in) * BN;
  }
};

// Tiles that the products are cut into: rows and columns, waves over both, steps
// that LDS holds (one is multiplied while the others are on their way),
// workgroups that a CU holds at once, and groups of such waves in a workgroup,
// which take a part of the steps each and add their sums up at the end (few
// tiles, a long contraction).
enum Tile { k320x256, k256x256, k192x256, k128x256, k128x128, k128x128by2, k64x64, k64x64by2, k64x64by4,
            k32x32by4, k32x32by8, kTiles };
struct TileShape {
  int m, n, wm, wn, stages, per_cu, groups;
};
constexpr TileShape kTileShapes[kTiles] = {
    {320, 256, 4, 4, 2, 1, 1}, {256, 256, 4, 4, 2, 1, 1}, {192, 256, 4, 4, 2, 1, 1}, {128, 256, 4, 4, 2, 1, 1},
    {128, 128, 2, 2, 2, 2, 1}, {128, 128, 2, 2, 2, 1, 2}, {64, 64, 2, 2, 4, 2, 1},   {64, 64, 2, 2, 4, 1, 2},   {64, 64, 2, 2, 2, 1, 4},
    {32, 32, 1, 1, 2, 2, 4},   {32, 32, 1, 1, 2, 1, 8}};
constexpr TileShape tile_shape(int tile, bool is_float, bool gated) {
  TileShape s = kTileShapes[tile];
  // the matrix instructions bound float: more workgroups instead of more steps in flight
  if (is_float && tile == k64x64) s.stages = 2, s.per_cu = 4;
  // two column blocks of each weight in a wave, so that a lane stores 16 bytes of halves
  if (gated && !is_float && s.m == 64) s.wm = 4, s.wn = 1;
  return s;
}
// Float tiles gain nothing above 128 x 128; the weights' gradients take no
// others of 256 columns than 256 x 256 (320 rows need more registers than there
// are).
template <typename T, bool kColA>
constexpr bool has_tile(int t) {
  if (t < k128x128) return sizeof(T) == 2 && (!kColA || t == k256x256);
  return true;
}

// Workgroup `id` of `count` of one product, with kTileBytes of LDS.
template <typename T, int kTile, bool kGatedTile>
constexpr int kTileBytes = tile_shape(kTile, sizeof(T) == 4, kGatedTile).groups *
                           tile_shape(kTile, sizeof(T) == 4, kGatedTile).stages * 128 *
                           (tile_shape(kTile, sizeof(T) == 4, kGatedTile).m +
                            tile_shape(kTile, sizeof(T) == 4, kGatedTile).n);
template <typename T, int kTile, bool kGatedTile>
constexpr int kTileThreads = 64 * tile_shape(kTile, sizeof(T) == 4, kGatedTile).groups *
                             tile_shape(kTile, sizeof(T) == 4, kGatedTile).wm *
                             tile_shape(kTile, sizeof(T) == 4, kGatedTile).wn;

template <typename T, int kTile, bool kColA, bool kColB, int kEpi>
__device__ __forceinline__ void gemm_tile(const Args& g, int id, int count, char* shared) {
  constexpr TileShape S = tile_shape(kTile, sizeof(T) == 4, kEpi == kGated);
  constexpr int BM = S.m, BN = S.n, WM = S.wm, WN = S.wn, kStages = S.stages, kGroups = S.groups;
  constexpr int NT = 64 * WM * WN, MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr bool kDual = kEpi == kGated;  // columns: BN/2 of b[0], then BN/2 of b[1]
  constexpr int BNC = kDual ? BN / 2 : BN;
  using OA = Operand<T, BM, kColA>;
  using OB = Operand<T, BN, kColB>;
  using LA = typename OA::template Loader<NT>;
  using LB = typename OB::template Loader<NT>;
  using Frag = typename std::conditional<sizeof(T) == 2, half8, terms::Split8<3>>::type;
  constexpr int kStep = Num<T>::kStep, kStageBytes = OA::kBytes + OB::kBytes;
  static_assert(!kDual || !kColB, "both sides of a gated product lie along the contraction");
  constexpr int kInFlight = LA::kLoads + LB::kLoads;
  static_assert(kStages == 2 || (LA::kUnits % NT == 0 && LB::kUnits % NT == 0), "as many loads in every wave");
  const int group = wave() / (WM * WN), w = wave() % (WM * WN), wm = w / WN, wn = w % WN;
  const int tid = threadIdx.x % NT;
  char* const smem = shared + group * kStages * kStageBytes;
  const Place at(g, id, count, BM, BNC);
  const long m0 = at.m0, n0 = at.n0;
  // this group's steps, and the step that its next loads are of: number k of
  // its part of the contraction, at pa and pb
  const int from = at.split * (int)g.each, to = min(from + (int)g.each, (int)g.steps);
  const int rounds = (to - from + kGroups - 1) / kGroups, s0 = from + group * rounds;
  const int todo = max(min(rounds, to - s0), 0), of_part = (int)g.steps / g.parts;
  constexpr bool kParts = kEpi == kLinear && !kColA;  // the contraction may have two
  const bool second = kParts && s0 >= of_part;
  int k = second ? s0 - of_part : s0;
  const long da = (kColA ? kStep * g.lda : kStep) * (long)sizeof(T), db = (kColB ? kStep * g.ldb : kStep) * (long)sizeof(T);
  auto start = [](const void* p, long first, bool col, long ld) {
    return static_cast<const char*>(p) + first * (col ? 1 : ld) * (long)sizeof(T);
  };
  const char* pa = start(g.a[second ? 1 : at.part], m0, kColA, g.lda) + k * da;
  const char* pb = start(g.b[second], n0, kColB, g.ldb) + k * db;
  const char* pu = kDual ? start(g.b[1], n0, false, g.ldb) + k * db : nullptr;
  const int tail = (int)(g.K - (of_part - 1) * (long)kStep);
  LA la;
  LB lb;
  la.init(g.M - m0, g.lda, tail, tid);
  lb.init(g.N - n0, g.ldb, tail, tid, BNC);
  auto load = [&](int stage) {
    const bool ends = k == of_part - 1;
    char* lds = smem + stage * kStageBytes;
#pragma unroll
    for (int it = 0; it < LA::kLoads; ++it) la.one(pa, ends, lds, it, w);
#pragma unroll
    for (int it = 0; it < LB::kLoads; ++it)
      lb.one(kDual && it >= LB::kLoads / 2 ? pu : pb, ends, lds + OA::kBytes, it, w);
    pa += da, pb += db, pu += db, ++k;
    if (kParts && k == of_part && g.parts > 1) {
      k = 0;
      pa = start(g.a[1], m0, kColA, g.lda);
      pb = start(g.b[1], n0, kColB, g.ldb);
    }
  };
  floatx4 acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = floatx4{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int s = 0; s < kStages - 1; ++s)
    if (s < todo) load(s);
  int stage = 0;
  for (int r = 0; r < rounds; ++r) {
    // this step's loads are done in every wave, and the buffer that the loads
    // below refill has been read by all of them
    if (kStages > 2 && r + kStages - 2 < todo) wait_loads<kInFlight * (kStages - 2)>();
    else wait_loads<0>();
    barrier();
    if (r + kStages - 1 < todo) load(stage == 0 ? kStages - 1 : stage - 1);
    if (kGroups > 1 && r >= todo) continue;  // the last group may have fewer steps
    const char* sa = smem + stage * kStageBytes;
    const char* sb = sa + OA::kBytes;
#pragma unroll
    for (int ks = 0; ks < kStep / 32; ++ks) {
      Frag fa[MI], fb[NI];
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) OA::read(sa, (wm * MI + mi) * 16, ks, fa[mi]);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        // gated: a wave's first NI/2 blocks are of b[0], the others, of the same columns, of b[1]
        const int blk = kDual ? (ni < NI / 2 ? wn * (NI / 2) + ni : BNC / 16 + wn * (NI / 2) + ni - NI / 2)
                              : wn * NI + ni;
        OB::read(sb, blk * 16, ks, fb[ni]);
      }
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = product(fb[ni], fa[mi], acc[mi][ni]);
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }

  if constexpr (kGroups > 1) {
    static_assert((kGroups - 1) * BM * BN * 4 <= kGroups * kStages * kStageBytes, "sums fit");
    floatx4* const sums = reinterpret_cast<floatx4*>(shared);
    __syncthreads();  // the buffers are read
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
        if (group > 0) sums[((group - 1) * MI * NI + mi * NI + ni) * NT + tid] = acc[mi][ni];
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int o = 0; o < kGroups - 1; ++o)
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) acc[mi][ni] += sums[(o * MI * NI + mi * NI + ni) * NT + tid];
  }

  // each lane: row lane % 16 of the row blocks, eight columns of each pair of column blocks;
  // gated, four of each block where they are 16 bytes or there is one block of each weight
  constexpr bool kFour = sizeof(T) == 4 || NI / 2 == 1;
  const int i = threadIdx.x & 15, q = (threadIdx.x >> 4) & 3, c8 = 16 * (q & 1) + 8 * (q >> 1);
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const long m = m0 + (wm * MI + mi) * 16 + i;
    if constexpr (kDual) {
#pragma unroll
      for (int p = 0; p < (kFour ? NI / 2 : 0); ++p) {
        float x[4], u[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = acc[mi][p][c], u[c] = acc[mi][NI / 2 + p][c];
        const long n = n0 + (wn * (NI / 2) + p) * 16 + 4 * q;
        if (m < g.M && n < g.N) finish_gated<T>(g, m, n, x, u);
      }
#pragma unroll
      for (int p = 0; p < (kFour ? 0 : NI / 4); ++p) {
        float x[8], u[8];
        pair8(acc[mi][2 * p], acc[mi][2 * p + 1], x);
        pair8(acc[mi][NI / 2 + 2 * p], acc[mi][NI / 2 + 2 * p + 1], u);
        const long n = n0 + wn * (NI / 2) * 16 + 32 * p + c8;
        if (m < g.M && n < g.N) finish_gated<T>(g, m, n, x, u);
      }
    } else {
#pragma unroll
      for (int p = 0; p < NI / 2; ++p) {
        float x[8];
        pair8(acc[mi][2 * p], acc[mi][2 * p + 1], x);
        const long n = n0 + wn * NI * 16 + 32 * p + c8;
        if (m < g.M && n < g.N) {
          if (kColA && g.splits > 1)
            store8(g.partial + ((long)at.split * g.mparts + at.part) * g.M * g.N + m * g.N + n, x);
          else
            finish<T>(g, at.part, m, n, x);
        }
      }
    }
  }
}

template <typename T, int kTile, bool kColA, bool kColB, int kEpi>
__global__ __launch_bounds__((kTileThreads<T, kTile, kEpi == kGated>)) void gemm_kernel(const Args g) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host's pass does not take the loads' builtin in a template
  __shared__ __attribute__((aligned(1024))) char shared[kTileBytes<T, kTile, kEpi == kGated>];
  gemm_tile<T, kTile, kColA, kColB, kEpi>(g, blockIdx.x, gridDim.x, shared);
#endif
}

// What a launch costs, in us. A step (128 bytes of every row) costs a CU about
// 0.28, the meeting of the waves and the latency of LDS, and 1.3 for each 256 x
// 256 half outputs; one wave alone on its SIMD (128 x 128, one workgroup on a CU)
// takes 1.6 times that. Float ones cost 7, as every wave splits its values into
// terms, and 5.5 with 128 x 128, which split each fewer times (4.6 by two groups,
// of which one splits while the other multiplies). Four or more groups that read
// both half operands turned need 0.4 more a step. A tile starts and ends in 2 and 5
// for as many outputs, and groups of waves add their sums up. Within 20% of what
// was measured over 100 to 25,600 rows of 100 to 4,096 values. Half, 25,600 x 2,048
// x 768 with 320, 256, 192 and 128 rows of 256 columns: 77, 107, 90 and 106 (0.94,
// 1.17, 1.57 and 2.34 rounds of the CUs); 4,000 x 1,024 x 1,024 with 128 x 128 16.1,
// by two groups 14.5, 64 x 64 17.3; 1,600 x 768 x 768 13.0, 11.7, 8.2; 130 x 768 x
// 768 with 128 x 128 11.8, 64 x 64 6.4, 32 x 32 by four groups 5.0. Float, 4,000 x
// 1,024 x 1,024 with 128 x 128 56.5, by two groups 50.5, 64 x 64 64.6; 1,600 x 768 x
// 768 43.0, 36.5, 29.3, with 32 x 32 by four groups 24.7. Weights' gradient, half,
// 768 x 768 over 1,600 with 64 x 64 10.7, by four groups 11.0, 32 x 32 18.2.
constexpr int kCus = 256;

inline long tile_count(const TileShape& s, long M, long N) { return ((M + s.m - 1) / s.m) * ((N + s.n - 1) / s.n); }

// One round of tiles, `on` workgroups on every CU; `turned`: both operands lie
// down the columns.
template <typename T>
float round_cost(const TileShape& s, long steps, long on, bool turned) {
  const float area = s.m * s.n / 65536.f;
  const bool square = s.m == 128 && s.n == 128, alone = square && s.groups == 1 && on == 1;
  const float per_step = sizeof(T) == 2 ? (alone ? 2.1f : 1.3f) : !square ? 7.f : s.groups == 1 ? 5.5f : 4.6f;
  const float meet = sizeof(T) == 2 && turned && s.groups >= 4 ? 0.68f : 0.28f;
  return (steps + s.groups - 1) / s.groups * (meet + per_step * area * on * s.groups) + 2.f + 5.f * area * on +
         (s.groups - 1) * (0.25f + 8.f * area);
}

// M x N outputs, `others` such products at once, `steps` steps each: the best
// tile, and what it costs in *cost.
template <typename T, bool kColA>
int best_tile(long M, long N, long others, long steps, float* cost = nullptr) {
  int best = -1;
  float least = 0.f;
  for (int t = 0; t < kTiles; ++t) {
    if (!has_tile<T, kColA>(t)) continue;
    const TileShape s = tile_shape(t, sizeof(T) == 4, false);
    const long count = tile_count(s, M, N) * others, slots = (long)kCus * s.per_cu;
    const long whole = count / slots, rest = count % slots;
    const float c = whole * round_cost<T>(s, steps, s.per_cu, kColA) +
                    (rest ? round_cost<T>(s, steps, (rest + kCus - 1) / kCus, kColA) : 0.f);
    if (best < 0 || c < least) least = c, best = t;
  }
  if (cost) *cost = least;
  return best;
}

// The tile of a forward product, or kTiles: skinny_kernel (gla_linear.hip), which takes
// up to 16 rows and 16 columns a workgroup (gated: eight of either weight). It runs for up
// to 16 rows where there are no more workgroups than CUs, or twice as many for up
// to four rows: more of them wait for their weights one after the other, where the
// tiles, of 32 to 256 columns, read ahead. us, it against the tiles, half: linear of one
// row x 768 x 4,096 4.2 and 5.2, 16 rows 4.7 and 5.3; x 8,192 5.6 and 6.5, 4 rows 6.1 and
// 6.5, 16 rows 7.3 and 6.6; x 16,384 8.3 and 7.7, 16 rows 11.7 and 7.8; x 65,536 23 and 24,
// 16 rows 37 and 24; one row x 2,048 x 16,384 17.0 and 15.0; 24 rows x 768 x 768 (as two
// such kernels' work) 4.4 and 4.3, 64 rows 6.8 and 4.3. Float, one row x 2,048 x 8,192 17.4
// and 17.6, 16 rows 22.8 and 18.6, 16 rows x 768 x 65,536 75 and 49. Gated, one row x 2,048
// x 4,096 9.9 and 12.2, 16 rows 12.7 and 12.3, x 8,192 15.8 and 14.8, 16 rows 22 and 15; 16
// rows x 768 x 2,048 5.0 and 5.2, 32 rows 5.7 and 5.2; float one row x 768 x 4,096 9.7 and
// 10.2, 16 rows 12.2 and 10.2.
constexpr int kFewRows = 16;
template <bool kDual>
constexpr int kFewCols = kDual ? 8 : 16;
template <typename T, int kEpi>
int forward_tile(long M, long N, long steps) {
  constexpr bool kDual = kEpi == kGated;
  if (M <= kFewRows && N <= kFewCols<kDual> * kCus * (M <= 4 ? 2 : 1)) return kTiles;
  return best_tile<T, false>(M, kDual ? 2 * N : N, 1, steps);
}

// Rows of a forward product per launch: at most 2^22, and 2^31 outputs. A tile has
// at most a thread for each of its outputs (the gated one of 32 columns, 16 of each
// weight, by eight groups), and a launch may have less than 2^32 threads.
inline long rows_at_once(long N) {
  return (1L << 31) / (N > 512 ? N : 512);
}

// One product on tiles of the given kind.
template <typename T, int kTile, bool kColA, bool kColB, int kEpi>
hipError_t launch_tiles(Args g, hipStream_t s) {
  constexpr TileShape S = tile_shape(kTile, sizeof(T) == 4, kEpi == kGated);
  g.tiles_m = (int)((g.M + S.m - 1) / S.m);
  g.tiles_n = (int)((g.N + (kEpi == kGated ? S.n / 2 : S.n) - 1) / (kEpi == kGated ? S.n / 2 : S.n));
  hipLaunchKernelGGL((gemm_kernel<T, kTile, kColA, kColB, kEpi>),
                     dim3((unsigned)(g.tiles_m * g.mparts * g.tiles_n * g.splits)),
                     dim3(kTileThreads<T, kTile, kEpi == kGated>), 0, s, g);
  return hipGetLastError();
}
template <typename T, bool kColA, bool kColB, int kEpi, int kTile = 0>
hipError_t launch_product(const Args& g, int tile, hipStream_t s) {
  if constexpr (kTile == kTiles) {
    return hipErrorInvalidValue;
  } else {
    if constexpr (has_tile<T, kColA>(kTile))
      if (tile == kTile) return launch_tiles<T, kTile, kColA, kColB, kEpi>(g, s);
    return launch_product<T, kColA, kColB, kEpi, kTile + 1>(g, tile, s);
  }
}

}  // namespace gemm
}  // namespace gla
