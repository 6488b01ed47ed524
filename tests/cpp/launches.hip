// How forward products are launched (csrc/gla_gemm.h), over every power of two of
// rows, values in and values out whose tensors fit 300 GB: prints the launches of
// 2^32 threads or more and returns their number.
#include <stdio.h>

#include "gla_gemm.h"

using namespace gla::gemm;

static int failed = 0;

template <typename T, int kEpi>
void look(long rows, long K, long N) {
  constexpr bool kDual = kEpi == kGated;
  const long es = sizeof(T), steps = (K * es + 127) / 128;
  if ((double)es * ((double)rows * (K + N) + (kDual ? 2 : 1) * (double)N * K) > 300e9) return;
  const long most = rows_at_once(N), M = rows < most ? rows : most;
  const int tile = forward_tile<T, kEpi>(M, N, steps);
  if (tile == kTiles) return;  // up to 16 rows: 512 threads for eight or 16 of up to 65,536 columns
  const TileShape s = tile_shape(tile, es == 4, kDual);
  const long columns = kDual ? s.n / 2 : s.n, tiles = ((M + s.m - 1) / s.m) * ((N + columns - 1) / columns);
  const long threads = tiles * 64 * s.groups * s.wm * s.wn;
  if (M < 1 || M > 1L << 22 || threads >= 1L << 32)
    ++failed, printf("%ld x %ld x %ld of %ld bytes%s: %ld rows, %ld threads\n", rows, K, N, es, kDual ? " gated" : "", M, threads);
}

int main() {
  for (long rows = 1; rows <= 1L << 31; rows *= 2)
    for (long K = 8; K <= 65536; K *= 2)
      for (long N = 8; N <= 65536; N *= 2) {
        look<gla::half_t, kLinear>(rows, K, N), look<gla::half_t, kGated>(rows, K, N);
        look<float, kLinear>(rows, K, N), look<float, kGated>(rows, K, N);
      }
  return failed;
}
