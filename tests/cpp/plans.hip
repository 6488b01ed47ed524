// What the products run on: for every line "call dtype rows K N" of the input (calls
// linear, gated, linear_bwd, gated_bwd; dtypes f16, f32) a line of kernels, each
// "call dtype part tile", with the tile's rows x columns and groups of waves, and
// whether the weights' rows are split.
#include <stdio.h>
#include <string.h>

#include "gla_gemm.h"
#include "gla_linear.h"

using namespace gla::gemm;

static void kernel(const char* call, const char* dtype, const char* part, int tile) {
  if (tile == kTiles) printf("%s %s %s few\n", call, dtype, part);
  else printf("%s %s %s %dx%dby%d\n", call, dtype, part, kTileShapes[tile].m, kTileShapes[tile].n, kTileShapes[tile].groups);
}

template <typename T>
void plan(const char* call, const char* dtype, long rows, int K, int N) {
  const long steps = (K * (long)sizeof(T) + 127) / 128;
  const int code = sizeof(T) == 2 ? 0 : 1;
  if (!strcmp(call, "linear")) return kernel(call, dtype, "y", forward_tile<T, kLinear>(rows, N, steps));
  if (!strcmp(call, "gated")) return kernel(call, dtype, "y", forward_tile<T, kGated>(rows, N, steps));
  const gla::LinearBwdLayout l =
      !strcmp(call, "linear_bwd") ? gla::linear_bwd_layout(rows, K, N, 1, code) : gla::gated_bwd_layout(rows, K, N, code);
  if (l.pair) {
    kernel(call, dtype, l.splits > 1 ? "pair,split" : "pair", l.tile_x);
  } else {
    kernel(call, dtype, "gx", l.tile_x);
    kernel(call, dtype, l.splits > 1 ? "gw,split" : "gw", l.tile_w);
  }
}

int main() {
  char call[16], dtype[8];
  long rows;
  int K, N;
  while (scanf("%15s %7s %ld %d %d", call, dtype, &rows, &K, &N) == 5) {
    if (!strcmp(dtype, "f16")) plan<gla::half_t>(call, dtype, rows, K, N);
    else plan<float>(call, dtype, rows, K, N);
    printf("\n");
  }
  return 0;
}
