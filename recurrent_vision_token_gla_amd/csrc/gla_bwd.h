// Host-side launch interface of the recurrence's backward pass (gla_bwd.hip).
// Arguments are already validated by the C-ABI layer.
#pragma once

#include "gla_launch.h"

namespace gla {

constexpr int kBwdChunk = 64;  // tokens per chunk of the backward pass

// Byte offsets inside the workspace of gla_bwd, per (batch, head, chunk): the
// chunk's forward summary U_n, replaced by the state S_n entering the chunk;
// its reverse summary R_n, replaced by D_n, the gradient of the state behind
// the chunk (summaries float [dk][dv]; states too, or for half inputs their two
// bf16 terms in the same 32 bits); and the chunk's decay a_n (float [dk]).
struct BwdLayout {
  size_t off_S, off_D, off_a, total;
};
BwdLayout bwd_layout(const Problem& p);

struct BwdArgs {
  const void *q, *k, *v, *gk, *go;
  void *gq, *gkey, *gv, *ggk;
  const float *s0, *gs_final;
  float* gs0;
};
// The whole backward pass for batch elements [b0, b0 + nb) (nb <=
// kMaxBatchPerLaunch); pointers are the full-problem bases.
hipError_t launch_bwd(const Problem& p, int b0, int nb, const DirPack& dirs, const BwdArgs& a,
                      char* ws, hipStream_t s);

}  // namespace gla
