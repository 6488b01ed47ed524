// Argument checks and the error detail shared by the C-ABI entry points
// (gla_api.hip, gla_train_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gla.h"
#include "gla_launch.h"

namespace gla {
namespace api {

inline thread_local char g_detail[256] = "";

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

inline int fail_hip(hipError_t e, const char* where) {
  snprintf(g_detail, sizeof(g_detail), "%s: %s", where, hipGetErrorString(e));
  return GLA_E_HIP;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Shape check shared by every entry point. Returns GLA_OK and fills `p`, or
// an error status. `empty` is set when there is nothing to compute.
inline int make_problem(int B, int H, int gh, int gw, int dk, int dv, int chunk, int dtype,
                        gla::Problem* p, bool* empty) {
  if (B < 0 || H < 0 || gh < 0 || gw < 0) return GLA_E_ARG;
  if (dtype != GLA_F16 && dtype != GLA_F32) return GLA_E_ARG;
  if ((dk != 32 && dk != 64) || (dv != 32 && dv != 64)) return GLA_E_UNSUPPORTED;
  if (chunk != 16 && chunk != 32 && chunk != 64) return GLA_E_UNSUPPORTED;
  const long long T = (long long)gh * gw;
  // element offsets are formed in 64-bit; T and the grid counts must fit int
  if (T > 0x7fffffffLL || (long long)B * T * H > (1LL << 40)) return GLA_E_UNSUPPORTED;
  *empty = (B == 0 || H == 0 || T == 0);
  p->B = B; p->H = H; p->gh = gh; p->gw = gw; p->T = (int)T;
  p->dk = dk; p->dv = dv; p->chunk = chunk; p->dtype = dtype;
  p->N = (int)((T + chunk - 1) / chunk);
  if (!*empty && (p->N > 0x7fffffff / 1 || H > 65535)) return GLA_E_UNSUPPORTED;
  return GLA_OK;
}

inline int check_dirs(const int32_t* dir, int B) {
  if (!dir) return GLA_E_ARG;
  for (int b = 0; b < B; ++b)
    if (dir[b] < GLA_L2R || dir[b] > GLA_B2T) return GLA_E_ARG;
  return GLA_OK;
}

inline gla::DirPack pack_dirs(const int32_t* dir, int b0, int nb) {
  gla::DirPack d;
  memset(&d, 0, sizeof(d));
  for (int i = 0; i < nb; ++i) d.w[i >> 4] |= (uint32_t)(dir[b0 + i] & 3) << (2 * (i & 15));
  return d;
}

inline int check_tensor(const void* t) { return (t && aligned(t, 16)) ? GLA_OK : GLA_E_ARG; }

// Some control word of a workspace prepared for the single pass lies in
// [p, p + n).
bool holds_control_words(const void* p, size_t n);

#define GLA_TRY(...)               \
  do {                             \
    const int rc_ = (__VA_ARGS__); \
    if (rc_ != GLA_OK) return rc_; \
  } while (0)

}  // namespace api
}  // namespace gla
