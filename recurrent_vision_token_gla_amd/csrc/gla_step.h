// Host-side launch interface of the single-token recurrence (gla_step.hip).
#pragma once

#include "gla_launch.h"

namespace gla {

struct StepArgs {
  int B, H, dk, dv, dtype;
  const void *q, *k, *v, *gk;
  void* out;
  float* state;
  long n_slots;
  const int32_t* slots;  // device memory, or nullptr: row b uses slot b
  Epilogue epi;          // the output gate, or no gate
};
hipError_t launch_step(const StepArgs& a, hipStream_t s);

}  // namespace gla
