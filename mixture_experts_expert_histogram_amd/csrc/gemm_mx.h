// Grouped products on microscaled 4-bit weights (gemm_mx.hip).
#pragma once
#include "gemm_common.h"

namespace moe {

// Expert weights in codes and scales.  Strides are bytes of codes: gate (up)
// row j of expert e starts gu_es e + gu_rs j after gu_g (gu_u); the scales
// follow the same strides over 16.
struct MxWeights {
  const void *gu_g, *gu_u, *gus_g, *gus_u, *Wd, *sd;
  long gu_es, gu_rs;
};

// LDS of a CU: the scales of a tile's 256 rows (K / 32 bytes each) and two
// stages of 64 rows of activations have to fit.
constexpr int MX_MAX_LDS = 160 * 1024;
constexpr int MX_MAX_K = 14336;

struct MxArgs {
  GArgs g;
  const void *gu_g, *gu_u, *gus_g, *gus_u, *Wd, *sd;
  long gu_es, gu_rs;
};

hipError_t launch_mx_gate_up(const GemmProblem& pb, const MxWeights& w, const void* X, void* a, hipStream_t s);
hipError_t launch_mx_down(const GemmProblem& pb, const MxWeights& w, const void* a, float* Yp, hipStream_t s);

}  // namespace moe
