// Arguments of the few-token kernels (few.hip).
#pragma once
#include "moe_internal.h"

namespace moe {

// Most tokens of a few-token call.
constexpr int FEW_MAX_T = 128;

// Strides are bytes.  Gate (up) row j of expert e starts gu_es e + gu_rs j
// after gu_g (gu_u); mx scales follow the same strides over 16 (a row of c
// code bytes has c / 16 scales).  Rows of Wd are d_rs bytes, H an expert.
struct FewArgs {
  const float* logits;  // [T,E], or null: ids and w are given
  const int32_t* ids;   // [T,K]
  const float* w;       // [T,K]
  int32_t* ids_out;     // with logits: where the choice goes (ids, w)
  float* w_out;
  const void* X;        // [T,H]
  const void* gu_g;
  const void* gu_u;
  const void* gus_g;
  const void* gus_u;
  const void* Wd;
  const void* sd;
  void* a;              // [S,I] in the activations' type
  float* y;             // [S,H]
  void* out;            // [T,H]
  int32_t* status;
  long gu_es, gu_rs, d_rs;
  int T, H, I, E, K, S;
  int act;
  float limit, alpha;
};
static_assert(sizeof(void*) == 8 && sizeof(long) == 8, "64-bit pointers and longs on host and device");

// kind: 0 bf16, 1 fp32, 2 microscaled 4-bit weights with bf16 activations.
hipError_t launch_few(int kind, const FewArgs& p, hipStream_t stream);

}  // namespace moe
