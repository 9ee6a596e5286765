// Arguments and launches of the norms before and after a block (norm.hip).
#pragma once
#include "moe_internal.h"

namespace moe {

constexpr int NORM_MAX_H = 16384;   // a row in the registers of 1024 threads
constexpr int NORM_GRID = 512;      // most workgroups of a backward pass (partial sums of the weights' gradients)

constexpr int NORM_SHORT = 256;     // threads of a backward workgroup of several rows
constexpr int NORM_ROWS = 1 << 21;  // most workgroups (rows) of a forward pass along x
constexpr int64_t NORM_MAX_T = int64_t(1) << 30;

struct NormArgs {
  const void* x;        // [T,H]: the residual stream before the step (forward), after it (backward)
  const void* h;        // [T,H] the block's output, or null: the norm before a block
  const void* w_post;   // [H] or null
  const void* w_next;   // [H] or null
  const void* gate;
  void* x_new;          // forward
  void* y;
  const void* d_new;    // backward: gradient of x_new (or null), of y
  const void* d_y;
  void* d_x;
  void* d_h;
  void* d_gate;
  float* d_w_post;
  float* d_w_next;
  float* part;          // [NORM_GRID][3][H] partial sums: next, post, gate
  int T, H, gate_kind;  // moe_gate_t
  float scale, eps;
};
static_assert(sizeof(void*) == 8, "64-bit pointers on host and device");

// dtype 0 bf16, 1 fp32
hipError_t launch_norm_fwd(int dtype, const NormArgs& p, hipStream_t s);
hipError_t launch_norm_bwd(int dtype, const NormArgs& p, hipStream_t s);

}  // namespace moe
