// Arguments and launches of the Newton-Schulz orthogonalisation (ortho.hip).
#pragma once
#include "moe_internal.h"

namespace moe {

constexpr int ORTHO_NARROW = 64;   // S below which the update's tiles have at most 128 rows and columns
constexpr int ORTHO_PARTS = 256;   // most partial sums of a matrix's squares

// Iterates X and Gram matrices are kept in fp16 with these factors, what X's
// rounding leaves in fp16 with ORTHO_LOW more.
constexpr float ORTHO_X = 64.f, ORTHO_P = 4096.f, ORTHO_LOW = 2048.f;

struct OrthoArgs {
  const void* g;        // [E,M,N] gradients
  const float* m;       // [E,M,N] momentum, or null: g is the update
  float* m_out;
  const void* w;        // [E,M,N] weights, or null: out receives the orthogonalised update
  void* out;            // out, or the new weights
  void *x0, *x1;        // fp16 [E,M,N]
  void *l0, *l1;        // fp16 [E,M,N]: what is left of X beside them
  void *p, *q;          // fp16 [E,S,S], S = min(M,N)
  float *pd, *qd;       // [E,S]: what the fp16 diagonals of P and Q leave out
  double* part;         // [E][ORTHO_PARTS]
  int E, M, N, S, steps;
  int g_f32, out_f32;
  int nesterov;
  float momentum, lr, keep;   // keep = 1 - decay
  float a, b, c, eps;
};
static_assert(sizeof(void*) == 8, "64-bit pointers on host and device");

hipError_t launch_ortho(const OrthoArgs& p, hipStream_t s);

}  // namespace moe
