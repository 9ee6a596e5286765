// Arguments and launches of the gated feed-forward block (ffn_fwd.hip,
// ffn_bwd.hip, ffn_few.hip).
#pragma once
#include "moe_internal.h"

namespace moe {

// Most tokens that the kernels for a few tokens take (weights read once, no
// tiles); more go to the dense products, in fp32 to those of one expert.  2880
// x 2880 bf16, both kernels in us: 16 tokens 24 against 26 on tiles of 64 x 64,
// 17 tokens 30 against 27, 64 tokens 51 against 33.  fp32, against the products of
// one expert: 2544 x 3712 64 tokens 100 against 526, 512 tokens 460 against 540,
// 1024 tokens 891 against 705; 2880 x 2880 494 against 490 and 936 against 660;
// 1048 x 712 59 against 175 and 97 against 179.
constexpr int FFN_FEW_BF16 = 16, FFN_FEW_F32 = 512;

struct FfnArgs {
  const void* x;        // [T,H]
  const void* gu_g;     // gate row j starts gu_rs j elements after gu_g, up row j after gu_u
  const void* gu_u;
  const void* gu;       // [2I,H], the rows in the layout's order
  const void* wd;       // [H,I]
  const float* gate;    // [T] logits, or null
  const void* add;      // [T,H], or null
  const void* dout;     // [T,H]
  void* a;              // [T,I]
  float* z;             // gate and up values in blocks (z_block), or null
  void* out;            // [T,H]
  void* dz;             // [T,2I] in the layout's order
  void* aw;             // [T,I]: sigmoid(gate) a
  void* dx;             // [T,H]
  float* dgate;         // [T], or null
  float* part;          // [T,parts]
  void* dgu;            // [2I,H]
  void* dwd;            // [H,I]
  long gu_rs;
  int T, H, I;
  int act, layout, grad_f32;
  float limit, alpha;
  int mt, nt, parts;    // tiles of the present product; partial sums of a row
};
static_assert(sizeof(void*) == 8 && sizeof(long) == 8, "64-bit pointers and longs on host and device");

// Floats of the saved gate and up values: blocks of 32 rows x 8 columns.
inline size_t ffn_z_floats(int64_t T, int64_t I) { return (size_t)((T + 31) / 32) * 32 * I * 2; }
// Most partial sums of a row that ffn_down_dgrad writes.
inline int64_t ffn_parts(int64_t I) { return 2 * ((I + 63) / 64); }

hipError_t launch_ffn_gate_up(FfnArgs p, hipStream_t s);      // a (if not null) and z (if not null)
hipError_t launch_ffn_down(FfnArgs p, hipStream_t s);         // out
hipError_t launch_ffn_down_dgrad(FfnArgs p, hipStream_t s);   // dz, aw, dgate
hipError_t launch_ffn_gate_up_dgrad(FfnArgs p, hipStream_t s);   // dx
hipError_t launch_ffn_wgrads(FfnArgs p, hipStream_t s);       // dgu, dwd
hipError_t launch_ffn_few(int dtype, FfnArgs p, hipStream_t s);  // out, by way of a
// ids[t] = 0 and w[t] = sigmoid(gate[t]) (1 without a gate): the block as a layer of one expert
hipError_t launch_ffn_one_expert(const float* gate, int T, int32_t* ids, float* w, hipStream_t s);
hipError_t launch_ffn_add(const float* add, const float* y, long n, float* out, hipStream_t s);   // out = add + y
// dgate[t] = s (1 - s) dw[t], s = sigmoid(gate[t])
hipError_t launch_ffn_dgate(const float* gate, const float* dw, int T, float* dgate, hipStream_t s);

}  // namespace moe
