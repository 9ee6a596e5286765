// Microscaled 4-bit weights on the device: E2M1 codes (two a byte, the
// element of the even column in the low half) with one E8M0 scale byte for 32
// consecutive columns of a row; the element is code * 2^(scale - 127), a scale
// of 255 makes the block NaN.
#pragma once
#include "gemm_common.h"

namespace moe {

constexpr int MX_BLOCK = 32;   // elements that share a scale

// 2^(s - 127) of a scale byte, with every byte in the exponent field's place:
// 0 is the subnormal 2^-127 and 255 a NaN.
__device__ __forceinline__ float mx_scale(uint32_t s) {
  return __builtin_bit_cast(float, s == 0 ? 0x00400000u : s == 255 ? 0x7fc00000u : s << 23);
}

// Four bytes of codes (8 elements) as bf16, times the block's scale: exact (2
// significant bits, subnormals included), infinite from 2^128 on.
__device__ __forceinline__ bf16x8_t mx_expand(uint32_t codes, float scale) {
  struct { bf16x2_t p[4]; } r;
  r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return __builtin_bit_cast(bf16x8_t, r);
}

}  // namespace moe
