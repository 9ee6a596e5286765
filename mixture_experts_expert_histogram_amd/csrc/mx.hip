// Weight rows to 4-bit microscaled floating point and back (the format of
// mx.h).  Rows are whole blocks of 32, so a tensor is one run of blocks.
//
// Both directions move each byte once: 265 M bf16 elements (531 + 133 + 8 MB)
// are quantised in 97 us and dequantised in 94, 6.9 and 7.1 TB/s, which is HBM's
// rate, a million fp32 ones in 3 us each, which is a launch, and 265 M fp32 ones
// (1062 + 141 MB) in 220 and 453, where a lane's 32 bytes are stored 16 at a
// time, half lines of a wave's run.  A thread takes 8
// elements (16 bytes of bf16, 32 of fp32, 4 bytes of codes), so that a wave's
// accesses are contiguous in every tensor; the 4 threads of a block find its
// largest magnitude by two quad permutes.
#include "mx.h"

namespace moe {
namespace {

constexpr int Q_THREADS = 256;
constexpr int Q_UNROLL = 4;   // 8-element groups of a thread in flight at once

typedef uint32_t u32x4_v __attribute__((ext_vector_type(4)));

template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}

template <typename T> struct Oct;   // 8 elements of a weight row
template <> struct Oct<uint16_t> {
  u32x4_v v;
  __device__ __forceinline__ void load(const void* p, long i) { v = __builtin_nontemporal_load((const u32x4_v*)p + i); }
  __device__ __forceinline__ uint32_t bits(int j) const { return j & 1 ? v[j >> 1] & 0xffff0000u : v[j >> 1] << 16; }
};
template <> struct Oct<float> {
  u32x4_v v[2];
  __device__ __forceinline__ void load(const void* p, long i) {
    v[0] = __builtin_nontemporal_load((const u32x4_v*)p + 2 * i);
    v[1] = __builtin_nontemporal_load((const u32x4_v*)p + 2 * i + 1);
  }
  __device__ __forceinline__ uint32_t bits(int j) const { return v[j >> 2][j & 3]; }
};

// One group of 8: m is the block's largest |element| as fp32 bits, whose
// exponent field is floor(log2) + 127 (0 for zeros and subnormals), so the
// scale byte is that field minus the code range's 2, at least 0.  Dividing by
// the scale is the exact product with 2^(127 - byte) (byte <= 252); the
// conversion rounds to nearest, ties to the even code, and magnitudes over 6
// to 6.  A block with an infinity or NaN gets scale 255 and zero codes.
template <typename T>
__device__ __forceinline__ void quantize_oct(const Oct<T>& x, uint32_t& codes, uint32_t& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, x.bits(j) & 0x7fffffffu);
  m = quad_max<0xB1>(m);   // quad_perm [1,0,3,2]
  m = quad_max<0x4E>(m);   // quad_perm [2,3,0,1]
  const uint32_t ex = m >> 23;
  const bool bad = ex == 255;
  scale = bad ? 255u : ex > 2 ? ex - 2 : 0u;
  const float inv = __builtin_bit_cast(float, (bad ? 127u : 254u - scale) << 23);
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    y[j] = __builtin_amdgcn_fmed3f(__builtin_bit_cast(float, x.bits(j)) * inv, -6.f, 6.f);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[0], y[1], 1.f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], 1.f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[4], y[5], 1.f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[6], y[7], 1.f, 3);
  codes = bad ? 0u : c;
}

// n8 = number of 8-element groups (a multiple of 4: the threads of a block are
// inside or outside together).
template <typename T>
__global__ __launch_bounds__(Q_THREADS) void mx_quantize_kernel(const void* __restrict__ w, long n8,
                                                                uint32_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
  const long step = (long)gridDim.x * Q_THREADS * Q_UNROLL;
  for (long i0 = (long)blockIdx.x * Q_THREADS * Q_UNROLL + threadIdx.x; i0 < n8; i0 += step) {
    Oct<T> x[Q_UNROLL];
#pragma unroll
    for (int u = 0; u < Q_UNROLL; ++u) x[u].load(w, min(i0 + u * Q_THREADS, n8 - 4 + (i0 & 3)));
#pragma unroll
    for (int u = 0; u < Q_UNROLL; ++u) {
      const long i = i0 + u * Q_THREADS;
      uint32_t c, s;
      quantize_oct<T>(x[u], c, s);
      if (i < n8) {
        codes[i] = c;
        if ((i & 3) == 0) scales[i >> 2] = (uint8_t)s;
      }
    }
  }
}

template <typename T>
__global__ __launch_bounds__(Q_THREADS) void mx_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales, long n8,
                                                                  void* __restrict__ w) {
  const long step = (long)gridDim.x * Q_THREADS * Q_UNROLL;
  for (long i0 = (long)blockIdx.x * Q_THREADS * Q_UNROLL + threadIdx.x; i0 < n8; i0 += step) {
    uint32_t c[Q_UNROLL], s[Q_UNROLL];
#pragma unroll
    for (int u = 0; u < Q_UNROLL; ++u) {
      const long i = min(i0 + u * Q_THREADS, n8 - 1);
      c[u] = codes[i];
      s[u] = scales[i >> 2];
    }
#pragma unroll
    for (int u = 0; u < Q_UNROLL; ++u) {
      const long i = i0 + u * Q_THREADS;
      if (i >= n8) continue;
      // the product is exact: a code has 2 significant bits, and 2^-127 times
      // the smallest one, 0.5, is a subnormal of both types (from 2^128 on,
      // bytes 253 and 254, it is infinite in both)
      const float sc = mx_scale(s[u]);
      float y[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 v = q == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.f, 0)
                        : q == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.f, 1)
                        : q == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.f, 2)
                                 : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.f, 3);
        y[2 * q] = v[0] * sc;
        y[2 * q + 1] = v[1] * sc;
      }
      if constexpr (sizeof(T) == 2) {
        const u32x4_v o = {pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7])};
        __builtin_nontemporal_store(o, (u32x4_v*)w + i);
      } else {
        typedef float f32x4_v __attribute__((ext_vector_type(4)));
        __builtin_nontemporal_store(f32x4_v{y[0], y[1], y[2], y[3]}, (f32x4_v*)w + 2 * i);
        __builtin_nontemporal_store(f32x4_v{y[4], y[5], y[6], y[7]}, (f32x4_v*)w + 2 * i + 1);
      }
    }
  }
}

int grid_of(long n8) {
  const long per = (long)Q_THREADS * Q_UNROLL;
  const long g = (n8 + per - 1) / per;
  return (int)(g < (1L << 20) ? g : (1L << 20));
}

}  // namespace

hipError_t launch_mx_quantize(int dtype, const void* w, long n, void* codes, void* scales, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  return run_kernel("mx_quantize", stream, [&] {
    if (dtype == 0)
      mx_quantize_kernel<uint16_t><<<grid_of(n / 8), Q_THREADS, 0, stream>>>(w, n / 8, (uint32_t*)codes,
                                                                             (uint8_t*)scales);
    else
      mx_quantize_kernel<float><<<grid_of(n / 8), Q_THREADS, 0, stream>>>(w, n / 8, (uint32_t*)codes,
                                                                          (uint8_t*)scales);
  });
}

hipError_t launch_mx_dequantize(int dtype, const void* codes, const void* scales, long n, void* w,
                                hipStream_t stream) {
  if (n == 0) return hipSuccess;
  return run_kernel("mx_dequantize", stream, [&] {
    if (dtype == 0)
      mx_dequantize_kernel<uint16_t><<<grid_of(n / 8), Q_THREADS, 0, stream>>>((const uint32_t*)codes,
                                                                               (const uint8_t*)scales, n / 8, w);
    else
      mx_dequantize_kernel<float><<<grid_of(n / 8), Q_THREADS, 0, stream>>>((const uint32_t*)codes,
                                                                            (const uint8_t*)scales, n / 8, w);
  });
}

}  // namespace moe
