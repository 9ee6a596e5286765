// The gated feed-forward block for few tokens: the time is that of reading 3 H I
// weights once, and for one token that of two launches and their first loads.
//
// A workgroup takes 16 weight rows (8 gate and 8 up rows, or 16 rows of Wd);
// its 8 waves split k in units of one 128-byte line a row, read straight into
// matrix-core fragments (16 rows x 64 contiguous bytes a load) against 16 token
// columns, D units in flight a wave.  The partial sums meet in LDS in wave order.
// Few rows a workgroup and all of its loads in flight at once are what fills
// the card with one matrix of 2880 x 2880 (16 tokens bf16: 24 us for both
// kernels).  13 tokens fp32, H 1048, I 712: 7.0 and 5.8 us for 9 MB, the two
// launches' start, first loads and end.  In fp32 up to four groups of 16 tokens
// share a workgroup's weights, and more tokens are more workgroups: 64 tokens of
// 2544 x 3712 56 and 44 us, 256 tokens 164 and 110 (53 TFLOP/s of the fp32 matrix
// rate's 157), bound by the token rows that every 16 weight rows read from L2.
#include "ffn_tiles.h"

namespace moe {
namespace dense {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int FEW_NW = 8;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)(((uint64_t)hi << 32) | lo), 0, (int)kNone, 0x00027000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// Units of NT x 16 token columns that fit in registers.
template <int NT> struct Depth { static constexpr int D = NT == 1 ? 6 : NT == 2 ? 4 : 2; };

// The dot products of this wave's units with 16 weight rows (byte offset wrow
// of this lane's row, lane % 16, from w) and NT x 16 tokens (rows of K elements
// from x), left in LDS: red[wave][token][row].
template <bool F32, int NT>
__device__ __forceinline__ void few_dot(__amdgpu_buffer_rsrc_t w, uint32_t wrow, __amdgpu_buffer_rsrc_t x, int T, int K,
                                        float* red, int wave, int lane) {
  constexpr int ESZ = F32 ? 4 : 2, D = Depth<NT>::D;
  const uint32_t bytes = (uint32_t)K * ESZ;
  const uint32_t mine = (lane >> 4) * 16;
  uint32_t xrow[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = n * 16 + (lane & 15);
    xrow[n] = t < T ? t * bytes : kNone;
  }
  struct Unit { u32x4 w[2], x[NT][2]; } ring[D];
  const auto load = [&](int u, Unit& r) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t o = u * 128 + q * 64 + mine;
      r.w[q] = load16(w, o < bytes ? wrow + o : kNone);
#pragma unroll
      for (int n = 0; n < NT; ++n) r.x[n][q] = load16(x, o < bytes && xrow[n] != kNone ? xrow[n] + o : kNone);
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(wave + d * FEW_NW, ring[d]);
  f32x4 acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int units = (int)((bytes + 127) / 128);
  for (int u = wave; u < units; u += D * FEW_NW) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (F32) {
            const f32x4 wf = __builtin_bit_cast(f32x4, ring[d].w[q]), xf = __builtin_bit_cast(f32x4, ring[d].x[n][q]);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[i], xf[i], acc[n], 0, 0, 0);
          } else {
            acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, ring[d].w[q]),
                                                             __builtin_bit_cast(bf16x8_t, ring[d].x[n][q]), acc[n], 0, 0, 0);
          }
        }
      load(u + (d + D) * FEW_NW, ring[d]);
      __builtin_amdgcn_sched_barrier(0);   // or every product of the ring moves before its reloads
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
    *(f32x4*)(red + ((wave * NT + n) * 16 + (lane & 15)) * 16 + 4 * (lane >> 4)) = acc[n];
  __syncthreads();
}
template <int NT>
__device__ __forceinline__ float few_sum(const float* red, int t, int row) {
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < FEW_NW; ++w) v += red[(w * NT * 16 + t) * 16 + row];
  return v;
}

// A workgroup's rows and tokens: its block of rows, and in t0 and nt its group of
// NT x 16 tokens.  The groups of a block of rows follow one another on one XCD
// (workgroup w runs on XCD w % 8), which reads the weights once.
template <int NT>
__device__ __forceinline__ int few_place(int T, int& t0, int& nt) {
  const int groups = (T + NT * 16 - 1) / (NT * 16), w = blockIdx.x >> 3, block = w / groups;
  t0 = (w - block * groups) * NT * 16;
  nt = min(T - t0, NT * 16);
  return block * 8 + (blockIdx.x & 7);
}

template <bool F32, int NT>
__global__ __launch_bounds__(FEW_NW * 64) void ffn_few_gate_up_kernel(FfnArgs p) {
  using T = std::conditional_t<F32, float, uint16_t>;
  __shared__ __align__(16) float red[FEW_NW * NT * 256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int t0, nt;
  const int j0 = few_place<NT>(p.T, t0, nt) * 8;
  if (j0 >= p.I) return;
  const long row = p.gu_rs * sizeof(T);
  // I is a multiple of 8: the workgroup's 8 columns exist
  const uint32_t wrow = (uint32_t)((lane & 7) * row) + (lane & 8 ? (uint32_t)((const char*)p.gu_u - (const char*)p.gu_g) : 0u);
  few_dot<F32, NT>(rsrc((const char*)p.gu_g + row * j0), wrow, rsrc((const T*)p.x + (size_t)t0 * p.H), nt, p.H, red, wave, lane);
  for (int o = threadIdx.x; o < 8 * nt; o += FEW_NW * 64) {
    const int j = o & 7, t = o >> 3;
    store_val<T>((T*)p.a + (size_t)(t0 + t) * p.I + j0 + j,
                 glu_fwd(few_sum<NT>(red, t, j), few_sum<NT>(red, t, 8 + j), p.act, p.limit, p.alpha));
  }
}

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }

template <bool F32, int NT>
__global__ __launch_bounds__(FEW_NW * 64) void ffn_few_down_kernel(FfnArgs p) {
  using T = std::conditional_t<F32, float, uint16_t>;
  __shared__ __align__(16) float red[FEW_NW * NT * 256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int t0, nt;
  const int h0 = few_place<NT>(p.T, t0, nt) * 16;
  if (h0 >= p.H) return;
  const uint32_t row = p.I * sizeof(T);
  few_dot<F32, NT>(rsrc((const char*)p.wd + (size_t)row * h0), row * min(lane & 15, p.H - 1 - h0),
                   rsrc((const T*)p.a + (size_t)t0 * p.I), nt, p.I, red, wave, lane);
  for (int o = threadIdx.x; o < 16 * nt; o += FEW_NW * 64) {
    const int h = o & 15, t = o >> 4;
    if (h0 + h >= p.H) continue;
    const size_t at = (size_t)(t0 + t) * p.H + h0 + h;
    const float ad = p.add ? as_float(((const T*)p.add)[at]) : 0.f;
    store_val<T>((T*)p.out + at, ad + row_gate(p.gate, t0 + t) * few_sum<NT>(red, t, h));
  }
}

// ------------------------------------------------------------------ up to four tokens
// A wave takes one activation column (its gate and its up row) or one output
// row, a lane 16 bytes of every kilobyte of a row: nothing is shared between
// waves, and at 2880 columns every load of the card is in flight at once, 11
// waves a CU.  2880 x 2880 bf16, one token: 7.3 and 4.6 us (4.6 and 3.6 TB/s)
// for the two kernels, where the 16-row workgroups took 12.5 and 6.6.
constexpr int ONE_CH = 6;   // kilobytes of a row in flight

template <bool F32>
__device__ __forceinline__ float dot16(u32x4 w, u32x4 x, float s) {
  const f32x4 wf = __builtin_bit_cast(f32x4, w), xf = __builtin_bit_cast(f32x4, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      s += wf[i] * xf[i];
    } else {
      s += __builtin_bit_cast(float, w[i] << 16) * __builtin_bit_cast(float, x[i] << 16);
      s += __builtin_bit_cast(float, w[i] & 0xffff0000u) * __builtin_bit_cast(float, x[i] & 0xffff0000u);
    }
  }
  return s;
}
// The dot products of R rows (of `bytes` bytes, from w[r]) with the first N of
// T tokens (rows of x), in every lane.
template <bool F32, int R, int N>
__device__ __forceinline__ void one_dot(const __amdgpu_buffer_rsrc_t (&w)[R], __amdgpu_buffer_rsrc_t x, int T, uint32_t bytes,
                                        int lane, float (&sum)[R][N]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < N; ++t) sum[r][t] = 0.f;
  for (uint32_t c0 = 0; c0 < bytes; c0 += ONE_CH * 1024) {
    u32x4 wv[R][ONE_CH], xv[N][ONE_CH];
#pragma unroll
    for (int c = 0; c < ONE_CH; ++c) {
      const uint32_t o = c0 + c * 1024 + lane * 16, at = o < bytes ? o : kNone;
#pragma unroll
      for (int r = 0; r < R; ++r) wv[r][c] = load16(w[r], at);
    }
#pragma unroll
    for (int c = 0; c < ONE_CH; ++c) {
      const uint32_t o = c0 + c * 1024 + lane * 16;
#pragma unroll
      for (int t = 0; t < N; ++t) xv[t][c] = load16(x, o < bytes && t < T ? t * bytes + o : kNone);
    }
#pragma unroll
    for (int c = 0; c < ONE_CH; ++c)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < N; ++t) sum[r][t] = dot16<F32>(wv[r][c], xv[t][c], sum[r][t]);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < N; ++t) sum[r][t] += __shfl_xor(sum[r][t], d);
}

template <bool F32, int N>
__global__ __launch_bounds__(256) void ffn_one_gate_up_kernel(FfnArgs p) {
  using T = std::conditional_t<F32, float, uint16_t>;
  const int lane = threadIdx.x & 63, j = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // I is a multiple of 8
  const __amdgpu_buffer_rsrc_t w[2] = {rsrc((const T*)p.gu_g + p.gu_rs * j), rsrc((const T*)p.gu_u + p.gu_rs * j)};
  float s[2][N];
  one_dot<F32, 2, N>(w, rsrc(p.x), p.T, p.H * sizeof(T), lane, s);
#pragma unroll
  for (int t = 0; t < N; ++t)
    if (lane == 0 && t < p.T) store_val<T>((T*)p.a + (size_t)t * p.I + j, glu_fwd(s[0][t], s[1][t], p.act, p.limit, p.alpha));
}

template <bool F32, int N>
__global__ __launch_bounds__(256) void ffn_one_down_kernel(FfnArgs p) {
  using T = std::conditional_t<F32, float, uint16_t>;
  const int lane = threadIdx.x & 63, h = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // so is H
  const __amdgpu_buffer_rsrc_t w[1] = {rsrc((const T*)p.wd + (size_t)p.I * h)};
  float ad[N], g[N];
#pragma unroll
  for (int t = 0; t < N; ++t) {
    const int tc = min(t, p.T - 1);
    ad[t] = p.add ? as_float(((const T*)p.add)[(size_t)tc * p.H + h]) : 0.f;
    g[t] = row_gate(p.gate, tc);
  }
  float s[1][N];
  one_dot<F32, 1, N>(w, rsrc(p.a), p.T, p.I * sizeof(T), lane, s);
#pragma unroll
  for (int t = 0; t < N; ++t)
    if (lane == 0 && t < p.T) store_val<T>((T*)p.out + (size_t)t * p.H + h, ad[t] + g[t] * s[0][t]);
}

template <bool F32, int N>
hipError_t run_one(const FfnArgs& p, hipStream_t s) {
  const hipError_t e = run_kernel("ffn_one_gate_up", s, [&] { ffn_one_gate_up_kernel<F32, N><<<p.I / 4, 256, 0, s>>>(p); });
  if (e != hipSuccess) return e;
  return run_kernel("ffn_one_down", s, [&] { ffn_one_down_kernel<F32, N><<<p.H / 4, 256, 0, s>>>(p); });
}

// Groups of 16 tokens of a workgroup, for that many blocks of rows (bf16: the one
// group): the fewest rounds of the card, times what a workgroup of them takes.
// fp32 down products, us with 1, 2 and 4: 32 blocks of k 8192, 64 tokens 35, 47
// and 75, 256 tokens 66, 49 and 77; 159 of k 3712, 64 tokens 50, 51 and 44.
template <bool F32>
int few_groups(int T, int blocks) {
  constexpr float time[] = {1.f, 1.36f, 2.15f};
  int best = 0;
  float least = 0.f;
  for (int i = 0; F32 && i < 3; ++i) {
    const float t = (float)((blocks * ((T + (16 << i) - 1) / (16 << i)) + 255) / 256) * time[i];
    if (i == 0 || t < least) best = i, least = t;
  }
  return 1 << best;
}
template <bool F32, class Run>
hipError_t with_groups(int T, int blocks, Run run) {
  const int n = few_groups<F32>(T, blocks);
  const int grid = (blocks + 7) / 8 * 8 * ((T + 16 * n - 1) / (16 * n));
  if constexpr (F32) {
    if (n == 4) return run(std::integral_constant<int, 4>{}, grid);
    if (n == 2) return run(std::integral_constant<int, 2>{}, grid);
  }
  return run(std::integral_constant<int, 1>{}, grid);
}

template <bool F32>
hipError_t few(const FfnArgs& p, hipStream_t s) {
  if (p.T == 1) return run_one<F32, 1>(p, s);
  if (p.T == 2) return run_one<F32, 2>(p, s);
  if (p.T <= 4) return run_one<F32, 4>(p, s);
  const hipError_t e = with_groups<F32>(p.T, p.I / 8, [&](auto n, int grid) {
    const auto k = ffn_few_gate_up_kernel<F32, decltype(n)::value>;
    return run_kernel("ffn_few_gate_up", s, [&] { k<<<grid, FEW_NW * 64, 0, s>>>(p); });
  });
  if (e != hipSuccess) return e;
  return with_groups<F32>(p.T, (p.H + 15) / 16, [&](auto n, int grid) {
    const auto k = ffn_few_down_kernel<F32, decltype(n)::value>;
    return run_kernel("ffn_few_down", s, [&] { k<<<grid, FEW_NW * 64, 0, s>>>(p); });
  });
}

// ------------------------------------------------------------------ the block as one expert (fp32, many tokens)
__global__ __launch_bounds__(256) void ffn_one_expert_kernel(const float* gate, int T, int32_t* ids, float* w) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= T) return;
  ids[t] = 0;
  w[t] = row_gate(gate, t);
}
__global__ __launch_bounds__(256) void ffn_add_kernel(const float* add, const float* y, long n4, float* out) {
  for (long i = blockIdx.x * 256l + threadIdx.x; i < n4; i += gridDim.x * 256l)
    *(f32x4*)(out + 4 * i) = *(const f32x4*)(add + 4 * i) + *(const f32x4*)(y + 4 * i);
}
__global__ __launch_bounds__(256) void ffn_dgate_kernel(const float* gate, const float* dw, int T, float* dgate) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t < T) dgate[t] = gate_slope(gate[t]) * dw[t];
}

}  // namespace dense

using namespace dense;

hipError_t launch_ffn_few(int dtype, FfnArgs p, hipStream_t s) { return dtype == 0 ? few<false>(p, s) : few<true>(p, s); }

hipError_t launch_ffn_one_expert(const float* gate, int T, int32_t* ids, float* w, hipStream_t s) {
  return run_kernel("ffn_one_expert", s, [&] { ffn_one_expert_kernel<<<(T + 255) / 256, 256, 0, s>>>(gate, T, ids, w); });
}
hipError_t launch_ffn_add(const float* add, const float* y, long n, float* out, hipStream_t s) {
  const long g = (n / 4 + 255) / 256;
  return run_kernel("ffn_add", s, [&] { ffn_add_kernel<<<(int)(g < 4096 ? g : 4096), 256, 0, s>>>(add, y, n / 4, out); });
}
hipError_t launch_ffn_dgate(const float* gate, const float* dw, int T, float* dgate, hipStream_t s) {
  return run_kernel("ffn_dgate", s, [&] { ffn_dgate_kernel<<<(T + 255) / 256, 256, 0, s>>>(gate, dw, T, dgate); });
}

}  // namespace moe
