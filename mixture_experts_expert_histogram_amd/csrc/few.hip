// The whole layer for a few tokens (decoding): one kernel for the gate_up
// projection with its activation, one for the down projection, one for the
// sum over a token's experts.
//
//   a[s]   = phi(Wgu[e_s] x_t)        s = t K + k, e_s = ids[s]
//   y[s]   = w_s Wd[e_s] a[s]
//   out[t] = sum_k y[t K + k]
//
// With a few tokens an expert holds one or two slots, and the time is that of
// reading the active experts' weights once: 2 flops a weight byte against the
// 300 where the matrix cores would bound it.  So nothing here is staged for
// reuse: a wave reads its 32 weight rows straight into matrix-core fragments
// (16 rows by k, every lane 16 bytes of one row) and multiplies them with up
// to 16 token columns, whose fragments come from L1/L2.  The lanes' share of k
// follows from the 16-byte loads (lane group g of 4 holds the g-th 16 bytes of
// a row's 64), and the token fragments are read in the same k order, so no
// operand is ever shuffled.  The waves of a workgroup take k units in turn
// and their partial sums meet in LDS in wave order.
//
// No routing pass precedes it: a workgroup finds its expert's slots by a scan
// over the ids (at most T K of them), in slot order.  Nothing depends on the
// order in which workgroups run, and no atomics are used.
//
// Loads are buffer loads whose offset is put past the buffer's end where a
// row, a token or a k chunk does not exist: they return zero without memory
// traffic and without a branch.
#include <type_traits>

#include "few.h"
#include "mx.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

enum { W_BF16 = 0, W_F32 = 1, W_MX = 2 };

constexpr uint32_t kPast = 0x80000000u;   // byte offset past every buffer

template <int KIND> struct Unit;   // 64 bytes of a weight row
template <> struct Unit<W_BF16> { static constexpr int K = 32, XQ = 1, XSZ = 2; };
template <> struct Unit<W_F32> { static constexpr int K = 16, XQ = 1, XSZ = 4; };
template <> struct Unit<W_MX> { static constexpr int K = 128, XQ = 4, XSZ = 2; };

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)(((uint64_t)hi << 32) | lo), 0, (int)kPast, 0x00027000);
}
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// Weight rows of one wave: two groups of 16 rows (gate and up rows of 16
// activation columns, or 32 output columns).  off is this lane's row (lane %
// 16) in bytes from the group's base; a mx row's scales have their own.
struct Rows {
  __amdgpu_buffer_rsrc_t w[2], s[2];
  uint32_t off[2], soff[2];
};

template <int KIND>
__device__ __forceinline__ f32x4 mma16(u32x4_t w, const u32x4_t* x, float scale, f32x4 acc) {
  if constexpr (KIND == W_BF16) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w), __builtin_bit_cast(bf16x8_t, x[0]),
                                                  acc, 0, 0, 0);
  } else if constexpr (KIND == W_F32) {
    const f32x4 wf = __builtin_bit_cast(f32x4, w), xf = __builtin_bit_cast(f32x4, x[0]);
#pragma unroll
    for (int q = 0; q < 4; ++q) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[q], xf[q], acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_expand(w[q], scale), __builtin_bit_cast(bf16x8_t, x[q]), acc, 0,
                                                    0, 0);
  }
  return acc;
}

// acc[group][n] += rows . x over this wave's k units (u = wave, wave + NW,
// ...), U units of loads in flight; xoff[n]: byte offset of this lane's token
// row of column tile n (kPast: no token).  Accumulator element v of a lane is
// weight row 4 (lane / 16) + v of the group, token column lane % 16.
template <int KIND, int NT, int U, int NW>
__device__ __forceinline__ void dot_rows(const Rows& r, __amdgpu_buffer_rsrc_t xr, const uint32_t (&xoff)[NT], int K,
                                         int wave, int lane, f32x4 (&acc)[2][NT]) {
  using UN = Unit<KIND>;
  constexpr int KL = UN::K / 4;   // k of a lane in a unit
  const int g = lane >> 4;
  const int nu = (K + UN::K - 1) / UN::K;
  for (int u0 = wave; u0 < nu; u0 += U * NW) {
    u32x4_t w[U][2], x[U][NT][UN::XQ];
    uint32_t sc[U][2];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = u0 + i * NW, k = u * UN::K + g * KL;
      const bool ok = k < K;   // K is a multiple of KL
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[i][h] = load16(r.w[h], ok ? r.off[h] + u * 64 + g * 16 : kPast);
        if constexpr (KIND == W_MX)
          sc[i][h] = __builtin_amdgcn_raw_buffer_load_b8(r.s[h], ok ? r.soff[h] + u * 4 + g : kPast, 0, 0);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < UN::XQ; ++q)
          x[i][n][q] = load16(xr, ok && xoff[n] != kPast ? xoff[n] + (k + q * 8) * UN::XSZ : kPast);
    }
    __builtin_amdgcn_sched_barrier(0);   // every load of the batch is issued before the first product waits
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float s = KIND == W_MX ? mx_scale(sc[i][h]) : 1.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[h][n] = mma16<KIND>(w[i][h], x[i][n], s, acc[h][n]);
      }
  }
}

// The slots of this workgroup's expert, ascending, in LDS: returns their
// number, or 0 when the workgroup has no work.  Grid row y stands for expert
// y when there are at least E slots, otherwise for the expert of slot y (and
// works if y is that expert's first slot).  Every thread of the workgroup
// calls it.
__device__ __forceinline__ int find_slots(const FewArgs& p, int& e, uint16_t* list, int* cnt) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  const bool by_slot = p.S < p.E;
  e = by_slot ? p.ids[blockIdx.y] : (int)blockIdx.y;
  if ((unsigned)e >= (unsigned)p.E) return 0;
  const uint64_t lower = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  int c = 0;
  for (int s0 = 0; s0 < p.S; s0 += blockDim.x) {
    const int s = s0 + tid;
    const bool hit = s < p.S && p.ids[s] == e;
    const uint64_t m = __ballot(hit);
    if (lane == 0) cnt[wave] = __popcll(m);
    __syncthreads();
    int at = c + __popcll(m & lower);
    for (int v = 0; v < nw; ++v) {
      at += v < wave ? cnt[v] : 0;
      c += cnt[v];
    }
    if (hit) list[at] = (uint16_t)s;
    __syncthreads();
  }
  if (by_slot && list[0] != blockIdx.y) return 0;
  return c;
}

template <int NT>
__device__ __forceinline__ void zero(f32x4 (&acc)[2][NT]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[h][n] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// The waves' partial sums in LDS: [wave][group][row 16][column 16 NT], read
// back summed in wave order.
template <int NT>
__device__ __forceinline__ void put_partial(float* red, int wave, int lane, const f32x4 (&acc)[2][NT]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *(f32x4*)(red + (((wave * 2 + h) * NT + n) * 16 + (lane & 15)) * 16 + 4 * (lane >> 4)) = acc[h][n];
}
// element (row j, token column c) of group h
template <int NT, int NW>
__device__ __forceinline__ float get_sum(const float* red, int h, int j, int c) {
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) v += red[(((w * 2 + h) * NT + (c >> 4)) * 16 + (c & 15)) * 16 + j];
  return v;
}

template <typename T> __device__ __forceinline__ void put(T* p, float v) { store_val<T>(p, v); }

template <int KIND> struct Elem { using T = uint16_t; };
template <> struct Elem<W_F32> { using T = float; };

// ---------------------------------------------------------------- gate_up
// One workgroup: 16 activation columns of one expert, for all its tokens in
// passes of 16 NT.
template <int KIND, int NT, int U, int NW>
__device__ __forceinline__ void gate_up_pass(const FewArgs& p, const Rows& r, int j0, int c0, int c,
                                             const uint16_t* list, float* red, int wave, int lane) {
  using T = typename Elem<KIND>::T;
  uint32_t xoff[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int i = c0 + n * 16 + (lane & 15);
    xoff[n] = i < c ? (uint32_t)(list[i] / p.K) * (uint32_t)(p.H * Unit<KIND>::XSZ) : kPast;
  }
  f32x4 acc[2][NT];
  zero<NT>(acc);
  dot_rows<KIND, NT, U, NW>(r, rsrc(p.X), xoff, p.H, wave, lane, acc);
  put_partial<NT>(red, wave, lane, acc);
  __syncthreads();
  T* a = (T*)p.a;
  for (int o = threadIdx.x; o < 256 * NT; o += NW * 64) {
    const int j = o & 15, t = o >> 4;
    if (c0 + t < c && j0 + j < p.I) {
      const float gv = get_sum<NT, NW>(red, 0, j, t), uv = get_sum<NT, NW>(red, 1, j, t);
      put<T>(a + (size_t)list[c0 + t] * p.I + j0 + j, glu_fwd(gv, uv, p.act, p.limit, p.alpha));
    }
  }
  __syncthreads();
}

template <int KIND, int NW>
__global__ __launch_bounds__(NW * 64) void few_gate_up_kernel(FewArgs p) {
  extern __shared__ char few_lds[];
  __shared__ int cnt[NW];
  __shared__ __align__(16) float red[NW * 2 * 2 * 256];
  uint16_t* list = (uint16_t*)few_lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (blockIdx.x == 0 && blockIdx.y == 0 && wave == 0) {   // slots with an id outside [0,E)
    int bad = 0;
    for (int s = lane; s < p.S; s += 64) bad += (unsigned)p.ids[s] >= (unsigned)p.E;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) bad += __shfl_xor(bad, d);
    if (lane == 0) p.status[0] = bad;
  }
  int e;
  const int c = find_slots(p, e, list, cnt);
  if (c == 0) return;
  const int j0 = blockIdx.x * 16;
  const int j = min(j0 + (lane & 15), p.I - 1) - j0;
  Rows r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    r.w[h] = rsrc((const char*)(h ? p.gu_u : p.gu_g) + p.gu_es * e + p.gu_rs * j0);
    r.off[h] = (uint32_t)(p.gu_rs * j);
    if constexpr (KIND == W_MX) {
      r.s[h] = rsrc((const char*)(h ? p.gus_u : p.gus_g) + (p.gu_es * e + p.gu_rs * j0) / 16);
      r.soff[h] = (uint32_t)(p.gu_rs * j / 16);
    }
  }
  if (c <= 16) {
    gate_up_pass<KIND, 1, (KIND == W_MX ? 3 : 8), NW>(p, r, j0, 0, c, list, red, wave, lane);
  } else {
    for (int c0 = 0; c0 < c; c0 += 32)
      gate_up_pass<KIND, 2, (KIND == W_MX ? 2 : 4), NW>(p, r, j0, c0, c, list, red, wave, lane);
  }
}

// ---------------------------------------------------------------- down
// One workgroup: 32 output columns of one expert's slots.
template <int KIND, int NT, int U, int NW>
__device__ __forceinline__ void down_pass(const FewArgs& p, const Rows& r, int h0, int c0, int c, const uint16_t* list,
                                          float* red, int wave, int lane) {
  uint32_t xoff[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int i = c0 + n * 16 + (lane & 15);
    xoff[n] = i < c ? (uint32_t)list[i] * (uint32_t)(p.I * Unit<KIND>::XSZ) : kPast;
  }
  f32x4 acc[2][NT];
  zero<NT>(acc);
  dot_rows<KIND, NT, U, NW>(r, rsrc(p.a), xoff, p.I, wave, lane, acc);
  put_partial<NT>(red, wave, lane, acc);
  __syncthreads();
  for (int o = threadIdx.x; o < 512 * NT; o += NW * 64) {
    const int j = o & 31, t = o >> 5;
    if (c0 + t < c && h0 + j < p.H) {
      const int s = list[c0 + t];
      p.y[(size_t)s * p.H + h0 + j] = p.w[s] * get_sum<NT, NW>(red, j >> 4, j & 15, t);
    }
  }
  __syncthreads();
}

template <int KIND, int NW>
__global__ __launch_bounds__(NW * 64) void few_down_kernel(FewArgs p) {
  extern __shared__ char few_lds[];
  __shared__ int cnt[NW];
  __shared__ __align__(16) float red[NW * 2 * 2 * 256];
  uint16_t* list = (uint16_t*)few_lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int e;
  const int c = find_slots(p, e, list, cnt);
  if (c == 0) return;
  const int h0 = blockIdx.x * 32;
  Rows r;
  const size_t es = (size_t)p.H * p.d_rs;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    r.w[h] = rsrc((const char*)p.Wd + es * e + p.d_rs * h0);
    r.off[h] = (uint32_t)(p.d_rs * (min(h0 + h * 16 + (lane & 15), p.H - 1) - h0));
    if constexpr (KIND == W_MX) {
      r.s[h] = rsrc((const char*)p.sd + (es * e + p.d_rs * h0) / 16);
      r.soff[h] = r.off[h] / 16;
    }
  }
  if (c <= 16) {
    down_pass<KIND, 1, (KIND == W_MX ? 3 : 8), NW>(p, r, h0, 0, c, list, red, wave, lane);
  } else {
    for (int c0 = 0; c0 < c; c0 += 32)
      down_pass<KIND, 2, (KIND == W_MX ? 2 : 4), NW>(p, r, h0, c0, c, list, red, wave, lane);
  }
}

// ---------------------------------------------------------------- sum over k
template <bool OUT_BF16>
__global__ __launch_bounds__(256) void few_combine_kernel(FewArgs p) {
  const int chunks = p.H / 4;
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= p.T * chunks) return;
  const int t = i / chunks, c = i - t * chunks;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < p.K; ++k) {
    const int s = t * p.K + k;
    if ((unsigned)p.ids[s] < (unsigned)p.E) v += *(const f32x4*)(p.y + (size_t)s * p.H + 4 * c);
  }
  if (OUT_BF16)
    store4<uint16_t>((uint16_t*)p.out + (size_t)t * p.H + 4 * c, v[0], v[1], v[2], v[3]);
  else
    store4<float>((float*)p.out + (size_t)t * p.H + 4 * c, v[0], v[1], v[2], v[3]);
}

template <int KIND>
hipError_t launch(const FewArgs& p, hipStream_t stream) {
  constexpr int NW = 4;
  const size_t lds = (size_t)p.S * sizeof(uint16_t);
  const int gy = p.S < p.E ? p.S : p.E;
  hipError_t err = run_kernel(KIND == W_MX ? "few_mx_gate_up" : "few_gate_up", stream, [&] {
    few_gate_up_kernel<KIND, NW><<<dim3((p.I + 15) / 16, gy), NW * 64, lds, stream>>>(p);
  });
  if (err != hipSuccess) return err;
  err = run_kernel(KIND == W_MX ? "few_mx_down" : "few_down", stream, [&] {
    few_down_kernel<KIND, NW><<<dim3((p.H + 31) / 32, gy), NW * 64, lds, stream>>>(p);
  });
  if (err != hipSuccess) return err;
  return run_kernel("few_combine", stream, [&] {
    const int grid = (p.T * (p.H / 4) + 255) / 256;
    if (KIND == W_F32) few_combine_kernel<false><<<grid, 256, 0, stream>>>(p);
    else few_combine_kernel<true><<<grid, 256, 0, stream>>>(p);
  });
}

}  // namespace

hipError_t launch_few(int kind, const FewArgs& p, hipStream_t stream) {
  switch (kind) {
    case W_BF16: return launch<W_BF16>(p, stream);
    case W_F32: return launch<W_F32>(p, stream);
    default: return launch<W_MX>(p, stream);
  }
}

}  // namespace moe
