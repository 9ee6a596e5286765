// Backward products of the gated feed-forward block, given d_out and the gate
// and up values (s = sigmoid(gate), 1 without a gate):
//
//   r = d_out Wd,  da = s r,  (dg, du) = phi'(g, u) da,  d_gate = s (1 - s) <r, a>
//   d_x = dZ Wgu,  d_Wgu = dZ^T x,  d_Wd = d_out^T (s a)
//
// dZ and s a are rounded to bf16 as the next products' operands; every sum is
// fp32.
#include "ffn_tiles.h"

namespace moe {
namespace dense {

// 8192 tokens, H 4096, I 8192: 666 us (825 TFLOP/s).  The tiles' ends read 1.07
// GB of gate and up values and write 0.6 GB, all workgroups at about the same
// time and so without matrix work beside them: some 280 us at 6 TB/s.  Starts
// put apart by a wait gained 30 us here and lost more in smaller calls.
// ACT: 0 swiglu, 1 clamped
template <class C, int ACT>
__global__ __launch_bounds__(256, 1) void ffn_down_dgrad_kernel(FfnArgs p) {
  FFN_PROLOGUE(C)
  KSrc<C::NBA> as;
  CSrc<C::NBB> bs;
  init_rows(as, p.dout, m0, p.T, p.H, wave, lane);
  bs.init(p.wd, p.I, n0, p.I, wave, lane);
  mainloop<C, bf16x8_t>(as, bs, p.H, lds, acc, wave, lane);
  const int I = p.I;
  const int r0 = m0 + wm * 32 * C::FM, r32 = lane & 31, c00 = n0 + wn * 32 * C::FN;
  float s[C::FM], sum[C::FM];
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    s[i] = row_gate(p.gate, min(r0 + 32 * i + r32, p.T - 1));
    sum[i] = 0.f;
  }
  // The fragment's gate and up values; blocks of rows or columns past the last
  // read the last one (what comes of it is not stored).
  struct Z { float4 g[4], u[4]; };
  const int last = ((p.T - 1) >> 5) << 5;
  each_fragment<C, Z, 2>(
      [&](int i, int j, Z& z) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int c = min(c00 + 32 * j + 8 * v, I - 8);
          z.g[v] = *(const float4*)z_block(p.z, min(r0 + 32 * i, last), c, I, 0, lane);
          z.u[v] = *(const float4*)z_block(p.z, min(r0 + 32 * i, last), c, I, 1, lane);
        }
      },
      [&](int i, int j, const Z& z) __attribute__((always_inline)) {
        const int row = r0 + 32 * i + r32, c0 = c00 + 32 * j;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float dg[2][4], du[2][4], a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 g4 = z.g[2 * q + h], u4 = z.u[2 * q + h];
            const float g[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
            float rv = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float r = acc[i][j][8 * q + 4 * h + e];
              const float v = glu_bwd_t<ACT>(g[e], u[e], s[i] * r, p.limit, p.alpha, dg[h][e], du[h][e]);
              rv += r * v;
              a[h][e] = s[i] * v;
            }
            if (c0 + 16 * q + 8 * h < I) sum[i] += rv;
          }
          const u32x4 av = pack_pair(a[0], a[1]);
          const int cc = c0 + 16 * q + 8 * (lane >> 5);
          const bool ok = row < p.T && cc < I;
          if (ok) *(u32x4*)((uint16_t*)p.aw + (size_t)row * I + cc) = av;
          uint16_t* dz = (uint16_t*)p.dz + (size_t)row * 2 * I;
          if (p.layout) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int ch = c0 + 16 * q + 8 * h + 4 * (lane >> 5);
              if (row < p.T && ch < I) store4x2<uint16_t>(dz + 2 * ch, dg[h], du[h]);
            }
          } else {
            const u32x4 gv = pack_pair(dg[0], dg[1]), uv = pack_pair(du[0], du[1]);
            if (ok) {
              *(u32x4*)(dz + cc) = gv;
              *(u32x4*)(dz + I + cc) = uv;
            }
          }
        }
      });
  if (!p.dgate) return;
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    const int row = r0 + 32 * i + r32;
    sum[i] += __shfl_xor(sum[i], 32);   // the other half of the row's columns
    if (lane < 32 && row < p.T) p.part[(size_t)row * p.parts + nt * 2 + wn] = sum[i];
  }
}

// dgate[t] = s (1 - s) times the sum of the row's partial sums, in order (7 us for
// 4096 tokens and 30 sums a row, of which a launch is about 4).
__global__ __launch_bounds__(256) void ffn_gate_reduce_kernel(FfnArgs p) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= p.T) return;
  float v = 0.f;
  for (int i = 0; i < p.parts; ++i) v += p.part[(size_t)t * p.parts + i];
  p.dgate[t] = gate_slope(p.gate[t]) * v;
}

// 8192 tokens, H 4096, I 8192: 757 us (1452 TFLOP/s, matrix cores 87 % busy).
template <class C>
__global__ __launch_bounds__(256, 1) void ffn_gate_up_dgrad_kernel(FfnArgs p) {
  FFN_PROLOGUE(C)
  KSrc<C::NBA> as;
  CSrc<C::NBB> bs;
  init_rows(as, p.dz, m0, p.T, 2 * p.I, wave, lane);
  bs.init(p.gu, p.H, n0, p.H, wave, lane);
  mainloop<C, bf16x8_t>(as, bs, 2 * p.I, lds, acc, wave, lane);
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    const int row = m0 + wm * 32 * C::FM + 32 * i + (lane & 31);
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = acc[i][j][8 * q + e];
        const u32x4 o = pack_pair(v, v + 4);
        const int cc = n0 + (wn * C::FN + j) * 32 + 16 * q + 8 * (lane >> 5);
        if (row < p.T && cc < p.H) *(u32x4*)((uint16_t*)p.dx + (size_t)row * p.H + cc) = o;
      }
  }
}

// dW [M,N] = P^T Q over the T tokens: P [T,M], Q [T,N], both read along their
// rows with transposing LDS reads.  16384 x 4096 and 4096 x 8192 over 8192 tokens:
// 774 and 387 us (1421 TFLOP/s, matrix cores 85 and 83 % busy).
struct WgradArgs {
  const void *P, *Q;
  void* dw;
  int M, N, T, mt, nt;
};
template <class C, bool F32>
__global__ __launch_bounds__(256, 1) void ffn_wgrad_kernel(WgradArgs p) {
  FFN_PROLOGUE(C)
  CSrc<C::NBA> as;
  CSrc<C::NBB> bs;
  as.init(p.P, p.M, m0, p.M, wave, lane);
  bs.init(p.Q, p.N, n0, p.N, wave, lane);
  mainloop<C, bf16x8_t>(as, bs, p.T, lds, acc, wave, lane);
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    const int row = m0 + wm * 32 * C::FM + 32 * i + (lane & 31);
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = acc[i][j][8 * q + e];
        const int c = n0 + (wn * C::FN + j) * 32 + 16 * q;
        if constexpr (F32) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int ch = c + 8 * h + 4 * (lane >> 5);
            if (row < p.M && ch < p.N) store4<float>((float*)p.dw + (size_t)row * p.N + ch, v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
          }
        } else {
          const u32x4 o = pack_pair(v, v + 4);
          const int cc = c + 8 * (lane >> 5);
          if (row < p.M && cc < p.N) *(u32x4*)((uint16_t*)p.dw + (size_t)row * p.N + cc) = o;
        }
      }
  }
}

template <class C, bool F32>
hipError_t run_wgrad(const WgradArgs& p, const char* name, hipStream_t s) {
  const auto k = ffn_wgrad_kernel<C, F32>;
  return run_kernel(name, s, [&] { k<<<tile_grid(p.mt, p.nt), C::NT, 0, s>>>(p); });
}

hipError_t wgrad(WgradArgs p, bool f32, const char* name, hipStream_t s) {
  hipError_t e = hipSuccess;
  with_tile(tile_kind(p.M, p.N, p.T), [&](auto c) {
    using C = decltype(c);
    p.mt = (p.M + C::BM - 1) / C::BM;
    p.nt = (p.N + C::BN - 1) / C::BN;
    e = f32 ? run_wgrad<C, true>(p, name, s) : run_wgrad<C, false>(p, name, s);
  });
  return e;
}

}  // namespace dense

using namespace dense;

hipError_t launch_ffn_down_dgrad(FfnArgs p, hipStream_t s) {
  hipError_t e = hipSuccess;
  with_tile(tile_kind(p.T, p.I, p.H), [&](auto c) {
    using C = decltype(c);
    p.mt = (p.T + C::BM - 1) / C::BM;
    p.nt = (p.I + C::BN - 1) / C::BN;
    p.parts = 2 * p.nt;
    const auto k = p.act ? ffn_down_dgrad_kernel<C, 1> : ffn_down_dgrad_kernel<C, 0>;
    e = run_kernel("ffn_down_dgrad", s, [&] { k<<<tile_grid(p.mt, p.nt), C::NT, 0, s>>>(p); });
  });
  if (e != hipSuccess || !p.dgate) return e;
  return run_kernel("ffn_gate_reduce", s, [&] { ffn_gate_reduce_kernel<<<(p.T + 255) / 256, 256, 0, s>>>(p); });
}

hipError_t launch_ffn_gate_up_dgrad(FfnArgs p, hipStream_t s) {
  hipError_t e = hipSuccess;
  with_tile(tile_kind(p.T, p.H, 2 * p.I), [&](auto c) {
    using C = decltype(c);
    p.mt = (p.T + C::BM - 1) / C::BM;
    p.nt = (p.H + C::BN - 1) / C::BN;
    const auto k = ffn_gate_up_dgrad_kernel<C>;
    e = run_kernel("ffn_gate_up_dgrad", s, [&] { k<<<tile_grid(p.mt, p.nt), C::NT, 0, s>>>(p); });
  });
  return e;
}

hipError_t launch_ffn_wgrads(FfnArgs p, hipStream_t s) {
  const hipError_t e = wgrad({p.dout, p.aw, p.dwd, p.H, p.I, p.T, 0, 0}, p.grad_f32, "ffn_wgrad_down", s);
  if (e != hipSuccess) return e;
  return wgrad({p.dz, p.x, p.dgu, 2 * p.I, p.H, p.T, 0, 0}, p.grad_f32, "ffn_wgrad_gate_up", s);
}

}  // namespace moe
