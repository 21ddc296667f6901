// pool.hip -- the adapters of many requests beside a shared projection:
//
//   T[m] = scale_a A_a x_m                 (a = the slot of token m)
//   Y[m] = Y0[m] + B_a T[m]                or, of a gated block's two weights,
//   H[m] = act(G0[m] + Bg_a Tg[m]) (P0[m] + Bu_a Tu[m])
//
// with Y0 the frozen product as fp32 parts of a split contraction.  One adapter
// for every token is a pool of one slot.
#include <algorithm>

#include "downs.h"
#include "gate.h"

namespace qlora {
namespace {

__global__ __launch_bounds__(256) void pool_down_kernel(PoolView p, const bf16_t* __restrict__ X, int64_t M, int64_t K,
                                                        float* __restrict__ T, bf16_t* __restrict__ U) {
  pool_down<4>(p, X, M, K, T, U, blockIdx.x);
}

// A thread takes one column of the result and TB tokens: the splits' parts in
// order, then its row of B times each token's T, 32 ranks of a run of tokens
// of one slot at a time (B's in registers, T's uniform).
template <int G, int TB>
__global__ __launch_bounds__(256) void pool_finish_kernel(PoolView p, const float* __restrict__ part, int splits,
                                                          int64_t M, int64_t N, const float* __restrict__ T, int act,
                                                          bf16_t* __restrict__ Y, bf16_t* __restrict__ GU) {
  const int tiles = (int)((N + 255) / 256);
  const int64_t n = (int64_t)(blockIdx.x % tiles) * 256 + threadIdx.x, m0 = (int64_t)(blockIdx.x / tiles) * TB, GN = G * N;
  const int GR = G * p.R, mt = (int)min((int64_t)TB, M - m0);
  if (n >= N) return;
  float acc[G][TB];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int i = 0; i < TB; ++i) acc[g][i] = 0.0f;
  for (int s = 0; s < splits; ++s)
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < TB; ++i)
        if (i < mt) acc[g][i] += part[((int64_t)s * M + m0 + i) * GN + g * N + n];
  for (int i0 = 0; p.R > 0 && i0 < mt;) {
    const int a = slot_of(p, m0 + i0);
    int i1 = i0 + 1;
    while (i1 < mt && slot_of(p, m0 + i1) == a) ++i1;
    const int r = a < 0 ? 0 : rank_of(p, a);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const bf16_t* b = p.B + ((int64_t)max(a, 0) * GN + g * N + n) * p.R;
      for (int j = 0; j < r; j += 8) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(b + j);
        float w[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[2 * e] = bf2f(v[e] & 0xFFFFu), w[2 * e + 1] = bf2f(v[e] >> 16);
#pragma unroll
        for (int i = 0; i < TB; ++i)
          if (i >= i0 && i < i1) {
            const float* t = T + (m0 + i) * GR + g * p.R + j;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[g][i] = fmaf(w[e], t[e], acc[g][i]);
          }
      }
    }
    i0 = i1;
  }
#pragma unroll
  for (int i = 0; i < TB; ++i)
    if (i < mt) {
      const int64_t m = m0 + i;
      if constexpr (G == 1) {
        Y[m * N + n] = (bf16_t)pack_bf16x2(acc[0][i], 0.0f);
      } else {
        Y[m * N + n] = (bf16_t)pack_bf16x2(gate_of(acc[0][i], acc[1][i], act), 0.0f);
        if (GU) {
          GU[m * GN + n] = (bf16_t)pack_bf16x2(acc[0][i], 0.0f);
          GU[m * GN + N + n] = (bf16_t)pack_bf16x2(acc[1][i], 0.0f);
        }
      }
    }
}

}  // namespace

hipError_t launch_pool_down(const PoolView& p, const bf16_t* X, int64_t M, int64_t K, float* T, bf16_t* U,
                            hipStream_t st) {
  hipLaunchKernelGGL(pool_down_kernel, dim3((unsigned)pool_down_blocks(p, M, 4)), dim3(256), 0, st, p, X, M, K, T, U);
  return hipGetLastError();
}

hipError_t launch_pool_finish(const PoolView& p, const float* part, int splits, int64_t M, int64_t N, const float* T,
                              int act, bf16_t* Y, bf16_t* GU, hipStream_t st) {
  constexpr int TB = 8;
  const dim3 grid((unsigned)((N + 255) / 256 * ((M + TB - 1) / TB)));
  if (p.G == 1)
    hipLaunchKernelGGL((pool_finish_kernel<1, TB>), grid, dim3(256), 0, st, p, part, splits, M, N, T, act, Y, GU);
  else
    hipLaunchKernelGGL((pool_finish_kernel<2, TB>), grid, dim3(256), 0, st, p, part, splits, M, N, T, act, Y, GU);
  return hipGetLastError();
}

}  // namespace qlora
