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
  __shared__ float red[2 * 4 * 16];
  pool_down<4, 4>(p, X, M, K, T, U, blockIdx.x, 0, red);
}

// A thread takes one column of the result and TB tokens: the parts in order,
// then its row of B times each token's T (uniform: scalar loads), a run of tokens
// of one slot sharing the row.  LINE: the parts of a streamed product, TB dividing
// its blocks of tokens.  Mostly latency: the loads of kR ranks of B and of kP
// parts are issued together.
template <int G, int TB, bool LINE>
__global__ __launch_bounds__(256) void pool_finish_kernel(PoolView p, const float* __restrict__ part, int splits,
                                                          const int32_t* __restrict__ counts, StreamLine line, int64_t M,
                                                          int64_t N, const float* __restrict__ T, int act,
                                                          bf16_t* __restrict__ Y, bf16_t* __restrict__ GU) {
  const uint32_t width = blockDim.x;   // columns: 64 or 256
  const uint32_t tiles = (uint32_t)((N + width - 1) / width), bm = blockIdx.x / tiles, bn = blockIdx.x - bm * tiles;
  const int64_t n = (int64_t)bn * width + threadIdx.x, m0 = (int64_t)bm * TB, GN = G * N;
  const int GR = G * p.R, mt = (int)min((int64_t)TB, M - m0);
  const int64_t nc = min(n, N - 1);
  constexpr int kR = TB == 1 ? 64 : 32, kP = TB == 1 ? 8 : TB == 2 ? 4 : LINE ? 2 : 1;
  int cnt[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    cnt[g] = splits;
    if constexpr (LINE) {
      static_assert(kStreamRows % 256 == 0, "a workgroup's columns are one tile's");
      cnt[g] = counts[((uint32_t)m0 / line.block * G + g) * line.tiles + (bn * width) / kStreamRows];
    }
  }
  float acc[G][TB];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int i = 0; i < TB; ++i) acc[g][i] = 0.0f;
  // the term of tokens i0 .. i1 - 1, of slot a and rank r: ranks j0 ..
  u32x4_t v[G][kR / 8];
  auto load_b = [&](int a, int r, int j0) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int q = 0; q < kR / 8; ++q) {
        v[g][q] = u32x4_t{0u, 0u, 0u, 0u};
        if (j0 + 8 * q < r)
          v[g][q] = *reinterpret_cast<const u32x4_t*>(p.B + ((int64_t)a * GN + g * N + nc) * p.R + j0 + 8 * q);
      }
  };
  auto term = [&](int i0, int i1, int r, int j0) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int q = 0; q < kR / 8; ++q) {
        if (j0 + 8 * q >= r) break;
        float w[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[2 * e] = bf2f(v[g][q][e] & 0xFFFFu), w[2 * e + 1] = bf2f(v[g][q][e] >> 16);
#pragma unroll
        for (int i = 0; i < TB; ++i)
          if (i >= i0 && i < i1) {
            const float* t = T + (m0 + i) * GR + g * p.R + j0 + 8 * q;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[g][i] = fmaf(w[e], t[e], acc[g][i]);
          }
      }
  };
  // the first slot's rows are asked for before the parts
  int a = p.R > 0 ? slot_of(p, m0) : -1, r = a < 0 ? 0 : rank_of(p, a);
  load_b(max(a, 0), r, 0);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const float* src = part + m0 * GN + g * N + nc;
    for (int s0 = 0; s0 < cnt[g]; s0 += kP) {
      float x[kP][TB];
#pragma unroll
      for (int k = 0; k < kP; ++k)
#pragma unroll
        for (int i = 0; i < TB; ++i) {
          x[k][i] = 0.0f;
          if (s0 + k < cnt[g] && i < mt) x[k][i] = src[((int64_t)(s0 + k) * M + i) * GN];
        }
#pragma unroll
      for (int k = 0; k < kP; ++k)
#pragma unroll
        for (int i = 0; i < TB; ++i) acc[g][i] += x[k][i];
    }
  }
  if (p.R > 0) {
    for (int i0 = 0;;) {
      int i1 = i0 + 1;
      while (i1 < mt && slot_of(p, m0 + i1) == a) ++i1;
      term(i0, i1, r, 0);
      for (int j0 = kR; j0 < r; j0 += kR) {
        load_b(a, r, j0);
        term(i0, i1, r, j0);
      }
      if ((i0 = i1) >= mt) break;
      a = slot_of(p, m0 + i0), r = a < 0 ? 0 : rank_of(p, a);
      load_b(max(a, 0), r, 0);
    }
  }
  if (n >= N) return;
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
  hipLaunchKernelGGL(pool_down_kernel, dim3((unsigned)pool_down_tasks(p.G * p.R, M, 4)), dim3(256), 0, st, p, X, M, K, T,
                     U);
  return hipGetLastError();
}

// After a streamed product a thread takes as few tokens as fill the card.
hipError_t launch_pool_finish(const PoolView& p, const float* part, int splits, const int32_t* counts,
                              const StreamLine* line, int64_t M, int64_t N, const float* T, int act, bf16_t* Y,
                              bf16_t* GU, hipStream_t st) {
  const int64_t tiles = (N + 255) / 256;
  const unsigned width = tiles * M < 1024 ? 64 : 256;
  auto go = [&](auto* fn, int tb) {
    hipLaunchKernelGGL(fn, dim3((unsigned)((N + width - 1) / width * ((M + tb - 1) / tb))), dim3(width), 0, st, p, part, splits, counts,
                       line ? *line : StreamLine{}, M, N, T, act, Y, GU);
    return hipGetLastError();
  };
  const int tb = !line ? 8 : tiles * M >= 4 * 1024 ? 4 : tiles * M >= 2 * 1024 ? 2 : 1;
  if (p.G == 1)
    return tb == 8   ? go(&pool_finish_kernel<1, 8, false>, 8)
           : tb == 4 ? go(&pool_finish_kernel<1, 4, true>, 4)
           : tb == 2 ? go(&pool_finish_kernel<1, 2, true>, 2)
                     : go(&pool_finish_kernel<1, 1, true>, 1);
  return tb == 8   ? go(&pool_finish_kernel<2, 8, false>, 8)
         : tb == 4 ? go(&pool_finish_kernel<2, 4, true>, 4)
         : tb == 2 ? go(&pool_finish_kernel<2, 2, true>, 2)
                   : go(&pool_finish_kernel<2, 1, true>, 1);
}

}  // namespace qlora
