// pool.hip -- the adapters of many requests beside a shared projection:
//
//   T[m] = scale_a A_a x_m                 (a = the slot of token m)
//   Y[m] = Y0[m] + B_a T[m]                or, of a gated block's two weights,
//   H[m] = act(G0[m] + Bg_a Tg[m]) (P0[m] + Bu_a Tu[m])
//
// with Y0 the frozen product as fp32 parts of a split contraction.  One adapter
// for every token is a pool of one slot.
#include <algorithm>

#include "gate.h"
#include "lds.h"
#include "pool.h"

namespace qlora {
namespace {

// A thread takes one column of the result and TB tokens: the parts in order,
// then its row of B times each token's T, the tokens of one slot sharing the row.
// LINE: the parts of a streamed product, at most `splits` of them, TB dividing its
// blocks of tokens, and T in `slices` parts; else T in one.  Mostly latency: T comes through LDS (as scalar loads, rank
// after rank, it took 2-4 us), and T, kR ranks of B and kP parts are asked for
// together, before it is known how many parts and ranks there are; what there is
// not is never used.
// 1 x 2 x 11008, rank 64 4.0 us; 32 tokens of as many slots of rank 16 beside 2 x
// 22016 rows 13 (17 MB of parts, 45 of B: 4.8 TB/s); 777 tokens mixed over 7 slots of
// rank 64, three parts of 5120 columns 25: the rows of B again for every eight tokens.
template <int G, int TB, bool LINE>
__global__ __launch_bounds__(256) void pool_finish_kernel(PoolView p, const float* __restrict__ part, int splits,
                                                          const int32_t* __restrict__ counts, StreamLine line, int64_t M,
                                                          int64_t N, const float* __restrict__ T, int slices, float scale,
                                                          bf16_t* __restrict__ U, int act, bf16_t* __restrict__ Y,
                                                          bf16_t* __restrict__ GU) {
  __shared__ __align__(16) float ts[TB * G * 128];   // [TB][G R]
  const uint32_t width = blockDim.x;   // columns: 64 or 256
  const uint32_t tiles = (uint32_t)((N + width - 1) / width), bm = blockIdx.x / tiles, bn = blockIdx.x - bm * tiles;
  const int64_t n = (int64_t)bn * width + threadIdx.x, m0 = (int64_t)bm * TB, GN = G * N;
  const int GR = G * p.R, mt = (int)min((int64_t)TB, M - m0);
  const int64_t nc = min(n, N - 1);
  constexpr int kR = TB == 1 ? 64 : 32, kP = TB == 1 ? 8 : TB == 2 ? 4 : 2;
  const uint32_t quads = (uint32_t)(mt * GR) / 4;
  // T: four of a row at a time, its parts in order
  auto load_t = [&](uint32_t e, float4 (&v)[kMaxSlices]) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kMaxSlices; ++k)
      if (LINE || k == 0) v[k] = *reinterpret_cast<const float4*>(T + ((int64_t)min(k, slices - 1) * M + m0) * GR + 4 * e);
  };
  float4 tv[kMaxSlices];
  if (threadIdx.x < quads) load_t(threadIdx.x, tv);
  // the slots of the tokens, and those not yet done
  int a[TB];
  uint32_t left = 0u;
#pragma unroll
  for (int i = 0; i < TB; ++i) {
    a[i] = p.R > 0 ? slot_of(p, min(m0 + i, M - 1)) : -1;
    if (a[i] >= 0 && i < mt) left |= 1u << i;
  }
  // ranks j0 .. of the rows of slot s
  u32x4_t v[G][kR / 8];
  auto load_b = [&](int s, int j0) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int q = 0; q < kR / 8; ++q)
        if (j0 + 8 * q < p.R)
          v[g][q] = *reinterpret_cast<const u32x4_t*>(p.B + ((int64_t)s * GN + g * N + nc) * p.R + j0 + 8 * q);
  };
  if (p.R > 0) load_b(max(a[0], 0), 0);
  int cnt[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    cnt[g] = splits;
    if constexpr (LINE) {
      static_assert(kStreamRows % 256 == 0, "a workgroup's columns are one tile's");
      cnt[g] = counts[((uint32_t)m0 / line.block * G + g) * line.tiles + (bn * width) / kStreamRows];
    }
  }
  float acc[G][TB], x[G][kP][TB];
  auto load_parts = [&](int g, int s0) __attribute__((always_inline)) {
    const float* src = part + m0 * GN + g * N + nc;
#pragma unroll
    for (int k = 0; k < kP; ++k)
#pragma unroll
      for (int i = 0; i < TB; ++i)
        x[g][k][i] = src[((int64_t)min(s0 + k, splits - 1) * M + min(i, mt - 1)) * GN];
  };
#pragma unroll
  for (int g = 0; g < G; ++g) load_parts(g, 0);
  auto put_t = [&](uint32_t e, const float4 (&v)[kMaxSlices]) __attribute__((always_inline)) {
    float4 t = v[0];
#pragma unroll
    for (int k = 1; k < kMaxSlices; ++k)
      if (LINE && k < slices) t = make_float4(t.x + v[k].x, t.y + v[k].y, t.z + v[k].z, t.w + v[k].w);
    *reinterpret_cast<float4*>(ts + 4 * e) = make_float4(t.x * scale, t.y * scale, t.z * scale, t.w * scale);
    if (U && bn == 0)
      *reinterpret_cast<uint2*>(U + m0 * GR + 4 * e) = make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
  };
  if (threadIdx.x < quads) put_t(threadIdx.x, tv);
  for (uint32_t e = threadIdx.x + width; e < quads; e += width) {
    load_t(e, tv);
    put_t(e, tv);
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int i = 0; i < TB; ++i) acc[g][i] = 0.0f;
    for (int s0 = 0; s0 < cnt[g]; s0 += kP) {
      if (s0 > 0) load_parts(g, s0);
#pragma unroll
      for (int k = 0; k < kP; ++k)
#pragma unroll
        for (int i = 0; i < TB; ++i) acc[g][i] = s0 + k < cnt[g] ? acc[g][i] + x[g][k][i] : acc[g][i];
    }
  }
  __syncthreads();
  for (bool first = true; left != 0u; first = false) {
    const int lead = __builtin_ctz(left), s = slot_of(p, m0 + lead), r = rank_of(p, s);
    uint32_t set = 0u;   // the tokens of this slot
#pragma unroll
    for (int i = 0; i < TB; ++i) set |= a[i] == s ? 1u << i : 0u;
    set &= left;
    for (int j0 = 0; j0 < r; j0 += kR) {
      if (!first || lead > 0 || j0 > 0) load_b(s, j0);
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
            if (set >> i & 1u) {
              const float4* t = reinterpret_cast<const float4*>(ts + i * GR + g * p.R + j0 + 8 * q);
              const float4 t0 = t[0], t1 = t[1];
              const float y[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[g][i] = fmaf(w[e], y[e], acc[g][i]);
            }
        }
    }
    left &= ~set;
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

// After a streamed product a thread takes as few tokens as fill the card, and more
// at higher ranks, whose rows of B weigh more than the parts: 209 tokens of 2256
// features at rank 128 17.7 us with one token, 11.6 with four.
hipError_t launch_pool_finish(const PoolView& p, const float* part, int splits, const int32_t* counts,
                              const StreamLine* line, int64_t M, int64_t N, const float* T, int slices, float scale,
                              bf16_t* U, int act, bf16_t* Y, bf16_t* GU, hipStream_t st) {
  const int64_t tiles = (N + 255) / 256;
  const unsigned width = tiles * M < 1024 ? 64 : 256;
  auto go = [&](auto* fn, int tb) {
    hipLaunchKernelGGL(fn, dim3((unsigned)((N + width - 1) / width * ((M + tb - 1) / tb))), dim3(width), 0, st, p, part,
                       splits, counts, line ? *line : StreamLine{}, M, N, T, slices, scale, U, act, Y, GU);
    return hipGetLastError();
  };
  const int64_t work = tiles * M * std::max(1, p.G * p.R / 32) / 1024;
  if (!line) return p.G == 1 ? go(&pool_finish_kernel<1, 8, false>, 8) : go(&pool_finish_kernel<2, 8, false>, 8);
  if (p.G == 1)
    return work >= 8   ? go(&pool_finish_kernel<1, 8, true>, 8)
           : work >= 4 ? go(&pool_finish_kernel<1, 4, true>, 4)
           : work >= 2 ? go(&pool_finish_kernel<1, 2, true>, 2)
                       : go(&pool_finish_kernel<1, 1, true>, 1);
  return work >= 8   ? go(&pool_finish_kernel<2, 8, true>, 8)
         : work >= 4 ? go(&pool_finish_kernel<2, 4, true>, 4)
         : work >= 2 ? go(&pool_finish_kernel<2, 2, true>, 2)
                     : go(&pool_finish_kernel<2, 1, true>, 1);
}

}  // namespace qlora
