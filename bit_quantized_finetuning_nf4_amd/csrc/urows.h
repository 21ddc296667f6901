// urows.h -- U = drop(X) A^T for few tokens or a small rank, without partial
// sums: a workgroup takes one rank row and up to four tokens and forms their
// fp32 dot products, each thread over every 256th group of eight columns.  A
// is read once per four tokens and X r times (from L2), so it pays while M K r
// is small; past that the MFMA product with split partials does (gemm.hip), a
// launch more, the partials' sum riding with the next one (ride.h) as this does.
// Four tokens: with 16 a workgroup brings 256 KiB at K
// = 8192 (16 tokens at rank 64 with their quantization and product: 15.8 us
// with four, 19.1 with eight, 26 with 16, 22.6 by MFMA).
#pragma once
#include "rng.h"

namespace qlora {

constexpr int kURowTokens = 4;

// What the bf16 h leaves of v; nothing where h is not finite (an infinity minus
// itself would make the gradient NaN where its sum is infinite).
__device__ __forceinline__ float rest_of(float v, uint32_t h) {
  return (h & 0x7F80u) == 0x7F80u ? 0.0f : v - bf2f(h);
}

template <bool DROP>
__device__ __forceinline__ void u_rows(const bf16_t* __restrict__ X, int64_t M, int64_t K, const bf16_t* __restrict__ A,
                                       int r, int block, bf16_t* __restrict__ U, bf16_t* __restrict__ parts, float s,
                                       const DropArgs& drop) {
  __shared__ float part[4][kURowTokens];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int j = block % r, m0 = block / r * kURowTokens;
  const int mt = min(kURowTokens, (int)M - m0);
  const int groups = (int)(K >> 3);
  [[maybe_unused]] DropKey key;
  if constexpr (DROP) key = drop_key(drop);
  float sum[kURowTokens];
#pragma unroll
  for (int i = 0; i < kURowTokens; ++i) sum[i] = 0.0f;
  // two groups of columns a turn, all their loads issued together
  for (int g0 = t; g0 < groups; g0 += 512) {
    uint4 a[2];
    u32x4_t x[2][kURowTokens];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int g = min(g0 + 256 * u, groups - 1);
      a[u] = reinterpret_cast<const uint4*>(A + (int64_t)j * K)[g];
#pragma unroll
      for (int i = 0; i < kURowTokens; ++i)
        x[u][i] = *reinterpret_cast<const u32x4_t*>(X + min((int64_t)m0 + i, M - 1) * K + 8 * g);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int g = g0 + 256 * u;
      if (g >= groups) break;
      const float a0 = bf2f(a[u].x & 0xFFFFu), a1 = bf2f(a[u].x >> 16), a2 = bf2f(a[u].y & 0xFFFFu),
                  a3 = bf2f(a[u].y >> 16), a4 = bf2f(a[u].z & 0xFFFFu), a5 = bf2f(a[u].z >> 16),
                  a6 = bf2f(a[u].w & 0xFFFFu), a7 = bf2f(a[u].w >> 16);
#pragma unroll
      for (int i = 0; i < kURowTokens; ++i)
        if (i < mt) {
          u32x4_t v = x[u][i];
          if constexpr (DROP) v = drop8(v, (uint32_t)(m0 + i) * (uint32_t)groups + (uint32_t)g, key);   // M K < 2^31
          float y = sum[i];
          y = fmaf(a0, bf2f(v.x & 0xFFFFu), y);
          y = fmaf(a1, bf2f(v.x >> 16), y);
          y = fmaf(a2, bf2f(v.y & 0xFFFFu), y);
          y = fmaf(a3, bf2f(v.y >> 16), y);
          y = fmaf(a4, bf2f(v.z & 0xFFFFu), y);
          y = fmaf(a5, bf2f(v.z >> 16), y);
          y = fmaf(a6, bf2f(v.w & 0xFFFFu), y);
          sum[i] = fmaf(a7, bf2f(v.w >> 16), y);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < kURowTokens; ++i)
    if (i < mt) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) sum[i] += __shfl_xor(sum[i], o);
      if (lane == 0) part[w][i] = sum[i];
    }
  __syncthreads();
  if (t < mt) {
    float v = (part[0][t] + part[1][t]) + (part[2][t] + part[3][t]);
    if constexpr (DROP) v *= drop.scale;
    const int64_t o = (int64_t)(m0 + t) * r + j;
    if (U) U[o] = (bf16_t)pack_bf16x2(v, 0.0f);
    v *= s;
#pragma unroll
    for (int k = 0; k < kTermParts; ++k)
      if (parts) {
        const uint32_t p = pack_bf16x2(v, 0.0f) & 0xFFFFu;
        parts[(int64_t)k * M * r + o] = (bf16_t)p;
        v = rest_of(v, p);
      }
  }
}

inline int u_rows_blocks(int64_t M, int r) { return r * (int)((M + kURowTokens - 1) / kURowTokens); }
// Where that takes less than the MFMA product: a workgroup's loads, and under
// the mask its Philox blocks, grow with M K r, the MFMA product's launch and
// its walk along K do not.  Fitted to both at 170 sizes each, 1 to 512 tokens,
// K 1024 to 22016, ranks 8 to 128, where it is within 0.1 % of the faster on
// the mean.  With the tokens' quantization and a 64-channel product, in us,
// here and by MFMA (then under the mask):
//    16 x  4096 r  64  10.2 12.6 (10.9 14.3)    128 x  4096 r 64  15.6 15.6 (20.7 17.4)
//     1 x 22016 r 128  15.6 22.5 (16.0 27.5)    256 x 12288 r 32  25.4 20.1 (37.9 23.7)
//   512 x  1024 r   8   9.3 10.8 (10.0 11.9)    512 x 22016 r 16  45.5 28.7 (58.3 32.0)
inline bool u_rows_ok(int64_t M, int64_t K, int r, bool drop) {
  if (M > 512) return false;
  return drop ? M * K * (r + 8) <= 14000000 + 2000 * K : M * K * (r + 10) <= 14000000 + 3400 * K;
}

}  // namespace qlora
