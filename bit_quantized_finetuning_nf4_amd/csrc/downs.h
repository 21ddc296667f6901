// downs.h -- T [M x G R] = scale_a A_a x_m (fp32), the tokens' own adapters'
// first half, for few tokens: a workgroup of WAVES waves takes one token and two
// rank rows of its slot a wave, in fp32 dot products.
#pragma once
#include "lds.h"
#include "pool.h"

namespace qlora {

inline int pool_down_blocks(const PoolView& p, int64_t M, int waves) {
  return (int)(M * ((p.G * p.R + 2 * waves - 1) / (2 * waves)));
}

// Workgroup `block`; U (may be null) is A_a x_m in bf16.
template <int WAVES>
__device__ __forceinline__ void pool_down(const PoolView& p, const bf16_t* __restrict__ X, int64_t M, int64_t K,
                                          float* __restrict__ T, bf16_t* __restrict__ U, int block) {
  const int GR = p.G * p.R, per = (GR + 2 * WAVES - 1) / (2 * WAVES);
  const int64_t m = block / per;
  const int t = threadIdx.x, lane = t & 63, j = (block % per) * 2 * WAVES + 2 * (t >> 6);
  if (j >= GR) return;
  const int a = slot_of(p, m);
  if (a < 0 || j % p.R >= rank_of(p, a)) return;   // ranks come in eights: both rows of a wave, or neither
  const bf16_t* A = p.A + ((int64_t)a * GR + j) * K;
  const bf16_t* x = X + m * K;
  float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 4
  for (int64_t k = 8 * lane; k < K; k += 512) {
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(x + k), a0 = *reinterpret_cast<const u32x4_t*>(A + k),
                  a1 = *reinterpret_cast<const u32x4_t*>(A + K + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = bf2f(v[e] & 0xFFFFu), hi = bf2f(v[e] >> 16);
      s0 = fmaf(bf2f(a0[e] & 0xFFFFu), lo, s0), s0 = fmaf(bf2f(a0[e] >> 16), hi, s0);
      s1 = fmaf(bf2f(a1[e] & 0xFFFFu), lo, s1), s1 = fmaf(bf2f(a1[e] >> 16), hi, s1);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s0 += __shfl_xor(s0, o), s1 += __shfl_xor(s1, o);
  if (lane < 2) {
    const float v = lane ? s1 : s0;
    const int64_t o = m * GR + j + lane;
    T[o] = v * scale_of(p, a);
    if (U) U[o] = (bf16_t)pack_bf16x2(v, 0.0f);
  }
}

}  // namespace qlora
