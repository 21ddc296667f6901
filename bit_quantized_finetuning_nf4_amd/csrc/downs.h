// downs.h -- T [M x G R] = scale_a A_a x_m (fp32), the first half of the tokens'
// own adapters, for few tokens: a task is four rank rows and TT tokens (one, or
// four), in fp32 dot products, the waves of a workgroup side by side along K.
// Tokens of one slot share the rows' loads; each other slot among the four is
// another pass.  A pass is mostly the latency of its loads, 3-5 us beside a
// product that streams at full rate.
#pragma once
#include "lds.h"
#include "pool.h"

namespace qlora {

constexpr int kDownRows = 4;
inline int pool_down_tasks(int GR, int64_t M, int tt) {
  return (int)((M + tt - 1) / tt) * (GR / kDownRows);   // G R % 8 == 0
}

// Task `task`; red holds 2 x WAVES x 16 floats of LDS, whose halves take turns:
// `turn` counts the workgroup's calls that returned true, those that used it.  U
// (may be null) is A_a x_m in bf16.
template <int WAVES, int TT>
__device__ __forceinline__ bool pool_down(const PoolView& p, const bf16_t* __restrict__ X, int64_t M, int64_t K,
                                          float* __restrict__ T, bf16_t* __restrict__ U, uint32_t task, uint32_t turn,
                                          float* red) {
  const uint32_t GR = (uint32_t)(p.G * p.R), per = GR / kDownRows;
  const int64_t m0 = (int64_t)(task / per) * TT;
  const uint32_t j = task % per * kDownRows, jr = j % (uint32_t)p.R;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  int slot[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) slot[i] = m0 + i < M ? __builtin_amdgcn_readfirstlane(slot_of(p, m0 + i)) : -1;
  float sum[TT][kDownRows];
#pragma unroll
  for (int i = 0; i < TT; ++i)
#pragma unroll
    for (int r = 0; r < kDownRows; ++r) sum[i][r] = 0.0f;
  bool any = false;
  constexpr int kUnroll = TT == 1 ? 4 : 2;
#pragma unroll
  for (int lead = 0; lead < TT; ++lead) {
    const int a = slot[lead];
    bool mine = a >= 0;
#pragma unroll
    for (int i = 0; i < lead; ++i) mine = mine && slot[i] != a;
    if (!mine || jr >= (uint32_t)rank_of(p, a)) continue;   // ranks come in eights
    any = true;
    // every load without a condition, so that all are in flight at once: a token
    // of another slot reads the leader's row, and its sums are dropped
    const bf16_t* A = p.A + ((int64_t)a * GR + j) * K;
    const bf16_t* x[TT];
    float s[TT][kDownRows];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      x[i] = X + (m0 + (slot[i] == a ? i : lead)) * K;
#pragma unroll
      for (int r = 0; r < kDownRows; ++r) s[i][r] = 0.0f;
    }
#pragma unroll kUnroll
    for (int64_t k = 8 * t; k < K; k += 512 * WAVES) {
      u32x4_t v[TT], b[kDownRows];
#pragma unroll
      for (int r = 0; r < kDownRows; ++r) b[r] = *reinterpret_cast<const u32x4_t*>(A + r * K + k);
#pragma unroll
      for (int i = 0; i < TT; ++i) v[i] = *reinterpret_cast<const u32x4_t*>(x[i] + k);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < TT; ++i) {
          const float lo = bf2f(v[i][e] & 0xFFFFu), hi = bf2f(v[i][e] >> 16);
#pragma unroll
          for (int r = 0; r < kDownRows; ++r) {
            s[i][r] = fmaf(bf2f(b[r][e] & 0xFFFFu), lo, s[i][r]);
            s[i][r] = fmaf(bf2f(b[r][e] >> 16), hi, s[i][r]);
          }
        }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int r = 0; r < kDownRows; ++r) sum[i][r] = slot[i] == a ? s[i][r] : sum[i][r];
  }
  if (!any) return false;   // the same in every wave
  float* mine = red + (turn & 1) * (WAVES * 16);
#pragma unroll
  for (int i = 0; i < TT; ++i)
    if (slot[i] >= 0) {
#pragma unroll
      for (int r = 0; r < kDownRows; ++r) {
        float s = sum[i][r];
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
        if (lane == 0) mine[w * 16 + 4 * i + r] = s;
      }
    }
  __syncthreads();
  const int i = t >> 2;
  if (t < 4 * TT && m0 + i < M) {
    const int a = slot_of(p, m0 + i);
    if (a >= 0 && jr < (uint32_t)rank_of(p, a)) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < WAVES; ++k) s += mine[k * 16 + t];
      const int64_t o = (m0 + i) * GR + j + (t & 3);
      T[o] = s * scale_of(p, a);
      if (U) U[o] = (bf16_t)pack_bf16x2(s, 0.0f);
    }
  }
  return true;
}

}  // namespace qlora
