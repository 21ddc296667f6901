// downs.h -- T [M x G R] = A_a x_m (fp32), the first half of the tokens' own
// adapters, for few tokens, as parts along K: a task is four rank rows, TT tokens
// (one, or four) and a slice of K, in fp32 dot products, one wave's work.  Tokens
// of one slot share the rows' loads; each other slot among the four is another
// pass.  A pass is mostly the latency of its loads: with a task for a whole
// workgroup of a streamed product, those that had one came 4 us after the others
// (8192 x 8192, 16 tokens of as many slots of rank 16: 22.0 us, 17.4 by waves).
#pragma once
#include "lds.h"
#include "pool.h"

namespace qlora {

constexpr int kDownRows = 4;
inline int64_t pool_down_tasks(int GR, int64_t M, int tt) { return (M + tt - 1) / tt * (GR / kDownRows); }   // G R % 8 == 0

// A wave's N sums over its lanes: afterwards lane l holds, in v[0], the sum whose
// number is the top bits of l (log2 N of them).  (By recursion: a loop that is not
// unrolled before its array is looked at would have the array put into LDS.)
template <int N, int O, int A>
__device__ __forceinline__ void wave_sums(float (&v)[A], int lane) {
  if constexpr (N > 1) {
    const bool up = (lane & O) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float keep = up ? v[i + N / 2] : v[i], give = up ? v[i] : v[i + N / 2];
      v[i] = keep + __shfl_xor(give, O);
    }
    wave_sums<N / 2, O / 2>(v, lane);
  } else if constexpr (O > 0) {
    v[0] += __shfl_xor(v[0], O);
    wave_sums<1, O / 2>(v, lane);
  }
}

// Task `task` of a wave: slice task % slices, `cols` columns (512 n) each, of the
// rest.  T [slices][M][G R]; a pool with scales has them in T.
template <int TT>
__device__ __forceinline__ void pool_down(const PoolView& p, const bf16_t* __restrict__ X, int64_t M, int64_t K,
                                          float* __restrict__ T, uint32_t task, uint32_t slices, uint32_t cols) {
  const uint32_t GR = (uint32_t)(p.G * p.R), per = GR / kDownRows;
  const uint32_t slice = task % slices, rest = task / slices;
  const int64_t m0 = (int64_t)(rest / per) * TT;
  const uint32_t j = rest % per * kDownRows, jr = j % (uint32_t)p.R;
  const int lane = threadIdx.x & 63;
  const int64_t k0 = (int64_t)slice * cols, k1 = min(K, k0 + cols);
  int slot[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) slot[i] = m0 + i < M ? __builtin_amdgcn_readfirstlane(slot_of(p, m0 + i)) : -1;
  float sum[TT * kDownRows];
#pragma unroll
  for (int i = 0; i < TT * kDownRows; ++i) sum[i] = 0.0f;
  bool any = false;
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
#pragma unroll 2
    for (int64_t kk = k0; kk < k1; kk += 512) {   // all lanes together; past the slice: zero
      const bool in = kk + 8 * lane < k1;
      const int64_t k = in ? kk + 8 * lane : k1 - 8;
      u32x4_t v[TT], b[kDownRows];
#pragma unroll
      for (int r = 0; r < kDownRows; ++r) b[r] = *reinterpret_cast<const u32x4_t*>(A + r * K + k);
#pragma unroll
      for (int i = 0; i < TT; ++i) v[i] = *reinterpret_cast<const u32x4_t*>(x[i] + k);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int r = 0; r < kDownRows; ++r) b[r][e] = in ? b[r][e] : 0u;
#pragma unroll
        for (int i = 0; i < TT; ++i) v[i][e] = in ? v[i][e] : 0u;
      }
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
      for (int r = 0; r < kDownRows; ++r) sum[i * kDownRows + r] = slot[i] == a ? s[i][r] : sum[i * kDownRows + r];
  }
  if (!any) return;
  wave_sums<TT * kDownRows, 32>(sum, lane);
  constexpr int kStep = 64 / (TT * kDownRows);   // lanes of a sum
  const int at = lane / kStep, i = at / kDownRows;
  if (lane % kStep == 0 && m0 + i < M) {
    const int a = slot_of(p, m0 + i);
    if (a >= 0 && jr < (uint32_t)rank_of(p, a))
      T[((int64_t)slice * M + m0 + i) * GR + j + at % kDownRows] = sum[0] * (p.scale ? p.scale[a] : 1.0f);
  }
}

}  // namespace qlora
