// gemm_i8.hip -- the product of 8-bit integers with one scale per token and
// one per output channel, and the LoRA tail:
//
//   Y[m][n] = sx[m] sw[n] sum_k Xq[m][k] Wq[n][k] + s sum_j U[m][j] B[n][j]
//
// The sum over k is exact: products of integers up to 127 in 32-bit sums, no
// overflow for K <= 131072 (127^2 K < 2^31).  It is rounded to fp32 when it
// is multiplied by the scales, and the adapter's product is added in fp32.
//
// The tile is the dense bf16 GEMM's (dense_tile.h): the operands stream the
// same bytes per MFMA, and each 32x32x32 integer MFMA does twice the work of
// the 32x32x16 bf16 one.  After the loop the sums become fp32 in the
// registers that held them.
#include <algorithm>

#include "dense_tile.h"

namespace qlora {
namespace {

// Integer sums of the tile to fp32, times both scales (lane layout of
// store_tile_lds).  Tokens and channels past the end take scale 0.
template <int FI>
__device__ __forceinline__ void scale_tile(const i32x16_t (&acc)[FI][4], f32x16_t (&out)[FI][4],
                                           const float* __restrict__ sx, const float* __restrict__ sw, int64_t M,
                                           int64_t N, int64_t m0, int64_t n0) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wr = w >> 1, wc = w & 1, lr = lane & 31, h = lane >> 5;
  float x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t m = m0 + 128 * wr + 32 * j + lr;
    x[j] = m < M ? sx[m] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t n = n0 + 32 * FI * wc + 32 * i + 8 * q + 4 * h;   // N % 8 == 0
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (n < N) v = *reinterpret_cast<const float4*>(sw + n);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        out[i][j][4 * q] = (float)acc[i][j][4 * q] * (x[j] * v.x);
        out[i][j][4 * q + 1] = (float)acc[i][j][4 * q + 1] * (x[j] * v.y);
        out[i][j][4 * q + 2] = (float)acc[i][j][4 * q + 2] * (x[j] * v.z);
        out[i][j][4 * q + 3] = (float)acc[i][j][4 * q + 3] * (x[j] * v.w);
      }
    }
}

// out += B (s U)^T over the rank, 32 at a time through 64-byte-row tiles, one
// chunk loaded into registers while the one before is multiplied.
template <int FI>
__device__ __forceinline__ void lora_tail(f32x16_t (&acc)[FI][4], const bf16_t* B, const bf16_t* U, int r, float s,
                                          int64_t M, int64_t N, int64_t m0, int64_t n0, char* smem) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wr = w >> 1, wc = w & 1;
  const FragOffs fo = frag_offs(lane);
  const int am64 = wc * 32 * FI * 64, bm64 = wr * 128 * 64;
  const int nt = (r + 31) / 32;
  TailRegs R;
  tail_load(R, B, false, N, r, n0, 0, 0, N, U, r, M, m0);
  for (int c = 0; c < nt; ++c) {
    char* buf = smem + (c & 1) * 2 * kOp;
    tail_store(buf, R, false, s);
    if (c + 1 < nt) tail_load(R, B, false, N, r, n0, 32 * (c + 1), 0, N, U, r, M, m0);
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int o = kk ? fo.o1 : fo.o0;
      bf16x8_t a[FI], b[4];
#pragma unroll
      for (int i = 0; i < FI; ++i) a[i] = rd16(buf + am64 + i * 2048 + o);
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = rd16(buf + kOp + bm64 + i * 2048 + o);
      mfma_block<FI, 4>(acc, a, b);
    }
  }
}

// Xq [M x ld], Wq [N x ld] bytes, ld = 128 npair_all; tiles of 64 FI channels
// x 256 tokens from channel n_begin on.
template <int FI>
__global__ __launch_bounds__(kThreads, 1) void i8_gemm_kernel(const int8_t* __restrict__ Wq,
                                                              const float* __restrict__ sw, int64_t N, int64_t ld,
                                                              const int8_t* __restrict__ Xq,
                                                              const float* __restrict__ sx, int64_t M,
                                                              const bf16_t* __restrict__ U,
                                                              const bf16_t* __restrict__ B, int r, float s,
                                                              bf16_t* __restrict__ Y, int64_t n_begin, int tiles_n,
                                                              int tiles_m) {
  extern __shared__ __align__(16) char smem[];
  int tn, tm;
  map_tile_grouped(xcd_tile_id(), tiles_n, tiles_m, tn, tm);
  const int64_t n0 = n_begin + (int64_t)tn * 64 * FI, m0 = (int64_t)tm * kTile;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6, wr = wv >> 1, wc = wv & 1;

  DenseOps f;
  f.w = __builtin_amdgcn_readfirstlane(wv);
  __builtin_assume(f.w >= 0 && f.w < 4);
  f.npair = (int)(ld >> 7);
  f.wr_ = make_rsrc(Wq, (uint32_t)(N * ld));
  f.xr = make_rsrc(Xq, (uint32_t)(M * ld));
  {
    const int c = (lane & 7) ^ ((4 * f.w + (lane >> 4)) & 7);   // see bf16_fwd_kernel
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      // rows past the end re-read the last row, never stored
      const int row = 8 * (4 * q + f.w) + (lane >> 3);
      if (q < 2 * FI) f.wo[q] = (uint32_t)(min(n0 + row, N - 1) * ld + c * 16);
      f.xo[q] = (uint32_t)(min(m0 + row, M - 1) * ld + c * 16);
    }
  }
  PairOffs po;
  {
    const int lr = lane & 31, h = lane >> 5;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) po.o[hf][kk] = pos128(lr, 4 * hf + 2 * kk + h);
  }
  const int am = wc * 32 * FI * 128, bm = wr * 128 * 128;

  i32x16_t acc[FI][4];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

#pragma unroll
  for (int d = 0; d < 2 * FI + 8; ++d) {
    pair_dma<FI>(smem, f, 0, d);
    pair_dma<FI>(smem + kPairSlot, f, 1, d);
  }
  QLORA_WAIT(0, 0);
  __builtin_amdgcn_s_barrier();
  Frags F;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < FI) F.a0[i] = rd16(smem + am + i * 32 * 128 + po.o[0][0]);
    F.b0[i] = rd16(smem + kPairOp + bm + i * 32 * 128 + po.o[0][0]);
  }
  for (int pr = 0; pr < f.npair; ++pr) {
    char* cur = smem + (pr & 1) * kPairSlot;
    char* nxt = smem + ((pr & 1) ^ 1) * kPairSlot;
    __builtin_amdgcn_sched_barrier(0);
    dense_slots<MmI8, FI, 0, 0>(cur, nxt, cur, f, pr, acc, F, am, bm, po);
    __builtin_amdgcn_sched_barrier(0);
    dense_slots<MmI8, FI, 1, 0>(cur, nxt, cur, f, pr, acc, F, am, bm, po);
  }
  // drain the DMAs still in flight (clamped re-loads) before reusing LDS
  QLORA_WAIT(0, 0);
  __builtin_amdgcn_s_barrier();

  f32x16_t out[FI][4];
  scale_tile<FI>(acc, out, sx, sw, M, N, m0, n0);
  if (r > 0) lora_tail<FI>(out, B, U, r, s, M, N, m0, n0, smem);
  store_tile_lds<FI>(out, Y, N, M, N, m0, n0, smem);
}

template <int FI>
hipError_t launch_fi(const I8Gemm& g, int64_t n_begin, int64_t n_rows, hipStream_t st) {
  const int tiles_n = (int)((n_rows + 64 * FI - 1) / (64 * FI)), tiles_m = (int)((g.M + kTile - 1) / kTile);
  auto* fn = &i8_gemm_kernel<FI>;
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), (int)kLdsPairs);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3(tiles_n * tiles_m), dim3(kThreads), kLdsPairs, st, g.Wq, g.sw, g.N, i8_row_bytes(g.K),
                     g.Xq, g.sx, g.M, g.U, g.B, g.r, g.s, g.Y, n_begin, tiles_n, tiles_m);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_gemm(const I8Gemm& g, hipStream_t st) { return launch_fi<4>(g, 0, g.N, st); }

}  // namespace qlora
