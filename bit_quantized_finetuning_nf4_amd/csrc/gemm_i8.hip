// gemm_i8.hip -- the product of 8-bit integers with one scale per token and
// one per output channel, and the LoRA tail:
//
//   Y[m][n] = sx[m] sw[n] sum_k Xq[m][k] Wq[n][k] + sum_j T[m][j] B[n][j]
//
// with T = s U as kTermParts bf16 matrices.
//
// The sum over k is exact: products of integers up to 127 in 32-bit sums, no
// overflow for K <= 131072 (127^2 K < 2^31); a split contraction leaves its
// parts as integers, which the sum kernel adds.  It is rounded to fp32 when it
// is multiplied by the scales, and the adapter's product is added in fp32.
//
// The tile is the dense bf16 GEMM's (dense_tile.h): the operands stream the
// same bytes per MFMA, and each 32x32x32 integer MFMA does twice the work of
// the 32x32x16 bf16 one.  After the loop the sums become fp32 in the
// registers that held them.  Bound by the lines a CU keeps in flight and by
// power: 4096 x 22016 x 8192 at rank 64 runs at 2.2 POPS (five whole rounds of
// 256 x 256 tiles 590 us and 1536 channels on 256 x 128 79 us); random operands
// in registers alone reach 3.4, the library's product of 16384^3 2.4.
#include <algorithm>
#include <cmath>

#include "dense_tile.h"

namespace qlora {
namespace {

// The scales of the tile's channels (1 KiB) and tokens (1 KiB) lie past the
// pair slots, DMA'd in the prologue, 0 past the end.
constexpr int kLdsScales = 2048;
__device__ __forceinline__ void scales_dma(char* dst, const float* sx, const float* sw, int64_t M, int64_t N, int64_t m0,
                                           int64_t n0, int w, int lane) {
  if (w == 0) dma16(make_rsrc(sw, (uint32_t)(N * 4)), dst, (uint32_t)((n0 + 4 * lane) * 4), 0u);
  if (w == 1) dma16(make_rsrc(sx, (uint32_t)(M * 4)), dst + 1024, (uint32_t)((m0 + 4 * lane) * 4), 0u);
}
// Integer sums of the tile to fp32, times both scales (lane layout of
// store_tile_lds).
template <int FI>
__device__ __forceinline__ void scale_tile(const i32x16_t (&acc)[FI][4], f32x16_t (&out)[FI][4], const char* scales) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wr = w >> 1, wc = w & 1, lr = lane & 31, h = lane >> 5;
  const float* sw = reinterpret_cast<const float*>(scales);
  const float* sx = reinterpret_cast<const float*>(scales + 1024);
  float x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = sx[128 * wr + 32 * j + lr];
#pragma unroll
  for (int i = 0; i < FI; ++i) {
    f32x4_t v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const f32x4_t*>(sw + 32 * FI * wc + 32 * i + 8 * q + 4 * h);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // through 16 vector registers, back into the accumulator registers that
      // held the sums: without the moves the compiler keeps the values in
      // vector registers, which spills
      float f[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] = scaled_sum(acc[i][j][e], v[e >> 2][e & 3], x[j]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float t;
        asm volatile("v_accvgpr_write_b32 %0, %1" : "=a"(t) : "v"(f[e]));
        out[i][j][e] = t;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// acc += the chunk at buf (weights at buf, tokens at buf + kOp).
template <int FI>
__device__ __forceinline__ void tail_mul(f32x16_t (&acc)[FI][4], const char* buf) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wr = w >> 1, wc = w & 1;
  const FragOffs fo = frag_offs(lane);
  const int am64 = wc * 32 * FI * 64, bm64 = wr * 128 * 64;
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

// acc += B T^T over the ranks of the parts, 32 at a time through 64-byte-row
// tiles, one chunk loaded into registers while the one before is multiplied.
template <int FI>
__device__ __forceinline__ void lora_tail(f32x16_t (&acc)[FI][4], const bf16_t* B, const bf16_t* T, int r, int64_t M,
                                          int64_t N, int64_t m0, int64_t n0, char* smem) {
  const int nt = (kTermParts * r + 31) / 32;
  TailRegs R;
  auto load = [&](int c) { tail_load_parts(R, B, false, N, r, n0, 32 * c, T, M, m0); };
  load(0);
  for (int c = 0; c < nt; ++c) {
    char* buf = smem + (c & 1) * 2 * kOp;
    tail_store(buf, R, false, 1.0f);
    if (c + 1 < nt) load(c + 1);
    __syncthreads();
    tail_mul<FI>(acc, buf);
  }
}

// Xq [M x ld], Wq [N x ld] bytes, whole 128-byte pairs; tiles of 64 FI channels
// x 256 tokens from channel n_begin on.  part != null: the grid holds the tiles
// once per split of the contraction, pps pairs each, and their integer sums go
// to part + split M N, the rest being the sum kernel's.
// TD: the LoRA tail by DMA.
template <int FI, bool TD>
__global__ __launch_bounds__(kThreads, 1) void i8_gemm_kernel(const int8_t* __restrict__ Wq,
                                                              const float* __restrict__ sw, int64_t N, int64_t ld,
                                                              const int8_t* __restrict__ Xq,
                                                              const float* __restrict__ sx, int64_t M,
                                                              const bf16_t* __restrict__ T,
                                                              const bf16_t* __restrict__ B, int r,
                                                              bf16_t* __restrict__ Y, int64_t n_begin, int tiles_n,
                                                              int tiles_m, int pps, int32_t* __restrict__ part) {
  extern __shared__ __align__(16) char smem[];
  int tn, tm;
  const int id = xcd_tile_id(), split = id / (tiles_n * tiles_m), p0 = split * pps;
  map_tile_grouped(id - split * tiles_n * tiles_m, tiles_n, tiles_m, tn, tm);
  const int64_t n0 = n_begin + (int64_t)tn * 64 * FI, m0 = (int64_t)tm * kTile;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6, wr = wv >> 1, wc = wv & 1;

  DenseOps f;
  f.w = __builtin_amdgcn_readfirstlane(wv);
  __builtin_assume(f.w >= 0 && f.w < 4);
  f.npair = min((int)(ld >> 7) - p0, pps);
  f.wr_ = make_rsrc(Wq, (uint32_t)(N * ld));
  f.xr = make_rsrc(Xq, (uint32_t)(M * ld));
  {
    const int c = (lane & 7) ^ ((4 * f.w + (lane >> 4)) & 7);   // see bf16_fwd_kernel
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      // rows past the end re-read the last row, never stored
      const int row = 8 * (4 * q + f.w) + (lane >> 3);
      if (q < 2 * FI) f.wo[q] = (uint32_t)(min(n0 + row, N - 1) * ld + p0 * 128 + c * 16);
      f.xo[q] = (uint32_t)(min(m0 + row, M - 1) * ld + p0 * 128 + c * 16);
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

  const bool tail = r > 0;
  scales_dma(smem + kLdsPairs, sx, sw, M, N, m0, n0, f.w, lane);
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
  if (part != nullptr) {
    store_tile_parts<FI>(acc, part + (int64_t)split * M * N, N, M, N, m0, n0);
    return;
  }
  // TD: the parts' chunks (32 ranks each) come into the pair slots, four at a
  // time, the first four while the sums become fp32
  const int nj = r / 32, nt = kTermParts * nj;
  auto tail_batch = [&](int c0) __attribute__((always_inline)) {
    for (int c = c0; c < min(c0 + 4, nt); ++c) {
      const int pt = c / nj;
      TailSrc ts;
      ts.wr = make_rsrc(B, (uint32_t)(N * r * 2));
      ts.tr = make_rsrc(T + pt * M * r, (uint32_t)(M * r * 2));
      ts.n0 = n0;
      ts.m0 = m0;
      ts.rows = N;
      ts.r = ts.ld = r;
      ts.col0 = 0;
      ts.bt = false;
      tail_dma(smem + (c - c0) * 2 * kOp, ts, c - pt * nj, f.w, lane);
    }
  };
  if (TD && tail) tail_batch(0);
  f32x16_t out[FI][4];
  scale_tile<FI>(acc, out, smem + kLdsPairs);
  if (tail) {
    if constexpr (TD) {
      for (int c0 = 0; c0 < nt; c0 += 4) {
        if (c0 > 0) {
          QLORA_WAIT(0, 0);
          __builtin_amdgcn_s_barrier();   // every wave is done with the batch before
          tail_batch(c0);
        }
        QLORA_WAIT(0, 0);
        __builtin_amdgcn_s_barrier();
        for (int c = c0; c < min(c0 + 4, nt); ++c) tail_mul<FI>(out, smem + (c - c0) * 2 * kOp);
      }
    } else {
      lora_tail<FI>(out, B, T, r, M, N, m0, n0, smem);
    }
  }
  store_tile_lds<FI>(out, Y, N, M, N, m0, n0, smem);
}

// Ranks k .. k + 7 of the two parts, counted as one rank of 2 r: of B's row (or
// 0 where the row is past the end), and of T's.
__device__ __forceinline__ bf16x8_t b_ranks(const bf16_t* __restrict__ B, int r, int64_t n, int64_t N, int kp) {
  static_assert(kTermParts == 2);
  const int k = kp >= r ? kp - r : kp;
  bf16x8_t v{};
  if (k < r && n < N) v = *reinterpret_cast<const bf16x8_t*>(B + n * r + k);
  return v;
}
__device__ __forceinline__ bf16x8_t t_ranks(const bf16_t* __restrict__ T, int r, int64_t m, int64_t M, int kp) {
  const int part = kp >= r ? 1 : 0, k = kp - part * r;
  bf16x8_t v{};
  if (k < r && m < M) v = *reinterpret_cast<const bf16x8_t*>(T + (part * M + m) * r + k);
  return v;
}
// Channels n .. n + 3 of a token of scale x: the integer sums t, scaled, and the
// adapter's, to its row at y.
__device__ __forceinline__ void put4(i32x4_t t, f32x4_t lo, float4 sc, float x, bf16_t* __restrict__ y, int64_t n) {
  const float y0 = scaled_sum(t[0], sc.x, x) + lo[0], y1 = scaled_sum(t[1], sc.y, x) + lo[1],
              y2 = scaled_sum(t[2], sc.z, x) + lo[2], y3 = scaled_sum(t[3], sc.w, x) + lo[3];
  *reinterpret_cast<uint2*>(y + n) = make_uint2(pack_bf16x2(y0, y1), pack_bf16x2(y2, y3));
}

// Y from the integer parts of a split product, 64 tokens x 64 channels a
// workgroup: thread t adds the parts of channels 4 (t mod 16) .. of tokens t / 16
// + 16 i, whole lines of the parts' and of Y's rows, the loads of S splits
// together; the adapter's term comes from four 16x16 MFMA blocks per wave
// through LDS meanwhile.  2048 x 4096 in two splits 27 us at rank 64 (read in the
// MFMA's layout, 16 tokens' half lines per instruction, 36); what it adds to a sum
// of fp32 parts, 13 us, the product saves in its own epilogue for the most part.
template <int S>
__global__ __launch_bounds__(kThreads) void i8_sum_kernel(const int32_t* __restrict__ part, int splits,
                                                          const float* __restrict__ sw, int64_t N,
                                                          const float* __restrict__ sx, int64_t M,
                                                          const bf16_t* __restrict__ T, const bf16_t* __restrict__ B,
                                                          int r, bf16_t* __restrict__ Y, int cols) {
  constexpr int kPitch = 68;
  __shared__ __align__(16) float term[64 * kPitch];
  const int64_t m0 = (int64_t)(blockIdx.x / cols) * 64, n0 = (int64_t)(blockIdx.x % cols) * 64;
  const int tok = threadIdx.x >> 4, ch = 4 * (threadIdx.x & 15);
  // tokens and channels past the end re-read the last ones, never stored
  const int64_t n = min(n0 + ch, N - 4);
  i32x4_t t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = i32x4_t{0, 0, 0, 0};
  for (int s0 = 0; s0 < splits; s0 += S) {
    i32x4_t v[S][4];
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = min(s0 + k, splits - 1) * M + min(m0 + tok + 16 * i, M - 1);
        v[k][i] = *reinterpret_cast<const i32x4_t*>(part + row * N + n);
      }
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const int in = s0 + k < splits ? -1 : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] += v[k][i] & in;
    }
  }
  if (r > 0) {
    // wave w: tokens 32 (w / 2) .., channels 32 (w mod 2) ..
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane & 15, g = lane >> 4;
    const int wm = 32 * (w >> 1), wn = 32 * (w & 1);
    f32x4_t lo[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) lo[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = 0; c < kTermParts * r; c += 64) {
      bf16x8_t fb[2][2], fu[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          fb[k][i] = b_ranks(B, r, n0 + wn + 16 * i + l, N, c + 32 * k + 8 * g);
          fu[k][i] = t_ranks(T, r, m0 + wm + 16 * i + l, M, c + 32 * k + 8 * g);
        }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            lo[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[k][i], fu[k][j], lo[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<f32x4_t*>(term + (wm + 16 * j + l) * kPitch + wn + 16 * i + 4 * g) = lo[i][j];
    __syncthreads();
  }
  const float4 sc = *reinterpret_cast<const float4*>(sw + n);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + tok + 16 * i;
    f32x4_t lo = {0.0f, 0.0f, 0.0f, 0.0f};
    if (r > 0) lo = *reinterpret_cast<const f32x4_t*>(term + (tok + 16 * i) * kPitch + ch);
    if (m < M && n0 + ch < N) put4(t[i], lo, sc, sx[m], Y + m * N, n);   // N % 8 == 0
  }
}
hipError_t launch_i8_sum(const I8Gemm& g, int splits, const int32_t* part, hipStream_t st) {
  const int cols = (int)((g.N + 63) / 64);
  auto* fn = splits <= 2 ? &i8_sum_kernel<2> : &i8_sum_kernel<4>;
  hipLaunchKernelGGL(fn, dim3((unsigned)((g.M + 63) / 64 * cols)), dim3(kThreads), 0, st, part, splits, g.sw,
                     g.N, g.sx, g.M, g.T, g.B, g.r, g.Y, cols);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Few tokens (M <= 16 MT): the weight is streamed once, straight into the
// MFMA layout, and nothing else matters.  A workgroup of 8 waves takes 16 R
// channels; the waves take the 128-byte lines of a row in turn, so all eight
// stream the same rows, and their integer sums meet in LDS (exact in any
// order).  16x16x64 MFMA: lane (l = lane & 15, g = lane >> 4) holds 16 bytes
// of channel l (A) or token l (B); a load instruction takes 64 contiguous
// bytes of 16 rows, the next one the other half of the same lines.  The
// tokens come from L2 in the same layout.  Loads run one batch of UP lines
// ahead of the products.  One token at 8192 x 8192: 13.8 us, 4.9 TB/s of
// weight; 16 at 8192 x 8192: 17.3 us, 3.9 TB/s.
// ---------------------------------------------------------------------------
constexpr int kSkWaves = 8;

__device__ __forceinline__ i32x4_t ld16(const int8_t* p) { return *reinterpret_cast<const i32x4_t*>(p); }

template <int R, int MT>
struct SkinnyBatch {
  i32x4_t a[R][2], b[MT][2];
};

template <int R, int MT, int UP>
__global__ __launch_bounds__(kSkWaves * 64, 1) void i8_skinny_kernel(const int8_t* __restrict__ Wq,
                                                                     const float* __restrict__ sw, int64_t N,
                                                                     int64_t ld, const int8_t* __restrict__ Xq,
                                                                     const float* __restrict__ sx, int64_t M,
                                                                     const bf16_t* __restrict__ T,
                                                                     const bf16_t* __restrict__ B, int r,
                                                                     bf16_t* __restrict__ Y) {
  __shared__ __align__(16) i32x4_t red[kSkWaves][R * MT][64];
  // the wave's number as a scalar: its branches must not mask lanes, which an
  // MFMA would ignore
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * R;
  const int8_t* wp[R];
  const int8_t* xp[MT];
#pragma unroll
  for (int i = 0; i < R; ++i) wp[i] = Wq + min(n0 + 16 * i + l, N - 1) * ld + 16 * g;   // rows past the end: never stored
#pragma unroll
  for (int j = 0; j < MT; ++j) xp[j] = Xq + min((int64_t)(16 * j + l), M - 1) * ld + 16 * g;
  const int lines = (int)(ld >> 7);

  i32x4_t acc[R][MT];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};

  typedef SkinnyBatch<R, MT> Line;
  auto load = [&](Line& v, int line) __attribute__((always_inline)) {   // a line past the end re-loads the last one
    const int64_t o = (int64_t)min(line, lines - 1) * 128;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int i = 0; i < R; ++i) v.a[i][c] = ld16(wp[i] + o + 64 * c);
#pragma unroll
      for (int j = 0; j < MT; ++j) v.b[j][c] = ld16(xp[j] + o + 64 * c);
    }
  };
  auto mul = [&](const Line& v) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v.a[i][c], v.b[j][c], acc[i][j], 0, 0, 0);
  };
  Line cur[UP], nxt[UP];
#pragma unroll
  for (int u = 0; u < UP; ++u) load(cur[u], w + kSkWaves * u);
  for (int base = w; base < lines; base += kSkWaves * UP) {
    const bool more = base + kSkWaves * UP < lines;
    if (more) {
#pragma unroll
      for (int u = 0; u < UP; ++u) load(nxt[u], base + kSkWaves * (UP + u));
    }
#pragma unroll
    for (int u = 0; u < UP; ++u)
      if (base + kSkWaves * u < lines) mul(cur[u]);
    if (more) {
#pragma unroll
      for (int u = 0; u < UP; ++u) cur[u] = nxt[u];
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) red[w][i * MT + j][lane] = acc[i][j];
  __syncthreads();
  // wave b < R MT finishes block b: D[channel][token], lane: token l, channels 4 g ..
#pragma unroll
  for (int b = 0; b < R * MT; b += kSkWaves) {
    const int blk = b + w;
    if (blk >= R * MT) break;
    const int i = blk / MT, j = blk % MT;
    i32x4_t t = red[0][blk][lane];
#pragma unroll
    for (int v = 1; v < kSkWaves; ++v) t += red[v][blk][lane];
    const int64_t nrow = n0 + 16 * i, m = 16 * j + l;
    f32x4_t lo = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = 0; c < kTermParts * r; c += 32)   // adapter: 16 channels x 16 tokens over the ranks of both parts
      lo = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b_ranks(B, r, nrow + l, N, c + 8 * g), t_ranks(T, r, m, M, c + 8 * g),
                                                   lo, 0, 0, 0);
    const int64_t n = nrow + 4 * g;
    if (m < M && n < N) put4(t, lo, *reinterpret_cast<const float4*>(sw + n), sx[m], Y + m * N, n);   // N % 8 == 0
  }
}

template <int R, int MT, int UP>
hipError_t launch_skinny(const I8Gemm& g, hipStream_t st) {
  hipLaunchKernelGGL((i8_skinny_kernel<R, MT, UP>), dim3((unsigned)((g.N + 16 * R - 1) / (16 * R))),
                     dim3(kSkWaves * 64), 0, st, g.Wq, g.sw, g.N, i8_row_bytes(g.K), g.Xq, g.sx, g.M, g.T, g.B, g.r,
                     g.Y);
  return hipGetLastError();
}

template <int FI>
hipError_t launch_fi(const I8Gemm& g, int64_t n_begin, int64_t n_rows, int splits, int32_t* part, hipStream_t st) {
  const int tiles_n = (int)((n_rows + 64 * FI - 1) / (64 * FI)), tiles_m = (int)((g.M + kTile - 1) / kTile);
  // the rank in whole chunks, T's parts and B within 32-bit byte offsets
  const bool td = g.r > 0 && g.r % 32 == 0 && g.M * g.r < ((int64_t)1 << 30) && g.N * g.r < ((int64_t)1 << 30);
  auto* fn = td ? &i8_gemm_kernel<FI, true> : &i8_gemm_kernel<FI, false>;
  constexpr size_t lds = kLdsPairs + kLdsScales;
  hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), (int)lds);
  if (e != hipSuccess) return e;
  const int npair = (int)(i8_row_bytes(g.K) / 128);
  hipLaunchKernelGGL(fn, dim3(tiles_n * tiles_m * splits), dim3(kThreads), lds, st, g.Wq, g.sw, g.N,
                     i8_row_bytes(g.K), g.Xq, g.sx, g.M, g.T, g.B, g.r, g.Y, n_begin, tiles_n, tiles_m,
                     (npair + splits - 1) / splits, splits > 1 ? part : nullptr);
  return hipGetLastError();
}

}  // namespace

// Up to 32 tokens: the streaming kernel, or tiles (split where that pays and
// there is room), whichever is estimated to take less.  The streaming kernel
// takes 16 channels a workgroup, or 32 where that still fills the card and
// there are enough tokens for their second reading to cost; a round of
// workgroups costs by its batches of lines, and whole rounds up to two (a
// workgroup fills a CU), less than whole ones past that.  Neither goes below
// the weight's bytes at 4.8 TB/s.  Measured in us at 57 sizes, where the choice
// is within 0.7 % of the faster on the mean (tokens x channels x K, streaming
// and tiles):
//   1 x 22016 x 8192    34.5  44.8     16 x 8192 x 8192    17.7  20.6
//   8 x 4096 x 16384    17.5  20.8     16 x 5120 x 13824   29.8  18.7
//   16 x 4096 x 4096     6.5   8.7     1 x 256 x 22016     14.1   9.7
//   24 x 4096 x 4096     7.4   9.1     32 x 5120 x 5120    25.8  11.4
//   20 x 8192 x 2048     6.2   7.5     32 x 22016 x 8192   54.5  46.2
namespace {

constexpr int64_t kSkinnyTokens = 32;
constexpr int kSplitCus = 256;   // the workspace is sized for it (choose_tile)

double skinny_cost(int64_t M, int64_t N, int64_t lines, int cus) {
  const bool wide = M > 8 && N >= 8192;   // 32 channels a workgroup
  const double x = (double)((N + (wide ? 31 : 15)) / (wide ? 32 : 16)) / cus;
  const double rounds = x <= (M > 8 && M <= 16 && wide ? 1.0 : 2.0) ? std::ceil(x) : 0.46 * (x + std::ceil(x));
  const double l16 = (double)((lines + 15) / 16 * 16);
  if (M > 16) return rounds * (wide ? 1.5 + 0.3 * l16 : 2.0 + 5.7 * (double)((lines + 31) / 32));
  const double round = M <= 8 ? 2.2 + 0.073 * l16 : wide ? 0.5 + 0.26 * l16 : 2.4 + 0.113 * l16;
  return std::max(rounds * round, (double)N * lines * 128.0 / 4.8e6 + 2.0);
}
bool use_skinny(int64_t M, int64_t N, int64_t lines, int cus, size_t part_bytes) {
  if (M > kSkinnyTokens) return false;
  const double cost = skinny_cost(M, N, lines, cus), least = (double)N * lines * 128.0 / 4.8e6 + 4.0;   // of tiles
  return cost <= least || cost <= choose_tile(M, N, lines, cus, part_bytes).cost + 1.5;
}

}  // namespace

// More tokens: tiles, the small ones or 256 x 64 FI; or whole rounds of 256 x
// 256 tiles and the rest of the channels apart.
hipError_t launch_i8_gemm(const I8Gemm& g, hipStream_t st, int32_t* part, size_t part_bytes) {
  const int cus = device_cu_count();
  const int64_t lines = i8_row_bytes(g.K) / 128;
  if (use_skinny(g.M, g.N, lines, cus, part ? part_bytes : 0)) {
    if (g.M <= 16) return g.M > 8 && g.N >= 8192 ? launch_skinny<2, 1, 2>(g, st) : launch_skinny<1, 1, 2>(g, st);
    return g.N < 8192 ? launch_skinny<1, 2, 4>(g, st) : launch_skinny<2, 2, 2>(g, st);
  }
  auto part_of = [&](const TileChoice& c, int64_t n_begin, int64_t n_rows) {
    if (c.tm == 256)
      return c.tn == 256   ? launch_fi<4>(g, n_begin, n_rows, c.splits, part, st)
             : c.tn == 192 ? launch_fi<3>(g, n_begin, n_rows, 1, nullptr, st)
                           : launch_fi<2>(g, n_begin, n_rows, 1, nullptr, st);
    TileGemm t{};
    t.W = g.Wq, t.X = g.Xq, t.sw = g.sw, t.sx = g.sx, t.N = g.N, t.row_bytes = i8_row_bytes(g.K), t.M = g.M;
    t.T = g.T, t.B = g.B, t.r = g.r, t.Y = g.Y, t.part = part;
    return launch_tile(t, c, n_begin, n_rows, st);
  };
  // (a split one: of all channels)
  auto whole = [&](const TileChoice& c) {
    const hipError_t e = part_of(c, 0, g.N);
    return e != hipSuccess || c.splits == 1 ? e : launch_i8_sum(g, c.splits, part, st);
  };
  const TileChoice one = choose_tile(g.M, g.N, lines, cus, part ? part_bytes : 0);
  const int64_t tiles_m = (g.M + 255) / 256, tiles = tiles_m * ((g.N + 255) / 256);
  if (tiles > cus && cus % tiles_m == 0) {
    const int64_t rounds = tiles / cus, n_full = rounds * (cus / tiles_m) * 256;
    if (n_full < g.N) {
      const TileChoice rest = choose_tile(g.M, g.N - n_full, lines, cus, 0);
      if ((double)rounds * full_round_cost(lines) + rest.cost < one.cost) {
        const hipError_t e = launch_fi<4>(g, 0, n_full, 1, nullptr, st);
        return e != hipSuccess ? e : part_of(rest, n_full, g.N - n_full);
      }
    }
  }
  return whole(one);
}

size_t i8_gemm_part_bytes(int64_t M, int64_t N, int64_t K) {
  const int64_t lines = i8_row_bytes(K) / 128;
  return use_skinny(M, N, lines, kSplitCus, (size_t)1 << 62) ? 0 : tile_part_bytes(M, N, lines);
}

}  // namespace qlora
