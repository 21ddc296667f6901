// gemm_bf16.hip -- dense bf16 GEMMs on a dequantized weight.
//
//   forward   Y = X Wd^T + s U B^T     (Wd = deq(W) as bf16, U = X A^T)
//
// deepfa.ir blog, "QLoRA's Working Process": the 4-bit weights are converted
// to BF16 for the computation.  These kernels take that bf16 weight from
// memory instead of decoding it inside the tile, so a weight is decoded once
// per product (by the dequant kernel) rather than once per 256-token tile.
//
// 256 threads (4 waves), 256 x 256 output tile, wave (wr, wc) a 128 x 128
// sub-tile (tokens 128 wr.., weight rows 128 wc..) in 256 accumulator
// registers, bf16 MFMA 32x32x16 with fp32 accumulation.  The contraction runs
// in pairs of 32-wide stages: a pair (64 columns: one 128-byte line of every
// row) comes into LDS by buffer->LDS DMA, each instruction moving 8 whole rows,
// one pair ahead and more (dense_tile.h); one barrier per pair.
//
//   dX        the same kernel on deq(W)^T: dX = dY (W^T)^T + s G (A^T)^T,
//             with A read column-wise in the LoRA tail;
//   dX under dropout   the adapter branch saw drop(X), so its product is
//             masked like X before it joins: dX = dY (W^T)^T + s drop'(G A);
//   groups    weight rows in groups of gn, each with its own adapter (the
//             stacked q/k/v or gate/up weights of one layer).
#include <algorithm>

#include "dense_tile.h"
#include "rng.h"

namespace qlora {
namespace {

// Forms of the LoRA tail: T one matrix, scaled by s as it is read; or T as
// kTermParts parts with s in them, the product as it is or masked.
enum TailForm : int { kTailScaled = 0, kTailParts = 1, kTailPartsDrop = 2 };

// Chunks of the masked LoRA tail of a tile: acc += drop'(T A), A [r x cols] read
// transposed.  The nt <= 4 chunks are in LDS (chunk c at 2 kOp c), so the
// products of four 32 x 32 blocks at a time are summed in registers of their
// own, masked by their bits (block 4 i + j of the wave at bits + 1 KiB (4 i +
// j)), and added: the tile keeps one set of accumulators.
// Masked dX of 4096 x 22016 x 8192 at rank 64 1.3 PFLOP/s; 2048 x 4096 x 4096
// 68 us (one round of 256 x 128 tiles, 1.0 PFLOP/s).  With a block at a time,
// its mask computed here, the whole backward of 3918 x 20856 x 800 at rank 128
// took 438 us, 383 this way (both with T in one part; the second adds 10 us
// there, 1.6 to the 68 and 7 to the 1140 of the others).
template <int FI>
__device__ __forceinline__ void masked_tail(f32x16_t (&acc)[FI][4], const char* smem, int nt, const char* bits) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wr = w >> 1, wc = w & 1;
  const FragOffs fo = frag_offs(lane);
  const char* tok = smem + kOp + wr * 128 * 64;
#pragma unroll
  for (int i = 0; i < FI; ++i) {   // four blocks at a time
    f32x16_t y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) y[j][e] = 0.0f;
    for (int c = 0; c < nt; ++c) {
      bf16x8_t b0[4], b1[4], f0, f1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        b0[j] = rd16(tok + c * 2 * kOp + j * 2048 + fo.o0);
        b1[j] = rd16(tok + c * 2 * kOp + j * 2048 + fo.o1);
      }
      const char* a0 = smem + c * 2 * kOp + tr_off<512>(wc * FI + i);
      tr_read2<2048, 2048>(a0, a0 + 16 * 512, f0, f1);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = mfma32x32x16(f0, b0[j], y[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = mfma32x32x16(f1, b1[j], y[j]);
    }
    uint32_t keep[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      keep[j] = *reinterpret_cast<const uint32_t*>(bits + 1024 * (4 * i + j) + 4 * threadIdx.x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // back into the accumulator registers at once: the compiler would keep
      // the sums in vector registers, and spill
      float f[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] = acc[i][j][e] + masked(y[j][e], keep[j], e);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float v;
        asm volatile("v_accvgpr_write_b32 %0, %1" : "=a"(v) : "v"(f[e]));
        acc[i][j][e] = v;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// FI: weight fragments per wave, so the tile is 64 FI weight rows x 256
// tokens (FI = 4, 3 or 2); its tiles start at weight row n_begin.
// Split contraction (part != null): the grid holds the tiles once per split;
// split p takes contraction pairs p pps .. (64-column pairs), split 0 alone
// adds the LoRA tail, and each split stores its fp32 sums at part + p M N
// ([M x N], row stride N) instead of Y.
// FORM kTailParts and kTailPartsDrop: U holds kTermParts parts, one adapter (gn
// = N, ldu = r), s is not used; kTailPartsDrop: dX (b_trans), masked by `drop`.
template <int FI, bool TD, int FORM>
__global__ __launch_bounds__(kThreads, 1) void bf16_fwd_kernel(const bf16_t* __restrict__ Wd, int64_t N, int64_t K,
                                                               const bf16_t* __restrict__ X, int64_t M,
                                                               const bf16_t* __restrict__ U,
                                                               const bf16_t* __restrict__ Bl, int b_trans, int r,
                                                               int ldu, int64_t gn, float s, bf16_t* __restrict__ Y,
                                                               int64_t n_begin, int tiles_n, int tiles_m, int pps,
                                                               float* __restrict__ part, DropArgs drop) {
  constexpr bool DR = FORM == kTailPartsDrop;
  extern __shared__ __align__(16) char smem[];
  int tn, tm;
  int id = xcd_tile_id();
  const int split = id / (tiles_n * tiles_m);
  map_tile_grouped(id - split * tiles_n * tiles_m, tiles_n, tiles_m, tn, tm);
  const int64_t n0 = n_begin + (int64_t)tn * 64 * FI, m0 = (int64_t)tm * kTile;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6, wr = wv >> 1, wc = wv & 1;

  DenseOps f;
  f.w = __builtin_amdgcn_readfirstlane(wv);
  __builtin_assume(f.w >= 0 && f.w < 4);
  const int p0 = split * pps;
  f.npair = min((int)(K >> 6) - p0, pps);
  f.wr_ = make_rsrc(Wd, (uint32_t)(N * K * 2));
  f.xr = make_rsrc(X, (uint32_t)(M * K * 2));
  {
    // lane j of DMA instruction q: row 8 (4 q + w) + (j >> 3), position j & 7
    // holding chunk (j & 7) ^ ((row >> 1) & 7) = (j & 7) ^ ((4 w + (j >> 4)) & 7)
    const int c = (lane & 7) ^ ((4 * f.w + (lane >> 4)) & 7);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      // rows past the end re-read the last row: finite data, never stored
      const int row = 8 * (4 * q + f.w) + (lane >> 3);
      if (q < 2 * FI) f.wo[q] = (uint32_t)(min(n0 + row, N - 1) * K * 2 + p0 * 128 + c * 16);
      f.xo[q] = (uint32_t)(min(m0 + row, M - 1) * K * 2 + p0 * 128 + c * 16);
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

  f32x16_t acc[FI][4];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // TD: the LoRA tail by DMA (the launch checked that the rank comes in whole
  // chunks, that no tile straddles two adapter groups and that the side
  // arrays fit 32-bit byte offsets); otherwise through registers
  const int64_t g0 = n0 / gn;
  const bool tail = r > 0 && split == 0;
  const bool tdma = TD && !DR && tail;
  // (built where used, so nothing of it stays live through the main loop)
  auto tail_src = [&](int part) __attribute__((always_inline)) {
    TailSrc ts;
    ts.wr = make_rsrc(Bl, (uint32_t)(N * r * 2));
    ts.tr = make_rsrc(FORM == kTailScaled ? U : U + part * M * r, (uint32_t)(M * ldu * 2));
    ts.n0 = n0;
    ts.m0 = m0;
    ts.rows = N;
    ts.r = r;
    ts.ld = ldu;
    ts.col0 = (int)(g0 * r);
    ts.bt = b_trans != 0;
    return ts;
  };
  // chunk c of the parts, one part's chunks after the other's
  [[maybe_unused]] auto part_dma = [&](char* dst, int c) __attribute__((always_inline)) {
    const int nj = r / 32, part = c / nj;
    tail_dma(dst, tail_src(part), c - part * nj, f.w, lane);
  };
  Frags F;
  // K % 64 == 0: whole pairs of 32-wide stages
  // DR: the mask of the wave's block b = 4 i + j, a word per lane past the pair
  // slots; only the thread that wrote it reads it
  [[maybe_unused]] DropKey key;
  [[maybe_unused]] uint32_t block00 = 0u, block_row = 0u;   // M N < 2^31
  if constexpr (DR) {
    key = drop_key(drop);
    block_row = (uint32_t)(N >> 3);
    block00 = (uint32_t)(m0 + 128 * wr + (lane & 31)) * block_row + (uint32_t)((n0 + 32 * FI * wc) >> 3);
  }
  [[maybe_unused]] auto put_bits = [&](int b) __attribute__((always_inline)) {
    *reinterpret_cast<uint32_t*>(smem + kLdsPairs + 1024 * b + 4 * t) =
        mask_bits(block00 + 32u * (uint32_t)(b & 3) * block_row + 4u * (uint32_t)(b >> 2), key);
  };
  if constexpr (DR) {
    // the masks need LDS of their own: two pair slots, pairs 0 and 1 first
#pragma unroll
    for (int d = 0; d < 2 * FI + 8; ++d) {
      pair_dma<FI>(smem, f, 0, d);
      pair_dma<FI>(smem + kPairSlot, f, 1, d);
    }
    QLORA_WAIT(0, 0);
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < FI) F.a0[i] = rd16(smem + am + i * 32 * 128 + po.o[0][0]);
      F.b0[i] = rd16(smem + kPairOp + bm + i * 32 * 128 + po.o[0][0]);
    }
    for (int pr = 0; pr < f.npair; ++pr) {
      char* cur = smem + (pr & 1) * kPairSlot;
      char* nxt = smem + ((pr & 1) ^ 1) * kPairSlot;
      __builtin_amdgcn_sched_barrier(0);
      dense_slots<MmBf16, FI, 0, 0>(cur, nxt, cur, f, pr, acc, F, am, bm, po);
      // one block's mask a pair, while the next pair's lines are on their way
      if (tail && pr < 4 * FI) put_bits(pr);
      __builtin_amdgcn_sched_barrier(0);
      dense_slots<MmBf16, FI, 1, 0>(cur, nxt, cur, f, pr, acc, F, am, bm, po);
    }
  } else {
    dense_halves<MmBf16, FI>(smem, f, acc, F, am, bm, po);
  }
  // drain the DMAs still in flight (clamped re-loads) before reusing LDS
  QLORA_WAIT(0, 0);
  __builtin_amdgcn_s_barrier();

  if constexpr (DR) {
    if (tail)
      for (int b = f.npair; b < 4 * FI; ++b) put_bits(b);   // a contraction of fewer pairs than blocks
  }
  const FragOffs fo = frag_offs(lane);
  const int am64 = wc * 32 * FI * 64, bm64 = wr * 128 * 64;
  // acc += the chunk at buf (weights at buf, tokens at buf + kOp); the tokens
  // are scaled by s as they are read when `raw`
  auto tail_chunk = [&](const char* buf, bool raw) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int o = kk ? fo.o1 : fo.o0;
      if (b_trans) {
        // transposed reads in asm blocks, so that the DMAs of later chunks
        // stay in flight (see tr_read2)
        const char* tb = buf + kk * 16 * 512;
        const int f0 = wc * FI;
        if constexpr (FI == 3) {
          tr_read3<2048, 2048, 2048>(tb + tr_off<512>(f0), tb + tr_off<512>(f0 + 1), tb + tr_off<512>(f0 + 2), F.a0[0],
                                     F.a0[1], F.a0[2]);
        } else {
#pragma unroll
          for (int i = 0; i < FI; i += 2)
            tr_read2<2048, 2048>(tb + tr_off<512>(f0 + i), tb + tr_off<512>(f0 + i + 1), F.a0[i], F.a0[i + 1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < FI; ++i) F.a0[i] = rd16(buf + am64 + i * 2048 + o);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x8_t b = rd16(buf + kOp + bm64 + i * 2048 + o);
        F.b0[i] = raw ? scale_frag(b, s) : b;
      }
#pragma unroll
      for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma32x32x16(F.a0[i], F.b0[j], acc[i][j]);
    }
  };
  if constexpr (DR) {
    if (tail) {
      // four chunks at a time through the pair slots
      const int nt = (kTermParts * r + 31) / 32;
      for (int b0 = 0; b0 < nt; b0 += 4) {
        const int bn = min(4, nt - b0);
        if (b0 > 0) __syncthreads();   // every wave is done with the batch before
        for (int c = 0; c < bn; ++c) {
          if constexpr (TD) {
            part_dma(smem + c * 2 * kOp, b0 + c);
          } else {
            TailRegs R;
            tail_load_parts(R, Bl, true, N, r, n0, 32 * (b0 + c), U, M, m0);
            tail_store(smem + c * 2 * kOp, R, true, 1.0f);
          }
        }
        QLORA_WAIT(0, 0);
        __syncthreads();
        masked_tail<FI>(acc, smem, bn, smem + kLdsPairs);
      }
    }
  } else if constexpr (TD) {
    if (tdma) {
      // five chunks at a time, each in a half slot
      constexpr bool raw = FORM == kTailScaled;
      const TailSrc ts = tail_src(0);
      const int nt = (raw ? 1 : kTermParts) * (r / 32);
      for (int b0 = 0; b0 < nt; b0 += 5) {
        const int bn = min(5, nt - b0);
        if (b0 > 0) {
          QLORA_WAIT(0, 0);
          __builtin_amdgcn_s_barrier();   // every wave is done with the batch before
        }
        for (int c = 0; c < bn; ++c) {
          if constexpr (raw)
            tail_dma(smem + c * 2 * kOp, ts, b0 + c, f.w, lane);
          else
            part_dma(smem + c * 2 * kOp, b0 + c);
        }
        QLORA_WAIT(0, 0);
        __builtin_amdgcn_s_barrier();
        for (int c = 0; c < bn; ++c) tail_chunk(smem + c * 2 * kOp, raw);
      }
    }
  } else if (tail) {
    // acc += B (s U)^T over the rank, 32 at a time, through 64-byte-row tiles.
    // Weight rows come in groups of gn, each with its own adapter: rows of
    // group g take columns g r .. of U (row stride ldu) and their rows of B;
    // a tile that straddles groups runs the tail once per group, with the
    // other groups' rows zero.  Chunks alternate between two tile pairs:
    // chunk c + 1 is loaded into registers while chunk c is multiplied, and
    // one barrier per chunk both publishes a chunk and retires the buffer
    // the next store overwrites (its readers finished before they stored
    // their part of the chunk in between).
    // (With T in parts there is one adapter.)
    const int64_t g_last = (min(n0 + 64 * FI, N) - 1) / gn;
    const int nj = (r + 31) / 32;
    const int nt = FORM == kTailScaled ? (int)(g_last - g0 + 1) * nj : (kTermParts * r + 31) / 32;
    TailRegs R;
    auto load = [&](int t) {
      if constexpr (FORM == kTailScaled) {
        const int64_t g = g0 + t / nj;
        tail_load(R, Bl, b_trans != 0, N, r, n0, 32 * (t % nj), g * gn, min((g + 1) * gn, N), U + g * r, ldu, M,
                  m0);
      } else {
        tail_load_parts(R, Bl, b_trans != 0, N, r, n0, 32 * t, U, M, m0);
      }
    };
    load(0);
    for (int t = 0; t < nt; ++t) {
      char* buf = smem + (t & 1) * 2 * kOp;
      tail_store(buf, R, b_trans != 0, FORM == kTailScaled ? s : 1.0f);
      if (t + 1 < nt) load(t + 1);
      __syncthreads();
      tail_chunk(buf, false);
    }
  }
  if (part != nullptr)
    store_tile_parts<FI>(acc, part + (int64_t)split * M * N, N, M, N, m0, n0);
  else
    store_tile_lds<FI>(acc, Y, N, M, N, m0, n0, smem);
}

}  // namespace

namespace {

// Tiles of 64 FI weight rows over rows [n_begin, n_begin + n_rows) of the
// N-row weight (N is every array's extent and leading dimension).
// Whether the launch's tiles can take the LoRA tail by DMA: the rank in whole
// 32-wide chunks, no tile across two adapter groups, and U (M x ldu) and B
// or A (N x r) within 32-bit byte offsets.
bool tail_by_dma(int64_t N, int64_t M, int r, int ldu, int64_t gn, int64_t n_begin, int tiles_n, int rows) {
  if (r <= 0 || r % 32 != 0 || M * ldu >= ((int64_t)1 << 30) || N * r >= ((int64_t)1 << 30)) return false;
  for (int t = 0; t < tiles_n; ++t) {
    const int64_t lo = n_begin + (int64_t)t * rows, hi = std::min(lo + rows, N) - 1;
    if (lo / gn != hi / gn) return false;
  }
  return true;
}

// splits > 1: the contraction in that many parts of whole 64-column pairs,
// fp32 sums to part (splits x M x N floats), not Y.
template <int FI>
hipError_t launch_fi(const bf16_t* Wd, int64_t N, int64_t K, const bf16_t* X, int64_t M, const bf16_t* U,
                     const bf16_t* B, bool b_trans, int r, int ldu, int64_t gn, float s, bf16_t* Y, int64_t n_begin,
                     int64_t n_rows, hipStream_t st, TailForm form, const DropArgs* drop, int splits = 1,
                     float* part = nullptr) {
  const int tiles_n = (int)((n_rows + 64 * FI - 1) / (64 * FI));
  const int tiles_m = (int)((M + kTile - 1) / kTile);
  const bool td = tail_by_dma(N, M, r, ldu, gn, n_begin, tiles_n, 64 * FI);
  auto* fn = form == kTailPartsDrop ? (td ? &bf16_fwd_kernel<FI, true, kTailPartsDrop>
                                          : &bf16_fwd_kernel<FI, false, kTailPartsDrop>)
             : form == kTailParts
                 ? (td ? &bf16_fwd_kernel<FI, true, kTailParts> : &bf16_fwd_kernel<FI, false, kTailParts>)
                 : (td ? &bf16_fwd_kernel<FI, true, kTailScaled> : &bf16_fwd_kernel<FI, false, kTailScaled>);
  const size_t lds = form == kTailPartsDrop ? kLdsPairs + 4096 * FI : kLdsHalves;
  hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), (int)lds);
  if (e != hipSuccess) return e;
  const int npair = (int)(K >> 6);
  const int pps = splits > 1 ? (npair + splits - 1) / splits : npair;
  hipLaunchKernelGGL(fn, dim3(tiles_n * tiles_m * splits), dim3(kThreads), lds, st, Wd, N, K, X, M, U, B,
                     (int)b_trans, r, ldu, gn, s, Y, n_begin, tiles_n, tiles_m, pps, splits > 1 ? part : nullptr,
                     drop ? *drop : DropArgs{});
  return hipGetLastError();
}

// Y [M x N] (bf16) = the sum of the splits' fp32 partials, added in split
// order; four values per thread (N % 4 == 0).
__global__ __launch_bounds__(kThreads) void split_sum_kernel(const float* __restrict__ part, int splits, int64_t n,
                                                             bf16_t* __restrict__ Y) {
  const int64_t i = 4 * ((int64_t)blockIdx.x * kThreads + threadIdx.x);
  if (i >= n) return;
  float4 a = *reinterpret_cast<const float4*>(part + i);
  for (int p = 1; p < splits; ++p) {
    const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)p * n + i);
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  *reinterpret_cast<uint2*>(Y + i) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
}

// Time of weight rows [n_begin, N) in 64 FI-row tiles, in units of one round
// of 256-row tiles: rounds x FI / 4, with a small charge for the narrower
// tiles' extra LDS reads per MFMA.
double tile_cost(int64_t rows, int64_t tiles_m, int fi, int cus) {
  const int64_t tiles = (rows + 64 * fi - 1) / (64 * fi) * tiles_m;
  const double eff = fi == 4 ? 1.0 : fi == 3 ? 1.06 : 1.12;
  return (double)((tiles + cus - 1) / cus) * fi / 4.0 * eff;
}
int best_fi(int64_t rows, int64_t tiles_m, int cus) {
  int best = 4;
  for (int fi = 3; fi >= 2; --fi)
    if (tile_cost(rows, tiles_m, fi, cus) < tile_cost(rows, tiles_m, best, cus)) best = fi;
  return best;
}

hipError_t launch_rows(int fi, const bf16_t* Wd, int64_t N, int64_t K, const bf16_t* X, int64_t M,
                       const bf16_t* U, const bf16_t* B, bool b_trans, int r, int ldu, int64_t gn, float s,
                       bf16_t* Y, int64_t n_begin, hipStream_t st, TailForm form, const DropArgs* drop) {
  const int64_t n_rows = N - n_begin;
  if (fi == 3) return launch_fi<3>(Wd, N, K, X, M, U, B, b_trans, r, ldu, gn, s, Y, n_begin, n_rows, st, form, drop);
  if (fi == 2) return launch_fi<2>(Wd, N, K, X, M, U, B, b_trans, r, ldu, gn, s, Y, n_begin, n_rows, st, form, drop);
  return launch_fi<4>(Wd, N, K, X, M, U, B, b_trans, r, ldu, gn, s, Y, n_begin, n_rows, st, form, drop);
}

}  // namespace

// Split contraction.  A shape with at most half as many 256 x 256 tiles as
// CUs, which would otherwise run narrower tiles, and a long contraction runs
// its 256 x 256 tiles twice, each over half the contraction, and adds the
// two fp32 partials: the 7B gate/up dX product (128 tiles, 22016 columns)
// took 411 us on 128-row tiles.  The CU count the size of the partials
// assumes is fixed (256), so that the workspace a caller queries does not
// depend on the device; the launch splits only if it has that room.
constexpr int kSplitCus = 256;
constexpr int64_t kSplitMinK = 16384;
int dense_splits(int64_t N, int64_t K, int64_t M, int cus) {
  const int64_t tiles = ((N + kTile - 1) / kTile) * ((M + kTile - 1) / kTile);
  return (K >= kSplitMinK && N % 4 == 0 && 2 * tiles <= cus) ? 2 : 1;
}

size_t dense_split_bytes(int64_t N, int64_t K, int64_t M) {
  const int sp = dense_splits(N, K, M, kSplitCus);
  return sp > 1 ? (size_t)sp * (size_t)M * (size_t)N * sizeof(float) : 0;
}

// The grid is sized for the CU count.  Weight rows are cut into a part that
// fills whole rounds of 256-row tiles and a remainder, whose tile width (256,
// 192 or 128 rows) minimizes its time; a shape with fewer 256-row tiles than
// CUs is all remainder, or a split contraction (above) when part has room.
namespace {

hipError_t launch_dense(const bf16_t* Wd, int64_t N, int64_t K, const bf16_t* X, int64_t M, const bf16_t* U,
                        int ldu, const bf16_t* B, bool b_trans, int r, int64_t gn, float s, bf16_t* Y,
                        hipStream_t st, float* part, size_t part_bytes, TailForm form, const DropArgs* drop) {
  const int cus = device_cu_count();
  const int64_t tiles_m = (M + kTile - 1) / kTile;
  const int64_t tiles_n = (N + kTile - 1) / kTile;
  const int sp = dense_splits(N, K, M, cus);
  if (sp > 1 && part != nullptr && part_bytes >= (size_t)sp * (size_t)M * (size_t)N * sizeof(float)) {
    hipError_t e = launch_fi<4>(Wd, N, K, X, M, U, B, b_trans, r, ldu, gn, s, Y, 0, N, st, form, drop, sp, part);
    if (e != hipSuccess) return e;
    const int64_t n = M * N;
    hipLaunchKernelGGL(split_sum_kernel, dim3((unsigned)((n / 4 + kThreads - 1) / kThreads)), dim3(kThreads), 0, st,
                       part, sp, n, Y);
    return hipGetLastError();
  }
  int64_t n_split = 0;   // rows of the whole-round part
  if (tiles_n * tiles_m > cus && cus % tiles_m == 0) {
    const int64_t per_round = cus / tiles_m;   // 256-row column tiles per round
    n_split = std::min(N, (tiles_n * tiles_m / cus) * per_round * kTile);
    if (n_split >= N || tile_cost(N - n_split, tiles_m, best_fi(N - n_split, tiles_m, cus), cus) >=
                            tile_cost(N - n_split, tiles_m, 4, cus))
      n_split = 0;   // nothing left over, or the remainder gains nothing from narrower tiles: one launch
  }
  if (n_split > 0) {
    hipError_t e = launch_fi<4>(Wd, N, K, X, M, U, B, b_trans, r, ldu, gn, s, Y, 0, n_split, st, form, drop);
    if (e != hipSuccess) return e;
    // the remainder's tiles address rows from n_split on, in the same arrays
    return launch_rows(best_fi(N - n_split, tiles_m, cus), Wd, N, K, X, M, U, B, b_trans, r, ldu, gn, s, Y, n_split,
                       st, form, drop);
  }
  return launch_rows(best_fi(N, tiles_m, cus), Wd, N, K, X, M, U, B, b_trans, r, ldu, gn, s, Y, 0, st, form, drop);
}

}  // namespace

hipError_t launch_bf16_group(const bf16_t* Wd, int64_t N, int64_t K, const bf16_t* X, int64_t M, const bf16_t* U,
                             int ldu, const bf16_t* B, bool b_trans, int r, int64_t gn, float s, bf16_t* Y,
                             hipStream_t st, float* part, size_t part_bytes) {
  return launch_dense(Wd, N, K, X, M, U, ldu, B, b_trans, r, gn, s, Y, st, part, part_bytes, kTailScaled, nullptr);
}

hipError_t launch_bf16_fwd(const bf16_t* Wd, int64_t N, int64_t K, const bf16_t* X, int64_t M, const bf16_t* U,
                           const bf16_t* B, bool b_trans, int r, float s, bf16_t* Y, hipStream_t st, float* part,
                           size_t part_bytes) {
  return launch_bf16_group(Wd, N, K, X, M, U, r, B, b_trans, r, N, s, Y, st, part, part_bytes);
}

hipError_t launch_split_sum(const float* part, int splits, int64_t n, bf16_t* Y, hipStream_t st) {
  hipLaunchKernelGGL(split_sum_kernel, dim3((unsigned)((n / 4 + kThreads - 1) / kThreads)), dim3(kThreads), 0, st, part,
                     splits, n, Y);
  return hipGetLastError();
}

size_t staged_part_bytes(int64_t N, int64_t K, int64_t M) {
  return std::max(tile_part_bytes(M, N, K / 64), dense_split_bytes(N, K, M));
}

double staged_cost(int64_t N, int64_t K, int64_t M) { return choose_tile(M, N, K / 64, kSplitCus, (size_t)1 << 62).cost; }

// The tiles of a product whose sums are left as fp32 parts, on a card of kSplitCus
// CUs: the parts' number has to be the one that the caller sized its workspace
// for.  Tiles of 256 tokens only in a split contraction (gemm_pool.hip).
namespace {
TileChoice parts_tile(int64_t N, int64_t K, int64_t M) {
  const TileChoice c = choose_tile(M, N, K / 64, kSplitCus, (size_t)1 << 62);
  return c.tm == 256 && c.splits == 1 ? choose_tile(M, N, K / 64, kSplitCus, (size_t)1 << 62, true) : c;
}
}  // namespace
bool dense_tiles(int64_t N, int64_t K, int64_t M) {
  const TileChoice c = choose_tile(M, N, K / 64, kSplitCus, (size_t)1 << 62);
  return c.tm == 256 && c.splits == 1;
}
size_t product_part_bytes(int64_t N, int64_t K, int64_t M) {
  return (size_t)parts_tile(N, K, M).splits * (size_t)M * (size_t)N * sizeof(float);
}
hipError_t launch_product_parts(const bf16_t* Wd, int64_t N, int64_t K, const bf16_t* X, int64_t M, float* part,
                                int* splits, hipStream_t st) {
  const TileChoice c = parts_tile(N, K, M);
  *splits = c.splits;
  if (c.tm == 256) {
    PoolGemm g{};
    g.Wd = Wd, g.N = N, g.K = K, g.M = M, g.X = X, g.pool.G = 1, g.part = part, g.splits = c.splits;
    return launch_pool_gemm(g, st);
  }
  TileGemm t{};
  t.W = Wd, t.X = X, t.N = N, t.row_bytes = 2 * K, t.M = M, t.part = part, t.keep = true;
  return launch_tile(t, c, 0, N, st);
}

hipError_t launch_staged(const bf16_t* Wd, int64_t N, int64_t K, const bf16_t* X, int64_t M, const bf16_t* T,
                         const bf16_t* B, bool b_trans, int r, const DropArgs* drop, bf16_t* Y, hipStream_t st,
                         float* part, size_t part_bytes, SplitSum* rest) {
  const TailForm form = drop ? kTailPartsDrop : kTailParts;
  const TileChoice c = choose_tile(M, N, K / 64, device_cu_count(), part ? part_bytes : 0);
  if (c.tm < 256) {
    TileGemm t{};
    t.W = Wd, t.X = X, t.N = N, t.row_bytes = 2 * K, t.M = M, t.T = T, t.B = B, t.r = r, t.b_trans = b_trans;
    t.dropped = drop != nullptr;
    if (drop) t.drop = *drop;
    t.Y = Y, t.part = part;
    t.keep = rest && c.splits > 1;
    if (t.keep) *rest = SplitSum{part, c.splits, M * N, Y};
    return launch_tile(t, c, 0, N, st);
  }
  if (c.splits > 1) {
    const hipError_t e = launch_fi<4>(Wd, N, K, X, M, T, B, b_trans, r, r, N, 1.0f, Y, 0, N, st, form, drop,
                                      c.splits, part);
    if (rest) *rest = SplitSum{part, c.splits, M * N, Y};
    return e != hipSuccess || rest ? e : launch_split_sum(part, c.splits, M * N, Y, st);
  }
  return launch_dense(Wd, N, K, X, M, T, r, B, b_trans, r, N, 1.0f, Y, st, part, part_bytes, form, drop);
}

}  // namespace qlora
