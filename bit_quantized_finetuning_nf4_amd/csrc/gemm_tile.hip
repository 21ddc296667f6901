// gemm_tile.hip -- the products of a middling number of tokens, or of few
// channels: Y = X W^T and the adapter's term, in tiles small enough to reach
// every CU, for bf16 and for 8-bit operands.
//
//   forward   Y = X W^T + T B^T             (B [N x r], T = s U)
//   dX        Y = X W^T + T A               (A [r x N], W a transposed weight, T = s G)
//   dX under dropout                        (T A masked as Y's own shape)
//
// T comes as kTermParts bf16 matrices, summed as one of twice the rank.
//
// TM tokens x TN channels per workgroup, waves 2 x 2 over the tile, a ring of
// NS stages of 128 bytes of all its rows, brought by buffer->LDS DMA.  The
// fragments of a 32-byte step are read one step ahead of their MFMAs.  The
// stage's barrier stands before its last step's MFMAs, which hide the first
// reads of the next stage: there every wave has read all of the stage, so the
// DMA of stage st + NS goes into its slot at once.
//
// What bounds it is the compute unit's DMA: about 90 cache lines in flight, so
// 17-22 bytes a clock at the latencies of operands that come from beyond L2
// (57 from L2 alone), whatever the depth of the ring; without its MFMAs and
// LDS reads the loop takes the same time.  So the tile is chosen by the bytes
// that the busiest CU brings (choose_tile), and where even the smallest tiles
// leave CUs idle the contraction is split: fp32 parts, added in order, or the
// 32-bit integers as they are, whose sum stays exact (gemm_i8.hip).
#include <algorithm>
#include <type_traits>

#include "dense_tile.h"
#include "rng.h"

namespace qlora {
namespace {

enum Tail : int { kTailFwd = 0, kTailDx = 1, kTailDxDrop = 2 };

struct TileArgs {
  TileGemm g;
  int64_t n_begin;
  int tiles_n, tiles_m, sps;   // sps: stages per split of the contraction
};

template <class MM, int TM, int TN, int NS, int TAIL>
__global__ __launch_bounds__(kThreads, 1) void tile_kernel(TileArgs p) {
  constexpr bool kI8 = std::is_same<MM, MmI8>::value;
  constexpr int FI = TN / 64, FJ = TM / 64;         // 32-row fragments per wave
  constexpr int kRows = TM + TN, kSlot = kRows * 128, kDma = kRows / 32;   // DMA instructions per wave and stage
  extern __shared__ __align__(16) char smem[];
  const TileGemm& g = p.g;
  int tn, tm;
  int id = xcd_tile_id();
  const int split = id / (p.tiles_n * p.tiles_m);
  map_tile_grouped(id - split * p.tiles_n * p.tiles_m, p.tiles_n, p.tiles_m, tn, tm);
  const int64_t M = g.M, N = g.N, ld = g.row_bytes;
  const int64_t n0 = p.n_begin + (int64_t)tn * TN, m0 = (int64_t)tm * TM;
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6), wr = w >> 1, wc = w & 1;
  const int lr = lane & 31, h = lane >> 5;
  const int s0 = split * p.sps, nst = min((int)(ld >> 7) - s0, p.sps);
  // weight rows 0 .. TN - 1, then token rows; instruction q of wave w brings
  // rows 8 (4 q + w) .. + 7; rows past the end re-read the last one, never
  // stored
  const rsrc_t wres = make_rsrc(g.W, (uint32_t)(N * ld)), xres = make_rsrc(g.X, (uint32_t)(M * ld));
  uint32_t off[kDma];
#pragma unroll
  for (int q = 0; q < kDma; ++q) {
    const int row = 8 * (4 * q + w) + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
    const int64_t src = q < TN / 32 ? min(n0 + row, N - 1) : min(m0 + row - TN, M - 1);
    off[q] = (uint32_t)(src * ld + 16 * c);
  }
  auto dma = [&](char* slot, int st, int q) __attribute__((always_inline)) {
    // past the end: re-loads the last stage, never read
    dma16(q < TN / 32 ? wres : xres, slot + 8 * (4 * q + w) * 128, off[q], (uint32_t)(s0 + min(st, nst - 1)) * 128u);
  };
  typename MM::acc_t acc[FI][FJ];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
#pragma unroll
  for (int a = 0; a < NS; ++a)
#pragma unroll
    for (int q = 0; q < kDma; ++q) dma(smem + a * kSlot, a, q);
  int o[4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) o[kk] = pos128(lr, 2 * kk + h);
  const int am = wc * 32 * FI * 128, bm = (TN + wr * 32 * FJ) * 128;
  bf16x8_t a[2][FI], b[2][FJ];
  auto read = [&](const char* base, int kk, int set) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FI; ++i) a[set][i] = rd16(base + am + i * 32 * 128 + o[kk]);
#pragma unroll
    for (int j = 0; j < FJ; ++j) b[set][j] = rd16(base + bm + j * 32 * 128 + o[kk]);
  };
  QLORA_WAIT((NS - 1) * kDma, 0);
  __builtin_amdgcn_s_barrier();
  read(smem, 0, 0);
  int slot = 0;
  for (int st = 0; st < nst; ++st) {
    char* cur = smem + slot * kSlot;
    slot = slot == NS - 1 ? 0 : slot + 1;
#pragma unroll
    for (int kk = 0; kk < 3; ++kk) {
      read(cur, kk + 1, (kk + 1) & 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) acc[i][j] = MM::mma(a[kk & 1][i], b[kk & 1][j], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    QLORA_WAIT((NS - 2) * kDma, 0);   // stage st + 1 has landed; this wave has read all of stage st
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(smem + slot * kSlot, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int x = 0; x < FI * FJ; ++x) {
      acc[x / FJ][x % FJ] = MM::mma(a[1][x / FJ], b[1][x % FJ], acc[x / FJ][x % FJ]);
#pragma unroll
      for (int q = 0; q < kDma; ++q)
        if (q * FI * FJ / kDma == x) dma(cur, st + NS, q);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  QLORA_WAIT(0, 0);   // no DMA still in flight, and
  __builtin_amdgcn_s_barrier();   // no wave still reads the ring: the results pass through it

  // D[channel][token]: lane (lr, h): token lr, channels 8 q + 4 h .. of a
  // block.  The adapter's product is summed on its own (it is masked, or added
  // to scaled integer sums), from global memory: 8 ranks of a part per lane half
  // and MFMA, the loads of the next 16 ranks of all blocks in flight meanwhile.
  const int r = split == 0 && !(kI8 && g.part) ? g.r : 0;
  [[maybe_unused]] float x[FJ];
  [[maybe_unused]] f32x4_t sc[FI][4];
  if constexpr (kI8) {
#pragma unroll
    for (int j = 0; j < FJ; ++j) x[j] = g.sx[min(m0 + 32 * (FJ * wr + j) + lr, M - 1)];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)   // N % 8 == 0
        sc[i][q] = *reinterpret_cast<const f32x4_t*>(g.sw + min(n0 + 32 * (FI * wc + i) + 8 * q + 4 * h, N - 4));
  }
  f32x16_t y[FI][FJ];
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) y[i][j][e] = 0.0f;
  if (r > 0) {
    constexpr int kB = TAIL == kTailFwd ? 4 : 8;   // words of a weight fragment as loaded
    uint32_t fb[2][FI][kB];
    u32x4_t fu[2][FJ];
    static_assert(kTermParts == 2);
    auto load = [&](int c, int set) __attribute__((always_inline)) {
      const int kp = c + 8 * h, part = kp >= r ? 1 : 0, k = kp - part * r;
      const bf16_t* T = g.T + (part ? M * g.r : 0);   // past both parts (r % 8 == 0), or the rows: zero
#pragma unroll
      for (int i = 0; i < FI; ++i) {
        const int64_t n = n0 + 32 * (FI * wc + i) + lr;
        const bool in = k < r && n < N;
        if constexpr (TAIL == kTailFwd) {
          u32x4_t v = {0u, 0u, 0u, 0u};
          if (in) v = *reinterpret_cast<const u32x4_t*>(g.B + n * g.r + k);
#pragma unroll
          for (int e = 0; e < 4; ++e) fb[set][i][e] = v[e];
        } else {   // A's rows: eight ranks of one column
#pragma unroll
          for (int e = 0; e < 8; ++e) fb[set][i][e] = in ? g.B[(int64_t)(k + e) * N + n] : 0u;
        }
      }
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        const int64_t m = m0 + 32 * (FJ * wr + j) + lr;
        fu[set][j] = u32x4_t{0u, 0u, 0u, 0u};
        if (k < r && m < M) fu[set][j] = *reinterpret_cast<const u32x4_t*>(T + m * g.r + k);
      }
    };
    auto mul = [&](int set) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < FI; ++i) {
        u32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (TAIL == kTailFwd)
            v[e] = fb[set][i][e];
          else
            v[e] = fb[set][i][2 * e] | fb[set][i][2 * e + 1] << 16;
        }
#pragma unroll
        for (int j = 0; j < FJ; ++j)
          y[i][j] = mfma32x32x16(__builtin_bit_cast(bf16x8_t, v), __builtin_bit_cast(bf16x8_t, fu[set][j]), y[i][j]);
      }
    };
    load(0, 0);
    for (int c = 0; c < kTermParts * r; c += 32) {
      load(c + 16, 1);
      mul(0);
      load(c + 32, 0);
      mul(1);
    }
  }
  if constexpr (TAIL == kTailDxDrop) {
    if (r > 0) {
      const DropKey key = drop_key(g.drop);
#pragma unroll
      for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) {
          const uint32_t m = (uint32_t)(m0 + 32 * (FJ * wr + j) + lr);
          const uint32_t bits = mask_bits(m * (uint32_t)(N >> 3) + (uint32_t)((n0 + 32 * (FI * wc + i)) >> 3), key);
#pragma unroll
          for (int e = 0; e < 16; ++e) y[i][j][e] = masked(y[i][j][e], bits, e);
        }
    }
  }
  // through LDS, so that whole lines of a token's row are stored: rows of TN
  // values and 16 bytes (a store of four channels of 32 tokens from the
  // registers is 64 pieces of lines, which L2 takes one at a time: with those,
  // and the adapter's loads a block at a time, 333 x 11008 x 4096 took 35.1 us
  // at rank 16 and 39.2 at rank 64, 30.4 and 31.3 this way; T's second part adds
  // nothing to the first and 1.8 to the second)
  auto value = [&](int i, int j, int q, int e) __attribute__((always_inline)) {
    if constexpr (kI8)
      return scaled_sum(acc[i][j][4 * q + e], sc[i][q][e], x[j]) + y[i][j][4 * q + e];
    else
      return acc[i][j][4 * q + e] + y[i][j][4 * q + e];
  };
  auto out = [&](auto* dst, int64_t row0, auto pack) __attribute__((always_inline)) {
    constexpr int kSize = (int)sizeof(*dst), kPitch = TN * kSize + 16, kRow = TN * kSize / 16;
#pragma unroll
    for (int j = 0; j < FJ; ++j)
#pragma unroll
      for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          pack(smem + (32 * (FJ * wr + j) + lr) * kPitch + (32 * (FI * wc + i) + 8 * q + 4 * h) * kSize, i, j, q);
    __syncthreads();
#pragma unroll
    for (int p = 0; p < TM * kRow / kThreads; ++p) {
      const int id = t + kThreads * p, row = id / kRow, c = id % kRow;
      const int64_t n = n0 + c * (16 / kSize);
      if (m0 + row < M && n < N)
        *reinterpret_cast<uint4*>(dst + (row0 + row) * N + n) = *reinterpret_cast<const uint4*>(smem + row * kPitch + 16 * c);
    }
  };
  if (g.part)
    out(static_cast<float*>(g.part), (int64_t)split * M + m0, [&](char* p, int i, int j, int q)
                                                                  __attribute__((always_inline)) {
      if constexpr (kI8)
        *reinterpret_cast<int4*>(p) = make_int4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                                acc[i][j][4 * q + 3]);
      else
        *reinterpret_cast<float4*>(p) = make_float4(value(i, j, q, 0), value(i, j, q, 1), value(i, j, q, 2),
                                                    value(i, j, q, 3));
    });
  else
    out(g.Y, m0, [&](char* p, int i, int j, int q) __attribute__((always_inline)) {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(value(i, j, q, 0), value(i, j, q, 1)),
                                                pack_bf16x2(value(i, j, q, 2), value(i, j, q, 3)));
    });
}

template <class MM, int TM, int TN, int NS, int TAIL>
hipError_t launch(TileGemm g, int splits, int64_t n_begin, int64_t n_rows, hipStream_t st) {
  auto* fn = &tile_kernel<MM, TM, TN, NS, TAIL>;
  constexpr int lds = NS * (TM + TN) * 128;
  static_assert(lds >= TM * (TN * 4 + 16), "the results pass through the ring");
  hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), lds);
  if (e != hipSuccess) return e;
  TileArgs p{g, n_begin, (int)((n_rows + TN - 1) / TN), (int)((g.M + TM - 1) / TM), 0};
  const int lines = (int)(g.row_bytes / 128);
  p.sps = (lines + splits - 1) / splits;
  if (splits == 1 && !g.keep) p.g.part = nullptr;
  hipLaunchKernelGGL(fn, dim3(p.tiles_n * p.tiles_m * splits), dim3(kThreads), lds, st, p);
  if ((e = hipGetLastError()) != hipSuccess || splits == 1 || g.keep || std::is_same<MM, MmI8>::value) return e;
  return launch_split_sum(static_cast<const float*>(g.part), splits, g.M * g.N, g.Y, st);
}

template <class MM, int TAIL>
hipError_t launch_shape(const TileGemm& g, const TileChoice& c, int64_t n_begin, int64_t n_rows, hipStream_t st) {
  if (c.tm == 192) return launch<MM, 192, 128, 3, TAIL>(g, c.splits, n_begin, n_rows, st);
  if (c.tm == 128) return launch<MM, 128, 128, 4, TAIL>(g, c.splits, n_begin, n_rows, st);
  if (c.tn == 128) return launch<MM, 64, 128, 3, TAIL>(g, c.splits, n_begin, n_rows, st);
  return launch<MM, 64, 64, 4, TAIL>(g, c.splits, n_begin, n_rows, st);
}

// A round of tiles of tm tokens x tn channels: the bytes of the tile's rows
// that a CU brings in a ns, and what a round costs beside them, in us.  Fitted
// to the 8-bit product's times at 34 sizes (33 to 4096 tokens, 512 to 22016
// channels and columns, seven shapes each; 8-19 % rms), where the shape that
// they choose is within 0.3 % of the fastest on the mean and 7 % at most.
struct Shape {
  int tm, tn;
  double rate, fixed;
};
constexpr Shape kShapes[] = {{64, 64, 71e3, 2.2},   {64, 128, 70e3, 3.2},  {128, 128, 69e3, 5.5}, {192, 128, 66e3, 5.5},
                             {256, 128, 59e3, 6.0}, {256, 192, 61e3, 8.8}, {256, 256, 58e3, 10.5}};
double round_cost(const Shape& t, int64_t lines) {
  return (double)(t.tm + t.tn) * 128.0 * (double)lines / t.rate + t.fixed;
}
constexpr int kMaxSplits = 32;
constexpr int kMinLines = 4;   // stages of a split, at least

}  // namespace

double full_round_cost(int64_t lines) { return round_cost(kShapes[6], lines); }

// The shape, and the split of the contraction, with the least time (256 x 192
// and 256 x 128 tiles are not split: where they would be, another shape is).
// Measured in us for 8-bit operands (tokens x channels x K):
//   128 x 8192 x 8192    64x64 24   64x128 32   128x128 40
//                        128x128 in four splits 23.5, in two 29
//   512 x 8192 x 22016   128x128 112   192x128 126   64x64 175
//                        256x256 in four splits 102, unsplit 231
//   333 x 11008 x 4096   192x128 29   256x128 39   128x128 41   256x256 49
//   768 x 11008 x 4096   256x192 49   256x256 52   192x128 58   64x64 69
//   2048 x 4096 x 22016  256x256 in two splits 161   256x128 186   128x128 209
//   40 x 840 x 19840     64x64 in eight splits 11.3, unsplit 34
// Rings of two stages lose (151 us against 115 with four, 128 x 128 at 512 x
// 8192 x 22016); past three or four nothing changes.  A split adds a launch and
// its parts' way through memory (mostly the last-level cache).
TileChoice choose_tile(int64_t M, int64_t N, int64_t lines, int cus, size_t part_bytes, bool small) {
  TileChoice best{0, 0, 1, 1e30};
  for (const Shape& t : kShapes) {
    if (small && t.tm == 256) break;
    const int64_t tiles = (M + t.tm - 1) / t.tm * ((N + t.tn - 1) / t.tn);
    for (int want = 1; want <= (t.tm == 256 && t.tn != 256 ? 1 : kMaxSplits); ++want) {
      if (want > 1 && (int64_t)want * kMinLines > lines) break;
      const int64_t sps = (lines + want - 1) / want;
      const int splits = (int)((lines + sps - 1) / sps);   // no split is empty
      if (splits != want) continue;
      const size_t bytes = (size_t)splits * (size_t)M * (size_t)N * sizeof(float);
      if (splits > 1 && bytes > part_bytes) break;
      double cost = (double)((tiles * splits + cus - 1) / cus) * round_cost(t, sps);
      if (splits > 1) cost += 1.0 + 0.3 * splits + (double)bytes / 3.3e6;
      if (cost <= best.cost) best = TileChoice{t.tm, t.tn, splits, cost};
    }
  }
  return best;
}

// Room for the split that choose_tile would take with room enough, on a card
// of kSplitCus CUs, so that the size does not depend on the device; with
// less, or with more CUs, it takes what fits.
constexpr int kSplitCus = 256;
size_t tile_part_bytes(int64_t M, int64_t N, int64_t lines) {
  const TileChoice c = choose_tile(M, N, lines, kSplitCus, (size_t)1 << 62);
  return c.splits > 1 ? (size_t)c.splits * (size_t)M * (size_t)N * sizeof(float) : 0;
}

hipError_t launch_tile(const TileGemm& g, const TileChoice& c, int64_t n_begin, int64_t n_rows, hipStream_t st) {
  if (g.sw) return launch_shape<MmI8, kTailFwd>(g, c, n_begin, n_rows, st);
  if (!g.b_trans) return launch_shape<MmBf16, kTailFwd>(g, c, n_begin, n_rows, st);
  return g.dropped ? launch_shape<MmBf16, kTailDxDrop>(g, c, n_begin, n_rows, st)
                   : launch_shape<MmBf16, kTailDx>(g, c, n_begin, n_rows, st);
}

}  // namespace qlora
