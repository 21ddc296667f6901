// gemm_pool.hip -- the dense product of many tokens with what belongs to it in one
// kernel: each token's own adapter, and for a gated block the activation and
// the product of its two halves.
//
//   Y = X Wd^T + T B^T          T = scale_a A_a x of the token's slot, B = B_a
//   H = act(G) o P              of a block's two weights, both so
//
// Wd: the dequantized weight; of a gated block's two, 16 rows of gate and 16 of up
// in turn: a wave's fragments 2 i and 2 i + 1 are the same features of both, and the
// two meet in a lane's registers.  The main loop is dense_quads (dense_tile.h): 256 x
// 64 FI tiles, both operands by buffer->LDS DMA.  A contraction in splits (of
// one weight, with one adapter or none) leaves fp32 sums, the adapter's steps shared
// out to the splits.
//
// The adapters' term follows from global memory, T as kTermParts bf16 parts: for
// each slot among the tile's tokens the ranks 32 at a time, the next ones' loads in
// flight, the tokens of other slots zero.  Tokens of one slot next to each other
// (prompts) make it one pass or two of a tile; the time grows with the slots of a
// tile, here and in T's kernel below (4096 tokens through 8192 x 8192 at rank 16:
// eight prompts 443 us, eight slots in turn 607, a slot to every token 4030; two of
// 22016 x 8192: 2270, 2600, 8570).  With a pool the 256-row tile's term has more live
// values than registers: 88 (one weight) and 133 (two) go to scratch and are read
// back in it; with one adapter and one weight 32 rest there during the term.  The
// main loop has none.
//
// 4096 x 8192 x 22016 with the adapters of eight prompts 1060 us (1.39 PFLOP/s), two
// weights of 22016 x 8192 and 4096 tokens, activation and saved projections
// included, 2105 (1.41): bound by power, as the plain product (937 and 1980 by the
// library).  333 tokens through two of 11008 x 4096 76: bound by the lines that a CU
// keeps in flight.  Joining the halves in a pass of their own took 5090 for the
// second, with dequantization (2290 now).
#include <algorithm>
#include <type_traits>

#include "dense_tile.h"
#include "gate.h"
#include "pool.h"

namespace qlora {
namespace {

__device__ __forceinline__ f32x4_t mfma16x16x32(const bf16x8_t& a, const bf16x8_t& b, const f32x4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

struct PoolGemmArgs {
  PoolGemm g;
  int64_t rows;            // of the stack
  int64_t n_begin;
  int tiles_n, tiles_m, splits, pps;   // pps: pairs of a split
};

// The slots among TOKENS tokens from m0 on, each once, in the order of their
// first tokens, to list[0 .. result - 1], and ids[i] the slot of token m0 + i; room
// holds 2 TOKENS + 8 ints of LDS that no wave reads any more.  All of a workgroup's
// waves call it, TOKENS threads at least.
template <int TOKENS>
__device__ __forceinline__ int tile_slots(const PoolView& p, int64_t m0, int64_t M, int* room) {
  int *ids = room, *list = room + TOKENS, *wave_count = room + 2 * TOKENS;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int a = t < TOKENS && m0 + t < M ? slot_of(p, m0 + t) : -1;
  if (t < TOKENS) ids[t] = a;
  __syncthreads();
  bool first = a >= 0 && (t == 0 || ids[t - 1] != a);   // else a run goes on
  if (__any(first)) {
    bool seen = false;
    for (int q = 0; q < 16 * (w + 1); ++q) {
      const int4 v = *reinterpret_cast<const int4*>(ids + 4 * q);
      seen |= (v.x == a && 4 * q < t) || (v.y == a && 4 * q + 1 < t) || (v.z == a && 4 * q + 2 < t) ||
              (v.w == a && 4 * q + 3 < t);
    }
    first = first && !seen;
  }
  const uint64_t mask = __ballot(first);
  if (lane == 0 && w < TOKENS / 64) wave_count[w] = __popcll(mask);
  __syncthreads();
  int at = __popcll(mask & ((1ull << lane) - 1)), count = 0;
#pragma unroll
  for (int i = 0; i < TOKENS / 64; ++i) {
    if (i < w) at += wave_count[i];
    count += wave_count[i];
  }
  if (first) list[at] = a;
  __syncthreads();
  return count;
}

template <int FI, int G, bool POOL>
__global__ __launch_bounds__(kThreads, 1) void pool_gemm_kernel(PoolGemmArgs p) {
  extern __shared__ __align__(16) char smem[];
  const PoolGemm& a = p.g;
  int tn, tm;
  const int id = xcd_tile_id(), split = id / (p.tiles_n * p.tiles_m), p0 = split * p.pps;
  map_tile_grouped(id - split * p.tiles_n * p.tiles_m, p.tiles_n, p.tiles_m, tn, tm);
  const int64_t n0 = p.n_begin + (int64_t)tn * 64 * FI, m0 = (int64_t)tm * kTile;
  const int64_t K = a.K, M = a.M, N = a.N;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6, wr = wv >> 1, wc = wv & 1, l16 = lane & 15, lg = lane >> 4;

  DenseOps f;
  f.w = __builtin_amdgcn_readfirstlane(wv);
  __builtin_assume(f.w >= 0 && f.w < 4);
  f.npair = min((int)(K >> 6) - p0, p.pps);
  f.wr_ = make_rsrc(a.Wd, (uint32_t)(p.rows * K * 2));
  f.xr = make_rsrc(a.X, (uint32_t)(M * K * 2));
  {
    const int c = (lane & 7) ^ ((4 * f.w + (lane >> 4)) & 7);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      // rows past the end re-read the last row: never stored
      const int row = 8 * (4 * q + f.w) + (lane >> 3);
      if (q < 2 * FI) f.wo[q] = (uint32_t)(min(n0 + row, p.rows - 1) * K * 2 + p0 * 128 + c * 16);
      f.xo[q] = (uint32_t)(min(m0 + row, M - 1) * K * 2 + p0 * 128 + c * 16);
    }
  }
  const int o[2] = {pos128(l16, lg), pos128(l16, 4 + lg)};
  const int am = wc * 32 * FI * 128, bm = wr * 128 * 128;
  constexpr int NA = 2 * FI;
  f32x4_t acc[NA][8];
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  dense_quads<FI>(smem, f, acc, am, bm, o);
  QLORA_WAIT(0, 0);   // the clamped re-loads still in flight
  __builtin_amdgcn_s_barrier();

  if (a.pool.R > 0) {
    const PoolView& pl = a.pool;
    const int first = POOL ? 0 : 32 * split, step = 32 * p.splits;   // one adapter's steps go round the splits
    const int GR = G * pl.R;
    int* ids = reinterpret_cast<int*>(smem);
    int* list = ids + kTile;
    const int slots = POOL ? tile_slots<kTile>(pl, m0, M, ids) : 1;
    int mine[8];   // the slots of the lane's tokens
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = 128 * wr + 16 * j + l16;
      mine[j] = POOL ? ids[at] : (m0 + at < M ? 0 : -1);
    }
    // the lane's rows of B (of one weight) and of T: byte offsets, past the end zero
    constexpr int FG = NA / G;
    constexpr uint32_t kNone = 0x80000000u;   // and no array reaches it (M G R at most 2^27, N R below 2^30)
    static_assert(kTermParts == 2);
    uint32_t brow[FG], trow[8];
#pragma unroll
    for (int i = 0; i < FG; ++i) {
      const int64_t row = n0 + 32 * FI * wc + 16 * G * i;
      const int64_t n = (G == 1 ? row : row >> 1) + l16;
      brow[i] = n < N ? (uint32_t)(n * pl.R + 8 * lg) * 2u : kNone;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) trow[j] = (uint32_t)(min(m0 + 128 * wr + 16 * j + l16, M - 1) * GR + 8 * lg) * 2u;
    const uint32_t part = (uint32_t)(M * GR) * 2u, bytes = (uint32_t)(N * pl.R) * 2u;
    const rsrc_t tr = make_rsrc(a.T, 2 * part);
    // a step: 32 ranks of one weight's fragments, by half of the tokens at a time
    u32x4_t b[2][FG], x[2][2][4];
    auto load_b = [&](int t, int slot, int r, int g, int k0) __attribute__((always_inline)) {
      const rsrc_t br = make_rsrc(pl.B + ((int64_t)slot * G + g) * N * pl.R, bytes);
      const bool in = k0 + 8 * lg < r;
#pragma unroll
      for (int i = 0; i < FG; ++i)
        b[t][i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(br, in ? brow[i] : kNone, 2 * k0, 0));
    };
    auto load_x = [&](int h2, int slot, int r, int g, int k0) __attribute__((always_inline)) {
      const bool in = k0 + 8 * lg < r;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t at = in && mine[4 * h2 + j] == slot ? trow[4 * h2 + j] : kNone;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          x[h2][e][j] = __builtin_bit_cast(
              u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(tr, at, 2 * (k0 + g * pl.R) + (e ? part : 0u), 0));
      }
    };
    // Tokens of other slots have zeros, which an infinity or a NaN of this slot's B
    // would still reach.  A step that holds one, in a wave whose tokens are not all
    // the slot's, is left out and comes in a second turn, summed apart and given to
    // the slot's own tokens alone.
    auto apart = [&](int t, bool mixed) __attribute__((always_inline)) {
      bool found = false;
      if (POOL && mixed) {
#pragma unroll
        for (int i = 0; i < FG; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            found |= (b[t][i][e] & 0x7F80u) == 0x7F80u || (b[t][i][e] & 0x7F800000u) == 0x7F800000u;
        found = __any(found);
      }
      return found;
    };
    bool again = false;
    auto mul = [&](int t, int h2, int g) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < FG; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mfma_acc<false>(__builtin_bit_cast(bf16x8_t, b[t][i]), __builtin_bit_cast(bf16x8_t, x[h2][e][j]),
                            acc[G * i + g][4 * h2 + j]);
    };
    // Whether the wave has tokens of the slot, and others.
    auto present = [&](int slot, bool& mixed) __attribute__((always_inline)) {
      bool some = mine[0] == slot, all = some;
#pragma unroll
      for (int j = 1; j < 8; ++j) some = some || mine[j] == slot, all = all && mine[j] == slot;
      mixed = !__all(all);
      return (bool)__any(some);
    };
    for (int e = 0; e < slots; ++e) {
      const int slot = POOL ? __builtin_amdgcn_readfirstlane(list[e]) : 0;
      bool mixed = false;
      if (POOL && !present(slot, mixed)) continue;
      const int r = POOL ? rank_of(pl, slot) : pl.R;
      if (first >= r) continue;
      load_b(0, slot, r, 0, first);
      load_x(0, slot, r, 0, first);
      for (int k0 = first; k0 < r; k0 += step)
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int t = G == 1 ? 0 : g, gn = g + 1 < G ? g + 1 : 0, kn = g + 1 < G ? k0 : k0 + step;
          load_x(1, slot, r, g, k0);
          const bool skip = apart(t, mixed);
          again = again || skip;
          if (!skip) mul(t, 0, g);
          if (G == 2) load_b(t ^ 1, slot, r, gn, kn);
          load_x(0, slot, r, gn, kn);
          if (!skip) mul(t, 1, g);
          if (G == 1) load_b(0, slot, r, gn, kn);
        }
    }
    mfma_done();
    if (POOL && again) {
      for (int e = 0; e < slots; ++e) {
        const int slot = __builtin_amdgcn_readfirstlane(list[e]);
        bool mixed;
        if (!present(slot, mixed)) continue;
        const int r = rank_of(pl, slot);
        for (int k0 = 0; k0 < r; k0 += 32)
#pragma unroll
          for (int g = 0; g < G; ++g) {
            load_b(0, slot, r, g, k0);
            if (!apart(0, mixed)) continue;
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              load_x(h2, slot, r, g, k0);
#pragma unroll
              for (int i = 0; i < FG; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  f32x4_t& to = acc[G * i + g][4 * h2 + j];
                  const bf16x8_t w = __builtin_bit_cast(bf16x8_t, b[0][i]);
                  f32x4_t y = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
                  y = mfma16x16x32(w, __builtin_bit_cast(bf16x8_t, x[h2][1][j]),
                                   mfma16x16x32(w, __builtin_bit_cast(bf16x8_t, x[h2][0][j]), y));
                  const bool own = mine[4 * h2 + j] == slot;
#pragma unroll
                  for (int v = 0; v < 4; ++v) to[v] = own ? to[v] + y[v] : to[v];
                }
            }
          }
      }
    }
  }
  if constexpr (G == 1 && !POOL) {
    if (a.part) {   // the sums as they are, [M x N] of each split
#pragma unroll
      for (int m = 0; m < NA; ++m)
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const int64_t row = m0 + 128 * wr + 16 * n + l16, col = n0 + 32 * FI * wc + 16 * m + 4 * lg;
          if (row < M && col < N)   // N % 8 == 0
            *reinterpret_cast<f32x4_t*>(a.part + ((int64_t)split * M + row) * N + col) = acc[m][n];
        }
      return;
    }
  }
  // Out through LDS: lane (l16, lg) of fragments (m, n) has token 16 n + l16, features 4
  // lg .. of 16 m.
  auto store = [&](auto&& value, auto per, bf16_t* out, int64_t ld, int64_t c0) __attribute__((always_inline)) {
    constexpr int P = decltype(per)::value;   // fragments of 16 features a wave stores
    constexpr int U = 8 * P, SM = U % 32 == 0 ? 31 : U % 16 == 0 ? 15 : 7;
    lds_free_for_output();
#pragma unroll
    for (int m = 0; m < P; ++m)
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const f32x4_t v = value(m, n);
        lds_put4<U, SM>(smem, wr * 128 + 16 * n + l16, wc * 4 * P + 4 * m + lg, v[0], v[1], v[2], v[3]);
      }
    __syncthreads();
    lds_tile_out<U, SM>(smem, out, ld, M, N, m0, c0);
  };
  if constexpr (G == 1) {
    store([&](int m, int n) { return acc[m][n]; }, std::integral_constant<int, NA>{}, a.Y, N, n0);
  } else {
    const std::integral_constant<int, FI> half{};
    const int64_t c0 = n0 >> 1;
    if (a.GU) {
      store([&](int m, int n) { return acc[2 * m][n]; }, half, a.GU, 2 * N, c0);
      store([&](int m, int n) { return acc[2 * m + 1][n]; }, half, a.GU + N, 2 * N, c0);
    }
    auto h = [&](auto act) __attribute__((always_inline)) {
      store([&](int m, int n) {
        f32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = act_of<decltype(act)::value>(acc[2 * m][n][e]) * acc[2 * m + 1][n][e];
        return v;
      }, half, a.Y, N, c0);
    };
    if (a.act == kActSilu)
      h(std::integral_constant<int, kActSilu>{});
    else
      h(std::integral_constant<int, kActGelu>{});
  }
}

template <int FI, int G, bool POOL>
hipError_t launch_tiles(const PoolGemm& g, int64_t rows, int64_t n_begin, int64_t n_rows, hipStream_t st) {
  auto* fn = &pool_gemm_kernel<FI, G, POOL>;
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), (int)kLdsHalves);
  if (e != hipSuccess) return e;
  PoolGemmArgs p{g, rows, n_begin, (int)((n_rows + 64 * FI - 1) / (64 * FI)), (int)((g.M + kTile - 1) / kTile),
                 g.part ? g.splits : 1, 0};
  p.pps = ((int)(g.K >> 6) + p.splits - 1) / p.splits;
  hipLaunchKernelGGL(fn, dim3(p.tiles_n * p.tiles_m * p.splits), dim3(kThreads), kLdsHalves, st, p);
  return hipGetLastError();
}
template <int G, bool POOL>
hipError_t launch_fi(int fi, const PoolGemm& g, int64_t rows, int64_t n_begin, int64_t n_rows, hipStream_t st) {
  if (fi == 3) return launch_tiles<3, G, POOL>(g, rows, n_begin, n_rows, st);
  if (fi == 2) return launch_tiles<2, G, POOL>(g, rows, n_begin, n_rows, st);
  return launch_tiles<4, G, POOL>(g, rows, n_begin, n_rows, st);
}

// Rounds of the card that `rows` rows in tiles of 64 fi take, in rounds of 256-row
// tiles, the narrower ones' extra reads charged as for the plain dense product.
int64_t pool_rows(int64_t N, int G) { return G == 1 ? N : (N + kPoolTurn - 1) / kPoolTurn * 2 * kPoolTurn; }
double rounds(int64_t rows, int64_t tiles_m, int fi, int cus) {
  const int64_t tiles = (rows + 64 * fi - 1) / (64 * fi) * tiles_m;
  return (double)((tiles + cus - 1) / cus) * fi / 4.0 * (fi == 4 ? 1.0 : fi == 3 ? 1.06 : 1.12);
}
// The first `whole` rows in 256-row tiles, whole rounds of them, the others in
// tiles of 64 fi: what takes the least time.  A gated block's rows come in turns of
// 32 (16 of each weight), and a tile may begin at any of them: every fi fits after
// whole rounds.  Two weights of 22016 x 8192 and 4096 tokens: 40960 rows in ten
// rounds, then the rest in tiles of 192.
struct PoolTiles {
  int64_t whole;
  int fi;
};
PoolTiles pool_tiles(int64_t N, int64_t M, int G, int cus) {
  const int64_t tiles_m = (M + kTile - 1) / kTile;
  PoolTiles best{0, 4};
  double least = 1e30;
  for (int fi = 4; fi >= 2; --fi) {
    const int64_t rows = pool_rows(N, G);
    const int64_t round = std::max<int64_t>(1, cus / tiles_m) * kTile;   // rows of a round of 256-row tiles
    for (int k = 0; k < 2; ++k) {
      const int64_t whole = k == 0 || fi == 4 || tiles_m > cus ? 0 : rows / round * round;
      const double cost = (double)(whole / round) + (rows > whole ? rounds(rows - whole, tiles_m, fi, cus) : 0.0);
      if (cost < least) least = cost, best = PoolTiles{whole, fi};
    }
  }
  return best;
}

}  // namespace

// ---------------------------------------------------------------------------
// T of many tokens: fp32 partial sums [splits][M][G R] of scale_a A_a x, 128 tokens
// and RP of the slot's G R rank rows per workgroup, once for each slot among the
// tokens.  Stages of 64 columns, one 128-byte line of every row, in a ring of four
// that a fifth wave fills (a CU keeps about 90 lines in flight, and their issue
// stalls there).  4096 x 22016 of eight prompts at rank 64 76 us (180 MB at 2.4 TB/s),
// 1200 x 5120 x 2 at rank 32 19: bound by those lines.  Each slot of a tile is a pass
// over its tokens' columns, all 128 multiplied.
// ---------------------------------------------------------------------------
namespace {

constexpr int kRing = 4, kAhead = kRing - 1, kUThreads = kThreads + 64, kUTokens = 128;
template <int RP>
struct UShape {
  static constexpr int kP = kUTokens * 128, kQ = RP * 128, kStage = kP + kQ, kQDma = kQ / 1024;
  static constexpr int kWait = (kAhead - 1) * (16 + kQDma) < 63 ? (kAhead - 1) * (16 + kQDma) : 63;
  static constexpr int kIds = kRing * kStage, kLds = kIds + (2 * kUTokens + 8) * 4;
};

template <int RP>
__global__ __launch_bounds__(kUThreads, 1) void pool_u_kernel(PoolView p, const bf16_t* __restrict__ X, int64_t M,
                                                              int64_t K, int stages_per_split, int tiles_m,
                                                              float* __restrict__ part) {
  using S = UShape<RP>;
  extern __shared__ __align__(16) char smem[];
  const int tm = blockIdx.x % tiles_m, sp = blockIdx.x / tiles_m, GR = p.G * p.R, j0 = blockIdx.y * RP;
  const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63, lr = lane & 31, h = lane >> 5;
  const int64_t m0 = (int64_t)tm * kUTokens;
  const int s0 = sp * stages_per_split, s1 = min((int)(K >> 6), s0 + stages_per_split);   // no split is empty
  int* ids = reinterpret_cast<int*>(smem + S::kIds);
  const int slots = tile_slots<kUTokens>(p, m0, M, ids);
  const rsrc_t pr = make_rsrc(X + m0 * K, (uint32_t)(min((int64_t)kUTokens, M - m0) * K * 2));   // rows past M: zero
  for (int e = blockIdx.z; e < slots; e += gridDim.z) {
    const int slot = __builtin_amdgcn_readfirstlane(ids[kUTokens + e]), rank = rank_of(p, slot);
    if (w == 4) {   // the wave that brings the stages
      const rsrc_t qr = make_rsrc(p.A + ((int64_t)slot * GR + j0) * K, (uint32_t)((int64_t)min(RP, GR - j0) * K * 2));
      uint32_t po[16], qo[S::kQDma];
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int row = 8 * q + (lane >> 3);
        po[q] = (uint32_t)(row * K * 2 + 16 * ((lane & 7) ^ ((row >> 1) & 7)));
      }
#pragma unroll
      for (int q = 0; q < S::kQDma; ++q) {   // rows past G R: zero, never stored
        const int row = 8 * q + (lane >> 3);
        qo[q] = (uint32_t)(row * K * 2 + 16 * ((lane & 7) ^ ((row >> 1) & 7)));
      }
      auto dma = [&](int st, int slot_) __attribute__((always_inline)) {
        const uint32_t ss = (uint32_t)min(st, s1 - 1) * 128u;   // past the split: its last stage again, never read
        char* base = smem + slot_ * S::kStage;
#pragma unroll
        for (int q = 0; q < 16; ++q) dma16(pr, base + q * 1024, po[q], ss);
#pragma unroll
        for (int q = 0; q < S::kQDma; ++q) dma16(qr, base + S::kP + q * 1024, qo[q], ss);
      };
#pragma unroll
      for (int b = 0; b < kAhead; ++b) dma(s0 + b, b);
      int ring = kRing - 1;
      for (int st = s0; st < s1; ++st) {
        QLORA_WAIT(S::kWait, 0);
        __builtin_amdgcn_s_barrier();   // stage st has landed, and stage st - 1 has been read
        dma(st + kAhead, ring);
        ring = ring == kRing - 1 ? 0 : ring + 1;
      }
      QLORA_WAIT(0, 0);
    } else {
      constexpr int FJ = RP / 32;
      f32x16_t acc[FJ];
#pragma unroll
      for (int f = 0; f < FJ; ++f)
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[f][k] = 0.0f;
      int ring = 0;
      for (int st = s0; st < s1; ++st) {
        QLORA_WAIT(63, 0);   // this wave's reads of stage st - 1
        __builtin_amdgcn_s_barrier();
        const char* base = smem + ring * S::kStage;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const bf16x8_t b = rd16(base + pos128(32 * w + lr, 2 * kk + h));
#pragma unroll
          for (int f = 0; f < FJ; ++f)
            acc[f] = mfma32x32x16(rd16(base + S::kP + pos128(32 * f + lr, 2 * kk + h)), b, acc[f]);
        }
        ring = ring == kRing - 1 ? 0 : ring + 1;
      }
      // D[j][m]: lane (lr, h): token m0 + 32 w + lr, ranks j0 + 32 f + 8 q + 4 h + 0..3
      const float sc = scale_of(p, slot);
      if (ids[32 * w + lr] == slot) {
        float* out = part + ((int64_t)sp * M + m0 + 32 * w + lr) * GR;
#pragma unroll
        for (int f = 0; f < FJ; ++f)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int j = j0 + 32 * f + 8 * q + 4 * h;
            if (j < GR && j % p.R < rank)
              *reinterpret_cast<float4*>(out + j) = make_float4(acc[f][4 * q] * sc, acc[f][4 * q + 1] * sc,
                                                                acc[f][4 * q + 2] * sc, acc[f][4 * q + 3] * sc);
          }
      }
    }
    __syncthreads();   // every wave is done with the ring
  }
}

struct USplit {
  int tiles, sps, splits;
};
// About one workgroup for each of 256 CUs (fixed: the workspace's size), at least
// eight stages each.
USplit u_split(int64_t M, int64_t K) {
  USplit s{(int)((M + kUTokens - 1) / kUTokens), 0, 0};
  const int nst = (int)(K >> 6), want = std::max(1, std::min((256 + s.tiles - 1) / s.tiles, nst / 8));
  s.sps = (nst + want - 1) / want;
  s.splits = (nst + s.sps - 1) / s.sps;
  return s;
}

}  // namespace

size_t pool_u_part_bytes(int64_t M, int64_t K, int GR) {
  return (size_t)u_split(M, K).splits * (size_t)M * (size_t)GR * sizeof(float);
}

hipError_t start_pool_u(const PoolView& p, const bf16_t* X, int64_t M, int64_t K, float* part, bf16_t* parts, float* T,
                        Ride* rest, hipStream_t st) {
  const USplit s = u_split(M, K);
  const int GR = p.G * p.R, rp = GR <= 64 ? 64 : 128;
  auto* fn = rp == 64 ? &pool_u_kernel<64> : &pool_u_kernel<128>;
  const int lds = rp == 64 ? UShape<64>::kLds : UShape<128>::kLds;
  hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), lds);
  if (e != hipSuccess) return e;
  // The slots of a tile go round the grid's third dimension: two workgroups, or as
  // many more as CUs would have nothing to do (393 tokens of 15 slots mixed, K 832: 42
  // us with two, 14 with sixteen).
  const int ranks = (GR + rp - 1) / rp, idle = 256 / (s.tiles * s.splits * ranks);
  const int turns = std::min(p.slots, std::max(2, std::min(16, idle)));
  hipLaunchKernelGGL(fn, dim3(s.tiles * s.splits, ranks, turns), dim3(kUThreads), lds, st, p, X, M, K, s.sps, s.tiles, part);
  // (of tokens and ranks without an adapter the sums mean nothing, and are not read)
  *rest = Ride{};
  rest->kind = kRideSum, rest->blocks = (int)((M * GR / 4 + 255) / 256);
  rest->part = part, rest->splits = s.splits, rest->n = M * GR, rest->scale = rest->s = 1.0f;
  rest->parts = parts, rest->full = T;
  return hipGetLastError();
}

hipError_t launch_pool_gemm(const PoolGemm& g, hipStream_t st) {
  const int G = g.pool.G;
  const bool many = g.pool.ids != nullptr && g.pool.R > 0;
  if (g.part && (G != 1 || many)) return hipErrorInvalidValue;
  const PoolTiles p = pool_tiles(g.N, g.M, G, device_cu_count());
  const int64_t rows = pool_rows(g.N, G);
  auto go = [&](int fi, int64_t begin, int64_t n) {
    if (G == 1) return many ? launch_fi<1, true>(fi, g, rows, begin, n, st) : launch_fi<1, false>(fi, g, rows, begin, n, st);
    return many ? launch_fi<2, true>(fi, g, rows, begin, n, st) : launch_fi<2, false>(fi, g, rows, begin, n, st);
  };
  if (g.part) return go(4, 0, rows);
  if (p.whole > 0) {
    const hipError_t e = go(4, 0, p.whole);
    if (e != hipSuccess || p.whole >= rows) return e;
  }
  return go(p.fi, p.whole, rows - p.whole);
}

}  // namespace qlora
