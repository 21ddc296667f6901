// stream.hip -- the frozen product of few tokens, X deq(W_g)^T for G 4-bit
// weights side by side, as fp32 parts; the adapters and what follows are the
// next launch's (pool.hip).  Their first half, A_a x, is done by the same launch.
//
// A weight enters the product as the value that it stands for, RNE_bf16(RN32(L
// t)): the sums have no other error than fp32's.
//
//   * Work.  A unit is 256 rows of the stack by 256 columns (a span), for 16 NT
//     tokens.  The units lie on a line, tile by tile, that the workgroups share
//     out evenly (StreamLine): each writes one part for each tile that its stretch
//     touches, and a tile's parts are those of consecutive workgroups.  Two
//     workgroups share a CU.  The adapters' tasks go to workgroups that have fewer
//     units, or none, before these.
//   * Codes.  Eight waves take two sets of 16 rows each.  Of a set's span a lane
//     loads 16 bytes twice, each load over eight whole 128-byte lines (loads over
//     sixteen rows stall in the vector L1's address translation); an exchange
//     between lanes 8 apart gives lane (c, g) the 16-byte chunks g and 4 + g of
//     its own row c.  The next unit's are in flight meanwhile.
//   * A code byte is two weights: a table in LDS gives their two fp32 levels (256
//     entries of 8 bytes, a copy for each lane of a half wave, so no two of its
//     lanes meet in a bank: 64 KiB), one product each with the block's scale, one
//     conversion for both: two vector instructions a weight, 0.7 more for the
//     rest.
//   * v_mfma_f32_16x16x32_bf16: A operand x (lane (token, g)), B operand the
//     weights (lane (row, g)).  Which columns a lane group holds does not matter
//     to the sum as long as both operands agree: group g of step (j, d) has
//     columns 128 j + 32 g + 8 d .. of the span.
//   * x in LDS, a span or half of one at a time, the next one's loads and stores
//     beside the products, one barrier each.
//
// One token through two weights of 22016 x 8192 50 us (186 MB at 3.7 TB/s), of 11008 x
// 4096 20, through 4096 x 4096 7.5: 5-7 us to start (table, first codes, the
// adapters' loads) and then 4.0-4.6 TB/s.  That is what launches this short reach;
// the decode kernel (gemv.hip) reads the same codes at 5.6-5.7 TB/s over a pass of
// 35 GB.  32 tokens 70: x's lines come with the codes', half as many; 64 tokens 104, as
// many.  The vector units are busy 43 % of the time at 32 tokens, LDS 28 %; the
// kernel of 32 tokens is at its 128 registers, and seven more are read back from
// scratch in the unit loop.  Units of 512 rows, which halve x's share, took as long at
// 32 tokens and longer at 64 (more to start with).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "downs.h"
#include "lds.h"
#include "pool.h"

namespace qlora {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves, kSets = 2;
constexpr int kSpan = 256;                   // columns of a unit
constexpr int kLut = 256 * 32 * 8;
static_assert(16 * kSets * kWaves == kStreamRows, "rows of a unit");
template <int NT>
struct XShape {
  static constexpr int kCols = NT == 1 ? 256 : 128;       // columns of a stage of x
  static constexpr int kRow = 2 * kCols;                  // bytes of a token's row
  static constexpr int kBytes = 16 * NT * kRow;           // of a stage: 8 KiB (NT 4: 16)
  static constexpr int kPieces = kBytes / 16 / kThreads;  // 16-byte pieces a thread brings
  static constexpr int kLds = kLut + 2 * kBytes;
};

typedef __attribute__((address_space(3))) u32x2_t lds_u64;
typedef __attribute__((address_space(3))) u32x4_t lds_u128;

struct StreamArgs {
  DeqSrcs w;              // G weights, N x K each
  int64_t N, K, M;
  const bf16_t* X;
  float* part;            // [slots][M][G N]
  int32_t* counts;        // parts of each tile
  int G, codebook[2], absfmt[2];
  StreamLine line;
  PoolView pool;          // R > 0: T
  StreamDowns downs;
  float* T;
};

__device__ __forceinline__ f32x4_t mfma16x16x32(const bf16x8_t& a, const bf16x8_t& b, const f32x4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// A barrier that waits for the LDS alone: __syncthreads would wait for every load
// in flight too, the next unit's codes among them.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Eight weights: pairs of levels times t, to bf16.
__device__ __forceinline__ bf16x8_t weights8(const u32x2_t (&l)[4], float t) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(u2f(l[i].x) * t, u2f(l[i].y) * t);
  return __builtin_bit_cast(bf16x8_t, u32x4_t{o[0], o[1], o[2], o[3]});
}

// RN32(q / 255) of a code in the low byte: the quotient by RN32(1 / 255) with its
// remainder put right, which is exact for each of the 256 (checked one by one in
// exact arithmetic).
__device__ __forceinline__ float q8_fast(uint32_t byte) {
  const float q = (float)(byte & 0xFFu), c = 0x1.010102p-8f, r = q * c;
  return fmaf(fmaf(-255.0f, r, q), c, r);
}

// Waves a SIMD: four, or two with the registers to read ahead.
template <int NT>
constexpr int kSimdWaves = NT == 4 ? 2 : 4;

template <int NT>
__global__ __launch_bounds__(kThreads, kSimdWaves<NT>) void stream_kernel(StreamArgs p) {
  using S = XShape<NT>;
  extern __shared__ __align__(16) char smem[];   // no static LDS: addressed from 0
  const StreamLine& L = p.line;
  const uint32_t wg = blockIdx.x;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, c = lane & 15, g = lane >> 4;
  if (p.downs.tasks > 0) {
    const int at = p.downs.index(L, wg);
    if (at >= 0)
      for (uint32_t i = (uint32_t)__builtin_amdgcn_readfirstlane(w) * p.downs.wgs + (uint32_t)at; i < p.downs.tasks;
           i += kWaves * p.downs.wgs) {
        if (p.downs.tt == 1)
          pool_down<1>(p.pool, p.X, p.M, p.K, p.T, i, p.downs.slices, p.downs.cols);
        else
          pool_down<4>(p.pool, p.X, p.M, p.K, p.T, i, p.downs.slices, p.downs.cols);
      }
    if (wg >= L.wgs) return;
  }
  const uint32_t u0 = L.unit(wg), u1 = L.unit(wg + 1);
  const int64_t K = p.K, N = p.N;
  const uint32_t nblk = (uint32_t)(K >> 6), row_bytes = (uint32_t)(K >> 1);

  // Where a stretch of units is: tile (of all token blocks and weights), span,
  // token block and tile within it, weight and rows.
  struct At {
    uint32_t tile, s, tb, in;
  };
  const uint32_t per_tb = L.tiles * (uint32_t)p.G;
  auto start = [&](uint32_t u) {
    At a;
    a.tile = u / L.spans, a.s = u - a.tile * L.spans, a.tb = a.tile / per_tb, a.in = a.tile - a.tb * per_tb;
    return a;
  };
  auto next = [&](At& a) __attribute__((always_inline)) {
    if (++a.s == L.spans) {
      a.s = 0, ++a.tile;
      if (++a.in == per_tb) a.in = 0, ++a.tb;
    }
  };

  // x: piece q of thread t is 16 bytes of token (t + 512 q) / (kCols / 8) of the
  // block, chunk i of its stage at i ^ (token & 15)
  constexpr int kRowPieces = S::kCols / 8;
  uint4 xv[S::kPieces];
  At xat = start(u0);
  uint32_t xunit = u0, xhalf = 0;
  const rsrc_t xr = make_rsrc(p.X, (uint32_t)(p.M * K * 2));   // M K < 2^31
  auto load_x = [&]() __attribute__((always_inline)) {   // the next stage; columns past K, tokens past M: zero
    const uint32_t col0 = xat.s * kSpan + xhalf * 128u;
#pragma unroll
    for (int q = 0; q < S::kPieces; ++q) {
      const uint32_t e = (uint32_t)(t + kThreads * q), col = col0 + 8u * (e % kRowPieces);
      const uint32_t m = xat.tb * 16u * NT + e / kRowPieces;
      xv[q] = buf_load16(xr, m < (uint32_t)p.M && col < (uint32_t)K ? (m * (uint32_t)K + col) * 2u : 0xFFFFFFF0u, 0u);
    }
    if (S::kCols == kSpan || ++xhalf == 2) {
      xhalf = 0;
      if (++xunit < u1) next(xat);   // past the last unit: the last one again
    }
  };
  auto put_x = [&](uint32_t buf) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < S::kPieces; ++q) {
      const uint32_t e = (uint32_t)(t + kThreads * q), tok = e / kRowPieces, i = e % kRowPieces;
      *(lds_u128*)(size_t)(kLut + buf * S::kBytes + tok * S::kRow + 16u * (i ^ (tok & 15u))) =
          u32x4_t{xv[q].x, xv[q].y, xv[q].z, xv[q].w};
    }
  };
  load_x();

  // Codes and block constants of the unit to come.  Rows past N read the last
  // one, never stored; a ragged last span reads into the next row, or past the
  // end (zero).
  At at = start(u0);
  rsrc_t cr, ar;
  const float* gs;
  uint32_t lo[kSets][2], row0;   // byte offset of the lane's loads in span 0; first row of the wave
  int fmt, quad;
  auto set_tile = [&](const At& a) __attribute__((always_inline)) {
    const uint32_t gi = a.in / L.tiles, n0 = (a.in - gi * L.tiles) * kStreamRows + 32u * (uint32_t)w;
    row0 = n0;
    const uint8_t *codes = p.w.codes[gi], *absmax = p.w.absmax_q[gi];
    gs = p.w.group_scale[gi];
    fmt = p.absfmt[gi];
    quad = (nblk & 3u) == 0 && ((uintptr_t)absmax & 3u) == 0;
    cr = make_rsrc(codes, (uint32_t)N * row_bytes);
    ar = make_rsrc(absmax, (uint32_t)N * nblk);
#pragma unroll
    for (int k = 0; k < kSets; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        lo[k][i] = min(n0 + 16 * k + 8 * i + (uint32_t)(c & 7), (uint32_t)N - 1u) * row_bytes +
                   64u * (uint32_t)(c >> 3) + 16u * (uint32_t)g;
  };
  uint4 code[kSets][2];
  auto load_codes = [&](uint32_t s) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kSets; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) code[k][i] = buf_load16(cr, lo[k][i], 128u * s);
  };
  // of four spans at once: lane (c, g) has the codes of span 4 f + g of row c, and
  // the two group scales of the 16 blocks (the second from block `cross` on)
  uint32_t aq[kSets], cross[kSets];
  float gl[kSets], gh[kSets];
  auto load_scales = [&](uint32_t f) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      const uint32_t first = min(row0 + 16 * k + (uint32_t)c, (uint32_t)N - 1u) * nblk + 16u * f, o = first + 4u * (uint32_t)g;
      if (quad) {
        aq[k] = __builtin_amdgcn_raw_buffer_load_b32(ar, o, 0, 0);
      } else {
        aq[k] = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) aq[k] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(ar, o + e, 0, 0) << (8 * e);
      }
      cross[k] = 256u - (first & 255u);
      gl[k] = gs[first >> 8];
      gh[k] = gs[min(first + 15u, (uint32_t)N * nblk - 1u) >> 8];
    }
  };
  set_tile(at);
  load_codes(at.s);
  load_scales(at.s >> 2);
  // the table: entry e of lane column l at 256 e + 8 l; e & 15 = 2 w + (lane >> 5),
  // e >> 4 = i
  auto build = [&](int cb) __attribute__((always_inline)) {
    const int wu = __builtin_amdgcn_readfirstlane(w);
    const uint32_t l0 = cb_level_bits(cb, 2 * wu), l1 = cb_level_bits(cb, 2 * wu + 1);
    const uint32_t lov = lane < 32 ? l0 : l1, to = (uint32_t)(2 * wu + (lane >> 5)) * 256u + 8u * (uint32_t)(lane & 31);
#pragma unroll
    for (int i = 0; i < 16; ++i) *(lds_u64*)(size_t)(to + 4096u * i) = u32x2_t{lov, cb_level_bits(cb, i)};
  };
  int cb = p.codebook[at.in / L.tiles];
  build(cb);
  put_x(0);
  load_x();
  const uint32_t col = 8u * (uint32_t)(lane & 31);
  uint32_t xa[4];   // x of step d: chunk 4 g + d of half a span
#pragma unroll
  for (int d = 0; d < 4; ++d) xa[d] = kLut + (uint32_t)c * S::kRow + 16u * (uint32_t)((4 * g + d) ^ c);
  f32x4_t acc[kSets][NT];
#pragma unroll
  for (int k = 0; k < kSets; ++k)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[k][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  uint32_t stage = 0;
  // Two waves a SIMD: the table and x read one set ahead of the products.  Four: a
  // set's at a time, the other waves hide their latency.
  constexpr bool kAhead = kSimdWaves<NT> == 2;
  constexpr uint32_t kSel[4] = {0x0C0C0400u, 0x0C0C0500u, 0x0C0C0600u, 0x0C0C0700u};

  for (uint32_t u = u0; u < u1; ++u) {
    const At here = at;
    // What the unit needs of the loads is taken first; then the next ones go into
    // the same registers.
    float ts[kSets][2];   // of the lane's two chunks: blocks 2 j + (g >> 1) of the span
    uint32_t V[kSets][2][4];
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      const uint32_t sp = here.s & 3u;
      const uint32_t q4 = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (c + 16 * (int)sp), (int)aq[k]) >> (8 * (g >> 1));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t b = 4u * sp + 2u * j + (uint32_t)(g >> 1);
        const float s2 = b >= cross[k] ? gh[k] : gl[k];
        float q = q8_fast(q4 >> (16 * j));
        if (fmt == kAbsFp8) q = fp8_value((q4 >> (16 * j)) & 0xFFu);
        ts[k][j] = q * s2;
      }
      if (here.s == L.spans - 1) {   // past the row: no weight (a scale of infinity there is another row's)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (4u * here.s + 2u * j + (uint32_t)(g >> 1) >= nblk) ts[k][j] = 0.0f;
      }
      const uint32_t a0[4] = {code[k][0].x, code[k][0].y, code[k][0].z, code[k][0].w},
                     a1[4] = {code[k][1].x, code[k][1].y, code[k][1].z, code[k][1].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {   // rows 0-7 of the set from load 0, rows 8-15 from load 1
        V[k][0][e] = (uint32_t)__builtin_amdgcn_update_dpp((int)a0[e], (int)a1[e], 0x118, 0xF, 0xC, false);   // row_shr:8
        V[k][1][e] = (uint32_t)__builtin_amdgcn_update_dpp((int)a1[e], (int)a0[e], 0x108, 0xF, 0x3, false);   // row_shl:8
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    const bool last = u + 1 == u1, leave = last || here.s + 1 == L.spans;
    int cb_next = cb;
    if (!last) {
      next(at);
      if (leave) {
        set_tile(at);
        cb_next = p.codebook[at.in / L.tiles];
      }
      load_codes(at.s);
      if (leave || (at.s & 3u) == 0) load_scales(at.s >> 2);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (S::kCols < kSpan || j == 0) {
        lds_barrier();   // this stage of x is in LDS, and the one before has been read
        put_x((stage + 1) & 1);
        load_x();
        ++stage;
      }
      const uint32_t xb = ((stage - 1) & 1) * S::kBytes + (S::kCols == kSpan ? 256u * j : 0u);
      bf16x8_t x[kAhead ? 2 : 1][NT];
      u32x2_t l[kAhead ? 2 : kSets][4];
      auto read_x = [&](int d) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
          x[kAhead ? d & 1 : 0][n] = __builtin_bit_cast(bf16x8_t, *(const lds_u128*)(size_t)(xa[d] + xb + 16u * n * S::kRow));
      };
      auto read_l = [&](int d, int k) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) l[kAhead ? k & 1 : k][i] = *(const lds_u64*)(size_t)perm(V[k][j][d], col, kSel[i]);
      };
      if constexpr (kAhead) {
        read_x(0);
        read_l(0, 0);
      }
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if constexpr (!kAhead) read_x(d);
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
          if constexpr (!kAhead) {
            read_l(d, k);
          } else if (k + 1 < kSets) {
            read_l(d, k + 1);
          } else if (d < 3) {
            read_x(d + 1);
            read_l(d + 1, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
          const bf16x8_t b = weights8(l[kAhead ? k & 1 : k], ts[k][j]);
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[k][n] = mfma16x16x32(x[kAhead ? d & 1 : 0][n], b, acc[k][n]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (leave) {   // lane (c, g): tokens 4 g .. 4 g + 3 of row c
      const uint32_t slot = wg - L.first(here.tile);
      if (here.s + 1 == L.spans && t == 0) p.counts[here.tile] = (int32_t)slot + 1;
      const int64_t GN = (int64_t)p.G * N, m0 = (int64_t)here.tb * 16 * NT;
      const uint32_t gi = here.in / L.tiles, n0 = (here.in - gi * L.tiles) * kStreamRows + 32u * (uint32_t)w;
      float* out = p.part + ((int64_t)slot * p.M + m0) * GN + gi * N;
#pragma unroll
      for (int k = 0; k < kSets; ++k) {
        const int64_t n = (int64_t)n0 + 16 * k + c;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = 16 * nt + 4 * g + e;
            if (m0 + m < p.M && n < N) out[m * GN + n] = acc[k][nt][e];
          }
          acc[k][nt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
      }
      if (cb_next != cb) {   // on to the other weight, of another codebook
        cb = cb_next;
        lds_barrier();
        build(cb);
        lds_barrier();
      }
    }
  }
}

}  // namespace

// Two workgroups for each of 256 CUs (of 64 tokens, one); fixed, not the device's
// count, so that the workspace does not depend on the device.
StreamPlan stream_plan(int64_t N, int64_t K, int64_t M, int G, int R) {
  StreamPlan s{};
  s.nt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  StreamLine& L = s.line;
  L.tiles = (uint32_t)((N + kStreamRows - 1) / kStreamRows);
  L.spans = (uint32_t)((K + kSpan - 1) / kSpan);
  L.block = 16 * s.nt;
  // (below 2^20: G N K and M K below 2^31, M at most 320)
  L.units = L.tiles * (uint32_t)G * (uint32_t)((M + L.block - 1) / L.block) * L.spans;
  L.wgs = std::min<uint32_t>(s.nt == 4 ? 256 : 512, L.units);
  const uint32_t least = L.units / L.wgs;
  s.slots = (int)((L.spans + least - 2) / least + 1);
  s.all_tiles = (int)(L.units / L.spans);
  // The tasks go where they cost least: a task takes about `per` + 3 turns of 512
  // columns, a unit ten of them, and what fits beside the other workgroups' units
  // is free.
  StreamDowns& d = s.downs;
  d.slices = 1, d.least = least;
  if (R > 0) {
    const uint32_t most = s.nt == 4 ? 256 : 512;
    const int64_t rows = (K + 511) / 512;
    d.tt = pool_down_tasks(G * R, M, 1) > (int64_t)kWaves * most ? 4 : 1;
    const int64_t n = pool_down_tasks(G * R, M, d.tt);
    const uint32_t rest = L.units % L.wgs, wgs[3] = {most - L.wgs, rest > 0 ? L.wgs - rest : 0, L.wgs};
    const int64_t free[3] = {10 * (int64_t)least, 10, 0};
    int64_t best = INT64_MAX;
    for (int c = 0; c < 3; ++c) {
      const int64_t waves = (int64_t)kWaves * wgs[c];
      if (waves == 0) continue;
      const int64_t want = std::max<int64_t>(1, std::min(std::min<int64_t>(kMaxSlices, rows), waves / n));
      const int64_t per = (rows + want - 1) / want, slices = (rows + per - 1) / per, tasks = n * slices;
      const int64_t cost = std::max<int64_t>(0, (tasks + waves - 1) / waves * (per + 3) - free[c]);
      if (cost >= best) continue;
      best = cost;
      d.where = (StreamTasks)c, d.wgs = (uint32_t)std::min<int64_t>(wgs[c], tasks);
      d.slices = (uint32_t)slices, d.cols = (uint32_t)(512 * per), d.tasks = (uint32_t)tasks;
      if (c != kTasksApart) d.wgs = wgs[c];
    }
  }
  return s;
}

hipError_t launch_stream(const Nf4View* W, const bf16_t* X, int64_t M, const PoolView& pool, const StreamPlan& s, float* T,
                         float* part, int32_t* counts, hipStream_t st) {
  StreamArgs a{};
  for (int g = 0; g < pool.G; ++g) {
    a.w.codes[g] = W[g].codes, a.w.absmax_q[g] = W[g].absmax_q, a.w.group_scale[g] = W[g].group_scale;
    a.codebook[g] = W[g].codebook, a.absfmt[g] = W[g].absfmt;
  }
  a.N = W[0].N, a.K = W[0].K, a.M = M, a.X = X, a.part = part, a.counts = counts, a.G = pool.G;
  a.line = s.line, a.pool = pool, a.downs = s.downs, a.T = T;
  // the kernel's table is addressed from 0: the compiler may have put nothing there
  static std::atomic<uint32_t> looked{0u};
  auto go = [&](auto* fn, int lds) {
    hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), lds);
    if (e != hipSuccess) return e;
    if (!(looked.load(std::memory_order_relaxed) & (uint32_t)s.nt)) {
      hipFuncAttributes at{};
      if ((e = hipFuncGetAttributes(&at, reinterpret_cast<const void*>(fn))) != hipSuccess) return e;
      if (at.sharedSizeBytes != 0) return hipErrorInvalidKernelFile;
      looked.fetch_or((uint32_t)s.nt, std::memory_order_relaxed);
    }
    hipLaunchKernelGGL(fn, dim3(s.line.wgs + (s.downs.where == kTasksApart ? s.downs.wgs : 0)), dim3(kThreads), lds, st, a);
    return hipGetLastError();
  };
  return s.nt == 1   ? go(&stream_kernel<1>, XShape<1>::kLds)
         : s.nt == 2 ? go(&stream_kernel<2>, XShape<2>::kLds)
                     : go(&stream_kernel<4>, XShape<4>::kLds);
}

}  // namespace qlora
