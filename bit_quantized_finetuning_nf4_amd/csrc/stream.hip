// stream.hip -- the frozen product of few tokens, X deq(W_g)^T for G 4-bit
// weights side by side, as fp32 parts of a split contraction; the adapters and
// what follows are the next launch's (pool.hip).  The passes over the tokens'
// own adapters (scale_a A_a x) are further workgroups of the same launch.
//
// A weight enters the product as the value that it stands for, RNE_bf16(RN32(L
// t)): the sums have no other error than fp32's.
//
//   * A workgroup takes 256 rows of the stack and a slice of the contraction;
//     its eight waves two sets of 16 rows each.  A span is 256 columns of a set:
//     two loads of 16 bytes a lane, each over eight whole 128-byte lines (loads
//     over sixteen rows stall in the vector L1's address translation); an
//     exchange between lanes 8 apart gives lane (c, g) the 16-byte chunks g and
//     4 + g of its own row c.  The next span's are in flight meanwhile.
//   * A code byte is two weights: a table in LDS gives their two fp32 levels (256
//     entries of 8 bytes, a copy for each lane of a half wave, so no two of its
//     lanes meet in a bank: 64 KiB), one product each with the block's scale, one
//     conversion for both.  About 2.4 vector instructions a weight, 6 TB/s of
//     codes at 2.1 GHz, and 5 to 8 bytes of LDS.
//   * v_mfma_f32_16x16x32_bf16: A operand x (lane (token, g)), B operand the
//     weights (lane (row, g)).  Which columns a lane group holds does not matter
//     to the sum as long as both operands agree: group g of step (j, d) has
//     columns 128 j + 32 g + 8 d .. of the span.
//   * x: 16 KiB of LDS, 512, 256 or 128 columns of 16, 32 or 64 tokens at a time,
//     so that two workgroups share a CU and one computes while the other waits.
#include <algorithm>
#include <type_traits>

#include "pool.h"
#include "lds.h"
#include "downs.h"

namespace qlora {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves, kSets = 2;
constexpr int kRows = 16 * kSets * kWaves;   // rows of the stack per workgroup
constexpr int kSpan = 256;                   // columns
constexpr int kLut = 256 * 32 * 8, kXBytes = 16384, kLds = kLut + kXBytes;

typedef __attribute__((address_space(3))) u32x2_t lds_u64;
typedef __attribute__((address_space(3))) u32x4_t lds_u128;

struct StreamArgs {
  DeqSrcs w;              // G weights, N x K each
  int64_t N, K, M;
  const bf16_t* X;
  float* part;            // [splits][M][G N]
  int G, tiles, splits, spans, tokens, absfmt[2];   // tiles of one weight; spans of a slice
  PoolView pool;          // R > 0: T [M x G R], U
  float* T;
  bf16_t* U;
  int downs;              // workgroups that form T, before the others
};

__device__ __forceinline__ f32x4_t mfma16x16x32(const bf16x8_t& a, const bf16x8_t& b, const f32x4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Lane group `sp`'s value in every group (lane by lane within the group).
template <int SP>
__device__ __forceinline__ uint32_t of_group(uint32_t x) {
  const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);   // [0 1 0 1], [2 3 2 3]
  const uint32_t y = SP < 2 ? h[0] : h[1];
  const auto q = __builtin_amdgcn_permlane16_swap(y, y, false, false);
  return (SP & 1) ? q[1] : q[0];
}

// Eight weights of one code dword: levels by byte pairs, times t, to bf16.
__device__ __forceinline__ bf16x8_t weights8(uint32_t c, uint32_t col, float t) {
  uint32_t o[4];
  constexpr uint32_t kSel[4] = {0x0C0C0400u, 0x0C0C0500u, 0x0C0C0600u, 0x0C0C0700u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x2_t v = *(const lds_u64*)(size_t)perm(c, col, kSel[i]);
    o[i] = pack_bf16x2(u2f(v.x) * t, u2f(v.y) * t);
  }
  return __builtin_bit_cast(bf16x8_t, u32x4_t{o[0], o[1], o[2], o[3]});
}

template <int CB, int NT>
__global__ __launch_bounds__(kThreads, 4) void stream_kernel(StreamArgs p) {
  extern __shared__ __align__(16) char smem[];   // no static LDS: addressed from 0
  constexpr int XC = 512 / NT, kXRow = 2 * XC;   // x columns staged at a time, bytes of a token's row
  int id = blockIdx.x;
  if (id < p.downs) {
    pool_down<kWaves>(p.pool, p.X, p.M, p.K, p.T, p.U, id);
    return;
  }
  id -= p.downs;
  const int tile = id % p.tiles;
  id /= p.tiles;
  const int slice = id % p.splits;
  id /= p.splits;
  const int g_ = id % p.G, tb = id / p.G;        // which weight, which 16 NT tokens
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, c = lane & 15, g = lane >> 4;
  const int64_t K = p.K, N = p.N, m0 = (int64_t)tb * 16 * NT;
  const int nblk = (int)(K >> 6), mt = (int)min((int64_t)16 * NT, p.M - m0);
  const uint8_t *codes = p.w.codes[g_], *absmax = p.w.absmax_q[g_];
  const float* gs = p.w.group_scale[g_];
  const int fmt = p.absfmt[g_];
  const int s0 = slice * p.spans, s1 = min((int)((K + kSpan - 1) / kSpan), s0 + p.spans);   // no slice is empty

  // x: piece q of thread t is 16 bytes of columns XC st .. of token (t + 512 q) /
  // (XC / 8), chunk i of it at i ^ (token & 15)
  const rsrc_t xr = make_rsrc(p.X + m0 * K, (uint32_t)(mt * K * 2));
  constexpr int kPieces = kXBytes / 16 / kThreads, kRowPieces = XC / 8;
  uint32_t xo[kPieces], xl[kPieces];
  bool xin[kPieces];
#pragma unroll
  for (int q = 0; q < kPieces; ++q) {
    const int e = t + kThreads * q, tok = e / kRowPieces, i = e % kRowPieces;
    xo[q] = (uint32_t)(tok * K * 2 + 16 * i);
    xin[q] = tok < mt;
    xl[q] = kLut + (uint32_t)tok * kXRow + 16u * (uint32_t)(i ^ (tok & 15));
  }
  uint4 xv[kPieces];
  auto load_x = [&](int st) __attribute__((always_inline)) {   // columns past K, and tokens past M: zero
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const int col = XC * st + 8 * ((t + kThreads * q) % kRowPieces);
      xv[q] = buf_load16(xr, xin[q] && col < K ? xo[q] + (uint32_t)(XC * st) * 2u : 0xFFFFFFF0u, 0u);
    }
  };
  load_x(s0 * kSpan / XC);

  // The row of set k: rows past N read the last one, never stored.
  const int n0 = tile * kRows + 32 * w;
  uint32_t lo[kSets][2];   // byte offsets of the lane's loads in span 0, by half block column
  int64_t rb[kSets];       // first block of row c
  const int64_t row_bytes = K >> 1;
  // 64-bit bases, 32-bit offsets: N K / 2 < 2^32
#pragma unroll
  for (int k = 0; k < kSets; ++k) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      lo[k][i] = (uint32_t)(min((int64_t)n0 + 16 * k + 8 * i + (c & 7), N - 1) * row_bytes) +
                 64u * (uint32_t)(c >> 3) + 16u * (uint32_t)g;
    rb[k] = min((int64_t)n0 + 16 * k + c, N - 1) * nblk;
  }
  const rsrc_t cr = make_rsrc(codes, (uint32_t)(N * row_bytes));
  auto load_codes = [&](uint4 (&v)[kSets][2], int s) __attribute__((always_inline)) {
    // a ragged last span reads into the next row, or past the end (zero): its scale is 0 there
    const uint32_t o = 128u * (uint32_t)min(s, s1 - 1);
#pragma unroll
    for (int k = 0; k < kSets; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) v[k][i] = buf_load16(cr, lo[k][i] + o, 0u);
  };
  // Block constants of four spans: lane (c, g) has the four of span 4 f + g of
  // row c, as bytes, and the two group scales that those spans' 16 blocks can have.
  const rsrc_t ar = make_rsrc(absmax, (uint32_t)(N * nblk));
  uint32_t aq[kSets];
  float gl[kSets], gh[kSets];
  auto load_scales = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      const int b = 4 * s + 4 * g;
      aq[k] = 0u;
      const uint32_t o = (uint32_t)(rb[k] + b);
#pragma unroll
      for (int e = 0; e < 4; ++e)   // past the arrays: zero
        aq[k] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(ar, o + e, 0, 0) << (8 * e);
      const int64_t first = rb[k] + 4 * s, last = min(first + 15, N * nblk - 1);
      gl[k] = gs[first >> 8];
      gh[k] = gs[last >> 8];
    }
  };

  uint4 ca[kSets][2], cb[kSets][2];
  load_codes(ca, s0);
  load_scales(s0);
  {   // the table: entry e of lane column l at 256 e + 8 l; e & 15 = 2 w + (lane >> 5), e >> 4 = i
    const int wu = __builtin_amdgcn_readfirstlane(w);
    const uint32_t l0 = cb_level_bits<CB>(2 * wu), l1 = cb_level_bits<CB>(2 * wu + 1);
    const uint32_t lov = lane < 32 ? l0 : l1, at = (uint32_t)(2 * wu + (lane >> 5)) * 256u + 8u * (uint32_t)(lane & 31);
#pragma unroll
    for (int i = 0; i < 16; ++i) *(lds_u64*)(size_t)(at + 4096u * i) = u32x2_t{lov, cb_level_bits<CB>(i)};
  }

  const uint32_t col = 8u * (uint32_t)(lane & 31);
  uint32_t xa[4];   // x of step d: chunk 4 g + d of a half span
#pragma unroll
  for (int d = 0; d < 4; ++d) xa[d] = kLut + (uint32_t)c * kXRow + 16u * (uint32_t)((4 * g + d) ^ c);
  f32x4_t acc[kSets][NT];
#pragma unroll
  for (int k = 0; k < kSets; ++k)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[k][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const bool up = (c & 8) != 0;

  // The stage of x that starts at column XC st is in registers; it goes to LDS,
  // and the next one's loads are issued.
  auto stage_x = [&](int st) __attribute__((always_inline)) {
    __syncthreads();   // every wave is done with the stage before
#pragma unroll
    for (int q = 0; q < kPieces; ++q) *(lds_u128*)(size_t)xl[q] = u32x4_t{xv[q].x, xv[q].y, xv[q].z, xv[q].w};
    load_x(st + 1);
    __syncthreads();
  };
  // Span s = 4 f + SP: `cur` its codes, `nxt` receives the next span's.
  uint32_t aqf[kSets];
  float glf[kSets], ghf[kSets];
  auto span = [&](auto sp, uint4 (&cur)[kSets][2], uint4 (&nxt)[kSets][2], int s) __attribute__((always_inline)) {
    constexpr int SP = decltype(sp)::value;
    if constexpr (XC >= kSpan) {
      if (s % (XC / kSpan) == 0 || s == s0) stage_x(s * kSpan / XC);
    }
    load_codes(nxt, s + 1);
    __builtin_amdgcn_sched_barrier(0);
    // scales of the lane's two chunks: blocks 2 j + (g >> 1) of the span
    float ts[kSets][2];
    uint32_t V[kSets][2][4];
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      const uint32_t q4 = of_group<SP>(aqf[k]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int b = 4 * s + 2 * j + (g >> 1);
        const float s2 = ((rb[k] + b) >> 8) == ((rb[k] + 4 * (s - SP)) >> 8) ? glf[k] : ghf[k];
        const float q = absmax_value((q4 >> (16 * j + 8 * (g >> 1))) & 0xFFu, fmt);
        ts[k][j] = b < nblk ? q * s2 : 0.0f;
      }
      const uint32_t a0[4] = {cur[k][0].x, cur[k][0].y, cur[k][0].z, cur[k][0].w},
                     a1[4] = {cur[k][1].x, cur[k][1].y, cur[k][1].z, cur[k][1].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {   // rows 0-7 of the set from load 0, rows 8-15 from load 1
        const uint32_t dn = (uint32_t)__builtin_amdgcn_mov_dpp((int)a1[e], 0x118, 0xF, 0xF, false);   // row_shr:8
        const uint32_t u = (uint32_t)__builtin_amdgcn_mov_dpp((int)a0[e], 0x108, 0xF, 0xF, false);    // row_shl:8
        V[k][0][e] = up ? dn : a0[e];
        V[k][1][e] = up ? a1[e] : u;
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (XC < kSpan) stage_x(2 * s + j);
      const uint32_t xb = XC > kSpan ? 512u * (uint32_t)(s & 1) + 256u * j : XC == kSpan ? 256u * j : 0u;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        bf16x8_t x[NT], b[kSets];
#pragma unroll
        for (int n = 0; n < NT; ++n)
          x[n] = __builtin_bit_cast(bf16x8_t, *(const lds_u128*)(size_t)(xa[d] + xb + 16u * n * kXRow));
#pragma unroll
        for (int k = 0; k < kSets; ++k) b[k] = weights8(V[k][j][d], col, ts[k][j]);
#pragma unroll
        for (int k = 0; k < kSets; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[k][n] = mfma16x16x32(x[n], b[k], acc[k][n]);
      }
    }
  };

  for (int s = s0; s < s1; s += 4) {
#pragma unroll
    for (int k = 0; k < kSets; ++k) aqf[k] = aq[k], glf[k] = gl[k], ghf[k] = gh[k];
    if (s + 4 < s1) load_scales(s + 4);
    span(std::integral_constant<int, 0>{}, ca, cb, s);
    if (s + 1 >= s1) break;
    span(std::integral_constant<int, 1>{}, cb, ca, s + 1);
    if (s + 2 >= s1) break;
    span(std::integral_constant<int, 2>{}, ca, cb, s + 2);
    if (s + 3 >= s1) break;
    span(std::integral_constant<int, 3>{}, cb, ca, s + 3);
  }

  // lane (c, g): tokens 4 g .. 4 g + 3 of row c
  const int64_t GN = (int64_t)p.G * N;
  float* out = p.part + ((int64_t)slice * p.M + m0) * GN + g_ * N;
#pragma unroll
  for (int k = 0; k < kSets; ++k) {
    const int64_t n = (int64_t)n0 + 16 * k + c;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = 16 * nt + 4 * g + e;
        if (m < mt && n < N) out[m * GN + n] = acc[k][nt][e];
      }
  }
}

}  // namespace

// Slices of the contraction: about two workgroups for each CU, of a whole span
// at least, no slice empty.  Fixed, not the device's count, so that the
// workspace does not depend on the device.
StreamPlan stream_plan(int64_t N, int64_t K, int64_t M, int G) {
  StreamPlan s{};
  s.nt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  s.tiles = (int)((N + kRows - 1) / kRows);
  s.tokens = (int)((M + 16 * s.nt - 1) / (16 * s.nt));
  const int spans = (int)((K + kSpan - 1) / kSpan);
  const int64_t wgs = (int64_t)s.tiles * G * s.tokens;
  int want = (int)std::min<int64_t>(std::min(spans, 16), std::max<int64_t>(1, (512 + wgs / 2) / wgs));
  s.spans = (spans + want - 1) / want;
  if (s.nt == 1 && s.spans > 1) s.spans += s.spans & 1;   // whole stages of x
  s.splits = (spans + s.spans - 1) / s.spans;
  return s;
}

hipError_t launch_stream(const Nf4View* W, const bf16_t* X, int64_t M, const PoolView& pool, float* T, bf16_t* U,
                         float* part, int* splits, hipStream_t st) {
  const StreamPlan s = stream_plan(W[0].N, W[0].K, M, pool.G);
  StreamArgs a{};
  for (int g = 0; g < pool.G; ++g) {
    a.w.codes[g] = W[g].codes, a.w.absmax_q[g] = W[g].absmax_q, a.w.group_scale[g] = W[g].group_scale;
    a.absfmt[g] = W[g].absfmt;
  }
  a.N = W[0].N, a.K = W[0].K, a.M = M, a.X = X, a.part = part, a.G = pool.G;
  a.tiles = s.tiles, a.splits = s.splits, a.spans = s.spans, a.tokens = s.tokens;
  a.pool = pool, a.T = T, a.U = U, a.downs = pool.R > 0 ? pool_down_blocks(pool, M, kWaves) : 0;
  *splits = s.splits;
  auto go = [&](auto* fn) {
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(fn, dim3((unsigned)(a.downs + s.tiles * s.splits * pool.G * s.tokens)), dim3(kThreads), kLds, st, a);
    return hipGetLastError();
  };
  auto by_tokens = [&](auto cb) {
    constexpr int CB = decltype(cb)::value;
    return s.nt == 1 ? go(&stream_kernel<CB, 1>) : s.nt == 2 ? go(&stream_kernel<CB, 2>) : go(&stream_kernel<CB, 4>);
  };
  if (W[0].codebook == kCbFp4) return by_tokens(std::integral_constant<int, kCbFp4>{});
  if (W[0].codebook == kCbInt4) return by_tokens(std::integral_constant<int, kCbInt4>{});
  return by_tokens(std::integral_constant<int, kCbNf4>{});
}

}  // namespace qlora
