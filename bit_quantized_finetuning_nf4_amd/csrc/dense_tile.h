// dense_tile.h -- the main loop and the LoRA-tail staging of the dense GEMMs
// (gfx950): 256 x 64 FI output tiles, both operands streamed as rows of
// 128-byte lines through LDS by buffer->LDS DMA: two pair slots (dense_slots), or a
// ring of five half slots (dense_halves, dense_quads), which takes all of the LDS.
//
// The loop moves bytes: a pair is 128 bytes of every row, 64 bf16 or 128
// 8-bit integers, and a fragment is 16 bytes of a row.  The operation MM
// names the matrix instruction and its accumulator: MmBf16 (32x32x16 bf16,
// fp32 sums) or MmI8 (32x32x32 8-bit integers, 32-bit integer sums).
#pragma once
#include "gemm_common.h"

namespace qlora {
namespace {

typedef __attribute__((__vector_size__(16 * sizeof(int)))) int i32x16_t;
typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4_t;

struct MmBf16 {
  typedef f32x16_t acc_t;
  static __device__ __forceinline__ acc_t mma(const bf16x8_t& a, const bf16x8_t& b, const acc_t& c) {
    return mfma32x32x16(a, b, c);
  }
};
// Lane (lr, h) of a fragment holds 16 consecutive bytes of row lr; both
// operands take the same bytes of a row, so their order in the contraction
// does not matter to the sum.
struct MmI8 {
  typedef i32x16_t acc_t;
  static __device__ __forceinline__ acc_t mma(const bf16x8_t& a, const bf16x8_t& b, const acc_t& c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0,
                                                 0, 0);
  }
};

// An integer sum times the scales of its channel and token, in this order: an
// integer times a number of any size loses no range downwards, and the scales'
// own product would leave fp32's range where the result is inside it (an
// infinity times a sum of 0 would be NaN, 2^-150 a 0 that no sum brings back).
// What is left is a channel's scale past 2^97, whose product with a sum may
// overflow before a small token scale is applied; mantissas and exponents apart
// would mend that too, and cost 2-4 % of a product.
__device__ __forceinline__ float scaled_sum(int t, float sw, float sx) { return (float)t * sw * sx; }

constexpr int kPairOp = kTile * 128;                    // 32 KiB: 256 rows x 64 bf16 (two stages)
constexpr int kPairSlot = 2 * kPairOp;                  // weight rows at 0, token rows at kPairOp
constexpr size_t kLdsPairs = 2 * (size_t)kPairSlot;     // 128 KiB: two pair slots
constexpr int kDGroup = 4;                              // token tiles per tile group (tile order)

// Pair slots hold two consecutive 32-wide stages (one 64-wide stage): rows of
// 128 bytes in the layout of pos128.  Chunks 0..3 are the even stage, 4..7 the
// odd one.

// Tile order of the dense GEMMs.  The eight XCDs receive contiguous ranges of
// tile ids (the hardware hands workgroups to XCDs round robin); ids run over
// groups of kDGroup token tiles, each group column-tile-major, so that the
// tiles one XCD holds at a time share a few token tiles and a few weight
// tiles and both stream through its L2.
// With the contraction split, ids run split-major: the tiles of one split
// (which share its column range of both operands) sit on the same XCDs.
__device__ __forceinline__ int xcd_tile_id() {
  const int nwg = (int)gridDim.x;
  int id = blockIdx.x;
  if ((nwg & 7) == 0) id = (id & 7) * (nwg >> 3) + (id >> 3);
  return id;
}
// With 16 token tiles or more a group holds 8 of them, so each weight tile
// streams through an XCD's L2 half as often (the weight is the larger
// operand of these products): at 4096 tokens the 65B products ran 1.4 %
// faster than with 4; at 2048 tokens (8 token tiles) 4 stays slightly ahead.
__device__ __forceinline__ void map_tile_grouped(int id, int tiles_c, int tiles_r, int& tc, int& tr) {
  const int grp = tiles_r >= 16 ? 2 * kDGroup : kDGroup;
  const int per_group = grp * tiles_c;
  const int g = id / per_group, first = g * grp;
  const int size = min(grp, tiles_r - first);
  const int local = id - g * per_group;
  tr = first + local % size;
  tc = local / size;
}

struct DenseOps {
  rsrc_t wr_, xr;           // weight rows, token rows
  uint32_t wo[8], xo[8];    // lane offsets of the eight DMA instructions per operand (pair 0)
  int npair, w;
};

// DMA of pair `pair` (64 columns of every row) of both operands into pair
// slot `dst`: weight instruction q < 2 FI and token instruction q < 8 of
// wave w fill rows 8 (4 q + w) .. +7 of their tile, 128 bytes each (lane j:
// row + (j >> 3), position j & 7).  DMA d of a pair is weight instruction d
// for d < 2 FI, token instruction d - 2 FI after.  Past the last pair the last
// one is re-loaded (never read).
template <int FI>
__device__ __forceinline__ void pair_dma(char* dst, const DenseOps& f, int pair, int d) {
  const uint32_t soff = (uint32_t)min(pair, f.npair - 1) * 128u;
  const bool wrow = d < 2 * FI;
  const int q = wrow ? d : d - 2 * FI;
  char* dd = dst + (wrow ? 0 : kPairOp) + 8 * (4 * q + f.w) * 128;
  if (wrow)
    dma16(f.wr_, dd, f.wo[q], soff);
  else
    dma16(f.xr, dd, f.xo[q], soff);
}

// Read offsets of the lane within a pair slot: stage half hf, k16 step kk ->
// chunk 4 hf + 2 kk + h of row lr.
struct PairOffs {
  int o[2][2];
};

// MFMA slot X (0 .. 8 FI - 1) of substep s: X = 4 FI kk + 4 i + j is
// fragment pair (i, j) of k16 step kk (FI weight fragments of 32 rows, four
// token fragments).  Stage s is half HF of the pair slot at cur; stage s+1 is
// the other half of cur (HF = 0) or half 0 of the next slot (HF = 1).
//   LDS reads   read q (fragments A0, B0, B1, B2, B3, A1, .., A(FI-1) in
//               that order) in slot rd_slot(q): step 1 of stage s; in slot
//               4 FI + rd_slot(q): step 0 of stage s+1, into the registers
//               step 0 of stage s has finished with.
//   barrier     odd substeps, before slot 4 FI: this wave's DMAs of the next
//               pair have landed and its reads of this pair have completed;
//               after it the next pair is visible to every wave and no wave
//               reads this pair's slot any more.
//   DMA         the pair after next into this pair's slot (2 FI weight-row,
//               then 8 token-row instructions of 8 whole 128-byte rows each):
//               the first FI + 4 in the odd substep's slots 4 FI .., every
//               other slot; the other FI + 4 in the next pair's even substep,
//               one every fourth slot.  Issued all in the odd substep's
//               second half, 16 instructions per wave in 16 MFMA slots
//               overran the texture address queue (its FIFO full about 10 %
//               of the cycles) and stalled issue; split, the product ran
//               about 7 % faster.
template <int FI>
constexpr int rd_slot(int q) { return q * 4 * FI / (FI + 4); }
template <int FI>
constexpr int dma_half = FI + 4;   // DMAs of a pair issued in its odd substep
template <int FI>
constexpr int dma_slot_a(int d) { return 4 * FI + d * 4 * FI / dma_half<FI>; }
template <int FI>
constexpr int dma_slot_b(int d) { return (d - dma_half<FI>) * 8 * FI / dma_half<FI>; }

template <class MM, int FI, int X, int HF>
__device__ __forceinline__ void dense_slot(const char* cur, const char* nxt, char* fill, const DenseOps& f,
                                           int pair, typename MM::acc_t (&acc)[FI][4], Frags& F, int am, int bm,
                                           const PairOffs& po) {
  constexpr int H = 4 * FI;   // slots per k16 step
  constexpr int kk = X / H, y = X % H, i = y >> 2, j = y & 3;
  if constexpr (HF == 1 && X == H) {
    QLORA_WAIT(0, 0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }
  if constexpr (kk == 0)
    acc[i][j] = MM::mma(F.a0[i], F.b0[j], acc[i][j]);
  else
    acc[i][j] = MM::mma(F.a1[i], F.b1[j], acc[i][j]);
#pragma unroll
  for (int q = 0; q < FI + 4; ++q) {
    if (rd_slot<FI>(q) != y) continue;
    const bool isA = q == 0 || q >= 5;
    const int fr = q == 0 ? 0 : q >= 5 ? q - 4 : q - 1;   // fragment index
    // step 1 of stage s (half HF of cur), or step 0 of stage s+1
    const char* slot = kk == 0 ? cur : (HF == 0 ? cur : nxt);
    const int o = kk == 0 ? po.o[HF][1] : po.o[HF ^ 1][0];
    const char* base = slot + (isA ? am : kPairOp + bm) + fr * 32 * 128 + o;
    if (isA) {
      if (kk == 0) F.a1[fr] = rd16(base); else F.a0[fr] = rd16(base);
    } else {
      if (kk == 0) F.b1[fr] = rd16(base); else F.b0[fr] = rd16(base);
    }
  }
  if constexpr (HF == 1 && kk == 1) {
#pragma unroll
    for (int d = 0; d < dma_half<FI>; ++d)
      if (dma_slot_a<FI>(d) == X) pair_dma<FI>(fill, f, pair + 2, d);
  }
  if constexpr (HF == 0) {
    // the rest of pair + 1's DMAs into nxt, which no wave reads before the
    // barrier of this pair (in the first pair they re-load what the
    // prologue loaded: the same bytes to the same place)
#pragma unroll
    for (int d = dma_half<FI>; d < 2 * FI + 8; ++d)
      if (dma_slot_b<FI>(d) == X) pair_dma<FI>(const_cast<char*>(nxt), f, pair + 1, d);
  }
  __builtin_amdgcn_sched_barrier(0);
}

template <class MM, int FI, int HF, int X>
__device__ __forceinline__ void dense_slots(const char* cur, const char* nxt, char* fill, const DenseOps& f,
                                            int pair, typename MM::acc_t (&acc)[FI][4], Frags& F, int am, int bm,
                                            const PairOffs& po) {
  if constexpr (X < 8 * FI) {
    dense_slot<MM, FI, X, HF>(cur, nxt, fill, f, pair, acc, F, am, bm, po);
    dense_slots<MM, FI, HF, X + 1>(cur, nxt, fill, f, pair, acc, F, am, bm, po);
  }
}

// The same loop through a ring of five half slots of 32 KiB, one operand of a pair
// each: pair p's weight rows are half 2 p, its token rows half 2 p + 1, and half q
// is in slot q mod 5.  Two pair slots leave the last lines of a pair a quarter of a
// pair's time to arrive; here, once a pair has been read, its two slots take the
// token rows of the pair after next and the weight rows of the one behind it, spread
// over the whole next pair, and the last lines that a barrier waits for have half a
// pair's time: the wave's 2 FI weight loads issued after them stay in flight.
// 4096 x 8192 x 22016 1.94 -> 1.56 cycles a matrix cycle (0.65 -> 0.81 of the time in
// the matrix units), 1200 -> 1138 us; 333 x 22016 x 4096 95 -> 82; the eight grouped
// products of the 65B layer set (gemm_bf16.hip), both in turn on one card, 1323 -> 1374
// TFLOP/s, the clock falling from 1.78 to 1.67 GHz.  A loop that waits
// for no load at all takes the same: the rest is issue, and the clock, which falls
// as the units fill.  It needs all of the LDS: for kernels that keep nothing else
// there.
constexpr size_t kLdsHalves = 5 * (size_t)kPairOp;
// Load d of the group that follows the barrier of pair p (8 of token rows, 2 FI of
// weight rows), in matrix instructions after it.
template <int FI>
constexpr int half_off(int d) { return d * 16 * FI / (2 * FI + 8); }
template <int FI>
__device__ __forceinline__ void half_dma(char* dst, const DenseOps& f, bool wrow, int pair, int q) {
  const uint32_t soff = (uint32_t)min(pair, f.npair - 1) * 128u;
  char* dd = dst + 8 * (4 * q + f.w) * 128;
  if (wrow)
    dma16(f.wr_, dd, f.wo[q], soff);
  else
    dma16(f.xr, dd, f.xo[q], soff);
}
template <int FI>
__device__ __forceinline__ void group_dma(char* dx, char* dw, const DenseOps& f, int p, int d) {
  if (d < 8)
    half_dma<FI>(dx, f, false, p + 2, d);
  else
    half_dma<FI>(dw, f, true, p + 3, d - 8);
}
// Where halves 2 p .. 2 p + 4 are.
struct Halves {
  char* s[5];
};
// dense_slot, the halves of pair `pair` at c.s[0] and c.s[1], the next at c.s[2] and
// c.s[3].
template <class MM, int FI, int X, int HF>
__device__ __forceinline__ void half_slot(const Halves& c, const DenseOps& f, int pair, typename MM::acc_t (&acc)[FI][4],
                                          Frags& F, int am, int bm, const PairOffs& po) {
  constexpr int H = 4 * FI;
  constexpr int kk = X / H, y = X % H, i = y >> 2, j = y & 3;
  if constexpr (HF == 1 && X == H) {
    QLORA_WAIT(2 * FI, 0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }
  if constexpr (kk == 0)
    acc[i][j] = MM::mma(F.a0[i], F.b0[j], acc[i][j]);
  else
    acc[i][j] = MM::mma(F.a1[i], F.b1[j], acc[i][j]);
#pragma unroll
  for (int q = 0; q < FI + 4; ++q) {
    if (rd_slot<FI>(q) != y) continue;
    const bool isA = q == 0 || q >= 5;
    const int fr = q == 0 ? 0 : q >= 5 ? q - 4 : q - 1;
    const bool nxt = kk == 1 && HF == 1;
    const int o = kk == 0 ? po.o[HF][1] : po.o[HF ^ 1][0];
    const char* base = c.s[(nxt ? 2 : 0) + (isA ? 0 : 1)] + (isA ? am : bm) + fr * 32 * 128 + o;
    if (isA) {
      if (kk == 0) F.a1[fr] = rd16(base); else F.a0[fr] = rd16(base);
    } else {
      if (kk == 0) F.b1[fr] = rd16(base); else F.b0[fr] = rd16(base);
    }
  }
  constexpr int off = HF == 0 ? H + X : X < H ? 3 * H + X : X - H;
#pragma unroll
  for (int d = 0; d < 2 * FI + 8; ++d)
    if (half_off<FI>(d) == off) {
      if constexpr (HF == 1 && X >= H)
        group_dma<FI>(c.s[0], c.s[1], f, pair, d);
      else
        group_dma<FI>(c.s[3], c.s[4], f, pair - 1, d);
    }
  __builtin_amdgcn_sched_barrier(0);
}
template <class MM, int FI, int HF, int X>
__device__ __forceinline__ void half_slots(const Halves& c, const DenseOps& f, int pair, typename MM::acc_t (&acc)[FI][4],
                                           Frags& F, int am, int bm, const PairOffs& po) {
  if constexpr (X < 8 * FI) {
    half_slot<MM, FI, X, HF>(c, f, pair, acc, F, am, bm, po);
    half_slots<MM, FI, HF, X + 1>(c, f, pair, acc, F, am, bm, po);
  }
}

// The whole loop: every pair's products into acc.  Ends with the clamped loads past
// the last pair still in flight.
template <class MM, int FI>
__device__ __forceinline__ void dense_halves(char* smem, const DenseOps& f, typename MM::acc_t (&acc)[FI][4], Frags& F,
                                             int am, int bm, const PairOffs& po) {
  Halves c;
#pragma unroll
  for (int q = 0; q < 5; ++q) c.s[q] = smem + q * kPairOp;
#pragma unroll
  for (int q = 0; q < 2 * FI; ++q) half_dma<FI>(c.s[0], f, true, 0, q);
#pragma unroll
  for (int q = 0; q < 8; ++q) half_dma<FI>(c.s[1], f, false, 0, q);
#pragma unroll
  for (int q = 0; q < 2 * FI; ++q) half_dma<FI>(c.s[2], f, true, 1, q);
  // as far as the pair before the first would have come
  constexpr int kBefore = (4 * FI * (2 * FI + 8) + 16 * FI - 1) / (16 * FI);
#pragma unroll
  for (int d = 0; d < kBefore; ++d) group_dma<FI>(c.s[3], c.s[4], f, -1, d);
  QLORA_WAIT(2 * FI + kBefore, 0);   // pair 0 has landed
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < FI) F.a0[i] = rd16(c.s[0] + am + i * 32 * 128 + po.o[0][0]);
    F.b0[i] = rd16(c.s[1] + bm + i * 32 * 128 + po.o[0][0]);
  }
  for (int pr = 0; pr < f.npair; ++pr) {
    __builtin_amdgcn_sched_barrier(0);
    half_slots<MM, FI, 0, 0>(c, f, pr, acc, F, am, bm, po);
    __builtin_amdgcn_sched_barrier(0);
    half_slots<MM, FI, 1, 0>(c, f, pr, acc, F, am, bm, po);
    c = Halves{{c.s[2], c.s[3], c.s[4], c.s[0], c.s[1]}};
  }
}

// The ring of half slots with 16 x 16 x 32 matrix instructions: a wave's 2 FI
// fragments of 16 weight rows by 8 of 16 tokens, a stage of 32 columns at a time.
// Slot X = 8 m + n of a stage is fragments (m, n).  Reads during a stage: at slot 0 its
// own last weight fragment; from slot 8 on the next stage's: token fragments into
// the other set, weight fragment m into the registers that slot 8 m + 7 was the
// last to use.  The odd stage's slot 8 waits for the next pair.
// The matrix units take as many cycles as with 32 x 32 x 16, but an accumulator is
// read and written half as often a product, and what is not spent so is clock:
// 4096 x 8192 x 22016 1155 -> 1073 us (1.80 and 1.85 million cycles), 4096 x 44032
// x 8192 2250 -> 2095.
struct Frags16 {
  bf16x8_t a[8], b[2][8];
};
// c += a b in place, in accumulation registers: with the builtin the compiler moves
// them about, 200 moves a pair.  It knows nothing of the instruction's latencies,
// then: operands come from loads, or (READY false) an instruction may have written
// them just before; what is not another product of c waits for mfma_done.
template <bool READY = true>
__device__ __forceinline__ void mfma_acc(const bf16x8_t& a, const bf16x8_t& b, f32x4_t& c) {
  if constexpr (READY)
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else
    asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma_done() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
template <int FI>
constexpr int quad_off(int d) { return d * 32 * FI / (2 * FI + 8); }
template <int FI>
constexpr int quad_rd(int q) { return 8 + q * (16 * FI - 10) / 8; }
template <int FI, int X, int HF>
__device__ __forceinline__ void quad_slot(const Halves& c, const DenseOps& f, int pair, f32x4_t (&acc)[2 * FI][8], Frags16& F,
                                          int am, int bm, const int (&o)[2]) {
  constexpr int NA = 2 * FI, S = 8 * NA, m = X / 8, n = X % 8;
  if constexpr (HF == 1 && X == 8) {
    QLORA_WAIT(2 * FI, 0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }
  mfma_acc(F.a[m], F.b[HF][n], acc[m][n]);
  if constexpr (X == 0) F.a[NA - 1] = rd16(c.s[0] + am + (NA - 1) * 16 * 128 + o[HF]);
  constexpr int w = HF == 0 ? 0 : 2;   // the next stage's halves
  if constexpr (n == 3 && m > 0) F.a[m - 1] = rd16(c.s[w] + am + (m - 1) * 16 * 128 + o[HF ^ 1]);
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (quad_rd<FI>(q) == X) F.b[HF ^ 1][q] = rd16(c.s[w + 1] + bm + q * 16 * 128 + o[HF ^ 1]);
  constexpr int off = HF == 0 ? S - 8 + X : X < 8 ? 2 * S - 8 + X : X - 8;   // from the barrier on
#pragma unroll
  for (int d = 0; d < 2 * FI + 8; ++d)
    if (quad_off<FI>(d) == off) {
      if constexpr (HF == 1 && X >= 8)
        group_dma<FI>(c.s[0], c.s[1], f, pair, d);
      else
        group_dma<FI>(c.s[3], c.s[4], f, pair - 1, d);
    }
  __builtin_amdgcn_sched_barrier(0);
}
template <int FI, int HF, int X>
__device__ __forceinline__ void quad_slots(const Halves& c, const DenseOps& f, int pair, f32x4_t (&acc)[2 * FI][8], Frags16& F,
                                           int am, int bm, const int (&o)[2]) {
  if constexpr (X < 16 * FI) {
    quad_slot<FI, X, HF>(c, f, pair, acc, F, am, bm, o);
    quad_slots<FI, HF, X + 1>(c, f, pair, acc, F, am, bm, o);
  }
}
// Loads of a group that come before its pair's last slot.
template <int FI>
constexpr int quads_before() {
  int n = 0;
  for (int d = 0; d < 2 * FI + 8; ++d) n += quad_off<FI>(d) < 16 * FI - 8;
  return n;
}
// The whole loop, as dense_halves.
template <int FI>
__device__ __forceinline__ void dense_quads(char* smem, const DenseOps& f, f32x4_t (&acc)[2 * FI][8], int am, int bm,
                                            const int (&o)[2]) {
  Halves c;
#pragma unroll
  for (int q = 0; q < 5; ++q) c.s[q] = smem + q * kPairOp;
#pragma unroll
  for (int q = 0; q < 2 * FI; ++q) half_dma<FI>(c.s[0], f, true, 0, q);
#pragma unroll
  for (int q = 0; q < 8; ++q) half_dma<FI>(c.s[1], f, false, 0, q);
#pragma unroll
  for (int q = 0; q < 2 * FI; ++q) half_dma<FI>(c.s[2], f, true, 1, q);
  constexpr int kBefore = quads_before<FI>();
#pragma unroll
  for (int d = 0; d < kBefore; ++d) group_dma<FI>(c.s[3], c.s[4], f, -1, d);
  QLORA_WAIT(2 * FI + kBefore, 0);   // pair 0 has landed
  __builtin_amdgcn_s_barrier();
  mfma_done();
  Frags16 F;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < 2 * FI - 1) F.a[i] = rd16(c.s[0] + am + i * 16 * 128 + o[0]);
    F.b[0][i] = rd16(c.s[1] + bm + i * 16 * 128 + o[0]);
  }
  for (int pr = 0; pr < f.npair; ++pr) {
    __builtin_amdgcn_sched_barrier(0);
    quad_slots<FI, 0, 0>(c, f, pr, acc, F, am, bm, o);
    __builtin_amdgcn_sched_barrier(0);
    quad_slots<FI, 1, 0>(c, f, pr, acc, F, am, bm, o);
    c = Halves{{c.s[2], c.s[3], c.s[4], c.s[0], c.s[1]}};
  }
  mfma_done();
}

// One 32-wide chunk of the LoRA tail, in registers: the weight half
// B'[row0 + row, j0 ..] (zero past the rank, and for rows outside [lo, hi))
// and the token half T[trow0 + row, j0 + 8 c ..] (T is trows x rank with
// row stride ld; zero past the rank and the last row).  Token half: thread t
// holds row (t + 256 e) >> 2, 16-byte chunk (t + 256 e) & 3.  Weight half:
// B' is B [rows x r], held like the tokens; or, with b_trans, the transpose
// of B [r x rows], read along its rows (coalesced): thread t holds B[j0 +
// (i >> 5)][row0 + 8 (i & 31) ..] for i = t + 256 e.
struct TailRegs {
  uint4 w[4], t[4];
};
__device__ __forceinline__ void tail_load(TailRegs& R, const bf16_t* Bm, bool b_trans, int64_t rows, int r,
                                          int64_t row0, int j0, int64_t lo, int64_t hi, const bf16_t* T,
                                          int64_t ld, int64_t trows, int64_t trow0) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int idx = threadIdx.x + kThreads * e;
    const int row = idx >> 2, c = idx & 3, col = j0 + 8 * c;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (!b_trans) {
      if (col < r && row0 + row >= lo && row0 + row < hi)
        v = *reinterpret_cast<const uint4*>(Bm + (row0 + row) * r + col);
    } else {
      // rows % 8 == 0 and lo, hi multiples of 8: the 8 rows are all in or all out
      const int j = j0 + (idx >> 5);
      const int64_t rr = row0 + 8 * (idx & 31);
      if (j < r && rr >= lo && rr < hi) v = *reinterpret_cast<const uint4*>(Bm + (int64_t)j * rows + rr);
    }
    R.w[e] = v;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (col < r && trow0 + row < trows) u = *reinterpret_cast<const uint4*>(T + (trow0 + row) * ld + col);
    R.t[e] = u;
  }
}
// The same for one adapter whose T is kTermParts bf16 matrices [trows x r], as a
// chunk of a rank of kTermParts r: ranks r .. are the second part's.
__device__ __forceinline__ void tail_load_parts(TailRegs& R, const bf16_t* Bm, bool b_trans, int64_t rows, int r,
                                                int64_t row0, int j0, const bf16_t* T, int64_t trows,
                                                int64_t trow0) {
  static_assert(kTermParts == 2);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int idx = threadIdx.x + kThreads * e;
    const int row = idx >> 2, col = j0 + 8 * (idx & 3), part = col >= r ? 1 : 0, k = col - part * r;
    R.w[e] = R.t[e] = make_uint4(0u, 0u, 0u, 0u);
    if (!b_trans) {
      if (k < r && row0 + row < rows) R.w[e] = *reinterpret_cast<const uint4*>(Bm + (row0 + row) * r + k);
    } else {
      const int j = j0 + (idx >> 5), kj = j >= r ? j - r : j;
      const int64_t rr = row0 + 8 * (idx & 31);
      if (kj < r && rr < rows) R.w[e] = *reinterpret_cast<const uint4*>(Bm + (int64_t)kj * rows + rr);
    }
    if (k < r && trow0 + row < trows)
      R.t[e] = *reinterpret_cast<const uint4*>(T + (part * trows + trow0 + row) * r + k);
  }
}
// The chunk into LDS: s T as a 64-byte-row tile at dst + kOp; the weights
// at dst, as a 64-byte-row tile or, with b_trans, as a tile of 32 rank rows
// x 256 weight rows (512-byte rows, 32-byte block b of rank row n at
// b ^ (n & 3)) for transposed fragment reads.
__device__ __forceinline__ void tail_store(char* dst, const TailRegs& R, bool b_trans, float s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int idx = threadIdx.x + kThreads * e;
    const int row = idx >> 2, c = idx & 3;
    if (!b_trans) {
      wr16(dst + spos(row, c), R.w[e]);
    } else {
      const int n = idx >> 5, sg = idx & 31;
      wr16(dst + n * 512 + 32 * ((sg >> 1) ^ (n & 3)) + 16 * (sg & 1), R.w[e]);
    }
    wr16(dst + kOp + spos(row, c), scale16(R.t[e], s));
  }
}

// The LoRA tail by DMA, for tiles inside one adapter group with the rank in
// whole 32-wide chunks.  A chunk takes 32 KiB of LDS in the layouts of
// tail_store, but the token half holds T itself (unscaled): s, where T does not
// hold it, is applied to each fragment as it is read, which rounds exactly as
// tail_store does.
struct TailSrc {
  rsrc_t wr, tr;         // weight half (B, or A with b_trans), token half (T)
  int64_t n0, m0, rows;  // first weight row, first token row, weight rows (N)
  int r, ld, col0;       // rank, T's row stride, T's first column (the group's)
  bool bt;
};
// DMA of chunk c (ranks 32 c ..) into dst: per wave 4 token and 4 weight
// instructions of 1 KiB.  Token rows / weight rows (no b_trans): the
// 256-row x 64-byte pattern of dma_row / dma_chunk.  With b_trans: rank rows
// n = 2 (4 w + q) + (lane >> 5) of 512 bytes, lane position pc = lane & 31
// holding 32-byte block (pc >> 1) ^ (n & 3), half pc & 1.  Rows past the
// arrays read zero (buffer range) or another row's finite values, which only
// reach outputs past M or N.
__device__ __forceinline__ void tail_dma(char* dst, const TailSrc& S, int c, int w, int lane) {
  const int j0 = 32 * c;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = dma_row(q, w, lane), ch = dma_chunk(lane);
    dma16(S.tr, dst + kOp + (64 * q + 16 * w) * 64,
          (uint32_t)(((S.m0 + row) * S.ld + S.col0 + j0 + 8 * ch) * 2), 0u);
    if (!S.bt) {
      dma16(S.wr, dst + (64 * q + 16 * w) * 64, (uint32_t)(((S.n0 + row) * S.r + j0 + 8 * ch) * 2), 0u);
    } else {
      const int n = 2 * (4 * w + q) + (lane >> 5), pc = lane & 31;
      const int e = 8 * (2 * ((pc >> 1) ^ (n & 3)) + (pc & 1));
      dma16(S.wr, dst + 1024 * (4 * w + q), (uint32_t)(((int64_t)(j0 + n) * S.rows + S.n0 + e) * 2), 0u);
    }
  }
}
__device__ __forceinline__ bf16x8_t scale_frag(bf16x8_t v, float s) {
  return __builtin_bit_cast(bf16x8_t, scale16(__builtin_bit_cast(uint4, v), s));
}

// The tile's sums as they are, fp32 or 32-bit integers (the lane layout of
// store_tile_lds): lane (lr, h) of wave (wr, wc) holds token row0 + 128 wr + 32 j
// + lr, columns col0 + 32 FI wc + 32 i + 8 q + 4 h + 0..3, stored as one 16-byte
// piece (cols % 4 == 0).
template <int FI, class ACC, class T>
__device__ __forceinline__ void store_tile_parts(const ACC (&acc)[FI][4], T* out, int64_t ld, int64_t rows,
                                                 int64_t cols, int64_t row0, int64_t col0) {
  typedef T piece_t __attribute__((ext_vector_type(4)));
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wr = w >> 1, wc = w & 1, lr = lane & 31, h = lane >> 5;
#pragma unroll
  for (int i = 0; i < FI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = row0 + 128 * wr + 32 * j + lr;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t col = col0 + 32 * FI * wc + 32 * i + 8 * q + 4 * h;
        if (row < rows && col < cols)
          *reinterpret_cast<piece_t*>(out + row * ld + col) =
              piece_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
      }
    }
}

}  // namespace
}  // namespace qlora
