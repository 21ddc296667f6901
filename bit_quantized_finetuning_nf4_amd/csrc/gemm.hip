// gemm.hip -- the four LoRA products of the QLoRA linear layer:
//
//   U = X A^T,  G = dY B            (contraction along the rows of X / dY)
//   dA = s G^T X,  dB = s dY^T U    (contraction over the tokens)
// (the fused NF4 GEMMs live in gemm_nf4.hip)
//
// deepfa.ir blog, "LoRA: Prerequisite" and "QLoRA's Working Process" (the
// 4-bit weights are dequantized to BF16 on the fly in the forward and
// backward passes, only the adapters are trained); glossary "QLoRA",
// Definition (weight gradients only for the LoRA matrices).
//
// All four read one large bf16 matrix (X or dY, M x K or M x N) once and a
// small one (A, B, G or U) with the rank r <= 128 on one side, so they are
// HBM streams with little arithmetic.  Both kernels below bring the large
// matrix into LDS by buffer->LDS DMA through a ring of six 32-row (or
// 32-column) stages, five stages ahead, one barrier per stage, and run a few
// bf16 MFMAs (32x32x16, fp32 accumulation) per stage.  The contraction is
// split over workgroups (about one per CU); each split writes fp32 partial
// sums and reduce_kernel adds them in a fixed order, so results do not
// depend on timing.  The rank side is padded to RP = 64 or 128 with values
// that only reach output columns >= r, which are never stored.
#include <algorithm>

#include "device.h"
#include "kernels.h"
#include "lds.h"
#include "ride.h"

namespace qlora {

namespace {

constexpr int kThreads = 256;
constexpr int kRing = 6;    // stages in the LDS ring
constexpr int kAhead = 5;   // stages DMA'd ahead of the one being multiplied

// DMA of a 32-row x (PB / 2)-column tile in the layout above: instruction q
// covers rows (512 / PB) q .. ; lane l writes byte 16 (l mod (PB / 16)) of
// its row, which holds global column 8 (2 ((p >> 1) ^ (row & 3)) + (p & 1))
// for p = l mod (PB / 16).
template <int PB>
__device__ __forceinline__ void tr_dma_coords(int q, int lane, int& row, int& col) {
  constexpr int kLanesPerRow = PB / 16;
  row = (64 / kLanesPerRow) * q + lane / kLanesPerRow;
  const int p = lane % kLanesPerRow;
  col = 8 * (2 * ((p >> 1) ^ (row & 3)) + (p & 1));
}

// ---------------------------------------------------------------------------
// Row contraction: out[m][j] = sum_c P[m][c] Q(c, j), 128 rows m per
// workgroup (wave w: rows 32 w .. +31, the MFMA B operand), all RP ranks j
// (the A operand), stages of 32 c.  P rows are DMA'd as 64-byte rows
// (16-byte chunk c of row m at c ^ ((m >> 2) & 3)).  Q is A [r x C] (QT =
// false: rows j, read like P) or B [C x r] (QT = true: rows c, read
// transposed).  Output D[j][m]: a lane holds four consecutive j of one m.
// ---------------------------------------------------------------------------
template <int RP, bool QT>
struct RowShape {
  static constexpr int kP = 128 * 64;                      // 8 KiB of P per stage
  static constexpr int kQ = RP * 64;                       // Q per stage (RP rows x 64 B, or 32 rows x 2 RP B)
  static constexpr int kStage = kP + kQ;
  static constexpr int kQDma = kQ / 1024 / 4;              // Q DMA instructions per wave per stage
  static constexpr int kLoads = 2 + kQDma;                 // all DMA instructions per wave per stage
};

template <int RP, bool QT>
__global__ __launch_bounds__(kThreads, 1) void rskinny_kernel(const bf16_t* __restrict__ P, int64_t M, int64_t C,
                                                              int64_t ldp, int64_t p_gs,
                                                              const bf16_t* __restrict__ Q, int r, int64_t q_gs,
                                                              int stages_per_split, int tiles_m, int ldo,
                                                              float* __restrict__ part) {
  using S = RowShape<RP, QT>;
  extern __shared__ __align__(16) char smem[];
  const int tm = blockIdx.x % tiles_m, sp = blockIdx.x / tiles_m, g = blockIdx.y;
  const int t = threadIdx.x, w = t >> 6, lane = t & 63, lr = lane & 31, h = lane >> 5;
  const int64_t m0 = (int64_t)tm * 128;
  const int nst = (int)((C + 31) / 32);
  const int s0 = sp * stages_per_split, s1 = min(nst, s0 + stages_per_split);
  P += g * p_gs;
  Q += g * q_gs;
  // P rows of this tile only (rows past M read as zero); Q whole
  const rsrc_t pr = make_rsrc(P + m0 * ldp, (uint32_t)(((min((int64_t)128, M - m0) - 1) * ldp + C) * 2));
  const rsrc_t qr = make_rsrc(Q, (uint32_t)((int64_t)r * C * 2));
  uint32_t po[2], qo[S::kQDma > 0 ? S::kQDma : 1];
  int pl[2], ql[S::kQDma > 0 ? S::kQDma : 1];
#pragma unroll
  for (int q = 0; q < 2; ++q) {   // P: instruction q of wave w fills rows 16 (2w + q) .. +15
    const int row = 16 * (2 * w + q) + (lane >> 2), ch = (lane & 3) ^ ((lane >> 4) & 3);
    po[q] = (uint32_t)(row * ldp * 2 + ch * 16);
    pl[q] = 16 * (2 * w + q) * 64;
  }
#pragma unroll
  for (int q = 0; q < S::kQDma; ++q) {
    const int gi = S::kQDma * w + q;   // 1 KiB piece of the stage's Q tile
    if constexpr (!QT) {               // rows j of A, 64 bytes per stage
      const int row = 16 * gi + (lane >> 2), ch = (lane & 3) ^ ((lane >> 4) & 3);
      qo[q] = (uint32_t)(row * C * 2 + ch * 16);
    } else {                           // rows c of B, 2 RP bytes, transposed layout
      int row, col;
      tr_dma_coords<2 * RP>(gi, lane, row, col);
      qo[q] = (uint32_t)(row * r * 2 + col * 2);
    }
    ql[q] = S::kP + gi * 1024;
  }
  auto dma = [&](int st, int slot) {
    const int ss = min(st, s1 - 1);    // past the split: re-load its last stage (never read)
    char* base = smem + slot * S::kStage;
#pragma unroll
    for (int q = 0; q < 2; ++q) dma16(pr, base + pl[q], po[q], (uint32_t)ss * 64u);
#pragma unroll
    for (int q = 0; q < S::kQDma; ++q)
      dma16(qr, base + ql[q], qo[q], QT ? (uint32_t)ss * 32u * (uint32_t)r * 2u : (uint32_t)ss * 64u);
  };

  constexpr int FJ = RP / 32;
  static_assert(!QT || FJ == 2 || FJ == 4, "transposed rank side: RP 64 or 128");
  f32x16_t acc[FJ];
#pragma unroll
  for (int f = 0; f < FJ; ++f)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[f][e] = 0.0f;

  if (s0 < s1) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) dma(s0 + a, a);
    int slot = 0;
    for (int st = s0; st < s1; ++st) {
      // stage st was issued kAhead - 1 stages before the last kAhead - 1 issues
      QLORA_WAIT((kAhead - 1) * S::kLoads, 0);
      __builtin_amdgcn_s_barrier();
      dma(st + kAhead, slot == 0 ? kRing - 1 : slot - 1);   // the slot stage st - 1 used
      const char* base = smem + slot * S::kStage;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        // P fragment (B operand): row 32 w + lr, the 8 columns that lane half h
        // takes in k16 step kk.  Both operands must agree on that: a 64-byte
        // row read takes chunk 2h + kk (columns 16 h + 8 kk ..), a transposed
        // read of 32 Q rows takes rows 16 kk + 8 h .. (chunk 2 kk + h)
        const int ch = QT ? 2 * kk + h : 2 * h + kk;
        bf16x8_t b = rd16(base + spos(32 * w + lr, ch));
        if (32 * st + 8 * ch >= C) b = bf16x8_t{};   // columns past C (C % 8 == 0)
        bf16x8_t a[FJ];
        if constexpr (!QT) {
#pragma unroll
          for (int f = 0; f < FJ; ++f) a[f] = rd16(base + S::kP + spos(32 * f + lr, 2 * h + kk));
        } else {
          // transposed reads in asm blocks (see tr_read2): FJ is 2 or 4
          constexpr int O = 4 * 2 * RP;
          const char* qb = base + S::kP + kk * 16 * 2 * RP;
#pragma unroll
          for (int f = 0; f < FJ; f += 2) tr_read2<O, O>(qb + tr_off<2 * RP>(f), qb + tr_off<2 * RP>(f + 1), a[f], a[f + 1]);
        }
#pragma unroll
        for (int f = 0; f < FJ; ++f) acc[f] = mfma32x32x16(a[f], b, acc[f]);
      }
      slot = slot == kRing - 1 ? 0 : slot + 1;
    }
    QLORA_WAIT(0, 0);
  }
  // D[j][m]: lane (lr, h) holds m = m0 + 32 w + lr, j = 32 f + 8 q + 4 h + 0..3,
  // stored at column g r + j of the split's [M x ldo] partial
  float* out = part + (int64_t)sp * M * ldo + (int64_t)g * r;
  const int64_t m = m0 + 32 * w + lr;
  if (m < M) {
#pragma unroll
    for (int f = 0; f < FJ; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int j = 32 * f + 8 * q + 4 * h;
        if (j < r)
          *reinterpret_cast<float4*>(out + m * ldo + j) =
              make_float4(acc[f][4 * q], acc[f][4 * q + 1], acc[f][4 * q + 2], acc[f][4 * q + 3]);
      }
  }
}

// ---------------------------------------------------------------------------
// The row contraction of one adapter by whole lines: stages of 64 columns, one
// 128-byte line of every row of P (a CU keeps about 90 lines in flight, and a
// request for half a line takes a place like a whole one: with 64-byte rows U
// of 4096 x 8192 at rank 64 took 26 us).  Rows in the layout of pos128; a ring
// of four stages.  A fifth wave issues the DMAs: their issue stalls while the
// lines in flight are at their limit, and would hold up the wave's masks and
// products.  Q is A [r x C], read like P, or (QT) B [C x r], 64 rows c a
// stage, read transposed.  DROP: P is drop(P), masked as its fragments are
// read: a fragment's 16 bytes are eight consecutive columns of one row, one
// Philox block (rng.h), and no two lanes read the same ones.  G of 2048 x 4096
// at rank 64 7 us, U of 4096 x 8192 under the mask 23.6 us.
// ---------------------------------------------------------------------------
constexpr int kWideRing = 4, kWideAhead = kWideRing - 1, kWideThreads = kThreads + 64;

template <int RP>
struct WideShape {
  static constexpr int kP = 128 * 128;                     // 16 KiB of P per stage
  static constexpr int kQ = RP * 128;                      // RP rows x 128 B, or 64 rows x 2 RP B
  static constexpr int kStage = kP + kQ;
  static constexpr int kQDma = kQ / 1024;                  // DMA instructions per stage
  // all but two stages have landed (the counter holds 63 at most)
  static constexpr int kWait = (kWideAhead - 1) * (16 + kQDma) < 63 ? (kWideAhead - 1) * (16 + kQDma) : 63;
};

template <int RP, bool QT, bool DROP>
__global__ __launch_bounds__(kWideThreads, 1) void rwide_kernel(const bf16_t* __restrict__ P, int64_t M, int64_t C,
                                                            const bf16_t* __restrict__ Q, int r, int stages_per_split,
                                                            int tiles_m, float* __restrict__ part, DropArgs drop) {
  using S = WideShape<RP>;
  extern __shared__ __align__(16) char smem[];
  const int tm = blockIdx.x % tiles_m, sp = blockIdx.x / tiles_m;
  const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63, lr = lane & 31, h = lane >> 5;
  const int64_t m0 = (int64_t)tm * 128;
  const int nst = (int)((C + 63) / 64);
  const int s0 = sp * stages_per_split, s1 = min(nst, s0 + stages_per_split);   // no split is empty
  // P rows of this tile only (rows past M read as zero); Q whole
  const rsrc_t pr = make_rsrc(P + m0 * C, (uint32_t)(min((int64_t)128, M - m0) * C * 2));
  const rsrc_t qr = make_rsrc(Q, (uint32_t)((int64_t)r * C * 2));
  if (w == 4) {   // the wave that brings the stages
    uint32_t po[16], qo[S::kQDma];
#pragma unroll
    for (int q = 0; q < 16; ++q) {   // rows 8 q .. + 7 of P
      const int row = 8 * q + (lane >> 3);
      po[q] = (uint32_t)(row * C * 2 + 16 * ((lane & 7) ^ ((row >> 1) & 7)));
    }
#pragma unroll
    for (int q = 0; q < S::kQDma; ++q) {   // 1 KiB pieces of the stage's Q tile
      if constexpr (!QT) {                 // rows j of A (past r: never stored)
        const int row = 8 * q + (lane >> 3);
        qo[q] = (uint32_t)(row * C * 2 + 16 * ((lane & 7) ^ ((row >> 1) & 7)));
      } else {                             // rows c of B
        int row, col;
        tr_dma_coords<2 * RP>(q, lane, row, col);
        qo[q] = (uint32_t)(row * r * 2 + col * 2);
      }
    }
    auto dma = [&](int st, int slot) __attribute__((always_inline)) {
      const int ss = min(st, s1 - 1);    // past the split: re-load its last stage (never read)
      char* base = smem + slot * S::kStage;
#pragma unroll
      for (int q = 0; q < 16; ++q) dma16(pr, base + q * 1024, po[q], (uint32_t)ss * 128u);
#pragma unroll
      for (int q = 0; q < S::kQDma; ++q)
        dma16(qr, base + S::kP + q * 1024, qo[q], QT ? (uint32_t)ss * 64u * (uint32_t)r * 2u : (uint32_t)ss * 128u);
    };
#pragma unroll
    for (int a = 0; a < kWideAhead; ++a) dma(s0 + a, a);
    int slot = kWideRing - 1;
    for (int st = s0; st < s1; ++st) {
      QLORA_WAIT(S::kWait, 0);
      __builtin_amdgcn_s_barrier();   // stage st has landed, and stage st - 1 has been read
      dma(st + kWideAhead, slot);     // the slot stage st - 1 used
      slot = slot == kWideRing - 1 ? 0 : slot + 1;
    }
    QLORA_WAIT(0, 0);
    return;
  }
  constexpr int FJ = RP / 32;
  f32x16_t acc[FJ];
#pragma unroll
  for (int f = 0; f < FJ; ++f)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[f][e] = 0.0f;
  [[maybe_unused]] DropKey key;
  [[maybe_unused]] uint32_t row_block = 0;   // M C < 2^31: block numbers in 32 bits
  if constexpr (DROP) {
    key = drop_key(drop);
    row_block = (uint32_t)(m0 + 32 * w + lr) * (uint32_t)(C >> 3);
  }
  int slot = 0;
  for (int st = s0; st < s1; ++st) {
    QLORA_WAIT(63, 0);   // this wave's reads of stage st - 1
    __builtin_amdgcn_s_barrier();
    const char* base = smem + slot * S::kStage;
    const bool ragged = 64 * (st + 1) > C;   // columns past C (C % 8 == 0)
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int ch = 2 * kk + h;   // both operands: columns 16 kk + 8 h ..
      bf16x8_t b = rd16(base + pos128(32 * w + lr, ch));
      bf16x8_t a[FJ];
      if constexpr (!QT) {
#pragma unroll
        for (int f = 0; f < FJ; ++f) a[f] = rd16(base + S::kP + pos128(32 * f + lr, ch));
      } else {
        // transposed reads in asm blocks (see tr_read2)
        constexpr int O = 4 * 2 * RP;
        const char* qb = base + S::kP + kk * 16 * 2 * RP;
#pragma unroll
        for (int f = 0; f < FJ; f += 2) tr_read2<O, O>(qb + tr_off<2 * RP>(f), qb + tr_off<2 * RP>(f + 1), a[f], a[f + 1]);
      }
      if (ragged && 64 * st + 8 * ch >= C) {   // the next row's: neither operand may bring its infinities
        b = bf16x8_t{};
#pragma unroll
        for (int f = 0; f < FJ; ++f) a[f] = bf16x8_t{};
      }
      if constexpr (DROP)
        b = __builtin_bit_cast(bf16x8_t, drop8(__builtin_bit_cast(u32x4_t, b), row_block + (uint32_t)(8 * st + ch), key));
#pragma unroll
      for (int f = 0; f < FJ; ++f) acc[f] = mfma32x32x16(a[f], b, acc[f]);
    }
    slot = slot == kWideRing - 1 ? 0 : slot + 1;
  }
  // D[j][m]: lane (lr, h) holds m = m0 + 32 w + lr, j = 32 f + 8 q + 4 h + 0..3
  float* out = part + (int64_t)sp * M * r;
  const int64_t m = m0 + 32 * w + lr;
  if (m < M) {
#pragma unroll
    for (int f = 0; f < FJ; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int j = 32 * f + 8 * q + 4 * h;
        if (j < r)
          *reinterpret_cast<float4*>(out + m * r + j) =
              make_float4(acc[f][4 * q], acc[f][4 * q + 1], acc[f][4 * q + 2], acc[f][4 * q + 3]);
      }
  }
}

// ---------------------------------------------------------------------------
// Token contraction: D = sum_m Big[m][c] Sm[m][j] for 128 columns c per
// workgroup (wave w: columns 32 w .. +31) and all RP ranks j, stages of 32
// tokens.  Both tiles are rows m, read transposed.  DB = false stores dA
// [r x C] (A operand = Big, D[c][j]: four consecutive c per lane); DB = true
// stores dB [C x r] (A operand = Sm, D[j][c]: four consecutive j per lane).
// PARTS = kGradParts: the rank side is an fp32 matrix as a sum of three bf16
// ones, sm_part elements apart, all multiplied into the same sums (dA is fp32:
// one bf16 G would leave it G's rounding of 2^-9, two 2^-18, above the sum's
// own error).
// DROP: Big is drop(Big).  A transposed fragment holds eight tokens of one
// column, eight different Philox blocks, so the mask is applied in LDS
// instead: each lane zeroes the dropped elements of the 16-byte pieces that
// its own wave's DMA brought (one block each), one stage ahead of the one
// being multiplied; the stage's barrier publishes them.
// dA and dB of 2048 x 4096 x 4096 at rank 64 15 us, of 4096 tokens at 22016 x
// 8192 87 us (247 MB of X and dY: 2.8 TB/s), bound by the lines a CU keeps in
// flight, G's parts among them; tiles of 256 columns, which halve G's share, by
// eight waves took 17 and 98 us.
// ---------------------------------------------------------------------------
template <int RP, int PARTS>
struct ColShape {
  static constexpr int kBig = 32 * 256;                    // 8 KiB: 32 rows x 128 columns
  static constexpr int kSm = 32 * 2 * RP;                  // 32 rows x RP ranks
  static constexpr int kStage = kBig + PARTS * kSm;
  static constexpr int kSmDma = kSm / 1024 / 4;
  static constexpr int kLoads = 2 + PARTS * kSmDma;
  // three parts: a shorter ring, so that two workgroups of a rank up to 64
  // share a CU (a CU keeps about 11 KiB of loads in flight whatever the ring)
  static constexpr int kRing = PARTS == 1 ? qlora::kRing : 4;
  static constexpr int kAhead = kRing - 1;
};

// Workgroup `block` of group g (of `groups`).
template <int RP, bool DB, int PARTS, bool DROP>
__device__ __forceinline__ void cskinny(int block, int g, int groups, char* smem, const bf16_t* __restrict__ Big, int64_t M,
                                        int64_t C, int64_t ldb, int64_t big_gs, const bf16_t* __restrict__ Sm, int r,
                                        int lds, int64_t sm_gs, int stages_per_split, int tiles_c,
                                        float* __restrict__ part, int64_t sm_part, const DropArgs& drop, float scale) {
  static_assert(PARTS == 1 || (PARTS == 3 && !DB && RP <= 128), "three-part rank side: dA of one adapter");
  using S = ColShape<RP, PARTS>;
  constexpr int kRing = S::kRing, kAhead = S::kAhead;
  const int tc = block % tiles_c, sp = block / tiles_c;
  const int t = threadIdx.x, w = t >> 6, lane = t & 63, lr = lane & 31, h = lane >> 5;
  const int64_t c0 = (int64_t)tc * 128;
  const int nst = (int)((M + 31) / 32);
  const int s0 = sp * stages_per_split, s1 = min(nst, s0 + stages_per_split);
  Big += g * big_gs;
  Sm += g * sm_gs;
  // rows past M read as zero
  const rsrc_t br = make_rsrc(Big, (uint32_t)(((M - 1) * ldb + C) * 2));
  rsrc_t sr[PARTS];
#pragma unroll
  for (int p = 0; p < PARTS; ++p) sr[p] = make_rsrc(Sm + p * sm_part, (uint32_t)(((M - 1) * lds + r) * 2));
  uint32_t bo[2], so[S::kSmDma];
  int bl[2], sl[S::kSmDma];
  [[maybe_unused]] DropKey key;
  [[maybe_unused]] uint32_t blk[2];   // Philox block of the lane's pieces in stage 0 (M C < 2^31)
  if constexpr (DROP) key = drop_key(drop);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    int row, col;
    tr_dma_coords<256>(2 * w + q, lane, row, col);
    bo[q] = (uint32_t)(row * ldb * 2 + (c0 + col) * 2);   // columns past C: never stored
    bl[q] = (2 * w + q) * 1024;
    if constexpr (DROP) blk[q] = (uint32_t)((row * C + c0 + col) >> 3);
  }
#pragma unroll
  for (int q = 0; q < S::kSmDma; ++q) {
    int row, col;
    tr_dma_coords<2 * RP>(S::kSmDma * w + q, lane, row, col);
    so[q] = (uint32_t)(row * lds * 2 + col * 2);   // ranks past r: never stored
    sl[q] = S::kBig + (S::kSmDma * w + q) * 1024;
  }
  auto dma = [&](int st, int slot) {
    const uint32_t ss = (uint32_t)min(st, s1 - 1);
    char* base = smem + slot * S::kStage;
#pragma unroll
    for (int q = 0; q < 2; ++q) dma16(br, base + bl[q], bo[q], ss * 32u * (uint32_t)ldb * 2u);
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
#pragma unroll
      for (int q = 0; q < S::kSmDma; ++q)
        dma16(sr[p], base + p * S::kSm + sl[q], so[q], ss * 32u * (uint32_t)lds * 2u);
  };
  // zero the dropped elements of this lane's pieces of stage st, in slot
  // `slot` (columns past C: masks of values that are never stored)
  [[maybe_unused]] auto mask = [&](int st, int slot) __attribute__((always_inline)) {
    char* base = smem + slot * S::kStage;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      char* p = base + bl[q] + 16 * lane;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p);
      *reinterpret_cast<u32x4_t*>(p) = drop8(v, blk[q] + (uint32_t)st * 4u * (uint32_t)C, key);
    }
  };

  constexpr int FJ = RP / 32;
  static_assert(FJ == 2 || FJ == 4 || FJ == 8, "RP 64, 128 or 256");
  f32x16_t acc[FJ];
#pragma unroll
  for (int f = 0; f < FJ; ++f)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[f][e] = 0.0f;
  const int bo_frag = tr_off<256>(w);

  if (s0 < s1) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) dma(s0 + a, a);
    int slot = 0;
    if constexpr (DROP) {
      QLORA_WAIT((kAhead - 1) * S::kLoads, 0);
      mask(s0, 0);
    }
    for (int st = s0; st < s1; ++st) {
      // (DROP: stage st + 1 as well, for the mask; it is the wave's own DMA)
      QLORA_WAIT((kAhead - (DROP ? 2 : 1)) * S::kLoads, 0);
      __builtin_amdgcn_s_barrier();
      dma(st + kAhead, slot == 0 ? kRing - 1 : slot - 1);
      const char* base = smem + slot * S::kStage;
      if constexpr (DROP) {
        if (st + 1 < s1) mask(st + 1, slot == kRing - 1 ? 0 : slot + 1);
      }
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        if constexpr (PARTS == 3) {
          // fourteen transposed reads per asm block (see tr_read7): the big
          // tile's fragment and two rank fragments of each part
          constexpr int O = 4 * 2 * RP;
          const char* sb = base + S::kBig + kk * 16 * 2 * RP;
#pragma unroll
          for (int f = 0; f < FJ; f += 2) {
            bf16x8_t bg, sm[3][2];
            tr_read7<4 * 256, S::kSm, O>(base + kk * 16 * 256 + bo_frag, sb + tr_off<2 * RP>(f),
                                         sb + tr_off<2 * RP>(f + 1), bg, sm);
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
              for (int e = 0; e < 2; ++e) acc[f + e] = mfma32x32x16(bg, sm[p][e], acc[f + e]);
          }
        } else {
          // transposed reads in asm blocks (see tr_read3): the big tile's
          // fragment and the first two rank fragments, then three at a time
          constexpr int O = 4 * 2 * RP;
          const char* sb = base + S::kBig + kk * 16 * 2 * RP;
          bf16x8_t bg, sm[FJ];
          tr_read3<4 * 256, O, O>(base + kk * 16 * 256 + bo_frag, sb + tr_off<2 * RP>(0), sb + tr_off<2 * RP>(1), bg,
                                  sm[0], sm[1]);
          if constexpr (FJ == 4) tr_read2<O, O>(sb + tr_off<2 * RP>(2), sb + tr_off<2 * RP>(3), sm[2], sm[3]);
          if constexpr (FJ == 8) {
#pragma unroll
            for (int f = 2; f < 8; f += 3)
              tr_read3<O, O, O>(sb + tr_off<2 * RP>(f), sb + tr_off<2 * RP>(f + 1), sb + tr_off<2 * RP>(f + 2), sm[f],
                                sm[f + 1], sm[f + 2]);
          }
#pragma unroll
          for (int f = 0; f < FJ; ++f)
            acc[f] = DB ? mfma32x32x16(sm[f], bg, acc[f]) : mfma32x32x16(bg, sm[f], acc[f]);
        }
      }
      slot = slot == kRing - 1 ? 0 : slot + 1;
    }
    QLORA_WAIT(0, 0);
  }
  // the split's partial holds all groups' outputs, group g at g C r
  float* out = part + ((int64_t)sp * groups + g) * C * r;
#pragma unroll
  for (int f = 0; f < FJ; ++f)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (!DB) {   // D[c][j]: c = c0 + 32 w + 8 q + 4 h + 0..3, j = 32 f + lr -> dA[j][c..]
        const int j = 32 * f + lr;
        const int64_t c = c0 + 32 * w + 8 * q + 4 * h;
        if (j < r && c < C)
          *reinterpret_cast<float4*>(out + j * C + c) =
              make_float4(acc[f][4 * q] * scale, acc[f][4 * q + 1] * scale, acc[f][4 * q + 2] * scale,
                          acc[f][4 * q + 3] * scale);
      } else {               // D[j][c]: j = 32 f + 8 q + 4 h + 0..3, c = c0 + 32 w + lr -> dB[c][j..]
        const int j = 32 * f + 8 * q + 4 * h;
        const int64_t c = c0 + 32 * w + lr;
        if (j < r && c < C)
          *reinterpret_cast<float4*>(out + c * r + j) =
              make_float4(acc[f][4 * q] * scale, acc[f][4 * q + 1] * scale, acc[f][4 * q + 2] * scale,
                          acc[f][4 * q + 3] * scale);
      }
    }
}

template <int RP, bool DB>
__global__ __launch_bounds__(kThreads, 1) void cskinny_kernel(const bf16_t* __restrict__ Big, int64_t M, int64_t C,
                                                              int64_t ldb, int64_t big_gs,
                                                              const bf16_t* __restrict__ Sm, int r, int lds,
                                                              int64_t sm_gs, int stages_per_split, int tiles_c,
                                                              float* __restrict__ part) {
  extern __shared__ __align__(16) char smem[];
  cskinny<RP, DB, 1, false>(blockIdx.x, blockIdx.y, gridDim.y, smem, Big, M, C, ldb, big_gs, Sm, r, lds, sm_gs,
                            stages_per_split, tiles_c, part, 0, DropArgs{}, 1.0f);
}

// Both gradients of one adapter in one launch, dA's workgroups first: apart
// they leave the card half idle at their starts and ends (2048 x 4096 x 4096
// at rank 64: 12.5 and 7.5 us).
struct GradArgs {
  const bf16_t *X, *dY, *G3, *U;
  int64_t M, N, K;
  int r, sps_a, tiles_a, blocks_a, sps_b, tiles_b;
  float *part_a, *part_b;   // dA, dB themselves where one split is all
  float scale_b;            // 1 where there are more (dA's is in G's parts)
  DropArgs drop;
};
template <int RP, bool DROP>
__global__ __launch_bounds__(kThreads, 1) void adapter_grads_kernel(GradArgs p) {
  extern __shared__ __align__(16) char smem[];
  const int id = blockIdx.x;
  if (id < p.blocks_a)
    cskinny<RP, false, 3, DROP>(id, 0, 1, smem, p.X, p.M, p.K, p.K, 0, p.G3, p.r, p.r, 0, p.sps_a, p.tiles_a, p.part_a,
                                p.M * p.r, p.drop, 1.0f);
  else
    cskinny<RP, true, 1, false>(id - p.blocks_a, 0, 1, smem, p.dY, p.M, p.N, p.N, 0, p.U, p.r, p.r, 0, p.sps_b,
                                p.tiles_b, p.part_b, 0, p.drop, p.scale_b);
}

__global__ __launch_bounds__(kThreads) void reduce_kernel(const float* __restrict__ part, int splits, int64_t n,
                                                          float scale, float* __restrict__ out_f32,
                                                          bf16_t* __restrict__ out_bf16,
                                                          bf16_t* __restrict__ out_bf16_2) {
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
  if (i >= n) return;
  const float4 acc = sum_splits(part, splits, n, i, scale);
  if (out_f32) *reinterpret_cast<float4*>(out_f32 + i) = acc;
  if (out_bf16 || out_bf16_2) {
    const uint2 p = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    if (out_bf16) *reinterpret_cast<uint2*>(out_bf16 + i) = p;
    if (out_bf16_2) *reinterpret_cast<uint2*>(out_bf16_2 + i) = p;
  }
}

template <int KIND>
__global__ __launch_bounds__(256) void ride_kernel(Ride a) {
  ride<KIND>(a, blockIdx.x);
}

// The reductions of dA and dB in one launch: elements [0, n0) of the
// output are out0 (partials at part0, splits0 of them), the next n1 are out1
// (part1, splits1); each sums its splits in order, as reduce_kernel does.
__global__ __launch_bounds__(kThreads) void reduce2_kernel(const float* __restrict__ part0, int splits0, int64_t n0,
                                                           float* __restrict__ out0,
                                                           const float* __restrict__ part1, int splits1, int64_t n1,
                                                           float* __restrict__ out1, float scale, float scale1) {
  int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
  const float* part = part0;
  float* out = out0;
  int splits = splits0;
  int64_t n = n0;
  if (i >= n0) {
    i -= n0;
    part = part1, out = out1, splits = splits1, n = n1, scale = scale1;
  }
  if (i >= n) return;
  const float4 acc = sum_splits(part, splits, n, i, scale);
  *reinterpret_cast<float4*>(out + i) = acc;
}

// Splits of the contraction (stages of 32) for about `target` workgroups,
// at least 32 stages each: shorter splits spend most of their time filling
// the ring and add partials (the 7B and 13B steps ran 1.1-1.4 % faster than
// with 8).  The target (256, one per CU of the part this is
// tuned for) was measured; it is fixed, not the device's CU count, because
// the workspace size a caller queries must not depend on which device is
// current.  It does not depend on the number of groups a launch covers
// either, so that a group call sums in the order of the per-linear calls.
struct Split {
  int tiles, sps, splits;
};
Split split_for(int64_t tiles, int64_t contraction, int target) {
  const int nst = (int)((contraction + 31) / 32);
  int want = (int)((target + tiles - 1) / tiles);
  want = std::max(1, std::min(want, std::max(1, nst / 32)));
  Split s;
  s.tiles = (int)tiles;
  s.sps = (nst + want - 1) / want;
  s.splits = (nst + s.sps - 1) / s.sps;
  return s;
}

Split kind_split(int64_t rows, int64_t cols, int64_t contraction, int kind) {
  // rows x cols is the output: kXAt, kDyB [M x r]; kGtX [r x K]; kDytU [N x r]
  const int64_t tiles = (kind == kGtX) ? (cols + 127) / 128 : (rows + 127) / 128;
  return split_for(tiles, contraction, 256);
}

hipError_t reduce(const float* part, int splits, int64_t n, float scale, float* out_f32, bf16_t* out_bf16,
                  bf16_t* out_bf16_2, hipStream_t st) {
  hipLaunchKernelGGL(reduce_kernel, dim3((unsigned)((n / 4 + kThreads - 1) / kThreads)), dim3(kThreads), 0, st,
                     part, splits, n, scale, out_f32, out_bf16, out_bf16_2);
  return hipGetLastError();
}

// Row contraction over G groups (grid y): group g reads P + g p_gs (rows of
// stride ldp, C columns) and Q + g q_gs, and writes columns g r .. of the
// [M x ldo] result.
struct RowArgs {
  const bf16_t* P;
  int64_t M, C, ldp, p_gs;
  const bf16_t* Q;
  int r;
  int64_t q_gs;
  int G, ldo;
};

template <int RP, bool QT>
hipError_t run_rows(const RowArgs& a, float* part, float scale, bf16_t* out, bf16_t* out2, hipStream_t st) {
  const Split sp = split_for((a.M + 127) / 128, a.C, 256);
  auto* fn = &rskinny_kernel<RP, QT>;
  const size_t lds = (size_t)kRing * RowShape<RP, QT>::kStage;
  hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3(sp.tiles * sp.splits, a.G), dim3(kThreads), lds, st, a.P, a.M, a.C, a.ldp, a.p_gs, a.Q,
                     a.r, a.q_gs, sp.sps, sp.tiles, a.ldo, part);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  return reduce(part, sp.splits, a.M * a.ldo, scale, nullptr, out, out2, st);
}

// Token contraction over G groups (grid y): group g reads Big + g big_gs
// (rows of stride ldb, C columns) and Sm + g sm_gs (rows of stride lds, r
// ranks), and writes the g-th C x r block of the result.
struct ColArgs {
  const bf16_t* Big;
  int64_t M, C, ldb, big_gs;
  const bf16_t* Sm;
  int r, lds;
  int64_t sm_gs;
  int G;
};

// The token-contraction product's partials (no reduction); *splits gets
// their count.
template <int RP, bool DB>
hipError_t run_cols(const ColArgs& a, float* part, int* splits, hipStream_t st) {
  const Split sp = split_for((a.C + 127) / 128, a.M, 256);
  auto* fn = &cskinny_kernel<RP, DB>;
  const size_t lds = (size_t)kRing * ColShape<RP, 1>::kStage;
  hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3(sp.tiles * sp.splits, a.G), dim3(kThreads), lds, st, a.Big, a.M, a.C, a.ldb,
                     a.big_gs, a.Sm, a.r, a.lds, a.sm_gs, sp.sps, sp.tiles, part);
  *splits = sp.splits;
  return hipGetLastError();
}

}  // namespace

size_t skinny_partial_bytes(int64_t rows, int64_t cols, int64_t contraction, int kind) {
  const Split sp = kind_split(rows, cols, contraction, kind);
  return (size_t)sp.splits * (size_t)rows * (size_t)cols * sizeof(float);
}

hipError_t launch_xat(const bf16_t* X, const bf16_t* A, int64_t M, int64_t K, int r, float* part, bf16_t* out,
                      bf16_t* out2, float scale, hipStream_t st) {
  const RowArgs a{X, M, K, K, 0, A, r, 0, 1, r};
  if (r <= 64) return run_rows<64, false>(a, part, scale, out, out2, st);
  if (r <= 128) return run_rows<128, false>(a, part, scale, out, out2, st);
  if (r <= 192) return run_rows<192, false>(a, part, scale, out, out2, st);
  return run_rows<256, false>(a, part, scale, out, out2, st);
}

hipError_t launch_dyb_group(const bf16_t* dY, int64_t ldy, const bf16_t* B, int64_t M, int64_t N, int r, int G,
                            float* part, bf16_t* out, float scale, hipStream_t st) {
  const RowArgs a{dY, M, N, ldy, N, B, r, N * r, G, G * r};
  if (r <= 64) return run_rows<64, true>(a, part, scale, out, nullptr, st);
  return run_rows<128, true>(a, part, scale, out, nullptr, st);
}

hipError_t launch_dyb(const bf16_t* dY, const bf16_t* B, int64_t M, int64_t N, int r, float* part, bf16_t* out,
                      float scale, hipStream_t st) {
  return launch_dyb_group(dY, N, B, M, N, r, 1, part, out, scale, st);
}

size_t grads_partial_bytes(int64_t M, int64_t N, int64_t K, int r, int G) {
  const size_t a = skinny_partial_bytes(G * r, K, M, kGtX);
  return (a + 255) / 256 * 256 + (size_t)G * skinny_partial_bytes(N, r, M, kDytU);
}

hipError_t launch_grads(const bf16_t* Gm, const bf16_t* X, const bf16_t* dY, int64_t ldy, const bf16_t* U, int ldu,
                        int64_t M, int64_t N, int64_t K, int r, int G, float* part, float* dA, float* dB, float scale,
                        hipStream_t st) {
  // dA [G r x K] = s G^T X in one pass over X (the stacked rank as one)
  const int ra = G * r;
  const ColArgs a{X, M, K, K, 0, Gm, ra, ra, 0, 1};
  int sa = 0, sb = 0;
  hipError_t e = ra <= 64    ? run_cols<64, false>(a, part, &sa, st)
                 : ra <= 128 ? run_cols<128, false>(a, part, &sa, st)
                             : run_cols<256, false>(a, part, &sa, st);
  if (e != hipSuccess) return e;
  // dB_g [N x r] = s dY_g^T U_g for every group, partials after dA's
  float* part_b = part + (skinny_partial_bytes(ra, K, M, kGtX) + 255) / 256 * 256 / sizeof(float);
  const ColArgs b{dY, M, N, ldy, N, U, r, ldu, r, G};
  e = r <= 64 ? run_cols<64, true>(b, part_b, &sb, st) : run_cols<128, true>(b, part_b, &sb, st);
  if (e != hipSuccess) return e;
  const int64_t na = (int64_t)ra * K, nb = (int64_t)G * N * r;
  hipLaunchKernelGGL(reduce2_kernel, dim3((unsigned)(((na + nb) / 4 + kThreads - 1) / kThreads)), dim3(kThreads), 0, st,
                     part, sa, na, dA, part_b, sb, nb, dB, scale, scale);
  return hipGetLastError();
}

// Splits of the products of an adapter under dropout and of the 8-bit linear:
// the count whose rounds x columns (or tokens) of a split, with 160 to fill the
// ring and 32 for each split's partials, are least.  dA of 2048 x 4096 at rank
// 64: 64 workgroups took 26 us, 256 take 12 us.  Masked dA waits for its LDS
// passes as much as for its loads, so two workgroups share a CU (512); U and G
// are bound by the CU's loads, and one does.  No device query, so that the
// workspace does not depend on the device.
namespace {

Split fill_split(int64_t tiles, int64_t contraction, int stage, int min_stages, int slots) {
  const int nst = (int)((contraction + stage - 1) / stage);
  Split best{(int)tiles, nst, 1};
  int64_t best_cost = INT64_MAX;
  for (int want = 1; want <= 32 && (want == 1 || want * min_stages <= nst); ++want) {
    const int sps = (nst + want - 1) / want, splits = (nst + sps - 1) / sps;
    const int64_t cost = (tiles * splits + slots - 1) / slots * sps * stage + 160 + 32 * splits;
    if (cost < best_cost) best_cost = cost, best = Split{(int)tiles, sps, splits};
  }
  return best;
}
Split rows_split(int64_t M, int64_t C) { return fill_split((M + 127) / 128, C, 64, 2, 256); }
Split cols_split(int64_t C, int64_t M) { return fill_split((C + 127) / 128, M, 32, 4, 512); }
size_t part_bytes(const Split& s, int64_t n) { return (size_t)s.splits * (size_t)n * sizeof(float); }

}  // namespace

size_t adapter_part_bytes(int64_t M, int64_t N, int64_t K, int r) {
  const size_t u = part_bytes(rows_split(M, K), M * r), g = part_bytes(rows_split(M, N), M * r);
  const size_t da = part_bytes(cols_split(K, M), (int64_t)r * K), db = part_bytes(cols_split(N, M), N * r);
  return std::max(std::max(u, g), (da + 255) / 256 * 256 + db);
}

size_t u_part_bytes(int64_t M, int64_t K, int r) {
  // (with or without the mask)
  return u_rows_ok(M, K, r, true) && u_rows_ok(M, K, r, false) ? 0 : part_bytes(rows_split(M, K), M * r);
}

namespace {

template <int RP, bool QT, bool DROP>
hipError_t wide_partials(const bf16_t* P, int64_t M, int64_t C, const bf16_t* Q, int r, const DropArgs& drop,
                         const Split& sp, float* part, hipStream_t st) {
  auto* fn = &rwide_kernel<RP, QT, DROP>;
  const size_t lds = (size_t)kWideRing * WideShape<RP>::kStage;
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3(sp.tiles * sp.splits), dim3(kWideThreads), lds, st, P, M, C, Q, r, sp.sps, sp.tiles,
                     part, drop);
  return hipGetLastError();
}

}  // namespace

namespace {

Ride sum_ride(RideKind kind, const float* part, const Split& sp, int64_t n, float scale, bf16_t* out, bf16_t* parts,
              float s) {
  Ride d{};
  d.kind = kind, d.blocks = (int)((n / 4 + 255) / 256);
  d.part = part, d.splits = sp.splits, d.n = n, d.scale = scale, d.out = out, d.parts = parts, d.s = s;
  return d;
}

}  // namespace

hipError_t start_xat_drop(const bf16_t* X, const bf16_t* A, int64_t M, int64_t K, int r, const DropArgs* drop,
                          float* part, bf16_t* out, bf16_t* parts, float s, Ride* rest, hipStream_t st) {
  const DropArgs d = drop ? *drop : DropArgs{};
  if (u_rows_ok(M, K, r, drop != nullptr)) {
    *rest = Ride{};
    rest->kind = drop ? kRideRowsDrop : kRideRows, rest->blocks = u_rows_blocks(M, r);
    rest->X = X, rest->A = A, rest->M = M, rest->K = K, rest->r = r, rest->drop = d;
    rest->out = out, rest->parts = parts, rest->s = s;
    return hipSuccess;
  }
  const Split sp = rows_split(M, K);
  *rest = sum_ride(kRideSum, part, sp, M * r, drop ? drop->scale : 1.0f, out, parts, s);
  return drop ? (r <= 64 ? wide_partials<64, false, true>(X, M, K, A, r, d, sp, part, st)
                         : wide_partials<128, false, true>(X, M, K, A, r, d, sp, part, st))
              : (r <= 64 ? wide_partials<64, false, false>(X, M, K, A, r, d, sp, part, st)
                         : wide_partials<128, false, false>(X, M, K, A, r, d, sp, part, st));
}

hipError_t start_dyb_parts(const bf16_t* dY, const bf16_t* B, int64_t M, int64_t N, int r, float* part, bf16_t* parts,
                           float s, Ride* rest, hipStream_t st) {
  const Split sp = rows_split(M, N);
  *rest = sum_ride(kRideSum3, part, sp, M * r, 1.0f, nullptr, parts, s);
  return r <= 64 ? wide_partials<64, true, false>(dY, M, N, B, r, DropArgs{}, sp, part, st)
                 : wide_partials<128, true, false>(dY, M, N, B, r, DropArgs{}, sp, part, st);
}

hipError_t launch_ride(const Ride& a, hipStream_t st) {
  auto* fn = a.kind == kRideRows       ? &ride_kernel<kRideRows>
             : a.kind == kRideRowsDrop ? &ride_kernel<kRideRowsDrop>
             : a.kind == kRideSum      ? &ride_kernel<kRideSum>
                                       : &ride_kernel<kRideSum3>;
  hipLaunchKernelGGL(fn, dim3((unsigned)a.blocks), dim3(256), 0, st, a);
  return hipGetLastError();
}

namespace {

template <int RP>
constexpr int grads_lds() {
  return std::max(ColShape<RP, 3>::kRing * ColShape<RP, 3>::kStage, ColShape<RP, 1>::kRing * ColShape<RP, 1>::kStage);
}

}  // namespace

hipError_t launch_adapter_grads(const bf16_t* G3, const bf16_t* X, const bf16_t* dY, const bf16_t* U, int64_t M,
                                int64_t N, int64_t K, int r, const DropArgs* drop, float* part, float* dA, float* dB,
                                float scale, hipStream_t st) {
  const Split sa = cols_split(K, M), sb = cols_split(N, M);
  const int64_t na = (int64_t)r * K, nb = N * r;
  float* part_b = part + (part_bytes(sa, na) + 255) / 256 * 256 / sizeof(float);
  const bool whole_a = sa.splits == 1, whole_b = sb.splits == 1;
  const GradArgs p{X, dY, G3, U, M, N, K, r, sa.sps, sa.tiles, sa.tiles * sa.splits, sb.sps, sb.tiles,
                   whole_a ? dA : part, whole_b ? dB : part_b, whole_b ? scale : 1.0f, drop ? *drop : DropArgs{}};
  auto* fn = r <= 64 ? (drop ? &adapter_grads_kernel<64, true> : &adapter_grads_kernel<64, false>)
                     : (drop ? &adapter_grads_kernel<128, true> : &adapter_grads_kernel<128, false>);
  const int lds = r <= 64 ? grads_lds<64>() : grads_lds<128>();
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(fn), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3(p.blocks_a + sb.tiles * sb.splits), dim3(kThreads), lds, st, p);
  const int64_t ra = whole_a ? 0 : na, rb = whole_b ? 0 : nb;
  if (ra + rb == 0) return hipGetLastError();
  hipLaunchKernelGGL(reduce2_kernel, dim3((unsigned)(((ra + rb) / 4 + kThreads - 1) / kThreads)), dim3(kThreads), 0, st,
                     part, sa.splits, ra, dA, part_b, sb.splits, rb, dB, 1.0f, scale);
  return hipGetLastError();
}

}  // namespace qlora
