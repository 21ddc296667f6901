// rng.h -- the counter-based generator of the dropout masks (gfx950).
//
// Philox-4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011: the fewest rounds that they found to
// pass every statistical test).  A block is a pure function of a 128-bit
// counter and a 64-bit key, so a mask is never stored: every kernel that
// needs it, in the forward or the backward pass, computes the same bits from
// the position of the element.
//
// Element e of a row-major tensor takes 16-bit half e mod 8 of the block at
// counter (e / 8, offset), key = seed: one block serves the 16 bytes that a
// lane loads.  The half is read as a signed number and the element is kept
// where it is at least `thr` = round(65536 p) - 32768, so p is met to 2^-17;
// 16 bits rather than 32 per element halve the generator's work, which is
// what bounds the masked kernels next to their loads (14 32 x 32 -> 64-bit
// products per block: 212 cycles a wave, 320 with separate high and low
// products).
#pragma once
#include "device.h"
#include "kernels.h"
#include "lds.h"

namespace qlora {

typedef short s16x2_t __attribute__((ext_vector_type(2)));

// The part of the counter and key that a whole call shares.
struct DropKey {
  uint32_t k0, k1, o0, o1;
  int thr;   // in (-32768, 32767]
};
// The offset is offset + *step where the caller keeps a step count on the
// device (a captured graph then draws new masks on each replay).
__device__ __forceinline__ DropKey drop_key(const DropArgs& d) {
  const uint64_t o = d.offset + (d.step ? *d.step : 0ull);
  return DropKey{(uint32_t)d.seed, (uint32_t)(d.seed >> 32), (uint32_t)o, (uint32_t)(o >> 32), d.thr};
}

// One round's half: {high word, low word} of a 32 x 32-bit product.
__device__ __forceinline__ uint2 mul_wide(uint32_t a, uint32_t b) {
  const uint64_t p = (uint64_t)a * b;
  return make_uint2((uint32_t)(p >> 32), (uint32_t)p);
}
struct PhiloxState {
  uint32_t c0, c1, c2, c3;
};
template <int ROUND>
__device__ __forceinline__ void philox_round(PhiloxState& s, const DropKey& k) {
  const uint2 a = mul_wide(s.c0, 0xD2511F53u), b = mul_wide(s.c2, 0xCD9E8D57u);
  s = PhiloxState{b.x ^ s.c1 ^ (k.k0 + (uint32_t)ROUND * 0x9E3779B9u), b.y,
                  a.x ^ s.c3 ^ (k.k1 + (uint32_t)ROUND * 0xBB67AE85u), a.y};
}
__device__ __forceinline__ PhiloxState philox_start(uint64_t block, const DropKey& k) {
  return PhiloxState{(uint32_t)block, (uint32_t)(block >> 32), k.o0, k.o1};
}
// The block's four words: elements 2 i and 2 i + 1 in the halves of word i.
__device__ __forceinline__ u32x4_t philox(uint64_t block, const DropKey& k) {
  PhiloxState s = philox_start(block, k);
  philox_round<0>(s, k);
  philox_round<1>(s, k);
  philox_round<2>(s, k);
  philox_round<3>(s, k);
  philox_round<4>(s, k);
  philox_round<5>(s, k);
  philox_round<6>(s, k);
  return u32x4_t{s.c0, s.c1, s.c2, s.c3};
}
// All ones in the halves of w that are kept: (thr - 1) - half saturates
// without changing its sign, which is negative exactly where half >= thr
// (thr > -32768: a call that drops nothing takes no mask).
__device__ __forceinline__ uint32_t keep_halves(uint32_t w, int thr) {
  const short t = (short)(thr - 1);
  const s16x2_t d = __builtin_elementwise_sub_sat(s16x2_t{t, t}, __builtin_bit_cast(s16x2_t, w));
  return __builtin_bit_cast(uint32_t, d >> 15);
}
// Eight consecutive bf16 with the dropped ones zeroed.
__device__ __forceinline__ u32x4_t drop8(u32x4_t v, uint64_t block, const DropKey& k) {
  const u32x4_t w = philox(block, k);
  return u32x4_t{v.x & keep_halves(w.x, k.thr), v.y & keep_halves(w.y, k.thr), v.z & keep_halves(w.z, k.thr),
                 v.w & keep_halves(w.w, k.thr)};
}

// The mask of a 32-channel x 32-token block in the layout of a 32x32 MFMA (lane
// (lr, h): token lr, channels 8 q + 4 h .. + 3 in elements 4 q ..), a bit per
// element: element e at bit 8 + e / 2 + 16 (e mod 2).  block0 is the Philox
// block of the token's first channel.  A lane holds half of a block's eight
// elements and its two lane halves the two halves, so the lower half computes
// the block of channel group 2 p, the upper one that of 2 p + 1, and
// v_permlane32_swap hands each half its four elements of both.
__device__ __forceinline__ uint32_t mask_bits(uint32_t block0, const DropKey& key) {
  const int h = (threadIdx.x >> 5) & 1;
  const short t = (short)(key.thr - 1);
  uint32_t bits = 0u;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const u32x4_t x = philox(block0 + (uint32_t)(2 * p + h), key);
    const auto x0 = __builtin_amdgcn_permlane32_swap(x.x, x.z, false, false);
    const auto x1 = __builtin_amdgcn_permlane32_swap(x.y, x.w, false, false);
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int d = 0; d < 2; ++d) {   // the signs of both halves' differences, as in keep_halves
        const s16x2_t v = __builtin_bit_cast(s16x2_t, d == 0 ? (uint32_t)x0[g] : (uint32_t)x1[g]);
        bits = bits >> 1 | (__builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(s16x2_t{t, t}, v)) & 0x80008000u);
      }
  }
  return bits;
}
__device__ __forceinline__ float masked(float v, uint32_t bits, int e) {
  return u2f(f2u(v) & (uint32_t)__builtin_amdgcn_sbfe((int)bits, 8 + e / 2 + 16 * (e & 1), 1));
}

}  // namespace qlora
