// ride.h -- the last step of a small adapter product (U = drop(X) A^T, G = dY
// B), and copies of rows padded to whole stages, as extra workgroups of the
// launch that comes next anyway, a dequantization or a quantization, which
// neither reads the product nor is read by it.  Alone such a step is a launch of
// 3-5 us that leaves most of the card idle: the backward of 2048 x 4096 x 4096 at
// rank 64 took 107 us with it apart and 104 this way, the NF4 forward of 256 x
// 1024 x 1024 at rank 8 24.9 and 21.1.
#pragma once
#include "urows.h"

namespace qlora {

// Elements i .. i + 3 of the splits' partials, summed in split order, times
// scale; the loads of eight splits are issued together.
__device__ __forceinline__ float4 sum_splits(const float* __restrict__ part, int splits, int64_t n, int64_t i,
                                             float scale) {
  float4 acc = *reinterpret_cast<const float4*>(part + i);
  for (int s0 = 1; s0 < splits; s0 += 8) {
    float4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = *reinterpret_cast<const float4*>(part + (int64_t)min(s0 + k, splits - 1) * n + i);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool in = s0 + k < splits;   // selects, not branches: a branch would sink its load
      acc.x = in ? acc.x + v[k].x : acc.x;
      acc.y = in ? acc.y + v[k].y : acc.y;
      acc.z = in ? acc.z + v[k].z : acc.z;
      acc.w = in ? acc.w + v[k].w : acc.w;
    }
  }
  return make_float4(acc.x * scale, acc.y * scale, acc.z * scale, acc.w * scale);
}

// Workgroup `block` (of a.blocks, 256 threads) of the step.
//   kRideSum   v = the splits' sum times scale: bf16 of v to out, s v as it is or
//              as two parts
//   kRideSum3  s v as three parts, together its fp32 value (the workgroups
//              after those that pad rows)
// Parts lie n elements apart, each the bf16 rounding of what those before it
// left.
//   kRideRows, kRideRowsDrop   U by rows (urows.h)
__device__ __forceinline__ void pad_block(const PadRows& p, int block) {
  const int64_t c0 = p.in ? 0 : p.cols >> 3, per = (p.ld >> 3) - c0;
  const int64_t id = (int64_t)block * 256 + threadIdx.x;
  if (id >= p.rows * per) return;
  const int64_t m = id / per, g = c0 + id - m * per;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (8 * g < p.cols) v = *reinterpret_cast<const uint4*>(p.in + m * p.cols + 8 * g);
  *reinterpret_cast<uint4*>(p.out + m * p.ld + 8 * g) = v;
}
template <int KIND>
__device__ __forceinline__ void ride(const Ride& a, int block) {
  if constexpr (KIND == kRideRows || KIND == kRideRowsDrop) {
    u_rows<KIND == kRideRowsDrop>(a.X, a.M, a.K, a.A, a.r, block, a.out, a.parts, a.s, a.drop);
  } else {
    if constexpr (KIND == kRideSum3) {
      if (block < a.pad[0].blocks) return pad_block(a.pad[0], block);
      block -= a.pad[0].blocks;
      if (block < a.pad[1].blocks) return pad_block(a.pad[1], block);
      block -= a.pad[1].blocks;
    }
    const int64_t i = ((int64_t)block * 256 + threadIdx.x) * 4;
    if (i >= a.n) return;
    float4 v = sum_splits(a.part, a.splits, a.n, i, a.scale);
    if (KIND == kRideSum && a.out)
      *reinterpret_cast<uint2*>(a.out + i) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    v = make_float4(v.x * a.s, v.y * a.s, v.z * a.s, v.w * a.s);
    if (KIND == kRideSum && a.full) *reinterpret_cast<float4*>(a.full + i) = v;
    if (!a.parts) return;
#pragma unroll
    for (int k = 0; k < (KIND == kRideSum3 ? kGradParts : kTermParts); ++k) {
      const uint2 p = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      *reinterpret_cast<uint2*>(a.parts + k * a.n + i) = p;
      v = make_float4(rest_of(v.x, p.x & 0xFFFFu), rest_of(v.y, p.x >> 16), rest_of(v.z, p.y & 0xFFFFu),
                      rest_of(v.w, p.y >> 16));
    }
  }
}

}  // namespace qlora
