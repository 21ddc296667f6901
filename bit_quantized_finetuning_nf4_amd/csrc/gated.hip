// gated.hip -- the elementwise gradient of a gated block:
//
//   dG = dH o P o act'(G),  dP = dH o act(G)
//
// from the saved projections GU = [G | P] (bf16), side by side in 16 bits as
// the backward products read them.  10 bytes an element and about 45 fp64
// operations (gate.h says why 64 bits): 2048 x 13824 60-67 us, 4.2-4.7 TB/s, memory.
#include "gate.h"
#include "kernels.h"
#include "lds.h"

namespace qlora {
namespace {

// A thread takes eight columns of a token.  dY [M x 2 Fp], Fp = F rounded up to
// 32: columns F .. Fp of both halves are zero, as are those of Wt [K x 2 Fp]
// (may be null), whose contraction they pad.  The last threads transpose A [r x K],
// eight ranks of a column each.
__global__ __launch_bounds__(256) void gated_grad_kernel(const bf16_t* __restrict__ dH, const bf16_t* __restrict__ GU,
                                                         int64_t M, int64_t F, int64_t Fp, int act,
                                                         bf16_t* __restrict__ dY, bf16_t* __restrict__ Wt, int64_t K,
                                                         const bf16_t* __restrict__ A, int r, bf16_t* __restrict__ At) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, per = Fp >> 3;
  if (id >= M * per) {
    const int64_t pieces = (Fp - F) >> 3, pads = Wt ? 2 * K * pieces : 0;
    int64_t z = id - M * per;
    if (z >= pads) {
      z -= pads;
      const int64_t j = z / K, k = z - j * K;
      if (!At || j >= r / 8) return;
      uint32_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = A[(8 * j + e) * K + k];
      *reinterpret_cast<uint4*>(At + k * r + 8 * j) =
          make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
      return;
    }
    const int64_t k = z / (2 * pieces), q = z - k * 2 * pieces, half = q / pieces;
    *reinterpret_cast<uint4*>(Wt + k * 2 * Fp + half * Fp + F + 8 * (q - half * pieces)) = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int64_t m = id / per, c = 8 * (id - m * per);
  uint4 og = make_uint4(0u, 0u, 0u, 0u), op = og;
  if (c < F) {   // F % 8 == 0
    const u32x4_t h = *reinterpret_cast<const u32x4_t*>(dH + m * F + c);
    const u32x4_t g = *reinterpret_cast<const u32x4_t*>(GU + m * 2 * F + c);
    const u32x4_t p = *reinterpret_cast<const u32x4_t*>(GU + m * 2 * F + F + c);
    uint32_t wg[4], wp[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // fp64 to fp32 to bf16 rounds twice; the first rounding moves a value
      // across a bf16 tie only from within 2^-24 of it, one in 2^16
      float rg[2], rp[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const double x = bf2f(b ? g[e] >> 16 : g[e] & 0xFFFFu), y = bf2f(b ? h[e] >> 16 : h[e] & 0xFFFFu),
                     u = bf2f(b ? p[e] >> 16 : p[e] & 0xFFFFu);
        double sigma, slope;
        gate_slope(x, act, sigma, slope);
        rg[b] = (float)(y * u * slope);
        rp[b] = (float)(y * (x * sigma));
      }
      wg[e] = pack_bf16x2(rg[0], rg[1]);
      wp[e] = pack_bf16x2(rp[0], rp[1]);
    }
    og = make_uint4(wg[0], wg[1], wg[2], wg[3]);
    op = make_uint4(wp[0], wp[1], wp[2], wp[3]);
  }
  *reinterpret_cast<uint4*>(dY + m * 2 * Fp + c) = og;
  *reinterpret_cast<uint4*>(dY + m * 2 * Fp + Fp + c) = op;
}

}  // namespace

hipError_t launch_gated_grad(const bf16_t* dH, const bf16_t* GU, int64_t M, int64_t F, int64_t Fp, int act, bf16_t* dY,
                             bf16_t* Wt, int64_t K, const bf16_t* A, int r, bf16_t* At, hipStream_t st) {
  const int64_t n = M * (Fp >> 3) + (Wt ? 2 * K * ((Fp - F) >> 3) : 0) + (At ? K * (r / 8) : 0);
  hipLaunchKernelGGL(gated_grad_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, dH, GU, M, F, Fp, act, dY,
                     Wt, K, A, r, At);
  return hipGetLastError();
}

}  // namespace qlora
