// dropout.hip -- elementwise dropout: y = x / (1 - p) where the generator
// keeps an element, 0 elsewhere (whatever x holds there).  The backward pass
// is the same map of dy under the same seed and offset.
//
// A stream: 2 bytes read and 2 written per element.  A thread takes groups of
// eight elements, one 16-byte load, one Philox block (rng.h) and one 16-byte
// store each, kUnroll groups with their loads issued together, so that
// the generator's products run while the loads are in flight.  4096 x 22016:
// 65.5 us, 5.5 TB/s (a large copy reaches 4.8: part of the input is still in
// the last-level cache from the call before); one row of 4096: 1.7 us, a launch.
#include "rng.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

__device__ __forceinline__ uint32_t scale2(uint32_t v, uint32_t keep, float s) {
  return pack_bf16x2(bf2f(v & 0xFFFFu) * s, bf2f(v >> 16) * s) & keep;
}

__global__ __launch_bounds__(kThreads) void dropout_kernel(const bf16_t* x, int64_t n, DropArgs d, bf16_t* y) {
  const DropKey key = drop_key(d);
  const uint32_t all = d.thr == -32768 ? ~0u : 0u;   // p = 0: keep_halves has no such threshold
  const int64_t groups = n >> 3;
  const int64_t g0 = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  u32x4_t v[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t g = g0 + i * kThreads;
    if (g < groups) v[i] = *reinterpret_cast<const u32x4_t*>(x + 8 * g);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t g = g0 + i * kThreads;
    if (g < groups) {
      const u32x4_t w = philox((uint64_t)g, key);
      const u32x4_t o = {scale2(v[i].x, keep_halves(w.x, key.thr) | all, d.scale),
                         scale2(v[i].y, keep_halves(w.y, key.thr) | all, d.scale),
                         scale2(v[i].z, keep_halves(w.z, key.thr) | all, d.scale),
                         scale2(v[i].w, keep_halves(w.w, key.thr) | all, d.scale)};
      *reinterpret_cast<u32x4_t*>(y + 8 * g) = o;
    }
  }
  // the last n mod 8 elements, one thread each
  const int rest = (int)(n & 7);
  if (blockIdx.x == 0 && (int)threadIdx.x < rest) {
    const u32x4_t w = philox((uint64_t)groups, key);
    const int e = threadIdx.x;
    const uint32_t word = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
    const uint32_t keep = (keep_halves(word, key.thr) | all) >> (16 * (e & 1)) & 0xFFFFu;
    y[8 * groups + e] = (bf16_t)(pack_bf16x2(bf2f(x[8 * groups + e]) * d.scale, 0.0f) & keep);
  }
}

}  // namespace

hipError_t launch_dropout(const bf16_t* x, int64_t n, const DropArgs& d, bf16_t* y, hipStream_t st) {
  const int64_t per = 8 * kThreads * kUnroll;
  hipLaunchKernelGGL(dropout_kernel, dim3((unsigned)((n + per - 1) / per)), dim3(kThreads), 0, st, x, n, d, y);
  return hipGetLastError();
}

}  // namespace qlora
