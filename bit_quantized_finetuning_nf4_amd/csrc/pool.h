// pool.h -- the adapters of many requests as the kernels see them.
#pragma once
#include "device.h"
#include "kernels.h"

namespace qlora {

// The slot of token m, or -1: an id outside the pool is no adapter.
__device__ __forceinline__ int slot_of(const PoolView& p, int64_t m) {
  const int a = p.ids ? p.ids[m] : 0;
  return (uint32_t)a < (uint32_t)p.slots ? a : -1;
}
// The ranks of slot a that are read: whole groups of eight, R at most.
__device__ __forceinline__ int rank_of(const PoolView& p, int a) {
  if (!p.rank) return p.R;
  const int r = p.rank[a];
  return r <= 0 ? 0 : r >= p.R ? p.R : (r + 7) & ~7;
}
__device__ __forceinline__ float scale_of(const PoolView& p, int a) { return p.scale ? p.scale[a] : p.s; }

}  // namespace qlora
