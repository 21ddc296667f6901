// i8.hip -- rows of 8-bit integers with one fp32 scale each, the format of
// the 8-bit linears: a weight's output channels and an input's tokens.
//
//   scale_m = RN32(amax_m / 127),  amax_m = max_k |x[m][k]|
//   q[m][k] = the integer nearest 127 x[m][k] / amax_m (ties to even)
//
// A row of zeros has scale 0.  A row that holds an infinity or a NaN has
// scale NaN and codes 0, so that it poisons its own products and no others.
// Rows are padded with zeros to whole 128-byte lines (i8_row_bytes), which
// the product kernels stream.
//
// All of it is bound by memory: a row is read once into registers, its largest
// magnitude found across the workgroup (or the wave, for short rows), and its
// codes stored 16 bytes a thread.  22016 x 8192: 94 us, 5.8 TB/s; the transposed
// dequantization of 5120 x 13824 45 us, 4.7 TB/s.
#include "lds.h"
#include "ride.h"

namespace qlora {
namespace {

constexpr float kRoundMagic = 12582912.0f;   // 1.5 * 2^23: x + magic rounds x to an integer, in the low mantissa bits

// The quotient 127 x / a of bf16 numbers, to fp32's rounding.  n = 127 x is
// exact (15 bits); one Newton step on q0 = n RN(1/a), with the remainder by
// fma, leaves an error below one ulp, and none where the quotient is an fp32
// number.  A quotient of two 8-bit significands (times 127) that is not
// half-way between integers differs from every such point by more than
// 2^-17, so the rounded integer is the exact quotient's; the half-way points
// (x = a / 2 gives 63.5) are fp32 numbers.
__device__ __forceinline__ float quotient(float n, float a, float inv) {
  const float q0 = n * inv;
  return fmaf(fmaf(-q0, a, n), inv, q0);
}
// Four codes, one per byte.
__device__ __forceinline__ uint32_t quant4(uint32_t lo, uint32_t hi, float f127, float a, float inv) {
  const uint32_t b0 = f2u(quotient(bf2f(lo & 0xFFFFu) * f127, a, inv) + kRoundMagic);
  const uint32_t b1 = f2u(quotient(bf2f(lo >> 16) * f127, a, inv) + kRoundMagic);
  const uint32_t b2 = f2u(quotient(bf2f(hi & 0xFFFFu) * f127, a, inv) + kRoundMagic);
  const uint32_t b3 = f2u(quotient(bf2f(hi >> 16) * f127, a, inv) + kRoundMagic);
  return perm(perm(b3, b2, 0x0C0C0400u), perm(b1, b0, 0x0C0C0400u), 0x05040100u);
}

__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}
__device__ __forceinline__ uint32_t max_abs(uint32_t m, uint4 v) {
  return max_halves(max_halves(max_halves(m, v.x & 0x7FFF7FFFu), max_halves(v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu)),
                    v.w & 0x7FFF7FFFu);
}

struct RowScale {
  float a, inv, f127;   // 127 x f / (a f): f a power of two that keeps both in range
  float scale;
};
// bits: the largest |x| of the row as a bf16 pattern (which orders like the
// numbers, infinity and NaN above them).
__device__ __forceinline__ RowScale row_scale(uint32_t bits) {
  const float a = bf2f(bits);
  RowScale r;
  const float f = a < 0x1p-60f ? 0x1p64f : a > 0x1p60f ? 0x1p-64f : 1.0f;
  r.a = a * f;
  r.inv = 1.0f / r.a;
  r.f127 = 127.0f * f;
  r.scale = a / 127.0f;
  if (bits == 0u) r.a = r.inv = r.f127 = 0.0f;
  if (bits >= 0x7F80u) {   // codes 0 for every element: 0 x fma chain is NaN, so select below
    r.a = r.inv = r.f127 = 0.0f;
    r.scale = __builtin_nanf("");
  }
  return r;
}

// Row m by TPR threads (a wave, or the whole workgroup), thread t of them; 16
// elements per thread and chunk, NCH chunks held in registers so that the row
// is read once; NCH = 0: longer rows, read twice (the second time mostly from
// cache).  wmax: four words of LDS (TPR == 256).
template <int TPR, int NCH>
__device__ __forceinline__ void quant_row(const bf16_t* __restrict__ X, int64_t m, int t, int64_t K, int64_t ld,
                                          int8_t* __restrict__ Q, float* __restrict__ scale, uint32_t* wmax) {
  const int lane = threadIdx.x & 63;
  const bf16_t* x = X + m * K;
  int8_t* q = Q + m * ld;
  const int64_t groups = K >> 3;     // K % 8 == 0
  auto load = [&](int64_t g) { return g < groups ? reinterpret_cast<const uint4*>(x)[g] : make_uint4(0u, 0u, 0u, 0u); };
  uint4 v[NCH > 0 ? 2 * NCH : 1];
  uint32_t mx = 0u;
  if constexpr (NCH > 0) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int64_t g = 2 * ((int64_t)c * TPR + t);
      v[2 * c] = load(g);
      v[2 * c + 1] = load(g + 1);
    }
#pragma unroll
    for (int c = 0; c < 2 * NCH; ++c) mx = max_abs(mx, v[c]);
  } else {
    for (int64_t g = t; g < groups; g += TPR) mx = max_abs(mx, load(g));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mx = max_halves(mx, (uint32_t)__shfl_xor((int)mx, o));
  if constexpr (TPR == 256) {
    if (lane == 0) wmax[threadIdx.x >> 6] = mx;
    __syncthreads();
    mx = max_halves(max_halves(wmax[0], wmax[1]), max_halves(wmax[2], wmax[3]));
  }
  const uint32_t bits = max(mx & 0xFFFFu, mx >> 16);
  const RowScale s = row_scale(bits);
  if (t == 0) scale[m] = s.scale;
  const bool live = bits != 0u && bits < 0x7F80u;
  auto store = [&](int64_t g, uint4 a, uint4 b) {   // groups g, g + 1: 16 codes
    if (8 * g >= ld) return;
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if (live)
      o = make_uint4(quant4(a.x, a.y, s.f127, s.a, s.inv), quant4(a.z, a.w, s.f127, s.a, s.inv),
                     quant4(b.x, b.y, s.f127, s.a, s.inv), quant4(b.z, b.w, s.f127, s.a, s.inv));
    *reinterpret_cast<uint4*>(q + 8 * g) = o;
  };
  if constexpr (NCH > 0) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) store(2 * ((int64_t)c * TPR + t), v[2 * c], v[2 * c + 1]);
  } else {
    for (int64_t g = 2 * t; 8 * g < ld; g += 2 * TPR) store(g, load(g), load(g + 1));
  }
}

// SUM: the first sum.blocks workgroups add up the partials of U (ride.h).
template <int TPR, int NCH, bool SUM>
__global__ __launch_bounds__(256) void quant_rows_kernel(const bf16_t* __restrict__ X, int64_t M, int64_t K,
                                                         int64_t ld, int8_t* __restrict__ Q,
                                                         float* __restrict__ scale, Ride sum) {
  __shared__ uint32_t wmax[4];
  if (SUM && (int)blockIdx.x < sum.blocks) {
    ride<kRideSum>(sum, blockIdx.x);
    return;
  }
  const int64_t m = ((int64_t)blockIdx.x - (SUM ? sum.blocks : 0)) * (256 / TPR) + threadIdx.x / TPR;
  if (TPR == 64 && m >= M) return;   // whole waves; TPR == 64 meets no barrier
  quant_row<TPR, NCH>(X, m, threadIdx.x % TPR, K, ld, Q, scale, wmax);
}

// What the product needs first, in one launch where U is small: workgroups
// 0 .. nu - 1 compute U = drop(X) A^T (urows.h), the others quantize one token
// each.  Either part alone would leave most of the card idle.
template <int NCH, bool DROP>
__global__ __launch_bounds__(256) void i8_prep_kernel(const bf16_t* __restrict__ X, int64_t M, int64_t K, int64_t ld,
                                                      const bf16_t* __restrict__ A, int r, int nu,
                                                      bf16_t* __restrict__ U, bf16_t* __restrict__ parts, float s,
                                                      int8_t* __restrict__ Q, float* __restrict__ scale,
                                                      DropArgs drop) {
  __shared__ uint32_t wmax[4];
  if ((int)blockIdx.x >= nu)
    quant_row<256, NCH>(X, (int)blockIdx.x - nu, threadIdx.x, K, ld, Q, scale, wmax);
  else
    u_rows<DROP>(X, M, K, A, r, blockIdx.x, U, parts, s, drop);
}

// deq = RNE_bf16(RN32(scale q)).
__device__ __forceinline__ uint32_t deq2(uint32_t v, int i, float s) {   // bytes i, i + 1 of v
  return pack_bf16x2((float)(int8_t)(v >> (8 * i)) * s, (float)(int8_t)(v >> (8 * i + 8)) * s);
}
__global__ __launch_bounds__(256) void i8_dequant_kernel(const int8_t* __restrict__ Q, const float* __restrict__ scale,
                                                         int64_t N, int64_t K, int64_t ld, bf16_t* __restrict__ out) {
  // eight columns per thread
  const int64_t per = K >> 3, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= N * per) return;
  const int64_t n = id / per, g = id - n * per;
  const uint2 c = *reinterpret_cast<const uint2*>(Q + n * ld + 8 * g);
  const float s = scale[n];
  *reinterpret_cast<uint4*>(out + n * K + 8 * g) =
      make_uint4(deq2(c.x, 0, s), deq2(c.x, 2, s), deq2(c.y, 0, s), deq2(c.y, 2, s));
}

// WdT [K x ldo] = deq(W)^T, columns N .. ldo - 1 zero (ldo = N rounded up to
// 64): 64 x 64 tiles through LDS.  Reads 64 bytes of 64 rows, writes 128
// bytes of 64 rows.
// The first rest.blocks workgroups (0: none) do what rides along (ride.h).
__global__ __launch_bounds__(256) void i8_dequant_t_kernel(const int8_t* __restrict__ Q,
                                                           const float* __restrict__ scale, int64_t N, int64_t K,
                                                           int64_t ld, bf16_t* __restrict__ out, int64_t ldo,
                                                           int tiles_k, Ride rest) {
  __shared__ __align__(16) uint32_t tile[64][33];   // [column][row pair], one word of padding
  const int id = (int)blockIdx.x - rest.blocks;
  if (id < 0) {
    ride<kRideSum3>(rest, blockIdx.x);
    return;
  }
  const int by = id / tiles_k;
  const int64_t k0 = (int64_t)(id - by * tiles_k) * 64, n0 = (int64_t)by * 64;
  const int t = threadIdx.x;
  {
    // thread: row pair t / 8 (rows 2 p, 2 p + 1), 8 columns at 8 (t mod 8)
    const int p = t >> 3, c = t & 7;
    const int64_t n = n0 + 2 * p;
    uint2 a = make_uint2(0u, 0u), b = make_uint2(0u, 0u);
    float sa = 0.0f, sb = 0.0f;
    // (k0 + 8 c < ld always: ld is a multiple of 128; columns past K hold 0)
    if (n < N) a = *reinterpret_cast<const uint2*>(Q + n * ld + k0 + 8 * c), sa = scale[n];
    if (n + 1 < N) b = *reinterpret_cast<const uint2*>(Q + (n + 1) * ld + k0 + 8 * c), sb = scale[n + 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t wa = i < 4 ? a.x : a.y, wb = i < 4 ? b.x : b.y;
      tile[8 * c + i][p] = pack_bf16x2((float)(int8_t)(wa >> (8 * (i & 3))) * sa, (float)(int8_t)(wb >> (8 * (i & 3))) * sb);
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int idx = t + 256 * e, k = idx >> 3, c = idx & 7;
    if (k0 + k < K)
      *reinterpret_cast<uint4*>(out + (k0 + k) * ldo + n0 + 8 * c) =
          make_uint4(tile[k][4 * c], tile[k][4 * c + 1], tile[k][4 * c + 2], tile[k][4 * c + 3]);
  }
}

unsigned blocks_of(int64_t threads) { return (unsigned)((threads + 255) / 256); }

}  // namespace

hipError_t launch_quant_rows(const bf16_t* X, int64_t M, int64_t K, int8_t* Q, float* scale, const Ride* sum,
                             hipStream_t st) {
  const int64_t ld = i8_row_bytes(K);
  const Ride d = sum ? *sum : Ride{};
  auto go = [&](auto* fn, auto* fn_sum, int rows_per_block) {
    hipLaunchKernelGGL((sum ? fn_sum : fn), dim3((unsigned)(d.blocks + (M + rows_per_block - 1) / rows_per_block)),
                       dim3(256), 0, st, X, M, K, ld, Q, scale, d);
  };
  if (ld <= 1024)
    go(&quant_rows_kernel<64, 1, false>, &quant_rows_kernel<64, 1, true>, 4);
  else if (ld <= 4096)
    go(&quant_rows_kernel<256, 1, false>, &quant_rows_kernel<256, 1, true>, 1);
  else if (ld <= 8192)
    go(&quant_rows_kernel<256, 2, false>, &quant_rows_kernel<256, 2, true>, 1);
  else if (ld <= 16384)
    go(&quant_rows_kernel<256, 4, false>, &quant_rows_kernel<256, 4, true>, 1);
  else if (ld <= 32768)
    go(&quant_rows_kernel<256, 8, false>, &quant_rows_kernel<256, 8, true>, 1);
  else
    go(&quant_rows_kernel<256, 0, false>, &quant_rows_kernel<256, 0, true>, 1);
  return hipGetLastError();
}

bool i8_prep_ok(int64_t M, int64_t K, int r, bool drop) { return u_rows_ok(M, K, r, drop) && i8_row_bytes(K) <= 32768; }

hipError_t launch_i8_prep(const bf16_t* X, int64_t M, int64_t K, const bf16_t* A, int r, const DropArgs* drop,
                          bf16_t* U, bf16_t* parts, float s, int8_t* Q, float* scale, hipStream_t st) {
  const int64_t ld = i8_row_bytes(K);
  const int nu = u_rows_blocks(M, r);
  auto go = [&](auto* fn) {
    hipLaunchKernelGGL(fn, dim3((unsigned)(nu + M)), dim3(256), 0, st, X, M, K, ld, A, r, nu, U, parts, s, Q,
                       scale, drop ? *drop : DropArgs{});
  };
  if (ld <= 4096)
    drop ? go(&i8_prep_kernel<1, true>) : go(&i8_prep_kernel<1, false>);
  else if (ld <= 8192)
    drop ? go(&i8_prep_kernel<2, true>) : go(&i8_prep_kernel<2, false>);
  else if (ld <= 16384)
    drop ? go(&i8_prep_kernel<4, true>) : go(&i8_prep_kernel<4, false>);
  else
    drop ? go(&i8_prep_kernel<8, true>) : go(&i8_prep_kernel<8, false>);
  return hipGetLastError();
}

hipError_t launch_i8_dequant(const int8_t* Q, const float* scale, int64_t N, int64_t K, bf16_t* out, hipStream_t st) {
  hipLaunchKernelGGL(i8_dequant_kernel, dim3(blocks_of(N * (K >> 3))), dim3(256), 0, st, Q, scale, N, K,
                     i8_row_bytes(K), out);
  return hipGetLastError();
}

hipError_t launch_i8_dequant_t(const int8_t* Q, const float* scale, int64_t N, int64_t K, bf16_t* out, int64_t ldo,
                               const Ride& rest, hipStream_t st) {
  const int tiles_k = (int)((K + 63) / 64);
  hipLaunchKernelGGL(i8_dequant_t_kernel, dim3((unsigned)(rest.blocks + tiles_k * ((N + 63) / 64))), dim3(256), 0, st,
                     Q, scale, N, K, i8_row_bytes(K), out, ldo, tiles_k, rest);
  return hipGetLastError();
}

}  // namespace qlora
