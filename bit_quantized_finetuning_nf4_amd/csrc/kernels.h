// kernels.h -- launch helpers implemented by the .hip files (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qlora.h"

namespace qlora {

typedef uint16_t bf16_t;

struct Nf4View {
  const uint8_t* codes;
  const uint8_t* absmax_q;
  const float* group_scale;
  int64_t N;  // rows
  int64_t K;  // cols, K % 64 == 0 on the GEMM/GEMV paths
  int codebook;  // 0 NF4, 1 FP4, 2 Int4 (the values of qlora_codebook)
  int absfmt;    // second-level format (the values of qlora_absmax_format)
};

// Dropout of one call: the mask's key and counter offset, the threshold on
// signed 16-bit halves and the factor 1 / (1 - p) of what is kept (rng.h).
struct DropArgs {
  uint64_t seed, offset;
  const uint64_t* step;   // device memory, may be null: added to offset
  int thr;
  float scale;
};

// y = drop(x) over n bf16 values (16-byte aligned; y may be x).
hipError_t launch_dropout(const bf16_t* x, int64_t n, const DropArgs& d, bf16_t* y, hipStream_t st);

// Compute units of the current device (256 if the query fails).
int device_cu_count();

// Raise kernel fn's dynamic-LDS limit to `bytes` (the most any of its
// launches asks for) on the current device, once per device.
hipError_t allow_lds(const void* fn, int bytes);
constexpr int kMaxLds = 160 * 1024;

// codebook: 0 NF4, 1 FP4, 2 Int4 (the values of qlora_codebook)
// One AdamW step over n parameters (p_bf16 may be null); see optim.hip.
hipError_t launch_adamw(float* p, bf16_t* p_bf16, const float* g, float* m, float* v, int64_t n, float lr,
                        float beta1, float beta2, float eps, float weight_decay, int step, hipStream_t st);

hipError_t launch_quantize(const bf16_t* W, int64_t numel, uint8_t* codes, uint8_t* absmax_q,
                           float* group_scale, int codebook, int absfmt, hipStream_t s);
hipError_t launch_dequant(const uint8_t* codes, const uint8_t* absmax_q, const float* group_scale,
                          int64_t numel, int codebook, int absfmt, bf16_t* out, hipStream_t s);

// WdT [K x N] = deq(W)^T (bf16) for W [N x K], K % 64 == 0, N < 65536 * 64;
// rows of WdT are ldo >= N elements apart (a column block of a wider matrix).
hipError_t launch_dequant_t(const uint8_t* codes, const uint8_t* absmax_q, const float* group_scale, int64_t N,
                            int64_t K, int codebook, int absfmt, bf16_t* out, int64_t ldo, hipStream_t s);

// launch_dequant of a whole weight (rest: kRideSum or kRideRowsDrop) and
// launch_dequant_t (rest: kRideSum3) with an adapter product's last step.
struct Ride;
hipError_t launch_dequant_ride(const Nf4View& W, bf16_t* out, const Ride& rest, hipStream_t s);
hipError_t launch_dequant_t_ride(const Nf4View& W, bf16_t* out, int64_t ldo, const Ride& rest, hipStream_t s);

// Up to kDeqMax weights of one shape (N x K), one codebook and one absmax
// format, dequantized by one launch: weight i to out + i out_gs, as
// launch_dequant (N K weights) or, transposed, as launch_dequant_t.
constexpr int kDeqMax = 8;
struct DeqSrcs {
  const uint8_t* codes[kDeqMax];
  const uint8_t* absmax_q[kDeqMax];
  const float* group_scale[kDeqMax];
};
hipError_t launch_dequant_group(const DeqSrcs& src, int n, int64_t N, int64_t K, int codebook, int absfmt,
                                bool transposed, bf16_t* out, int64_t ldo, int64_t out_gs, hipStream_t s);

// Y = X deq(W)^T + s * U * B^T  (U already holds X A^T in bf16; r may be 0).
// parts: U is the sum of that many matrices [M x r], one after the other.
hipError_t launch_fwd(const Nf4View& W, const bf16_t* X, int64_t M, const bf16_t* U, const bf16_t* B,
                      int r, float s, bf16_t* Y, hipStream_t st, int parts = 1);

// dX = dY deq(W) + s * G * A  (G = dY B in bf16; r may be 0)
hipError_t launch_dx(const Nf4View& W, const bf16_t* dY, int64_t M, const bf16_t* G, const bf16_t* A,
                     int r, float s, bf16_t* dX, hipStream_t st);

// Dense bf16 product on a weight already in bf16, Wd [N x K]:
// Y [M x N] = X Wd^T + s * U * B'^T (r may be 0), where B' [N x r] is B, or,
// with b_trans, the transpose of B [r x N].  The backward runs it on the
// transposed weight: dX = dY (W^T)^T + s G (A^T)^T.  part (part_bytes of
// fp32 scratch, may be null) lets shapes with few tiles and a long
// contraction split it (dense_split_bytes(N, K, M) bytes are enough).
hipError_t launch_bf16_fwd(const bf16_t* Wd, int64_t N, int64_t K, const bf16_t* X, int64_t M, const bf16_t* U,
                           const bf16_t* B, bool b_trans, int r, float s, bf16_t* Y, hipStream_t st,
                           float* part = nullptr, size_t part_bytes = 0);
// The same over a stack of weights with one adapter each: weight rows come in
// groups of gn (the last may be shorter), and the rows of group g take
// columns g r .. g r + r - 1 of U (row stride ldu) in the tail.  gn = N and
// ldu = r is launch_bf16_fwd.
hipError_t launch_bf16_group(const bf16_t* Wd, int64_t N, int64_t K, const bf16_t* X, int64_t M, const bf16_t* U,
                             int ldu, const bf16_t* B, bool b_trans, int r, int64_t gn, float s, bf16_t* Y,
                             hipStream_t st, float* part = nullptr, size_t part_bytes = 0);
// Scratch for a split contraction of the dense product Y [M x N] over K
// (0 when such a shape is not split).
size_t dense_split_bytes(int64_t N, int64_t K, int64_t M);

// Skinny products with a deterministic split-contraction reduction.
// out_bf16 / out_f32 (either may be null) receive scale * result.
size_t skinny_partial_bytes(int64_t rows, int64_t cols, int64_t contraction, int kind);
enum SkinnyKind { kXAt = 0, kDyB = 1, kGtX = 2, kDytU = 3 };
hipError_t launch_xat(const bf16_t* X, const bf16_t* A, int64_t M, int64_t K, int r, float* part,
                      bf16_t* out, bf16_t* out2, float scale, hipStream_t st);
hipError_t launch_dyb(const bf16_t* dY, const bf16_t* B, int64_t M, int64_t N, int r, float* part,
                      bf16_t* out, float scale, hipStream_t st);
// G groups: group g reads columns g N .. of dY [M x ldy] and B + g N r, and
// writes columns g r .. of out [M x G r]; partials: skinny_partial_bytes(M,
// G r, N, kDyB).
hipError_t launch_dyb_group(const bf16_t* dY, int64_t ldy, const bf16_t* B, int64_t M, int64_t N, int r, int G,
                            float* part, bf16_t* out, float scale, hipStream_t st);
// The adapter gradients: dA [G r x K] = scale G^T X (Gm [M x G r], X [M x
// K]) and, per group g, dB_g = scale dY_g^T U_g (columns g N .. of dY [M x
// ldy], columns g r .. of U [M x ldu]) into dB + g N r; the two split
// reductions run as one launch.  Partials: grads_partial_bytes(M, N, K, r, G).
size_t grads_partial_bytes(int64_t M, int64_t N, int64_t K, int r, int G);
hipError_t launch_grads(const bf16_t* Gm, const bf16_t* X, const bf16_t* dY, int64_t ldy, const bf16_t* U, int ldu,
                        int64_t M, int64_t N, int64_t K, int r, int G, float* part, float* dA, float* dB, float scale,
                        hipStream_t st);

// The same products for an adapter under dropout and for callers that need
// fp32-accurate gradients: drop may be null (no mask); r <= 128.  Partials:
// u_part_bytes for the first alone, adapter_part_bytes for all of them.
size_t u_part_bytes(int64_t M, int64_t K, int r);
size_t adapter_part_bytes(int64_t M, int64_t N, int64_t K, int r);
// The last step of such a product, left to the caller: workgroups of a launch
// that neither reads nor writes what it does (ride.h), or launch_ride.
enum RideKind : int { kRideSum, kRideSum3, kRideRows, kRideRowsDrop };
// out [rows x ld]: in [rows x cols] (null: nothing copied) and zero columns
// cols .. ld - 1; cols, ld % 8 == 0.
struct PadRows {
  const bf16_t* in;
  bf16_t* out;
  int64_t rows, cols, ld;
  int blocks;
};
inline PadRows pad_rows(const bf16_t* in, int64_t rows, int64_t cols, bf16_t* out, int64_t ld) {
  return PadRows{in, out, rows, cols, ld, (int)((rows * (in ? ld >> 3 : (ld - cols) >> 3) + 255) / 256)};
}
//
// What such a product gives: out [M x r] bf16 (may be null), and parts (may be
// null), s times it as the sum of bf16 matrices [M x r], one after the other:
// kTermParts of them, or (kRideSum3) kGradParts.  The dense products take the
// adapter's side in that form: one bf16 would leave Y and dX an error of 2^-9
// of the adapter's term, as large as the rounding of the result; two leave
// 2^-17.  s is applied in fp32, before the split.
constexpr int kTermParts = 2, kGradParts = 3;
struct Ride {
  RideKind kind;
  int blocks;                 // workgroups of 256
  bf16_t *out, *parts;
  float* full;                // kRideSum: s times the sum in fp32 (may be null)
  float s;
  const float* part;          // sums of partials
  int splits;
  int64_t n;
  float scale;
  const bf16_t *X, *A;        // U by rows
  int64_t M, K;
  int r;
  DropArgs drop;
  PadRows pad[2];             // kRideSum3: padded copies, too
};
hipError_t launch_ride(const Ride& a, hipStream_t st);
// U = drop(X) A^T, to out and parts: all but *rest (kRideSum, kRideRows or
// kRideRowsDrop).
hipError_t start_xat_drop(const bf16_t* X, const bf16_t* A, int64_t M, int64_t K, int r, const DropArgs* drop,
                          float* part, bf16_t* out, bf16_t* parts, float s, Ride* rest, hipStream_t st);
// s G = s dY B as kGradParts parts: all but *rest (kRideSum3).
hipError_t start_dyb_parts(const bf16_t* dY, const bf16_t* B, int64_t M, int64_t N, int r, float* part, bf16_t* parts,
                           float s, Ride* rest, hipStream_t st);
// dA [r x K] = G^T drop(X) with G3 as above (s in it, and 1 / (1 - p) too),
// dB [N x r] = scale dY^T U.
hipError_t launch_adapter_grads(const bf16_t* G3, const bf16_t* X, const bf16_t* dY, const bf16_t* U, int64_t M,
                                int64_t N, int64_t K, int r, const DropArgs* drop, float* part, float* dA, float* dB,
                                float scale, hipStream_t st);

// The small tiles or the 256-token kernels, whichever is estimated faster: Y
// [M x N] = X Wd^T + T B'^T, T in kTermParts parts; with b_trans and drop (may
// be null) the adapter's term masked as the M x N tensor was (dX), its scale in
// T.  K % 64 == 0; part as for launch_bf16_fwd, staged_part_bytes are enough.
size_t staged_part_bytes(int64_t N, int64_t K, int64_t M);
double staged_cost(int64_t N, int64_t K, int64_t M);   // us, estimated
// Whether the 256-token tiles are estimated the fastest, unsplit.
bool dense_tiles(int64_t N, int64_t K, int64_t M);
// Splits of a dense product of few 256-token tiles and a long contraction (1: none).
int dense_splits(int64_t N, int64_t K, int64_t M, int cus);
// X Wd^T alone as *splits fp32 parts [M x N].  product_part_bytes are enough.
size_t product_part_bytes(int64_t N, int64_t K, int64_t M);
hipError_t launch_product_parts(const bf16_t* Wd, int64_t N, int64_t K, const bf16_t* X, int64_t M, float* part,
                                int* splits, hipStream_t st);
// rest (may be null): the sum of a split contraction's parts is left to the caller.
struct SplitSum {
  const float* part;
  int splits;   // 0: nothing left
  int64_t n;
  bf16_t* out;
};
hipError_t launch_staged(const bf16_t* Wd, int64_t N, int64_t K, const bf16_t* X, int64_t M, const bf16_t* T,
                         const bf16_t* B, bool b_trans, int r, const DropArgs* drop, bf16_t* Y, hipStream_t st,
                         float* part, size_t part_bytes, SplitSum* rest = nullptr);

// The same of G stacked adapters of rank r (a gated block's two): columns g N ..
// of dY [M x ldy] and B + g N r give columns g r .. of G's parts [M x G r].
size_t group_dyb_part_bytes(int64_t M, int64_t N, int r, int G);
hipError_t start_dyb_parts_group(const bf16_t* dY, int64_t ldy, const bf16_t* B, int64_t M, int64_t N, int r, int G,
                                 float* part, bf16_t* parts, float s, Ride* rest, hipStream_t st);
// dA [G r x K] and dB [G N x r] (group g: columns g dy_gs .. of dY, g r .. of U),
// and the sum that another product left.
size_t group_grads_part_bytes(int64_t M, int64_t N, int64_t K, int r, int G);
hipError_t launch_adapter_grads_group(const bf16_t* G3, const bf16_t* X, const bf16_t* dY, int64_t ldy, int64_t dy_gs,
                                      const bf16_t* U, int64_t M, int64_t N, int64_t K, int r, int G, float* part,
                                      float* dA, float* dB, float scale, const SplitSum& left, hipStream_t st);

// The adapters of a call: S slots of rank R for each of G weights side by side,
// A [S x G R x K], B [S x G N x R]; token m takes slot ids[m] (ids null: slot 0),
// none where that is no slot.  scale null: s; rank null: R for all (pool.h).
struct PoolView {
  const bf16_t *A, *B;
  const float* scale;
  const int32_t* rank;
  const int32_t* ids;
  float s;
  int slots, R, G;   // R == 0: no adapters
};
// The work of a streamed product (stream.hip): units, `spans` of them to a tile,
// shared out evenly to `wgs` workgroups in order; units x wgs < 2^32.
constexpr int kStreamRows = 256;
struct StreamLine {
  uint32_t tiles, spans, units, wgs, block;   // tiles of one weight and token block; tokens of a block
  // the first unit of workgroup w, and the workgroup of unit u
  __host__ __device__ uint32_t unit(uint32_t w) const { return w * units / wgs; }
  __host__ __device__ uint32_t of(uint32_t u) const { return ((u + 1) * wgs - 1) / units; }
  // the first workgroup of a tile
  __host__ __device__ uint32_t first(uint32_t tile) const { return of(tile * spans); }
};
// The adapters' first half as tasks of waves (downs.h): `slices` of K, `cols` wide;
// done by `wgs` workgroups: others than the product's, those that have one unit
// less than the rest (`least`), or all of them.
constexpr int kMaxSlices = 4;
enum StreamTasks : int { kTasksApart, kTasksLight, kTasksAll };
struct StreamDowns {
  uint32_t tasks, slices, cols, wgs, least;
  int tt;   // tokens of a task
  StreamTasks where;
  // the number of workgroup w among them, or -1
  __host__ __device__ int index(const StreamLine& l, uint32_t w) const {
    if (where == kTasksApart) return w < l.wgs ? -1 : (int)(w - l.wgs);
    if (where == kTasksAll) return (int)w;
    const uint32_t u = l.unit(w);
    return l.unit(w + 1) - u == least ? (int)(w - (u - w * least)) : -1;   // less those before it that have one more
  }
};
struct StreamPlan {
  int nt, slots;   // slots: parts of a tile at most
  int all_tiles;   // of all weights and token blocks
  StreamLine line;
  StreamDowns downs;
};
StreamPlan stream_plan(int64_t N, int64_t K, int64_t M, int G, int R);
// The G frozen products as parts [slots][M][G N], counts[t] of
// those of tile t (token block, weight, kStreamRows rows), and T as parts
// [downs.slices][M][G R], with the scales of a pool that has them, in the same
// launch.
hipError_t launch_stream(const Nf4View* W, const bf16_t* X, int64_t M, const PoolView& pool, const StreamPlan& plan,
                         float* T, float* part, int32_t* counts, hipStream_t st);
// Y [M x N] from fp32 parts [M x G N] of the frozen products, `splits` of them or
// (counts not null) as launch_stream leaves them, `splits` of a tile at most, and the adapters' term; G ==
// 2: act(first) second, and the two themselves to GU [M x 2 N] (may be null).
// T [M x G R] is scale times the sum of `slices` parts, that sum in bf16 to U (may
// be null).
hipError_t launch_pool_finish(const PoolView& p, const float* part, int splits, const int32_t* counts,
                              const StreamLine* line, int64_t M, int64_t N, const float* T, int slices, float scale,
                              bf16_t* U, int act, bf16_t* Y, bf16_t* GU, hipStream_t st);
// The products of many tokens with the adapters' term, and of a gated block's two
// weights with its activation, from a dequantized stack (gemm_pool.hip): G == 1
// Wd [N x K]; G == 2 kPoolTurn rows of each in turn, N rounded up to kPoolRows of
// each, as launch_dequant_pair leaves them.  T: kTermParts parts [M x G R].  part
// not null (G == 1, one adapter or none): the sum as `splits` fp32 parts [M x N].
struct PoolGemm {
  const bf16_t* Wd;
  int64_t N, K, M;
  const bf16_t *X, *T;
  PoolView pool;
  int act;
  bf16_t *Y, *GU;
  float* part;
  int splits;
};
constexpr int64_t kPoolRows = 32, kPoolTurn = 16;
inline int64_t pool_stack_rows(int64_t N, int G) { return G == 1 ? N : (N + kPoolRows - 1) / kPoolRows * kPoolRows * 2; }
// 32-bit offsets of T and of a slot's B, R ranks of G weights each.
inline bool pool_term_ok(int64_t M, int64_t N, int64_t R, int G) {
  return M <= ((int64_t)1 << 27) / (G * R) && N < ((int64_t)1 << 30) / R;
}
hipError_t launch_pool_gemm(const PoolGemm& g, hipStream_t st);
// T [M x G R] of a pool's adapters, as parts or in fp32 (T; either may be null),
// through `part` (pool_u_part_bytes): all but *rest (kRideSum).
size_t pool_u_part_bytes(int64_t M, int64_t K, int GR);
hipError_t start_pool_u(const PoolView& p, const bf16_t* X, int64_t M, int64_t K, float* part, bf16_t* parts, float* T,
                        Ride* rest, hipStream_t st);
// The same of one adapter, or of two of rank r / 2 stacked (r <= 256): s X A^T, and
// X A^T in bf16 to out (may be null).
size_t xat_part_bytes(int64_t M, int64_t K, int r);
hipError_t start_xat_parts(const bf16_t* X, const bf16_t* A, int64_t M, int64_t K, int r, float* part, bf16_t* out,
                           bf16_t* parts, float* T, float s, Ride* rest, hipStream_t st);
// Two weights N x K as one stack in turns of `turn` rows; those past N are left
// as they were.  N K < 2^31.  With *rest of kRideSum, possibly empty.
hipError_t launch_dequant_pair(const Nf4View* W, int turn, bf16_t* out, const Ride& rest, hipStream_t st);
// The two transposed, weight z to columns z half .. of out [K x 2 half]; those past
// N of each are left as they were.  rest: of kRideSum3, possibly empty.
hipError_t launch_dequant_t_pair(const Nf4View* W, bf16_t* out, int64_t half, const Ride& rest, hipStream_t st);
// dY [M x 2 Fp] = [dG | dP] of a gated block (gated.hip), zero from column F of
// each half on, as Wt [K x 2 Fp] is made (may be null); and At [K x r] = A^T (may be
// null, r % 8 == 0).
hipError_t launch_gated_grad(const bf16_t* dH, const bf16_t* GU, int64_t M, int64_t F, int64_t Fp, int act, bf16_t* dY,
                             bf16_t* Wt, int64_t K, const bf16_t* A, int r, bf16_t* At, hipStream_t st);

// Rows of 8-bit integers with one scale each (i8.hip): bytes from one row to
// the next, and the passes over them.
inline int64_t i8_row_bytes(int64_t cols) { return (cols + 127) / 128 * 128; }
constexpr int64_t kI8MaxCols = 131072;   // 127^2 cols fits a 32-bit sum
// Q [M x i8_row_bytes(K)], scale [M] from X [M x K], K % 8 == 0.
// sum: null, or a step of kRideSum to take along.
hipError_t launch_quant_rows(const bf16_t* X, int64_t M, int64_t K, int8_t* Q, float* scale, const Ride* sum,
                             hipStream_t st);
// U = drop(X) A^T, to U (may be null) and parts as above (r may be 0, drop
// null), and X quantized, in one launch, where i8_prep_ok.
bool i8_prep_ok(int64_t M, int64_t K, int r, bool drop);
hipError_t launch_i8_prep(const bf16_t* X, int64_t M, int64_t K, const bf16_t* A, int r, const DropArgs* drop,
                          bf16_t* U, bf16_t* parts, float s, int8_t* Q, float* scale, hipStream_t st);
hipError_t launch_i8_dequant(const int8_t* Q, const float* scale, int64_t N, int64_t K, bf16_t* out, hipStream_t st);
// out [K x ldo] = deq^T, ldo = N rounded up to 64, the columns past N zero;
// rest: of kRideSum3, possibly empty.
hipError_t launch_i8_dequant_t(const int8_t* Q, const float* scale, int64_t N, int64_t K, bf16_t* out, int64_t ldo,
                               const Ride& rest, hipStream_t st);

// Y [M x N] = sx sw^T o (Xq Wq^T) + T B^T (r may be 0), T in kTermParts parts.
struct I8Gemm {
  const int8_t* Wq;
  const float* sw;
  int64_t N, K;
  const int8_t* Xq;
  const float* sx;
  int64_t M;
  const bf16_t* T;
  const bf16_t* B;
  int r;
  bf16_t* Y;
};
// part (part_bytes of scratch, may be null) lets shapes of few tiles split their
// contraction into 32-bit integer parts; i8_gemm_part_bytes is enough.
size_t i8_gemm_part_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_i8_gemm(const I8Gemm& g, hipStream_t st, int32_t* part, size_t part_bytes);

// Tiles of a middling product (gemm_tile.hip).  Rows of W [N] and X [M] are
// row_bytes apart, whole 128-byte lines; sw and sx: 8-bit operands.  The
// adapter's term: T, kTermParts parts [M x r], with B [N x r], or with b_trans A
// [r x N], masked by `drop` if `dropped`.  A split contraction leaves fp32 parts of everything in
// `part`, which launch_tile adds up; of 8-bit operands the integer sums alone,
// which the caller does.
struct TileGemm {
  const void* W;
  const void* X;
  const float* sw;
  const float* sx;
  int64_t N, row_bytes, M;
  const bf16_t* T;
  const bf16_t* B;
  int r;
  bool b_trans, dropped;
  DropArgs drop;
  bf16_t* Y;
  void* part;
  bool keep;   // leave the fp32 parts, of one split too, to the caller
};
struct TileChoice {
  int tm, tn, splits;   // tm == 256: one of the 256-token kernels
  double cost;          // us, estimated
};
double full_round_cost(int64_t lines);   // of 256 x 256 tiles
// small: of the tiles below 256 tokens.
TileChoice choose_tile(int64_t M, int64_t N, int64_t lines, int cus, size_t part_bytes, bool small = false);
size_t tile_part_bytes(int64_t M, int64_t N, int64_t lines);
hipError_t launch_tile(const TileGemm& g, const TileChoice& c, int64_t n_begin, int64_t n_rows, hipStream_t st);
// Y [n] bf16 = the sum of the splits' fp32 parts, in order.
hipError_t launch_split_sum(const float* part, int splits, int64_t n, bf16_t* Y, hipStream_t st);

// The paged optimizer's layout and step (paged.hip).
bool paged_plan(const qlora_paged_tensor* t, int nt, size_t dev_bytes, qlora_paged_layout* L);
hipError_t paged_adamw(const qlora_paged_tensor* t, int nt, char* ws, const qlora_paged_layout& L, float lr,
                       float b1, float b2, float eps, float wd, int step, int flags, hipStream_t st,
                       hipStream_t copy_stream);

// Decode of one to 16 tokens per linear.
struct GemvJob {
  const uint8_t* codes;
  const uint8_t* absmax_q;
  const float* group_scale;
  const bf16_t* x;
  const bf16_t* A;
  const bf16_t* B;
  bf16_t* y;
  float* u;  // m x r fp32 scratch (A x per token)
  int32_t N;
  int32_t K;
  int32_t r;
  float s;
  int32_t m;  // tokens: x is [m x K], y [m x N]
};
// gemv_prepare writes the job table (jobs, per-workgroup tile segments and
// the u = A x map) into `table` (device memory of at least
// gemv_table_bound(njobs, max rows) bytes) by one host-to-device copy on
// `st`; gemv_run then launches u = A x (one launch for the one-token jobs,
// one for the others) and the NF4 GEMV (one launch per kind of job present:
// one token or several, with absmax rows read two or four bytes at a time or
// byte by byte).
size_t gemv_table_bound(int njobs, int64_t max_rows);
size_t gemv_lds_bytes(int64_t K);
// What gemv_run needs besides the table in device memory.
constexpr int kGvKinds = 4;   // launches per call: batch-1 and several tokens, two absmax layouts each
struct GemvLaunch {
  void* table;
  uint64_t seg_off[kGvKinds], rng_off[kGvKinds], down_off;
  int32_t groups[kGvKinds], max_steps[2];   // max_steps: the two one-token launches
  int32_t n_down, n_rows;                    // u = A x map entries, the first n_rows of them one per adapter row
  int32_t codebook;  // shared by every job of the call: 4-bit codebook | second-level format << 8
};
hipError_t gemv_prepare(const GemvJob* jobs, int njobs, int codebook, void* table, size_t table_bytes,
                        GemvLaunch* out, hipStream_t st);
hipError_t gemv_run(const GemvLaunch& L, hipStream_t st);

}  // namespace qlora
