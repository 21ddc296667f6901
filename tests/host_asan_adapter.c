/* The dropout and 8-bit entry points' argument checks under host
 * AddressSanitizer: as tests/host_asan_driver.c, only calls that are refused
 * before any HIP call, with descriptors on the heap in blocks of exactly their
 * size.  Prints "host asan adapter OK" when every status is the expected one.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "qlora.h"

static int failures = 0;

#define EXPECT(call, want)                                                            \
  do {                                                                                \
    int got_ = (int)(call);                                                           \
    if (got_ != (int)(want)) {                                                        \
      fprintf(stderr, "line %d: %s -> %d, expected %d\n", __LINE__, #call, got_, (int)(want)); \
      ++failures;                                                                     \
    }                                                                                 \
  } while (0)

static uint16_t* bf(int i) { return (uint16_t*)(uintptr_t)(0x10000 * (i + 1)); }

static qlora_nf4_weight* nf4(int64_t rows, int64_t cols) {
  qlora_nf4_weight* w = calloc(1, sizeof(*w));
  w->rows = rows, w->cols = cols, w->blocksize = 64, w->group_blocks = 256;
  w->codes = (uint8_t*)bf(0), w->absmax_q = (uint8_t*)bf(1), w->group_scale = (float*)bf(2);
  return w;
}
static qlora_i8_rows* rows8(int64_t rows, int64_t cols) {
  qlora_i8_rows* q = calloc(1, sizeof(*q));
  q->rows = rows, q->cols = cols, q->codes = (int8_t*)bf(0), q->scale = (float*)bf(1);
  return q;
}
static qlora_drop* drop(double p, uintptr_t step) {
  qlora_drop* d = calloc(1, sizeof(*d));
  d->p = p, d->seed = 1, d->offset = 2, d->step = (const uint64_t*)step;
  return d;
}

int main(void) {
  const double bad_p[] = {-0.1, 1.0, 2.0, NAN, INFINITY, -INFINITY};
  qlora_nf4_weight *w = nf4(128, 256), *odd = nf4(132, 256), *narrow = nf4(128, 200), *wide = nf4(8, 64);
  qlora_i8_rows *q = rows8(64, 256), *k12 = rows8(64, 12), *long_row = rows8(64, 131080), *n60 = rows8(60, 256),
                *k128 = rows8(64, 128), *huge = rows8((int64_t)1 << 24, 131072), *none = rows8(0, 256);
  qlora_drop *d = drop(0.1, 0), *d_odd = drop(0.1, 0x10004);
  uint8_t* ws = (uint8_t*)bf(9);
  const size_t big = (size_t)1 << 40;

  EXPECT(qlora_dropout(NULL, 8, d, bf(1), NULL), QLORA_E_NULL);
  EXPECT(qlora_dropout(bf(0), 8, NULL, bf(1), NULL), QLORA_E_NULL);
  EXPECT(qlora_dropout(bf(0) + 1, 8, d, bf(1), NULL), QLORA_E_ALIGN);
  EXPECT(qlora_dropout(bf(0), 8, d_odd, bf(1), NULL), QLORA_E_ALIGN);
  EXPECT(qlora_dropout(bf(0), 0, d, bf(1), NULL), QLORA_E_SHAPE);
  EXPECT(qlora_dropout(bf(0), INT64_MAX, d, bf(1), NULL), QLORA_E_SHAPE);
  for (int i = 0; i < 6; ++i) {
    qlora_drop* b = drop(bad_p[i], 0);
    EXPECT(qlora_dropout(bf(0), 8, b, bf(1), NULL), QLORA_E_UNSUPPORTED);
    EXPECT(qlora_linear_fwd_drop(w, bf(0), 4, bf(1), bf(2), 8, 16.0f, b, bf(3), NULL, ws, big, NULL), QLORA_E_UNSUPPORTED);
    EXPECT(qlora_linear_bwd_drop(w, bf(0), bf(4), 4, bf(1), bf(2), 8, 16.0f, NULL, b, bf(3), (float*)bf(5),
                                 (float*)bf(6), ws, big, NULL),
           QLORA_E_UNSUPPORTED);
    EXPECT(qlora_i8_linear_fwd(q, bf(0), 4, bf(1), bf(2), 8, 16.0f, b, bf(3), NULL, ws, big, NULL), QLORA_E_UNSUPPORTED);
    EXPECT(qlora_i8_linear_bwd(q, bf(0), bf(4), 4, bf(1), bf(2), 8, 16.0f, NULL, b, bf(3), (float*)bf(5), (float*)bf(6),
                               ws, big, NULL),
           QLORA_E_UNSUPPORTED);
    free(b);
  }
  qlora_nf4_weight* bad_w[] = {odd, narrow};
  for (int i = 0; i < 2; ++i) {
    EXPECT(qlora_linear_fwd_drop(bad_w[i], bf(0), 4, bf(1), bf(2), 8, 16.0f, d, bf(3), NULL, ws, big, NULL),
           QLORA_E_UNSUPPORTED);
    EXPECT(qlora_linear_bwd_drop(bad_w[i], bf(0), bf(4), 4, bf(1), bf(2), 8, 16.0f, NULL, d, bf(3), (float*)bf(5),
                                 (float*)bf(6), ws, big, NULL),
           QLORA_E_UNSUPPORTED);
  }
  EXPECT(qlora_linear_fwd_drop(w, bf(0), 4, bf(1), bf(2), 8, 16.0f, d, bf(3), NULL, ws, 64, NULL), QLORA_E_WORKSPACE);
  EXPECT(qlora_linear_fwd_drop(w, bf(0), 4, NULL, NULL, 0, 16.0f, d, bf(3), NULL, ws, big, NULL), QLORA_E_UNSUPPORTED);
  EXPECT(qlora_linear_fwd_drop(wide, bf(0), 1 << 24, bf(1), bf(2), 128, 16.0f, d, bf(3), NULL, ws, big, NULL),
         QLORA_E_UNSUPPORTED);
  EXPECT(qlora_linear_bwd_drop(w, bf(0), bf(4), 4, bf(1), bf(2), 8, 16.0f, NULL, d, bf(3), NULL, NULL, ws, big, NULL),
         QLORA_E_NULL);

  qlora_i8_rows* bad_q[] = {k12, long_row, huge};
  for (int i = 0; i < 3; ++i) {
    EXPECT(qlora_i8_quantize(bf(0), bad_q[i], NULL), QLORA_E_UNSUPPORTED);
    EXPECT(qlora_i8_dequant(bad_q[i], bf(0), NULL), QLORA_E_UNSUPPORTED);
    EXPECT(qlora_i8_matmul(q, bad_q[i], bf(0), NULL), QLORA_E_UNSUPPORTED);
    EXPECT(qlora_i8_linear_fwd(bad_q[i], bf(0), 4, NULL, NULL, 0, 1.0f, NULL, bf(3), NULL, ws, big, NULL),
           QLORA_E_UNSUPPORTED);
  }
  EXPECT(qlora_i8_quantize(bf(0), none, NULL), QLORA_E_SHAPE);
  EXPECT(qlora_i8_matmul(q, n60, bf(0), NULL), QLORA_E_UNSUPPORTED);
  EXPECT(qlora_i8_matmul(k128, q, bf(0), NULL), QLORA_E_SHAPE);
  EXPECT(qlora_i8_matmul(NULL, q, bf(0), NULL), QLORA_E_NULL);
  EXPECT(qlora_i8_linear_fwd(q, bf(0), 4, NULL, NULL, 0, 1.0f, d, bf(3), NULL, ws, big, NULL), QLORA_E_UNSUPPORTED);
  EXPECT(qlora_i8_linear_fwd(q, bf(0), 4, NULL, NULL, 0, 1.0f, NULL, bf(3), NULL, ws, 64, NULL), QLORA_E_WORKSPACE);
  EXPECT(qlora_i8_linear_fwd(q, bf(0), INT64_MAX, NULL, NULL, 0, 1.0f, NULL, bf(3), NULL, ws, big, NULL), QLORA_E_SHAPE);
  EXPECT(qlora_i8_linear_bwd(q, NULL, bf(4), 4, NULL, NULL, 0, 1.0f, NULL, NULL, bf(3), (float*)bf(5), NULL, ws, big,
                             NULL),
         QLORA_E_SHAPE);

  const int ops[] = {QLORA_OP_FWD_DROP, QLORA_OP_BWD_DROP, QLORA_OP_I8_FWD, QLORA_OP_I8_BWD};
  const int64_t sizes[] = {INT64_MIN, -8, 0, 1, 8, 64, 131072, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX};
  for (int o = 0; o < 4; ++o)
    for (int a = 0; a < 10; ++a)
      for (int b = 0; b < 10; ++b)
        for (int c = 0; c < 10; ++c) {   // never a trap, and nothing for sizes that no call takes
          const size_t n = qlora_workspace_bytes((qlora_op)ops[o], sizes[a], sizes[b], sizes[c], 8, 0);
          if (sizes[a] <= 0 || sizes[b] <= 0 || sizes[c] <= 0 || sizes[a] > INT32_MAX || sizes[c] > INT32_MAX)
            EXPECT(n, 0);
        }
  for (int i = 0; i < 10; ++i)
    if (sizes[i] <= 0 || sizes[i] > 131072) EXPECT(qlora_i8_row_bytes(sizes[i]), 0);

  free(w), free(odd), free(narrow), free(wide), free(q), free(k12), free(long_row), free(n60), free(k128), free(huge);
  free(none), free(d), free(d_odd);
  if (failures) return 1;
  printf("host asan adapter OK\n");
  return 0;
}
