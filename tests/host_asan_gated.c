/* The gated block's and the adapter pools' argument checks under host
 * AddressSanitizer: as tests/host_asan_driver.c, only calls that are refused
 * before any HIP call, with descriptors on the heap in blocks of exactly their
 * size.  Prints "host asan gated OK" when every status is the expected one.
 */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

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

/* `n` weights, in a block of exactly their size */
static qlora_nf4_weight* weights(int n, int64_t rows, int64_t cols) {
  qlora_nf4_weight* w = calloc((size_t)n, sizeof(*w));
  for (int i = 0; i < n; ++i) {
    w[i].rows = rows, w[i].cols = cols, w[i].blocksize = 64, w[i].group_blocks = 256;
    w[i].codes = (uint8_t*)bf(0), w[i].absmax_q = (uint8_t*)bf(1), w[i].group_scale = (float*)bf(2);
  }
  return w;
}
static qlora_adapter_pool* pool(int64_t slots, int64_t rows, int64_t cols, int32_t rank) {
  qlora_adapter_pool* p = calloc(1, sizeof(*p));
  p->slots = slots, p->rows = rows, p->cols = cols, p->rank = rank;
  p->A = bf(3), p->B = bf(4), p->scale = (float*)bf(5);
  return p;
}

int main(void) {
  const size_t big = (size_t)1 << 60;
  uint8_t* ws = (uint8_t*)bf(9);
  int32_t* ids = (int32_t*)bf(8);
  qlora_nf4_weight *one = weights(1, 128, 256), *two = weights(2, 128, 256), *odd = weights(2, 132, 256),
                   *narrow = weights(2, 128, 200), *none = weights(2, 0, 256), *huge = weights(2, (int64_t)1 << 26, 256),
                   *longer = weights(2, 64, (int64_t)1 << 40), *unlike = weights(2, 128, 256);
  unlike[1].rows = 136;
  qlora_adapter_pool *p1 = pool(4, 128, 256, 16), *p2 = pool(4, 256, 256, 16);

  /* many and gated_many */
  EXPECT(qlora_many_fwd(NULL, bf(6), 4, p1, ids, bf(7), ws, big, NULL), QLORA_E_NULL);
  EXPECT(qlora_many_fwd(one, bf(6), 4, NULL, ids, bf(7), ws, big, NULL), QLORA_E_NULL);
  EXPECT(qlora_many_fwd(one, bf(6), 4, p1, NULL, bf(7), ws, big, NULL), QLORA_E_NULL);
  EXPECT(qlora_many_fwd(one, bf(6), 0, p1, NULL, bf(7), ws, big, NULL), QLORA_E_SHAPE);
  EXPECT(qlora_many_fwd(one, bf(6), INT64_MAX, p1, ids, bf(7), ws, big, NULL), QLORA_E_SHAPE);
  EXPECT(qlora_many_fwd(one, bf(6), INT64_MIN, p1, ids, bf(7), ws, big, NULL), QLORA_E_SHAPE);
  EXPECT(qlora_many_fwd(one, bf(6), 0x7FFFFFFF, p1, ids, bf(7), ws, big, NULL), QLORA_E_UNSUPPORTED);
  EXPECT(qlora_many_fwd(one, bf(6), 4, p1, ids, bf(7), ws, 0, NULL), QLORA_E_WORKSPACE);
  EXPECT(qlora_many_fwd(odd, bf(6), 4, p1, ids, bf(7), ws, big, NULL), QLORA_E_UNSUPPORTED);
  EXPECT(qlora_many_fwd(one, bf(6), 4, p2, ids, bf(7), ws, big, NULL), QLORA_E_SHAPE);
  EXPECT(qlora_gated_many_fwd(two, bf(6), 4, p1, ids, 0, bf(7), ws, big, NULL), QLORA_E_SHAPE);
  EXPECT(qlora_gated_many_fwd(two, bf(6), 4, p2, ids, 2, bf(7), ws, big, NULL), QLORA_E_UNSUPPORTED);
  EXPECT(qlora_gated_many_fwd(unlike, bf(6), 4, p2, ids, 0, bf(7), ws, big, NULL), QLORA_E_SHAPE);
  EXPECT(qlora_gated_many_fwd(narrow, bf(6), 4, p2, ids, 0, bf(7), ws, big, NULL), QLORA_E_UNSUPPORTED);
  const int64_t slots[] = {0, -1, INT64_MIN, 65537, INT64_MAX};
  for (int i = 0; i < 5; ++i) {
    qlora_adapter_pool* p = pool(slots[i], 128, 256, 16);
    EXPECT(qlora_many_fwd(one, bf(6), 4, p, ids, bf(7), ws, big, NULL), i < 3 ? QLORA_E_SHAPE : QLORA_E_UNSUPPORTED);
    free(p);
  }
  const int32_t ranks[] = {0, -8, 4, 136, INT32_MIN, INT32_MAX};
  for (int i = 0; i < 6; ++i) {
    qlora_adapter_pool* p = pool(4, 128, 256, ranks[i]);
    EXPECT(qlora_many_fwd(one, bf(6), 4, p, ids, bf(7), ws, big, NULL), QLORA_E_UNSUPPORTED);
    free(p);
    if (ranks[i] == 0) continue;   /* no adapters */
    EXPECT(qlora_gated_fwd(two, bf(6), 4, bf(3), bf(4), ranks[i], 16.0f, 0, bf(7), NULL, NULL, ws, big, NULL),
           QLORA_E_UNSUPPORTED);
    EXPECT(qlora_gated_bwd(two, bf(6), bf(7), bf(8), 4, bf(3), bf(4), ranks[i], 16.0f, 0, NULL, bf(5), (float*)bf(10),
                           (float*)bf(11), ws, big, NULL),
           QLORA_E_UNSUPPORTED);
  }

  /* gated, forward and backward */
  qlora_nf4_weight* bad[] = {odd, narrow, huge, longer, none, unlike};
  for (int i = 0; i < 6; ++i) {
    const int f = (int)qlora_gated_fwd(bad[i], bf(6), 64, bf(3), bf(4), 8, 16.0f, 0, bf(7), NULL, NULL, ws, big, NULL);
    const int b = (int)qlora_gated_bwd(bad[i], bf(6), bf(7), bf(8), 64, bf(3), bf(4), 8, 16.0f, 0, NULL, bf(5), (float*)bf(10),
                                       (float*)bf(11), ws, big, NULL);
    EXPECT(f, i < 4 ? QLORA_E_UNSUPPORTED : QLORA_E_SHAPE);
    EXPECT(b, f);
  }
  EXPECT(qlora_gated_fwd(NULL, bf(6), 4, NULL, NULL, 0, 0.0f, 0, bf(7), NULL, NULL, ws, big, NULL), QLORA_E_NULL);
  EXPECT(qlora_gated_fwd(two, bf(6), 0, NULL, NULL, 0, 0.0f, 0, bf(7), NULL, NULL, ws, big, NULL), QLORA_E_SHAPE);
  EXPECT(qlora_gated_fwd(two, bf(6), 4, NULL, NULL, 0, 0.0f, 0, bf(7), bf(8) + 1, NULL, ws, big, NULL), QLORA_E_ALIGN);
  EXPECT(qlora_gated_bwd(two, bf(6), bf(7), NULL, 4, NULL, NULL, 0, 0.0f, 0, NULL, bf(5), NULL, NULL, ws, big, NULL),
         QLORA_E_NULL);
  EXPECT(qlora_gated_bwd(two, bf(6), bf(7), bf(8), 4, NULL, NULL, 0, 0.0f, 0, NULL, bf(5), (float*)bf(10), NULL, ws, big, NULL),
         QLORA_E_SHAPE);

  /* workspaces: never a size that wrapped round */
  const int ops[] = {QLORA_OP_GATED_FWD, QLORA_OP_GATED_BWD, QLORA_OP_MANY_FWD, QLORA_OP_GATED_MANY_FWD};
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 63, 64, 65, 2048, 65536, 1 << 24, (int64_t)1 << 31, INT64_MAX};
  const int32_t rs[] = {0, 8, 128};
  for (int o = 0; o < 4; ++o)
    for (int a = 0; a < 12; ++a)
      for (int b = 0; b < 12; ++b)
        for (int c = 0; c < 12; ++c)
          for (int r = 0; r < 3; ++r) {
            const size_t n = qlora_workspace_bytes(ops[o], sizes[a], sizes[b], sizes[c], rs[r], 0);
            if (n > ((size_t)1 << 42)) ++failures, fprintf(stderr, "op %d: %zu bytes\n", ops[o], n);
            if ((a < 3 || b < 3 || c < 3) && n != 0) ++failures, fprintf(stderr, "op %d: a workspace for nothing\n", ops[o]);
          }

  free(one), free(two), free(odd), free(narrow), free(none), free(huge), free(longer), free(unlike), free(p1), free(p2);
  if (failures == 0) printf("host asan gated OK\n");
  return failures != 0;
}
