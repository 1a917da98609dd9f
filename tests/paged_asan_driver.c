/* Calls the paged cache's entry points with arguments that the host checks
 * reject (or with nothing to do), for a run under AddressSanitizer: exits 0
 * when each returned the expected status. */
#include <stdio.h>

#include "mova.h"

static int bad = 0;

static void expect(const char* what, int got, int want) {
  if (got != want) {
    fprintf(stderr, "%s: %d, expected %d\n", what, got, want);
    bad = 1;
  }
}

#define P ((void*)(1u << 20))

int main(void) {
  int32_t* i = (int32_t*)P;
  int64_t* s = (int64_t*)P;
  float* f = (float*)P;
  const size_t big = (size_t)1 << 40;

  expect("plan B", mova_paged_plan(i, i, -1, 8, 16, 10, i, i, 40, i, i + 1, i + 8, i, s, i, 0),
         MOVA_ERR_INVALID_ARG);
  expect("plan requests", mova_paged_plan(i, i, 2049, 8, 16, 10, i, i, 40, i, i + 1, i + 8, i, s, i, 0),
         MOVA_ERR_UNSUPPORTED);
  expect("plan count", mova_paged_plan(i, i, 4, 8, 16, 10, i, i, 40, i, i, i + 8, i, s, i, 0),
         MOVA_ERR_INVALID_ARG);
  expect("plan table", mova_paged_plan(i, i, 4, 8, 16, 10, NULL, i, 40, i, i + 1, i + 8, i, s, i, 0),
         MOVA_ERR_INVALID_ARG);

  expect("store empty", mova_kv_store_paged(P, P, 0, 8, 128, P, P, 0, NULL, NULL, 10, 16, s, P, 0),
         MOVA_OK);
  expect("store scale", mova_kv_store_paged(P, P, 8, 8, 128, P, P, 0, f, NULL, 10, 16, s, P, 0),
         MOVA_ERR_INVALID_ARG);
  expect("store width", mova_kv_store_paged(P, P, 8, 129, 128, P, P, 1, f, f, 10, 16, s, P, 0),
         MOVA_ERR_UNSUPPORTED);
  expect("store bounds", mova_kv_store_paged(NULL, P, 8, 8, 128, NULL, P, 1, f, f, 10, 16, s, P, 0),
         MOVA_ERR_INVALID_ARG);

  expect("select empty",
         mova_block_select(P, P, 40, 16, i, 10, i, 0, 32, 8, 128, 8, 1, 2, i, NULL, 0, 0), MOVA_OK);
  expect("select keep",
         mova_block_select(P, P, 40, 16, i, 10, i, 4, 32, 8, 128, 2, 2, 2, i, P, big, 0),
         MOVA_ERR_INVALID_ARG);
  expect("select workspace",
         mova_block_select(P, P, 40, 16, i, 10, i, 4, 32, 8, 128, 8, 1, 2, i, P, 16, 0),
         MOVA_ERR_WORKSPACE);
  for (int b = 1; b <= 2048; b *= 2)
    for (int h = 1; h <= 64; h *= 2)
      for (int keep = 1; keep < 5000; keep *= 7) {
        if (mova_block_select_workspace_bytes(b, 4 * h, h, 128, 3000, 16, keep) == (size_t)-1 ||
            mova_attention_workspace_bytes(b, 4 * h, h, 128, 3000, 16, keep) == (size_t)-1)
          bad = 1;
      }

  expect("attention empty",
         mova_attention_paged(P, P, P, 1, f, f, 40, 16, i, 10, i, i, 4, 0, 32, 8, 128, 0.1f, 0, P, f,
                              NULL, 0, 0),
         MOVA_OK);
  expect("attention list",
         mova_attention_paged(P, P, P, 1, f, f, 40, 16, i, 10, i, NULL, 4, 4, 32, 8, 128, 0.1f, 0, P,
                              f, P, big, 0),
         MOVA_ERR_INVALID_ARG);
  expect("attention heads",
         mova_attention_paged(P, P, P, 1, f, f, 40, 16, i, 10, i, i, 4, 4, 33, 8, 128, 0.1f, 0, P, f,
                              P, big, 0),
         MOVA_ERR_UNSUPPORTED);
  expect("attention workspace",
         mova_attention_paged(P, P, P, 1, f, f, 40, 16, i, 10, i, i, 4, 4, 32, 8, 128, 0.1f, 0, P, f,
                              P, 16, 0),
         MOVA_ERR_WORKSPACE);
  if (!bad) printf("paged asan driver: ok\n");
  return bad;
}
