/* Calls the chunk attention's and the block upkeep's entry points with
 * arguments that the host checks reject (or with nothing to do), for a run under
 * AddressSanitizer: exits 0 when each returned the expected status. */
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
  float* f = (float*)P;
  const size_t big = (size_t)1 << 40;

  expect("chunk empty",
         mova_attention_chunk_paged(P, P, P, 1, f, f, 40, 16, i, 10, i, i, i, 0, 4, 32, 8, 128, 0.1f,
                                    0, P, f, NULL, 0, 0),
         MOVA_OK);
  expect("chunk window",
         mova_attention_chunk_paged(P, P, P, 1, f, f, 40, 16, i, 10, i, i, i, 9, 4, 32, 8, 128, 0.1f,
                                    -1, P, f, P, big, 0),
         MOVA_ERR_INVALID_ARG);
  expect("chunk heads",
         mova_attention_chunk_paged(P, P, P, 1, f, f, 40, 16, i, 10, i, i, i, 9, 4, 33, 8, 128, 0.1f,
                                    0, P, f, P, big, 0),
         MOVA_ERR_UNSUPPORTED);
  expect("chunk workspace",
         mova_attention_chunk_paged(P, P, P, 1, f, f, 40, 16, i, 10, i, i, i, 9, 4, 32, 8, 128, 0.1f,
                                    0, (char*)P + 4096, f, P, 16, 0),
         MOVA_ERR_WORKSPACE);
  for (int b = 1; b <= 2048; b *= 2)
    for (int h = 1; h <= 64; h *= 2)
      for (int t = 1; t <= 1 << 24; t *= 16)
        for (int d = 64; d <= 256; d *= 2)
          if (mova_attention_chunk_workspace_bytes(t, b, 4 * h, h, d, 100, 16) == (size_t)-1) bad = 1;

  expect("fork pairs", mova_paged_fork(i, i, i, 2049, i, 4, 16, 10, i, i, 40, i, i + 1, i, 40, i + 8, i,
                                       i, 0),
         MOVA_ERR_UNSUPPORTED);
  expect("fork lens", mova_paged_fork(i, i, NULL, 3, i, 4, 16, 10, i, i, 40, i, i + 1, i, 40, i, i, i,
                                      0),
         MOVA_ERR_INVALID_ARG);
  expect("free count", mova_paged_free(i, i, 4, 16, 10, i, i, 40, i, i, i, 40, i + 8, P, big, 0),
         MOVA_ERR_INVALID_ARG);
  expect("free blocks", mova_paged_free(i, i, 4, 16, 10, i, i, 40, i, i + 1, i, (1 << 20) + 1, i + 8, P,
                                        big, 0),
         MOVA_ERR_UNSUPPORTED);
  expect("free workspace", mova_paged_free(i, i, 4, 16, 10, i, i, 40, i, i + 1, i, 40, i + 8, P, 16, 0),
         MOVA_ERR_WORKSPACE);
  expect("compact limit",
         mova_paged_compact(i, 4, 16, 10, i, i, i, i, 40, i, i + 1, i, i, 40, -1, i, i, i, i, P, big, 0),
         MOVA_ERR_INVALID_ARG);
  expect("compact workspace",
         mova_paged_compact(i, 4, 16, 10, i, i, i, i, 40, i, i + 1, i, i, 40, 0, i, i, i, i, P, 16, 0),
         MOVA_ERR_WORKSPACE);
  for (int nb = 0; nb <= 1 << 20; nb = 3 * nb + 1)
    if (mova_paged_free_workspace_bytes(nb) == (size_t)-1 ||
        mova_paged_compact_workspace_bytes(nb) == (size_t)-1)
      bad = 1;
  expect("copy none", mova_paged_copy(i, i, 0, NULL, P, P, NULL, 0, 40, 16, 8, 128, 0), MOVA_OK);
  expect("copy pools", mova_paged_copy(i, i, 3, NULL, NULL, NULL, NULL, 0, 40, 16, 8, 128, 0),
         MOVA_ERR_INVALID_ARG);
  if (!bad) printf("chunk asan driver: ok\n");
  return bad;
}
