/* A C11 client of the paged cache: it includes only sv_cache.h, takes the
 * address of every entry point the header declares and exercises their
 * host-only paths (frequencies, workspace sizes, argument checks).  One "name
 * value" line per result on stdout. */
#include <stdio.h>

#include "sv_cache.h"

typedef void (*any_fn)(void);

int main(void) {
  const struct {
    const char *name;
    any_fn fn;
  } entry[] = {
      {"sv_rotary_turns", (any_fn)sv_rotary_turns},
      {"sv_rotary", (any_fn)sv_rotary},
      {"sv_cache_append", (any_fn)sv_cache_append},
      {"sv_paged_attention_workspace", (any_fn)sv_paged_attention_workspace},
      {"sv_paged_attention", (any_fn)sv_paged_attention},
      {"sv_cache_commit", (any_fn)sv_cache_commit},
  };
  for (size_t k = 0; k < sizeof(entry) / sizeof(entry[0]); ++k)
    printf("linked %s %d\n", entry[k].name, entry[k].fn != NULL);
  const double f[2] = {6.283185307179586477 / 4, -6.283185307179586477 / 8};
  uint64_t turns[2];
  printf("turns %d\n", sv_rotary_turns(f, 2, turns));
  printf("quarter %d\n", turns[0] == (uint64_t)1 << 62);
  printf("back %d\n", turns[1] == (uint64_t)7 << 61);
  printf("struct_bytes %zu\n", sizeof(sv_paged_cache));
  printf("attention_ws %zu\n", sv_paged_attention_workspace(64, 9, 32, 8, 128, 8192, 1024));
  printf("attention_ws_bad %zu\n", sv_paged_attention_workspace(64, 9, 32, 7, 128, 8192, 1024));
  printf("rotary_null %d\n", sv_rotary(NULL, 0, NULL, 0, SV_DT_F32, NULL, 64, 0, 0, 1.0f, NULL, NULL, NULL, 1, 1, 1, 64, NULL));
  printf("append_null %d\n", sv_cache_append(NULL, NULL, 0, 1, NULL, NULL, NULL, NULL, NULL, 0, NULL, 0, NULL, 0, NULL, 0, SV_DT_BF16,
                                             NULL, 0, 0, 1.0f, 1, 1, 0, NULL));
  printf("attention_null %d\n", sv_paged_attention(NULL, 0, SV_DT_BF16, NULL, NULL, 0, 1, NULL, 0, NULL, NULL, NULL, 1, 1, 8, 8, 1.0f,
                                                   NULL, NULL, NULL, 0, NULL));
  printf("commit_null %d\n", sv_cache_commit(NULL, 1, 0, NULL, 0, 1, NULL, NULL, 0, 0, NULL, 1, 1, NULL, NULL));
  return 0;
}
