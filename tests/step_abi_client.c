/* A C11 client of the step operators: it includes only sv_step.h, takes the
 * address of every entry point the header declares and exercises their
 * host-only paths (workspace sizes, argument checks).  One "name value" line
 * per result on stdout. */
#include <stdio.h>

#include "sv_step.h"

typedef void (*any_fn)(void);

int main(void) {
  const struct {
    const char *name;
    any_fn fn;
  } entry[] = {
      {"sv_adjust_logits", (any_fn)sv_adjust_logits},
      {"sv_lmhead_quant", (any_fn)sv_lmhead_quant},
      {"sv_lmhead_quant_workspace", (any_fn)sv_lmhead_quant_workspace},
      {"sv_attention_workspace", (any_fn)sv_attention_workspace},
      {"sv_attention", (any_fn)sv_attention},
  };
  for (size_t k = 0; k < sizeof(entry) / sizeof(entry[0]); ++k)
    printf("linked %s %d\n", entry[k].name, entry[k].fn != NULL);
  printf("attention_ws %zu\n", sv_attention_workspace(64, 9, 32, 8, 128, 8192, 1024));
  printf("attention_ws_bad %zu\n", sv_attention_workspace(64, 9, 32, 7, 128, 8192, 1024));
  printf("adjust_null %d\n", sv_adjust_logits(NULL, 0, NULL, 0, SV_DT_BF16, NULL, 0, NULL, NULL, 2, 1, 100, NULL, 0, 0, NULL,
                                              NULL, NULL, NULL, NULL, NULL, NULL, 0, NULL, 0, 0, NULL));
  printf("lmhead_null %d\n", sv_lmhead_quant(NULL, 0, SV_DT_F16, NULL, NULL, NULL, 1, 64, 100, 64, NULL, 0, SV_DT_F32, NULL, 0, NULL));
  printf("lmhead_dtype %d\n", sv_lmhead_quant(NULL, 0, SV_DT_F32, NULL, NULL, NULL, 1, 64, 100, 64, NULL, 0, SV_DT_F32, NULL, 0, NULL));
  printf("attention_null %d\n", sv_attention(NULL, 0, SV_DT_BF16, NULL, NULL, 0, 0, 64, NULL, NULL, 0, 0, NULL, NULL, NULL,
                                             1, 1, 8, 8, 64, 10, 1.0f, NULL, NULL, NULL, 0, NULL));
  return 0;
}
