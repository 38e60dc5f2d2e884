/* A plain C99 caller of the cache operators: includes the public header, links the shared
 * library and exercises what needs no GPU. Prints one "name value" line per check;
 * tests/test_cache_edges_cpu.py compiles it, runs it and compares with the Python binding. */
#include <stddef.h>
#include <stdio.h>
#include <string.h>

#include "magicpig.h"

int main(void) {
  /* never dereferenced: every call below fails validation before touching memory */
  void* fake = (void*)(size_t)(1u << 20);
  mp_cache_config c;
  mp_rotary r;
  uint64_t bytes = 0;
  memset(&c, 0, sizeof c);
  memset(&r, 0, sizeof r);
  c.batch = 2;
  c.kv_heads = 2;
  c.q_heads = 8;
  c.head_dim = 128;
  c.page_size = 4096;
  c.n_pages = 20;
  c.max_pages = 8;
  c.dtype = MP_DTYPE_BF16;
  r.rot_dim = 128;
  r.eps = 1e-6f;
  printf("sizeof_cache_config %u\n", (unsigned)sizeof c);
  printf("offset_dtype %u\n", (unsigned)offsetof(mp_cache_config, dtype));
  printf("sizeof_rotary %u\n", (unsigned)sizeof r);
  printf("offset_eps %u\n", (unsigned)offsetof(mp_rotary, eps));
  printf("check_ok %d\n", mp_cache_config_check(&c));
  printf("check_null %d\n", mp_cache_config_check(NULL));
  printf("chunk_bytes_rc %d\n", mp_chunk_workspace_bytes(&c, 2, 1, 5000, &bytes));
  printf("chunk_bytes %llu\n", (unsigned long long)bytes);
  printf("evict_bytes_rc %d\n", mp_evict_workspace_bytes(&c, 5000, 100, &bytes));
  printf("evict_bytes %llu\n", (unsigned long long)bytes);
  printf("append_rotary %d\n", mp_cache_append(&c, NULL, fake, 1024, fake, 256, fake, 256, NULL, NULL, (const double*)fake, NULL,
                                               (const int32_t*)fake, (const int32_t*)fake, 5, fake, fake, (const int32_t*)fake, fake,
                                               NULL, NULL));
  printf("append_empty %d\n", mp_cache_append(&c, &r, fake, 1024, fake, 256, fake, 256, NULL, NULL, (const double*)fake, NULL,
                                              (const int32_t*)fake, (const int32_t*)fake, 0, fake, fake, (const int32_t*)fake, fake, NULL,
                                              NULL));
  printf("attention_scratch %d\n",
         mp_chunk_attention(&c, fake, (const int32_t*)fake, (const int32_t*)fake, 2, 1, 5000, fake, fake, (const int32_t*)fake, fake,
                            (float*)fake, fake, 0, NULL, NULL));
  printf("weights_capacity %d\n", mp_cache_weights(&c, fake, (const float*)fake, (const int32_t*)fake, (const int32_t*)fake, 2, 1, 40000, fake,
                                                   (const int32_t*)fake, (float*)fake, NULL, NULL));
  printf("evict_budget %d\n",
         mp_cache_evict(&c, &c, fake, fake, (const int32_t*)fake, (const int32_t*)fake, 5000, (const float*)fake, 4, 64, 60, fake, fake,
                        (const int32_t*)fake, NULL, (int32_t*)fake, NULL, fake, 1u << 30, NULL, NULL));
  printf("bits %u %u\n", (unsigned)MP_STATUS_BAD_PAGE, (unsigned)MP_STATUS_BAD_LENGTH);
  return 0;
}
