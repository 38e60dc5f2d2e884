/* The planning of a step, the attention over shared prefixes and the rotation of cached keys from a C99
 * caller: prints what the calls that need no GPU answer, for the test to compare. */
#include <stdio.h>
#include <string.h>

#include "magicpig.h"

int main(void) {
  mp_cache_config c;
  mp_rotary r;
  uint64_t bytes = 0;
  char* const at = (char*)(1 << 20); /* never dereferenced: validation fails first */
  void* const fake = at;
  int32_t* const ints = (int32_t*)fake;
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
  printf("plan_overlap %d\n", mp_cache_plan(&c, ints, NULL, ints, ints, 5, ints, ints, ints, ints, ints, NULL, NULL, NULL, NULL, NULL));
  printf("plan_sequences %d\n", MP_PLAN_SEQUENCES);
  printf("prefix_bytes_rc %d\n", mp_prefix_workspace_bytes(&c, &c, 2, 1, 5000, 2, 9000, &bytes));
  printf("prefix_bytes %llu\n", (unsigned long long)bytes);
  printf("prefix_scratch %d\n",
         mp_prefix_attention(&c, &c, fake, ints, ints, 2, 1, 5000, fake, fake, ints, ints, ints, 2, 9000, fake, fake, ints, fake, (float*)fake,
                             fake, 0, NULL, NULL));
  printf("rotate_capacity %d\n", mp_cache_rotate(&c, &r, fake, ints, ints, 40000, NULL, NULL, NULL, NULL, 1, 0, 1.0f, NULL, NULL));
  printf("rotate_nothing %d\n", mp_cache_rotate(&c, &r, fake, ints, ints, 400, NULL, NULL, NULL, NULL, 1, 0, 1.0f, NULL, NULL));
  printf("bit %u\n", (unsigned)MP_STATUS_NO_ROOM);
  return 0;
}
