// Host run of the groups' index arithmetic (csrc/mp_cache.cuh): whatever cu_group, cu_q and the lengths
// hold, a group's rows and slots lie inside their buffers, and proper ones come out as they are. Prints
// "ok" or the first failure.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "mp_cache.cuh"

using namespace mp;

static uint32_t rng_state = 4711;
static uint32_t rnd() {
  rng_state = rng_state * 1664525u + 1013904223u;
  return rng_state >> 8;
}
static int wild(int limit) {  // mostly near the limits, sometimes far outside
  switch (rnd() % 8) {
    case 0: return int(rnd()) - 8000000;
    case 1: return INT32_MAX;
    case 2: return INT32_MIN;
    case 3: return -1;
    case 4: return limit;
    case 5: return limit + 1;
    default: return int(rnd() % uint32_t(limit + 1));
  }
}

#define CHECK(x)                                                   \
  do {                                                             \
    if (!(x)) {                                                    \
      std::printf("failed: %s (line %d, trial %d)\n", #x, __LINE__, trial); \
      return 1;                                                    \
    }                                                              \
  } while (0)

int main() {
  for (int trial = 0; trial < 200000; ++trial) {
    const bool proper = trial % 2;
    const int batch = 1 + rnd() % 6, groups = 1 + rnd() % 4, cols = 1 + rnd() % 5, ps = 16 * (1 + rnd() % 8), total = rnd() % 50;
    std::vector<int32_t> cu(batch + 1), cg(groups + 1), lens(groups);
    const int max_q = proper ? total + 1 : 1 + rnd() % 20, max_kv = 1 + rnd() % (cols * ps);
    for (auto& v : cu) v = wild(total);
    for (auto& v : cg) v = wild(batch);
    for (auto& v : lens) v = wild(max_kv);
    if (proper) {
      cu[0] = cg[0] = 0;
      for (int b = 1; b <= batch; ++b) cu[b] = cu[b - 1] + int(rnd() % uint32_t(total - cu[b - 1] + 1));
      for (int g = 1; g <= groups; ++g) cg[g] = cg[g - 1] + int(rnd() % uint32_t(batch - cg[g - 1] + 1));
      for (auto& v : lens) v = int(rnd() % uint32_t(max_kv + 1));
    }
    uint32_t status = 0;
    CacheArgs c;
    c.batch = groups;
    c.kvh = 2;
    c.group = 3;
    c.d = 64;
    c.page_size = ps;
    c.n_pages = 9;
    c.cols = cols;
    c.page_shift = -1;
    c.table = nullptr;
    c.cu_q = cu.data();
    c.kv_len = lens.data();
    c.total_q = total;
    c.max_q = max_q;
    c.max_kv = max_kv;
    c.status = &status;
    CHECK(c.cu_group == nullptr);  // what the other operators leave it at
    c.cu_group = cg.data();
    c.sequences = batch;
    for (int g = 0; g < groups; ++g) {
      const Seq s = group_of(c, g);
      CHECK(s.n >= 0 && s.n <= max_kv && s.m >= 0 && s.m <= max_q);
      CHECK(s.row0 >= 0 && s.row0 + s.m <= total);
      CHECK(s.first == s.n && s.seen() == s.n);  // every row sees every slot
      if (proper) CHECK(s.row0 == cu[cg[g]] && s.row0 + s.m == cu[cg[g + 1]] && s.n == lens[g]);
    }
    if (proper) CHECK(status == 0);
  }
  std::printf("ok\n");
  return 0;
}
