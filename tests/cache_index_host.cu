// Host run of the cache operators' index arithmetic (csrc/mp_cache.cuh): sequences and
// page numbers read from device memory may hold anything, and whatever they hold, every
// row and slot that comes out lies inside its buffer. Prints "ok" or the first failure.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "mp_cache.cuh"

using namespace mp;

static uint32_t rng_state = 12345;
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
    const int batch = 1 + rnd() % 4, kvh = 1 + rnd() % 3, cols = 1 + rnd() % 5, ps = 16 * (1 + rnd() % 8);
    const int pages = 1 + rnd() % 9, total = rnd() % 50, max_q = 1 + rnd() % 20;
    const int max_kv = 1 + rnd() % (cols * ps);
    std::vector<int32_t> table(batch * cols), cu(batch + 1), kv(batch);
    for (auto& v : table) v = wild(pages);
    for (auto& v : cu) v = wild(total);
    for (auto& v : kv) v = wild(max_kv);
    uint32_t status = 0;
    CacheArgs c;
    c.batch = batch;
    c.kvh = kvh;
    c.group = 2;
    c.d = 64;
    c.page_size = ps;
    c.n_pages = pages;
    c.cols = cols;
    c.page_shift = -1;
    for (int i = 0; i < 31; ++i)
      if (ps == 1 << i) c.page_shift = i;
    c.table = table.data();
    c.cu_q = cu.data();
    c.kv_len = kv.data();
    c.total_q = total;
    c.max_q = max_q;
    c.max_kv = max_kv;
    c.status = &status;
    bool proper = cu[0] >= 0;
    for (int b = 0; b < batch; ++b) {
      const Seq s = seq_of(c, b);
      CHECK(s.n >= 0 && s.n <= max_kv && s.m >= 0 && s.m <= max_q);
      CHECK(s.row0 >= 0 && s.row0 + s.m <= total);
      const bool cut = s.n != kv[b] || s.row0 != cu[b] || int64_t(s.row0) + s.m != cu[b + 1];
      CHECK(!cut || (status & MP_STATUS_BAD_LENGTH));
      proper = proper && cu[b + 1] >= cu[b];
      const int64_t end = int64_t(pages) * kvh * ps * c.d;
      for (int i = 0; i < 3 && s.n > 0; ++i) {
        const int slot = int(rnd() % uint32_t(s.n)), h = int(rnd() % uint32_t(kvh));
        const int64_t at = slot_read(c, b, h, slot);
        CHECK(at >= 0 && at + c.d <= end);
        const int p = table[b * cols + slot / ps];
        CHECK((p >= 0 && p < pages) || (status & MP_STATUS_BAD_PAGE));
        if (p >= 0 && p < pages) CHECK(at == ((int64_t(p) * kvh + h) * ps + slot % ps) * c.d);
      }
    }
    for (int r = 0; r < total; ++r) {
      const int b = seq_at(c, r);
      CHECK(b >= -1 && b < batch);
      if (b >= 0) CHECK(cu[b] <= r && r < cu[b + 1]);
      if (b < 0 && proper)
        for (int i = 0; i < batch; ++i) CHECK(!(cu[i] <= r && r < cu[i + 1]));
    }
  }
  std::printf("ok\n");
  return 0;
}
