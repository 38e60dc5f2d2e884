// Host run of seq_of (csrc/mp_cache.cuh): whatever the lengths and limits, every row that a
// call takes sees the slots up to its own, cut at the call's limits, and a cut moves no row to
// another slot. Prints "ok" or the first failure.
#include <algorithm>
#include <cstdio>
#include <vector>

#include "mp_cache.cuh"

using namespace mp;

static uint32_t rng_state = 987;
static uint32_t rnd() {
  rng_state = rng_state * 1664525u + 1013904223u;
  return rng_state >> 8;
}
static int wild(int limit) {
  switch (rnd() % 8) {
    case 0: return int(rnd()) - 8000000;
    case 1: return INT32_MAX;
    case 2: return INT32_MIN;
    case 3: return limit;
    case 4: return limit + int(rnd() % 9);
    default: return int(rnd() % uint32_t(limit + 1));
  }
}

int main() {
  for (int trial = 0; trial < 400000; ++trial) {
    CacheArgs c = {};
    c.batch = 1 + rnd() % 3;
    c.kvh = 1;
    c.group = 1;
    c.d = 64;
    c.page_size = 16;
    c.cols = trial % 7 == 0 ? 1 << 26 : 1 + rnd() % 6;  // up to 2^30 slots
    c.n_pages = 4;
    c.page_shift = 4;
    c.total_q = trial % 7 == 1 ? 1 << 30 : rnd() % 60;
    c.max_q = trial % 7 == 1 ? 1 << 30 : 1 + rnd() % 40;
    const int slots = c.cols * c.page_size;
    c.max_kv = trial % 3 ? 1 + int(rnd() % uint32_t(slots)) : slots;
    std::vector<int32_t> cu(c.batch + 1), kv(c.batch);
    for (auto& v : cu) v = wild(c.total_q);
    if (trial % 2) std::sort(cu.begin(), cu.end());
    for (auto& v : kv) v = wild(c.max_kv);
    c.cu_q = cu.data();
    c.kv_len = kv.data();
    for (int b = 0; b < c.batch; ++b) {
      const Seq s = seq_of(c, b);
      const int64_t cut = std::max<int64_t>(0, std::min<int64_t>(kv[b], std::min<int64_t>(c.max_kv, slots)));
      int64_t most = 0;
      for (int k = 0; k < 8 && s.m > 0; ++k) {
        const int i = k == 0 ? 0 : k == 1 ? s.m - 1 : int(rnd() % uint32_t(s.m));
        const int64_t slot = int64_t(kv[b]) - cu[b + 1] + s.row0 + i;
        const int64_t want = std::max<int64_t>(0, std::min(cut, slot + 1));
        const int see = std::min(s.n, s.first + i + 1);  // in 32 bits, as the kernels have it
        if (std::max(0, see) != want) {
          std::printf("trial %d: row %d of %d sees %d slots, not %lld\n", trial, i, s.m, see, (long long)want);
          return 1;
        }
        most = std::max(most, want);
      }
      if (s.m > 0 && most != s.seen()) {
        std::printf("trial %d: %d slots seen, the last row sees %lld\n", trial, s.seen(), (long long)most);
        return 1;
      }
    }
  }
  std::printf("ok\n");
  return 0;
}
