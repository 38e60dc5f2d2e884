// Host run of the join's index arithmetic (csrc/mp_prefix.h): a kernel whose waits ran out leaves numbers of pieces
// unwritten, and whatever the workspace held in their place, every row of the sums that is named lies inside it.
// Proper numbers lead to as many rows as they say. Prints "ok" or the first failure.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "mp_prefix.h"

using namespace mp;

static uint32_t rng_state = 815;
static uint32_t rnd() {
  rng_state = rng_state * 1664525u + 1013904223u;
  return rng_state >> 8;
}
static int32_t left_over() {  // of an earlier call: sums, numbers, anything
  switch (rnd() % 6) {
    case 0: return INT32_MIN;
    case 1: return INT32_MAX;
    case 2: return int32_t(rnd() % 8) - 4;
    case 3: {
      const float x = (rnd() % 2 ? -1.f : 1.f) * (0.5f + float(rnd() % 1000) / 500.f);
      int32_t v;
      std::memcpy(&v, &x, 4);
      return v;
    }
    default: return int32_t(rnd() << 8 | rnd() % 256);
  }
}

#define CHECK(x)                                                          \
  do {                                                                    \
    if (!(x)) {                                                           \
      std::printf("failed: %s (line %d, trial %d)\n", #x, __LINE__, trial); \
      return 1;                                                           \
    }                                                                     \
  } while (0)

// Every row of the two sequences of one group, over sums of `total` rows.
template <bool TILES>
int walk(int trial, const CacheArgs& c, const Slices& sl, int prefix_rows, int64_t total, bool proper, int want) {
  const int qh = c.kvh * c.group;
  const Seq group = {0, prefix_rows, 100, 100};
  for (int b = 0; b < 2; ++b) {
    const Seq s = {b * 3, 3, 50, 47};
    for (int i = 0; i < 3 * qh + 2; ++i) {
      RowSums<TILES> r;
      r.place(c, sl, s, b, group, 0, i, 3 * qh);
      r.find(sl);
      CHECK((r.row < 0) == (i >= 3 * qh));
      CHECK(r.there >= 0 && r.all >= r.there);
      CHECK(int64_t(r.all) <= int64_t(sl.shared) + sl.own + 2 * sl.slots);
      for (int k = 0; k < r.all; ++k) {
        const int64_t at = r.at(sl, int64_t(c.total_q) * qh, k);
        CHECK(at >= 0 && at < total);
      }
      if (proper && r.row >= 0) CHECK(r.all - r.there == want && r.there == (b * 3 + i / qh < prefix_rows ? want : 0));
    }
  }
  return 0;
}

int main() {
  for (int trial = 0; trial < 60000; ++trial) {
    const bool proper = trial % 4 == 0;
    CacheArgs c;
    c.kvh = 1 + rnd() % 3;
    c.group = 1 + rnd() % 5;
    c.total_q = 6 + rnd() % 3;
    Slices sl;
    sl.pre_tiles = rnd() % 2;
    sl.own_tiles = rnd() % 2;
    sl.shared = sl.pre_tiles ? 1 : 1 + rnd() % 9;
    sl.own = sl.own_tiles ? 1 : 1 + rnd() % 9;
    sl.own_rows = sl.own_tiles ? kTileRows : 4 << rnd() % 3;
    sl.pre_rows = sl.pre_tiles ? kTileRows : 4 << rnd() % 3;
    const bool by_group = !sl.pre_tiles && rnd() % 2;  // prefixes in slices
    sl.own_keys = c.total_q * c.group / sl.own_rows + 3;
    sl.pre_keys = by_group ? 0 : c.total_q * c.group / sl.pre_rows + 3;
    sl.slot_rows = 6 * c.group;
    sl.slots = 2 + rnd() % 12;
    const int64_t rows = int64_t(c.total_q) * c.kvh * c.group;
    sl.cut = (sl.shared + sl.own) * rows;
    const int want = proper ? 1 : 0;
    std::vector<int64_t> own(sl.own_keys * c.kvh), pre((sl.pre_keys ? sl.pre_keys : 1) * c.kvh);  // two numbers each
    for (auto* v : {&own, &pre})
      for (auto& x : *v) {
        const int32_t y[2] = {proper ? want : left_over(), proper ? want : left_over()};
        std::memcpy(&x, y, 8);
      }
    sl.own_pieces = reinterpret_cast<int32_t*>(own.data());
    sl.pre_pieces = reinterpret_cast<int32_t*>(pre.data());
    const int64_t total = sl.cut + int64_t(sl.slots) * sl.slot_rows;
    const int prefix_rows = rnd() % 7;
    if (sl.pre_tiles || sl.own_tiles ? walk<true>(trial, c, sl, prefix_rows, total, proper, want)
                                     : walk<false>(trial, c, sl, prefix_rows, total, proper, want))
      return 1;
  }
  std::printf("ok\n");
  return 0;
}
