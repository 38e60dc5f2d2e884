// Prefixes in slices on large tiles, and beside them the own slots: the rules, and heads of 128.
#include "mp_prefix_tc.cuh"

namespace mp {

// Tiles of groups of at most max_q rows in all their KV heads, of total_q rows altogether.
static int64_t prefix_tiles(const mp_cache_config* c, int total_q, int max_q) {
  const int64_t group = c->q_heads / c->kv_heads, each = (max_q * group + kRows - 1) / kRows;
  return c->kv_heads * std::min(c->batch * each, c->batch + total_q * group / kRows);
}
// Slices are taken where a group's rows fit one half, and otherwise where there are at most half as many
// tiles as SMs: more keep each other's keys in L2 as they are, and equal runs leave no CTA idle.
bool prefix_in_slices(const mp_cache_config* c, int total_q, int max_q) {
  return int64_t(max_q) * (c->q_heads / c->kv_heads) <= 128 || 2 * prefix_tiles(c, total_q, max_q) <= device_sm_count();
}
// Two pieces a CTA where all groups have as many tiles as the largest, one a CTA at most.
int prefix_slices(const mp_cache_config* c, int max_q, int max_kv) {
  const int sms = device_sm_count(), tiles = int((int64_t(max_q) * (c->q_heads / c->kv_heads) + kRows - 1) / kRows);
  const int most = std::min((max_kv + kKeys - 1) / kKeys, (sms + c->kv_heads - 1) / c->kv_heads);
  return std::max(1, std::min(most, int((2 * int64_t(sms) + int64_t(c->kv_heads) * tiles - 1) / (int64_t(c->kv_heads) * tiles))));
}

cudaError_t launch_prefix_slices_64(const PrefixArgs& a, const PrefixFew& few, int rows, cudaStream_t st);
cudaError_t launch_prefix_slices(const PrefixArgs& a, const PrefixFew& few, int rows, cudaStream_t st) {
  return a.c.d == 128 ? launch_slices_of<128>(a, few, rows, st) : launch_prefix_slices_64(a, few, rows, st);
}

}  // namespace mp
