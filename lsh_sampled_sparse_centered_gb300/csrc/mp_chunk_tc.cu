// Host side of the attention on large tiles: a chunk over its slots, and groups' prefixes beside them.
#include "mp_chunk_tc.cuh"

namespace mp {

// One CTA per SM, or fewer when the limits leave fewer runs of units than that.
int chunk_tc_ctas(int batch, int kvh, int group, int max_q, int max_kv) {
  const int64_t tiles = (int64_t(max_q) * group + kRows - 1) / kRows;
  const double units = double(std::min(batch, kGroup)) * kvh * double(tiles) * ((max_kv + kKeys - 1) / kKeys);
  return int(std::max(1.0, std::min(double(device_sm_count()), units / kMinRun + 1.0)));
}

uint64_t chunk_tc_workspace(const mp_cache_config* c, int max_q, int max_kv) {
  const int group = c->q_heads / c->kv_heads, ctas = chunk_tc_ctas(c->batch, c->kv_heads, group, max_q, max_kv);
  const uint64_t rows = uint64_t(2 * ctas) * slot_rows_of(group, max_q);
  return align256(uint64_t(ctas) * sizeof(Cut)) + align256(rows * 8) + align256(rows * c->head_dim * 4);
}

static int both_ctas(int own, int pre) { return std::min(own + pre, device_sm_count()); }
uint64_t both_tc_rows(const mp_cache_config* own, int max_q, int max_kv, const mp_cache_config* pre, int max_group_q, int max_prefix) {
  const mp_cache_config* any = own ? own : pre;
  const int group = any->q_heads / any->kv_heads;
  const int ctas = both_ctas(own ? chunk_tc_ctas(own->batch, own->kv_heads, group, max_q, max_kv) : 0,
                             pre ? chunk_tc_ctas(pre->batch, pre->kv_heads, group, max_group_q, max_prefix) : 0);
  const int launches = ((own ? own->batch : 0) + (pre ? pre->batch : 0) + kGroup - 1) / kGroup;
  return uint64_t(2 * ctas) * launches * slot_rows_of(group, std::max(own ? max_q : 1, pre ? max_group_q : 1));
}

cudaError_t launch_chunk_tc(const ChunkArgs& a, void* workspace, cudaStream_t st) {
  const CacheCall& c = a.c;
  const int ctas = chunk_tc_ctas(c.batch, c.kvh, c.group, c.max_q, c.max_kv), slot_rows = slot_rows_of(c.group, c.max_q);
  return c.d == 128 ? launch<128, kChunk, 0>(a, {}, c.batch, ctas, slot_rows, workspace, st)
                    : launch<64, kChunk, 0>(a, {}, c.batch, ctas, slot_rows, workspace, st);
}

cudaError_t launch_both_tc(const PrefixArgs& a, bool own, const PrefixArgs* shared, const TilePieces& at, cudaStream_t st) {
  const CacheArgs& c = a.c;
  Extra<kBoth> x = {};
  int own_ctas = 0, pre_ctas = 0, units = 0, max_q = 1;
  if (own) {
    units = c.batch;
    own_ctas = chunk_tc_ctas(c.batch, c.kvh, c.group, c.max_q, c.max_kv);
    max_q = c.max_q;
  }
  if (shared) {
    const CacheArgs& p = shared->c;
    x.pre.c = p;
    x.pre.groups = p.batch;
    x.pre.box = box_rows(p.table, p.page_size);
    const uint64_t rows = uint64_t(p.n_pages) * p.kvh * p.page_size;
    if (!make_map(&x.k, shared->keys, p.d, rows, 64, x.pre.box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&x.v, shared->values, p.d, rows, 64, x.pre.box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
    units += p.batch;
    pre_ctas = chunk_tc_ctas(p.batch, p.kvh, p.group, p.max_q, p.max_kv);
    max_q = std::max(max_q, p.max_q);
  }
  x.pre.own_slice = a.own_slice;
  x.pre.pre_keys = at.pre_keys;
  x.pre.own_keys = at.own_keys;
  x.pre.pre_pieces = at.pre_pieces;
  x.pre.own_pieces = at.own_pieces;
  const int slot_rows = slot_rows_of(c.group, max_q), ctas = both_ctas(own_ctas, pre_ctas);
  return c.d == 128 ? launch<128, kBoth, 0>(a, x, units, ctas, slot_rows, nullptr, st)
                    : launch<64, kBoth, 0>(a, x, units, ctas, slot_rows, nullptr, st);
}

}  // namespace mp
