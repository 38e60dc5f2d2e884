// The attention over shared prefixes: what its translation units share.
#pragma once

#include "mp_cache.cuh"

namespace mp {

constexpr int kFewRows = 32;  // query rows of a KV head that go through k_prefix_few

// Units with few rows: groups over their prefixes (none: groups = 0) and sequences over their own slots.
struct PrefixFew {
  ChunkArgs pre, own;  // part and ml: slices [..][total_q][q_heads]
  int groups;
  bool own_units;
  int most_shared, most_own;          // pieces of a unit
  int32_t *pre_pieces, *own_pieces;   // [groups or batch][kv_heads]
};
cudaError_t launch_prefix_few(const PrefixFew& a, int rows, cudaStream_t st);
// The most pieces of a unit, and the most that this times total_q comes to for limits that are at most these.
int prefix_few_pieces(const mp_cache_config* c, int total_q, int max_kv);
int64_t prefix_few_rows_most(const mp_cache_config* c, int total_q, int max_kv);

}  // namespace mp
