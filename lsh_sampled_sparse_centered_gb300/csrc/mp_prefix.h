// The attention over shared prefixes: what its translation units share.
#pragma once

#include "mp_cache.cuh"

namespace mp {

constexpr int kFewRows = 32;    // query rows of a unit of k_prefix_few
constexpr int kFewRows32 = 16;  // and of k_prefix_few32

// Units: up to 32 rows each of groups over their prefixes (none: groups = 0) and of sequences over their own slots.
struct PrefixFew {
  ChunkArgs pre, own;  // part and ml: slices [..][total_q][q_heads]
  int groups;
  bool own_units;
  int most_shared, most_own;          // pieces of a unit
  int pre_blocks, own_blocks;         // units of a group or sequence and KV head, at most
  int32_t *pre_pieces, *own_pieces;   // [groups or batch][kv_heads][blocks]
};
cudaError_t launch_prefix_few(const PrefixFew& a, int rows, cudaStream_t st);
// The prefixes of `a` in slices on large tiles, and beside them the own slots of `few` (no groups).
cudaError_t launch_prefix_slices(const ChunkArgs& a, const PrefixFew& few, int rows, cudaStream_t st);
cudaError_t launch_prefix_few32(const PrefixFew& a, int rows, cudaStream_t st);  // fp32, up to kFewRows32 rows
// Whether a pass with these limits goes through it.
bool prefix_is_few(const mp_cache_config* c, int max_q, int max_kv);
inline int few_blocks(int group, int max_q) { return int((int64_t(max_q) * group + kFewRows - 1) / kFewRows); }
// The most pieces of a unit, and the most that this times total_q comes to for limits that are at most these.
int prefix_few_pieces(const mp_cache_config* c, int total_q, int max_kv);
int64_t prefix_few_rows_most(const mp_cache_config* c, int total_q, int max_kv);

}  // namespace mp
