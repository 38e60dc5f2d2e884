// The attention over shared prefixes: what its translation units share.
#pragma once

#include "mp_cache.cuh"

namespace mp {

// Units: blocks of rows of groups over their prefixes (none: groups = 0) and of sequences over their own slots.
struct PrefixFew {
  ChunkArgs pre, own;  // part and ml: slices [..][total_q][q_heads]
  int groups;
  bool own_units;
  int most_shared, most_own;          // pieces of a unit
  int pre_keys, own_keys;             // numbers of pieces that a KV head has place for
  int32_t *pre_pieces, *own_pieces;   // [kv_heads][keys]: at piece_key()
};
// Where the number of pieces of a block of rows is kept: block `block` (of `rows` rows each) of the group or
// sequence `unit` whose first packed row is `row0`. No two of them meet where no packed row is in two.
#ifdef __CUDACC__
__host__ __device__ __forceinline__ int piece_key(int row0, int group, int rows, int block, int unit) { return row0 * group / rows + block + unit; }
#endif
inline int64_t piece_keys(const mp_cache_config* c, int total_q, int rows) { return int64_t(total_q) * (c->q_heads / c->kv_heads) / rows + c->batch + 1; }

cudaError_t launch_prefix_few(const PrefixFew& a, int rows, cudaStream_t st);  // bf16, in blocks of 8, 16 or (d = 64) 32 rows
// The prefixes of `a` in slices on large tiles, and beside them the own slots of `few` (no groups).
cudaError_t launch_prefix_slices(const ChunkArgs& a, const PrefixFew& few, int rows, cudaStream_t st);
cudaError_t launch_prefix_few32(const PrefixFew& a, int rows, cudaStream_t st);  // fp32, up to 4, 8 or 16 rows
cudaError_t launch_prefix_simt(const PrefixFew& a, cudaStream_t st);             // fp32, in blocks of kChunkRows
// Whether prefixes with these limits go through launch_prefix_few, in blocks of `rows`.
bool prefix_is_few(const mp_cache_config* c, int max_q, int max_kv, int rows);
// The most pieces of a unit, and the most that this times total_q comes to for limits that are at most these.
int prefix_few_pieces(const mp_cache_config* c, int total_q, int max_kv);
int64_t prefix_few_rows_most(const mp_cache_config* c, int total_q, int max_kv);

}  // namespace mp
