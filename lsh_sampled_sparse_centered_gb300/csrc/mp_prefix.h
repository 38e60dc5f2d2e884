// The attention over shared prefixes: what its translation units share.
#pragma once

#include "mp_cache.cuh"

namespace mp {

// Units: blocks of rows of groups over their prefixes (none: groups = 0) and of sequences over their own slots.
struct PrefixFew {
  PrefixArgs pre, own;  // part and ml: slices [..][total_q][q_heads]
  int groups;
  bool own_units;
  int most_shared, most_own;          // pieces of a unit
  int pre_keys, own_keys;             // numbers of pieces that a KV head has place for
  int32_t *pre_pieces, *own_pieces;   // [kv_heads][keys]: at piece_key()
#if MP_CHECK
  bool stall;  // a warp waits for bytes that never come (bf16)
#endif
};
// Where the number of pieces of a block of rows is kept: block `block` (of `rows` rows each) of the group or
// sequence `unit` whose first packed row is `row0`. No two of them meet where no packed row is in two.
#ifdef __CUDACC__
__host__ __device__ __forceinline__ int piece_key(int row0, int group, int rows, int block, int unit) { return row0 * group / rows + block + unit; }
#endif
inline int64_t piece_keys(const mp_cache_config* c, int total_q, int rows) { return int64_t(total_q) * (c->q_heads / c->kv_heads) / rows + c->batch + 1; }

cudaError_t launch_prefix_few(const PrefixFew& a, int rows, cudaStream_t st);  // bf16, in blocks of 8, 16 or (d = 64) 32 rows
// The prefixes of `a` in slices on large tiles, and beside them the own slots of `few` (no groups).
cudaError_t launch_prefix_slices(const PrefixArgs& a, const PrefixFew& few, int rows, cudaStream_t st);
cudaError_t launch_prefix_few32(const PrefixFew& a, int rows, cudaStream_t st);  // fp32, up to 4, 8 or 16 rows
cudaError_t launch_prefix_simt(const PrefixFew& a, cudaStream_t st);             // fp32, in blocks of kChunkRows
// Whether prefixes with these limits go through launch_prefix_few, in blocks of `rows`.
bool prefix_is_few(const mp_cache_config* c, int max_q, int max_kv, int rows);
// The most pieces of a unit, and the most that this times total_q comes to for limits that are at most these.
int prefix_few_pieces(const mp_cache_config* c, int total_q, int max_kv);
int64_t prefix_few_rows_most(const mp_cache_config* c, int total_q, int max_kv);

#ifdef __CUDACC__
// Slices of the two passes, and their numbers per (group or sequence, KV head) where these differ.
struct Slices {
  int shared, own;
  int32_t *pre_pieces, *own_pieces;
  int pre_keys, own_keys, pre_rows, own_rows;  // at piece_key() of blocks of so many rows (pre_keys = 0: one for [group][KV head])
  // Large tiles: their pieces instead, two numbers each (TilePieces). A cut tile's are slots of `slot_rows` rows
  // each, `slots` in all, from row `cut` of the sums on: the first piece's slot s, then s + 1, s + 3, ...
  bool pre_tiles, own_tiles;
  int slot_rows, slots;
  int64_t cut;
};

// Where the sums of a query row are: slices [0, there) of the prefix, [there, all) of the own slots.
// TILES: some passes are large tiles'.
template <bool TILES>
struct RowSums {
  int row;  // among all rows, which are 32-bit together; -1: none
  int there, all;
  const int32_t *there_at, *all_at;  // where their numbers are, if they differ
  int tile[2];                       // the row's place in its tile of the prefix, of the own slots
  int64_t from[2];                   // the first slice's row of the sums, where its tile is cut
  bool cut[2];

  // Row i of the `mine` rows of sequence b, `s`, whose group is `g`.
  __host__ __device__ __forceinline__ void place(const CacheCall& c, const Slices& sl, const Seq& s, int b, const Seq& g, int group, int i, int mine) {
    const int qh = c.kvh * c.group;
    const bool live = i < mine;
    row = live ? s.row0 * qh + i : -1;
    const int token = i / qh, in = i - token * qh, h = in / c.group, in_head = in - h * c.group, t = s.row0 + token;
    const bool shared = live && g.row0 <= t && t < g.row0 + g.m;
    const int at0 = (t - g.row0) * c.group + in_head, at1 = token * c.group + in_head;  // among the group's and the sequence's
    there = shared ? sl.shared : 0;
    all = live ? sl.own : 0;
    there_at = !shared || !sl.pre_pieces ? nullptr
               : sl.pre_pieces + (sl.pre_keys ? int64_t(h) * sl.pre_keys + piece_key(g.row0, c.group, sl.pre_rows, at0 / sl.pre_rows, group)
                                              : int64_t(group) * c.kvh + h);
    all_at = !live || !sl.own_pieces ? nullptr
             : sl.own_pieces + int64_t(h) * sl.own_keys + piece_key(s.row0, c.group, sl.own_rows, at1 / sl.own_rows, b);
    if (TILES) {
      tile[0] = at0 % kTileRows;
      tile[1] = at1 % kTileRows;
      // numbers of tiles are twice as long
      if (there_at && sl.pre_tiles) there_at += there_at - sl.pre_pieces;
      if (all_at && sl.own_tiles) all_at += all_at - sl.own_pieces;
    }
  }
  // Behind the kernels that wrote the numbers.
  __host__ __device__ __forceinline__ void find(const Slices& sl) {
    cut[0] = cut[1] = false;
    auto look = [&](const int32_t* at, bool tiles, int& n, int64_t& begin, bool& is_cut, int in_tile) {
      if (!at) return;
      // Numbers that a kernel whose waits ran out did not write are whatever the workspace held: they lead to sums
      // that are there, or to none.
      if (!TILES || !tiles) {
        n = max(0, min(n, *at));
        return;
      }
      const int2 v = *reinterpret_cast<const int2*>(at);
      n = v.x < 0 || v.x > sl.slots || (v.x > 1 && (v.y < 1 || v.y >= sl.slots || v.y + 2 * v.x - 3 >= sl.slots)) ? 0 : v.x;
      is_cut = n > 1;
      begin = sl.cut + int64_t(v.y - 1) * sl.slot_rows + in_tile;
    };
    look(there_at, sl.pre_tiles, there, from[0], cut[0], tile[0]);
    look(all_at, sl.own_tiles, all, from[1], cut[1], tile[1]);
    all += there;
  }
  // The rows of the sums; `rows` are all query rows.
  __host__ __device__ static __forceinline__ int64_t total(const Slices& sl) { return sl.cut + int64_t(sl.slots) * sl.slot_rows; }
  // The row of them that slice i is.
  __host__ __device__ __forceinline__ int64_t at(const Slices& sl, int64_t rows, int i) const {
    const bool own = i >= there;
    const int n = own ? i - there : i;
    if (TILES && (own ? cut[1] : cut[0])) return (own ? from[1] : from[0]) + int64_t(n > 0 ? 2 * n : 1) * sl.slot_rows;
    return (own ? n + sl.shared : n) * rows + row;
  }
};
#endif

}  // namespace mp
