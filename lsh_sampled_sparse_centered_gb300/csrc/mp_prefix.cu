// Attention of a batch whose sequences share prefixes: the join of its two passes, and the host side.
//
// The softmax over a row's prefix and its own slots is the join of two: every partial result is an
// unnormalised sum with its reference and its weights' sum (fp32), whatever slots it covers. So one pass
// goes over the prefixes, whose rows are those of all the sequences of a group: each prefix is read once,
// and the products have as many rows as the group has. The other goes over the sequences' own slots, as
// the attention of a chunk does. The last kernel joins both passes' slices: memory bound where there are
// many rows, and otherwise a chain of lookups (sequence, group, pieces) and loads, which it keeps short by
// having the loads of all a row's slices in flight.
#include "mp_cache_host.h"
#include "mp_prefix.h"
#include "mp_tc.cuh"

namespace mp {
namespace {

// The running join of a row: four of its columns.
struct Joined {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);

  template <int N>
  __device__ __forceinline__ void add(const float2 (&v)[N], const float4 (&x)[N]) {
    float top = m;
#pragma unroll
    for (int k = 0; k < N; ++k) top = fmaxf(top, v[k].x);
    const float ref = top == -INFINITY ? 0.f : top, before = exp2f(m - ref);  // 0 while nothing was seen
    m = top;
    l *= before;
    o.x *= before;
    o.y *= before;
    o.z *= before;
    o.w *= before;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const bool any = v[k].y != 0.f;  // a slice that saw nothing has written no sum
      const float by = any ? exp2f(v[k].x - ref) : 0.f;
      l = fmaf(v[k].y, by, l);
      o.x = any ? fmaf(x[k].x, by, o.x) : o.x;
      o.y = any ? fmaf(x[k].y, by, o.y) : o.y;
      o.z = any ? fmaf(x[k].z, by, o.z) : o.z;
      o.w = any ? fmaf(x[k].w, by, o.w) : o.w;
    }
  }
  template <typename T, int D>
  __device__ __forceinline__ void write(const PrefixArgs& a, int64_t row, int e) const {
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    if (a.lse && e == 0) a.lse[row] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * D + e) = make_uint2(bf2(o.x * inv, o.y * inv), bf2(o.z * inv, o.w * inv));
    else
      *reinterpret_cast<float4*>(static_cast<T*>(a.out) + row * D + e) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  }
};

// The group that sequence b is in, if it is in one.
__device__ __forceinline__ int group_at(const CacheArgs& prefix, int b) {
  int lo = 0, hi = prefix.batch;  // cu_group[lo] <= b is kept where it holds for 0
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix.cu_group[mid] <= b) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Joins the slices' (m, l, sum) of a sequence's query rows, in their order, where they are few: WARPS warps share
// the slices of 128 / D rows (D / 4 lanes a row, 16 bytes a lane), so that all their loads are in flight together.
// Grid: rows of a sequence x sequences, so that what has to be looked up does not hang on a row.
template <typename T, int D, int WARPS, bool TILES>
__global__ void __launch_bounds__(256, 4) k_prefix_join(const PrefixArgs a, const CacheArgs prefix, const Slices sl) {
  constexpr int kLanes = D / 4, kAtOnce = 4;
  __shared__ float4 so[8][32];
  __shared__ float2 sml[8][32];
  const CacheCall& c = a.c;
  const int qh = c.kvh * c.group, b = blockIdx.y;
  const int64_t rows = int64_t(c.total_q) * qh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = lane % kLanes * 4;
  const Seq s = seq_of(c, b);
  const int group = group_at(prefix, b);
  const Seq g = group_of(prefix, group);
  RowSums<TILES> r;
  r.place(c, sl, s, b, g, group, int(blockIdx.x * (8 / WARPS) + warp / WARPS) * (32 / kLanes) + lane / kLanes, s.m * qh);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  r.find(sl);
  Joined j;
  const int most = __reduce_max_sync(0xffffffffu, r.all);
  for (int i0 = warp % WARPS * kAtOnce; i0 < most; i0 += WARPS * kAtOnce) {
    float2 v[kAtOnce];
    float4 x[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      bool live = i0 + k < r.all;
      const int64_t at = live ? r.at(sl, rows, i0 + k) : 0;
      live = live && inside(at >= 0 && at < r.total(sl), c.status);
      v[k] = live ? *reinterpret_cast<const float2*>(a.ml + at * 2) : make_float2(-INFINITY, 0.f);
      x[k] = live ? *reinterpret_cast<const float4*>(a.part + at * D + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    j.add(v, x);
  }
  // the warps' parts, in their order
  so[warp][lane] = j.o;
  sml[warp][lane] = make_float2(j.m, j.l);
  __syncthreads();
  if (warp % WARPS != 0 || r.row < 0) return;
  float2 v[WARPS];
  float4 x[WARPS];
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    v[w] = sml[warp + w][lane];
    x[w] = so[warp + w][lane];
  }
  Joined all;
  all.add(v, x);
  all.template write<T, D>(a, r.row, e);
}

// The same where they are many: a warp looks up `each` rows at once, one a lane (what a row has to look up is
// more instructions than its join: 1264 tokens of 32 heads 37 and 31 us), and then joins them one after the other.
template <typename T, int D, bool TILES>
__global__ void __launch_bounds__(256, 4) k_prefix_join_many(const PrefixArgs a, const CacheArgs prefix, const Slices sl, const int each) {
  constexpr int kLanes = D / 4, kAtOnce = 4, kTogether = 32 / kLanes;
  const CacheCall& c = a.c;
  const int qh = c.kvh * c.group, b = blockIdx.y;
  const int64_t rows = int64_t(c.total_q) * qh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = lane % kLanes * 4;
  const Seq s = seq_of(c, b);
  const int group = group_at(prefix, b), mine = s.m * qh;
  const Seq g = group_of(prefix, group);
  int first = int(blockIdx.x * 8 + warp) * each;
  RowSums<TILES> own;
  own.place(c, sl, s, b, g, group, first + lane, lane < each ? mine : 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  while (first < mine) {
    own.find(sl);
    for (int i = 0; i < each && first + i < mine; i += kTogether) {
      const int src = i + lane / kLanes;
      RowSums<TILES> r;
      r.row = __shfl_sync(0xffffffffu, own.row, src);
      r.there = __shfl_sync(0xffffffffu, own.there, src);
      r.all = __shfl_sync(0xffffffffu, own.all, src);
      if (TILES) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          r.from[k] = __shfl_sync(0xffffffffu, own.from[k], src);
          r.cut[k] = __shfl_sync(0xffffffffu, int(own.cut[k]), src);
        }
      }
      Joined j;
      const int most = __reduce_max_sync(0xffffffffu, r.all);
      for (int i0 = 0; i0 < most; i0 += kAtOnce) {
        float2 v[kAtOnce];
        float4 x[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          bool live = i0 + k < r.all;
          const int64_t at = live ? r.at(sl, rows, i0 + k) : 0;
          live = live && inside(at >= 0 && at < r.total(sl), c.status);
          v[k] = live ? *reinterpret_cast<const float2*>(a.ml + at * 2) : make_float2(-INFINITY, 0.f);
          x[k] = live ? *reinterpret_cast<const float4*>(a.part + at * D + e) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        j.add(v, x);
      }
      if (r.row >= 0) j.template write<T, D>(a, r.row, e);
    }
    first += int(gridDim.x) * 8 * each;
    own.place(c, sl, s, b, g, group, first + lane, lane < each ? mine : 0);
  }
}

template <typename T, int D, bool TILES>
cudaError_t join(const PrefixArgs& a, const CacheArgs& prefix, const Slices& sl, cudaStream_t st) {
  const int together = 32 / (D / 4), qh = a.c.kvh * a.c.group;
  // Four warps a row where there are at most 16 rows an SM, eight where there are at most two (32 tokens of 32
  // heads: 76, 69 and 71 us a call with one, four and eight, four tokens: 18.7, 16.6 and 15.0; 1500 rows: 53 and 49
  // with one and four, 4000 rows: 43 and 50); otherwise as many rows a warp as leave each SM 64 of these batches.
  const int64_t sms = device_sm_count(), warps = int64_t(a.c.total_q) * qh / together;
  const bool few = warps <= sms * 16, least = warps <= sms * 2;
  int each = together;
  while (each < 32 && warps * together > sms * 32 * 2 * each) each *= 2;
  cudaLaunchConfig_t cfg = {};
  const int cta_rows = few ? together * (least ? 1 : 2) : 8 * each;
  cfg.gridDim = dim3(unsigned((int64_t(a.c.max_q) * qh + cta_rows - 1) / cta_rows), a.c.batch);
  // and as many CTAs as fit, twice, which take several such batches
  if (!few) cfg.gridDim.x = unsigned(std::min<int64_t>(cfg.gridDim.x, std::max<int64_t>(1, 8 * sms / a.c.batch)));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (!few) return cudaLaunchKernelEx(&cfg, k_prefix_join_many<T, D, TILES>, a, prefix, sl, int(each));
  return least ? cudaLaunchKernelEx(&cfg, k_prefix_join<T, D, 8, TILES>, a, prefix, sl) : cudaLaunchKernelEx(&cfg, k_prefix_join<T, D, 4, TILES>, a, prefix, sl);
}

cudaError_t launch_join(const PrefixArgs& a, const CacheArgs& prefix, const Slices& sl, int dtype, cudaStream_t st) {
  using B = __nv_bfloat16;
  if (sl.pre_tiles || sl.own_tiles) return a.c.d == 128 ? join<B, 128, true>(a, prefix, sl, st) : join<B, 64, true>(a, prefix, sl, st);
  if (dtype == MP_DTYPE_BF16) return a.c.d == 128 ? join<B, 128, false>(a, prefix, sl, st) : join<B, 64, false>(a, prefix, sl, st);
  return a.c.d == 128 ? join<float, 128, false>(a, prefix, sl, st) : join<float, 64, false>(a, prefix, sl, st);
}

// How the passes go, and the rows of a block where they are cut into runs (kFew, kSimt).
enum Kind {
  kFew,    // few rows per KV head: launch_prefix_few, fp32 launch_prefix_few32
  kSimt,   // fp32 with more: launch_prefix_simt
  kTiles,  // bf16 with more: large tiles, joined to one slice
  kSlices  // prefixes on large tiles in slices, and the own slots (kFew) beside them
};
struct Plan {
  Kind own, shared;
  int own_rows, pre_rows;
};
int few_rows(int64_t rows, int least) { return rows <= least ? least : (rows <= 2 * least ? 2 * least : 4 * least); }

// bf16: a block of 32 rows takes more registers than a warp has with d = 128, and beside large tiles, whose
// warps have 208, with d = 64 too. us a call, 32/8 heads, with up to 32 rows in blocks beside slices, and with
// large tiles for both from 17 rows on:
//   32 sequences of 32 rows, 300 own slots, 4000 shared, d = 128     129    68       d = 64   47    53
//   the same over 1500 own slots                                     212    95                74    68
//   64 sequences of 20 rows, 1500 own slots, 60000 shared            975   333               440   250
// and up to 16 rows in blocks, with large tiles from 9 on:
//   32 sequences of 12 rows, 300 own slots, 4000 shared, d = 128      39    58                37    45
// Where all rows are as few as a block's, both passes take it whatever the lengths (d = 64: up to 32 rows).
// Own slots in blocks and prefixes on large tiles without slices, or the other way round, are two launches.
Plan plan_of(const mp_cache_config* c, const mp_cache_config* p, int total_q, int max_q, int max_group_q, int max_prefix) {
  const int64_t group = c->q_heads / c->kv_heads, own = max_q * group, pre = max_group_q * group, both = std::max(own, pre);
  if (c->dtype != MP_DTYPE_BF16) {
    constexpr int kMost = 16;
    const int rows = few_rows(pre <= kMost ? (own <= kMost ? both : pre) : own, 4);
    return {own <= kMost ? kFew : kSimt, pre <= kMost ? kFew : kSimt, own <= kMost ? rows : kChunkRows, pre <= kMost ? rows : kChunkRows};
  }
  const int most = c->head_dim == 128 ? 16 : 32;
  if (both <= most) return {kFew, kFew, few_rows(both, 8), few_rows(both, 8)};
  const int rows = few_rows(own, 8);
  const bool few = own <= most && prefix_is_few(p, max_group_q, max_prefix, rows);
  if (few || (own <= 16 && prefix_in_slices(p, total_q, max_group_q))) return {kFew, few ? kFew : kSlices, rows, rows};
  if (own <= 16) return {kFew, kTiles, rows, kTileRows};
  return {kTiles, kTiles, kTileRows, kTileRows};
}
// The most slices of a pass.
int slices_of(Kind kind, const mp_cache_config* c, int total_q, int max_q, int max_kv) {
  if (kind == kTiles) return 1;
  if (kind != kSlices) return prefix_few_pieces(c, total_q, max_kv);
  // as many fewer where most packed rows belong to no sequence
  return std::max(1, int(prefix_slices(c, max_q, max_kv) * part_rows(c, total_q, max_q) / total_q));
}
// The most that slices_of() * total_q comes to for limits that are at most these.
uint64_t slice_rows_most(const mp_cache_config* c, int total_q, int max_q, int max_kv, bool prefix) {
  const int group = c->q_heads / c->kv_heads;
  uint64_t most = prefix_few_rows_most(c, total_q, max_kv);
  // large tiles: the slices go by the tiles of a group, one where they are many
  for (int64_t tiles = 1; prefix && c->dtype == MP_DTYPE_BF16; ++tiles) {
    const int q = int(std::min<int64_t>(max_q, std::max<int64_t>(1, tiles * 256 / group))), s = prefix_slices(c, q, max_kv);
    most = std::max(most, uint64_t(s) * part_rows(c, total_q, q));
    if (s == 1 || q == max_q) break;
  }
  return most;
}
uint64_t sums_bytes(const mp_cache_config* c, uint64_t slice_rows) { return align256(slice_rows * c->q_heads * c->head_dim * 4); }
uint64_t ml_bytes(const mp_cache_config* c, uint64_t slice_rows) { return align256(slice_rows * c->q_heads * 2 * 4); }
// Numbers of pieces (two for large tiles), and for any plan.
uint64_t pieces_bytes(const mp_cache_config* c, int total_q, int rows) {
  return align256(uint64_t(piece_keys(c, total_q, rows)) * c->kv_heads * (rows == kTileRows ? 8 : 4));
}
uint64_t pieces_bytes_most(const mp_cache_config* c, int total_q) { return align256(uint64_t(piece_keys(c, total_q, 4)) * c->kv_heads * 8); }

// Rows of cut tiles as packed rows, which have a sum for each query head.
uint64_t cut_rows(const mp_cache_config* c, uint64_t rows) { return (rows + c->q_heads - 1) / c->q_heads; }

int check(const mp_cache_config* c, const mp_cache_config* p, int total_q, int max_q, int max_kv, int max_group_q, int max_prefix) {
  int rc = check_cache(c);
  if (rc != MP_OK) return rc;
  if ((rc = check_cache(p)) != MP_OK) return rc;
  if (p->kv_heads != c->kv_heads || p->q_heads != c->q_heads || p->head_dim != c->head_dim || p->dtype != c->dtype) return MP_ERR_INVALID_ARG;
  if (c->batch + p->batch > 65535) return MP_ERR_UNSUPPORTED;  // one grid's z
  if ((rc = check_limits(c, total_q, max_q, max_kv)) != MP_OK) return rc;
  return check_limits(p, total_q, max_group_q, max_prefix);
}

}  // namespace
}  // namespace mp

using namespace mp;

extern "C" {

int mp_prefix_workspace_bytes(const mp_cache_config* cfg, const mp_cache_config* prefix_cfg, int32_t total_q, int32_t max_q,
                              int32_t max_kv, int32_t max_group_q, int32_t max_prefix, uint64_t* bytes) {
  const int rc = check(cfg, prefix_cfg, total_q, max_q, max_kv, max_group_q, max_prefix);
  if (rc != MP_OK) return rc;
  if (!bytes) return MP_ERR_INVALID_ARG;
  *bytes = 0;
  if (total_q == 0) return MP_OK;
  max_q = std::min(max_q, total_q);
  max_group_q = std::min(max_group_q, total_q);
  uint64_t rows = slice_rows_most(cfg, total_q, max_q, max_kv, false) + slice_rows_most(prefix_cfg, total_q, max_group_q, max_prefix, true);
  if (cfg->dtype == MP_DTYPE_BF16) rows += cut_rows(cfg, both_tc_rows(cfg, max_q, max_kv, prefix_cfg, max_group_q, max_prefix));
  *bytes = pieces_bytes_most(cfg, total_q) + pieces_bytes_most(prefix_cfg, total_q) + sums_bytes(cfg, rows) + ml_bytes(cfg, rows);
  return MP_OK;
}

int mp_prefix_attention(const mp_cache_config* cfg, const mp_cache_config* prefix_cfg, const void* q, const int32_t* cu_q,
                        const int32_t* kv_len, int32_t total_q, int32_t max_q, int32_t max_kv, const void* keys,
                        const void* values, const int32_t* page_table, const int32_t* cu_group, const int32_t* prefix_len,
                        int32_t max_group_q, int32_t max_prefix, const void* prefix_keys, const void* prefix_values,
                        const int32_t* prefix_table, void* out, float* lse, void* workspace, size_t workspace_bytes,
                        uint32_t* status, void* stream) {
  int rc = check(cfg, prefix_cfg, total_q, max_q, max_kv, max_group_q, max_prefix);
  if (rc != MP_OK) return rc;
  if ((rc = check_pages(cfg, page_table)) != MP_OK) return rc;
  if ((rc = check_pages(prefix_cfg, prefix_table)) != MP_OK) return rc;
  if (!cu_q || !kv_len || !keys || !values || !cu_group || !prefix_len || !prefix_keys || !prefix_values) return MP_ERR_INVALID_ARG;
  if (total_q == 0) return MP_OK;
  if (!q || !out) return MP_ERR_INVALID_ARG;
  for (const void* p : {q, keys, values, prefix_keys, prefix_values, static_cast<const void*>(out)})
    if (!aligned16(p)) return MP_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(cu_q), static_cast<const void*>(kv_len), static_cast<const void*>(page_table),
                        static_cast<const void*>(cu_group), static_cast<const void*>(prefix_len),
                        static_cast<const void*>(prefix_table), static_cast<const void*>(lse), static_cast<const void*>(status)})
    if (!aligned4(p)) return MP_ERR_INVALID_ARG;
  max_q = std::min(max_q, total_q);
  max_group_q = std::min(max_group_q, total_q);
  const Plan plan = plan_of(cfg, prefix_cfg, total_q, max_q, max_group_q, max_prefix);
  const int own_slices = slices_of(plan.own, cfg, total_q, max_q, max_kv), slices = slices_of(plan.shared, prefix_cfg, total_q, max_group_q, max_prefix);
  const bool own_tiles = plan.own == kTiles, shared_tiles = plan.shared == kTiles;
  const uint64_t tile_rows = own_tiles || shared_tiles ? both_tc_rows(own_tiles ? cfg : nullptr, max_q, max_kv, shared_tiles ? prefix_cfg : nullptr,
                                                                      max_group_q, max_prefix)
                                                       : 0;
  const uint64_t whole = uint64_t(own_slices + slices) * total_q, rows = whole + cut_rows(cfg, tile_rows), sums = sums_bytes(cfg, rows),
                 own_pieces = pieces_bytes(cfg, total_q, plan.own_rows), pre_pieces = pieces_bytes(prefix_cfg, total_q, plan.pre_rows);
  const uint64_t need = own_pieces + pre_pieces + sums + ml_bytes(cfg, rows);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return MP_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MP_ERR_SCRATCH;
  if (injected("prefix")) return MP_ERR_INJECTED;

  char* ws = static_cast<char*>(workspace);
  Slices sl;
  sl.shared = slices;
  sl.own = own_slices;
  sl.own_pieces = reinterpret_cast<int32_t*>(ws);
  sl.pre_pieces = reinterpret_cast<int32_t*>(ws + own_pieces);
  sl.own_keys = int(piece_keys(cfg, total_q, plan.own_rows));
  sl.pre_keys = plan.shared == kSlices ? 0 : int(piece_keys(prefix_cfg, total_q, plan.pre_rows));
  sl.own_rows = plan.own_rows;
  sl.pre_rows = plan.pre_rows;
  sl.own_tiles = own_tiles;
  sl.pre_tiles = shared_tiles;
  sl.slot_rows = int(std::min<int64_t>(kTileRows, int64_t(std::max(own_tiles ? max_q : 1, shared_tiles ? max_group_q : 1)) *
                                                      (cfg->q_heads / cfg->kv_heads)));
  sl.slots = int(tile_rows / sl.slot_rows);
  sl.cut = int64_t(whole) * cfg->q_heads;
  ws += own_pieces + pre_pieces;
  PrefixArgs p, a;
  static_cast<CacheCall&>(a.c) = cache_args(cfg, page_table, cu_q, kv_len, total_q, max_q, max_kv, status);
  a.q = q;
  a.keys = keys;
  a.values = values;
  a.out = nullptr;
  a.lse = nullptr;
  a.splits = 1;
  a.joined = false;
  a.cuts = nullptr;
#if MP_CHECK
  a.stall = injected("prefix_wait");
#endif
  p = a;
  static_cast<CacheCall&>(p.c) = cache_args(prefix_cfg, prefix_table, cu_q, prefix_len, total_q, max_group_q, max_prefix, status);
  p.c.cu_group = cu_group;
  p.c.sequences = cfg->batch;
  p.keys = prefix_keys;
  p.values = prefix_values;
  p.pieces = sl.pre_pieces;
  const int64_t slice = int64_t(total_q) * cfg->q_heads;
  p.part = reinterpret_cast<float*>(ws);
  p.ml = reinterpret_cast<float*>(ws + sums);
  a.part = p.part + slices * slice * cfg->head_dim;
  a.ml = p.ml + slices * slice * 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaGetLastError();
  a.splits = own_slices;
  p.splits = slices;
  // the passes that are cut into runs, both in one launch where both are of a kind
  for (Kind kind : {kSimt, kFew}) {
    if (plan.own != kind && plan.shared != kind) continue;
    const bool beside = kind == kFew && plan.shared == kSlices, bf16 = cfg->dtype == MP_DTYPE_BF16;
    PrefixFew few;
#if MP_CHECK
    few.stall = injected("prefix_few_wait");
#endif
    few.pre = p;
    few.own = a;
    few.groups = plan.shared == kind ? prefix_cfg->batch : 0;
    few.own_units = plan.own == kind;
    few.most_shared = slices;
    few.most_own = own_slices;
    few.pre_keys = sl.pre_keys;
    few.own_keys = sl.own_keys;
    few.pre_pieces = sl.pre_pieces;
    few.own_pieces = sl.own_pieces;
    const int block = plan.own == kFew ? plan.own_rows : plan.pre_rows;
    ProfScope ps(st, beside ? K_PREFIX_ATTEND : (kind == kFew ? K_PREFIX_FEW : K_CHUNK_ATTEND));
    const cudaError_t e = beside          ? launch_prefix_slices(p, few, block, st)
                          : kind == kSimt ? launch_prefix_simt(few, st)
                          : bf16          ? launch_prefix_few(few, block, st)
                                          : launch_prefix_few32(few, block, st);
    if (e != cudaSuccess) return MP_ERR_CUDA;
  }
  // large tiles: likewise, in equal runs of all of them
  if (own_tiles || shared_tiles) {
    PrefixArgs both = a;
    both.state = p.part;
    both.state_ml = p.ml;
    both.own_slice = slices * slice;
    both.part = p.part + sl.cut * cfg->head_dim;
    both.ml = p.ml + sl.cut * 2;
    const TilePieces at = {sl.pre_keys, sl.own_keys, reinterpret_cast<int2*>(sl.pre_pieces), reinterpret_cast<int2*>(sl.own_pieces)};
    ProfScope ps(st, K_PREFIX_ATTEND);
    if (launch_both_tc(both, own_tiles, shared_tiles ? &p : nullptr, at, st) != cudaSuccess) return MP_ERR_CUDA;
  }
  a.out = out;
  a.lse = lse;
  a.part = p.part;
  a.ml = p.ml;
  ProfScope ps(st, K_PREFIX_JOIN);
  return launch_join(a, p.c, sl, cfg->dtype, st) == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}

}  // extern "C"
