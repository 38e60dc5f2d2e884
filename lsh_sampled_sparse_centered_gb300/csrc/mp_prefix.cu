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

// Slices of the two passes, and their numbers per (group or sequence, KV head) where these differ.
struct Slices {
  int shared, own;
  int32_t *pre_pieces, *own_pieces;
  int pre_keys, own_keys, pre_rows, own_rows;  // at piece_key() of blocks of so many rows (pre_keys = 0: one for [group][KV head])
};

// A join of many rows (1264 tokens of 32 heads in two slices: 22 us with four rows and two CTAs, 16 so):
constexpr int kRowsALane = 2;
constexpr int kResident = 4;  // CTAs of an SM
// and CTAs that fit go this many times into the grid: each looks up its sequence once for several rows (six chunks
// of 33 to 517 tokens, the whole call with 1, 2 and 4: 280, 272 and 274 us; a CTA for every 16 rows: 278).
constexpr int kRounds = 2;
// One of few rows: several warps a row, with four slices each in flight.
constexpr int kFewAtOnce = 4;

// Joins the slices' (m, l, sum) of a sequence's query rows, in their order. A warp takes ROWS rows (of
// D / 4 lanes each, 16 bytes a lane) and has the loads of kAtOnce slices of each in flight; with WARPS > 1
// as many warps share the slices of their rows, so that all of them are in flight together. The first
// `shared` slices are of the prefix, the `own` behind them of the own slots; where their numbers are kept
// per (group or sequence, KV head, block of rows), as many of them are there. Rows without a prefix have
// none of it.
// Grid: rows of a sequence x sequences, so that what has to be looked up does not hang on a row.
template <typename T, int D, int ROWS, int WARPS>
__global__ void __launch_bounds__(256, WARPS == 4 || ROWS > 128 / D ? kResident : 2) k_prefix_join(const ChunkArgs a, const CacheArgs prefix, const Slices sl) {
  constexpr int kLanes = D / 4, kTurns = ROWS * kLanes / 32, kAtOnce = WARPS > 1 ? kFewAtOnce : (kTurns == 1 ? 8 : 2);
  static_assert(WARPS == 1 || kTurns == 1);
  __shared__ float4 so[WARPS > 1 ? 8 : 1][32];
  __shared__ float2 sml[WARPS > 1 ? 8 : 1][32];
  const CacheArgs& c = a.c;
  const int qh = c.kvh * c.group, b = blockIdx.y;
  const int64_t rows = int64_t(c.total_q) * qh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / kLanes, e = lane % kLanes * 4;
  const Seq s = seq_of(c, b);
  int lo = 0, hi = prefix.batch;  // cu_group[lo] <= b is kept where it holds for 0
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix.cu_group[mid] <= b) lo = mid;
    else hi = mid;
  }
  const Seq g = group_of(prefix, lo);
  const int mine = s.m * qh, step = int(gridDim.x) * (8 / WARPS) * ROWS;  // all rows together are 32-bit
  int first = int(blockIdx.x * (8 / WARPS) + warp / WARPS) * ROWS;
  do {
    float m[kTurns], l[kTurns];
    float4 o[kTurns];
    int64_t row[kTurns];
    int there[kTurns], all[kTurns];  // slices of the row's prefix, and with those of its own slots
    const int32_t *there_at[kTurns], *all_at[kTurns];  // or where their numbers are
#pragma unroll
    for (int j = 0; j < kTurns; ++j) {
      const int i = first + j * (32 / kLanes) + sub;
      const bool live = i < mine;
      row[j] = live ? int64_t(s.row0) * qh + i : -1;
      const int token = i / qh, in = i - token * qh, h = in / c.group, in_head = in - h * c.group, t = s.row0 + token;
      const bool shared = live && g.row0 <= t && t < g.row0 + g.m;
      there[j] = shared ? sl.shared : 0;
      all[j] = live ? sl.own : 0;
      there_at[j] = !shared || !sl.pre_pieces ? nullptr
                    : sl.pre_pieces + (sl.pre_keys ? int64_t(h) * sl.pre_keys + piece_key(g.row0, c.group, sl.pre_rows,
                                                                                           ((t - g.row0) * c.group + in_head) / sl.pre_rows, lo)
                                                   : int64_t(lo) * c.kvh + h);
      all_at[j] = !live || !sl.own_pieces ? nullptr
                  : sl.own_pieces + int64_t(h) * sl.own_keys + piece_key(s.row0, c.group, sl.own_rows, (token * c.group + in_head) / sl.own_rows, b);
      m[j] = -INFINITY;
      l[j] = 0.f;
      o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (WARPS == 1 && first >= mine) return;
    int most = 0;
#pragma unroll
    for (int j = 0; j < kTurns; ++j) {
      if (there_at[j]) there[j] = min(there[j], *there_at[j]);
      if (all_at[j]) all[j] = min(all[j], *all_at[j]);
      all[j] += there[j];
      most = max(most, all[j]);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    for (int i0 = warp % WARPS * kAtOnce; i0 < most; i0 += WARPS * kAtOnce) {
      float2 v[kTurns][kAtOnce];
      float4 x[kTurns][kAtOnce];
#pragma unroll
      for (int j = 0; j < kTurns; ++j) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const int i = i0 + k;
          const bool live = i < all[j];
          const int64_t at = live ? (i < there[j] ? i : i - there[j] + sl.shared) * rows + row[j] : 0;
          v[j][k] = live ? *reinterpret_cast<const float2*>(a.ml + at * 2) : make_float2(-INFINITY, 0.f);
          x[j][k] = live ? *reinterpret_cast<const float4*>(a.part + at * D + e) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int j = 0; j < kTurns; ++j) {
        float top = m[j];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, v[j][k].x);
        const float ref = top == -INFINITY ? 0.f : top, before = exp2f(m[j] - ref);  // 0 while nothing was seen
        m[j] = top;
        l[j] *= before;
        o[j].x *= before;
        o[j].y *= before;
        o[j].z *= before;
        o[j].w *= before;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const bool any = v[j][k].y != 0.f;  // a slice that saw nothing has written no sum
          const float by = any ? exp2f(v[j][k].x - ref) : 0.f;
          l[j] = fmaf(v[j][k].y, by, l[j]);
          o[j].x = any ? fmaf(x[j][k].x, by, o[j].x) : o[j].x;
          o[j].y = any ? fmaf(x[j][k].y, by, o[j].y) : o[j].y;
          o[j].z = any ? fmaf(x[j][k].z, by, o[j].z) : o[j].z;
          o[j].w = any ? fmaf(x[j][k].w, by, o[j].w) : o[j].w;
        }
      }
    }
    if (WARPS > 1) {  // the warps' parts, in their order
      so[warp][lane] = o[0];
      sml[warp][lane] = make_float2(m[0], l[0]);
      __syncthreads();
      if (warp % WARPS != 0) return;
      float2 v[WARPS];
      float4 x[WARPS];
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        v[w] = sml[warp + w][lane];
        x[w] = so[warp + w][lane];
        top = fmaxf(top, v[w].x);
      }
      const float ref = top == -INFINITY ? 0.f : top;
      m[0] = top;
      l[0] = 0.f;
      o[0] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float by = v[w].y == 0.f ? 0.f : exp2f(v[w].x - ref);
        l[0] = fmaf(v[w].y, by, l[0]);
        o[0].x = fmaf(x[w].x, by, o[0].x);
        o[0].y = fmaf(x[w].y, by, o[0].y);
        o[0].z = fmaf(x[w].z, by, o[0].z);
        o[0].w = fmaf(x[w].w, by, o[0].w);
      }
    }
#pragma unroll
    for (int j = 0; j < kTurns; ++j) {
      if (row[j] < 0) continue;
      const float inv = l[j] == 0.f ? 0.f : 1.0f / l[j];
      if (a.lse && e == 0) a.lse[row[j]] = l[j] == 0.f ? -INFINITY : m[j] * 0.6931471805599453f + logf(l[j]);
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row[j] * D + e) = make_uint2(bf2(o[j].x * inv, o[j].y * inv), bf2(o[j].z * inv, o[j].w * inv));
      else
        *reinterpret_cast<float4*>(static_cast<T*>(a.out) + row[j] * D + e) = make_float4(o[j].x * inv, o[j].y * inv, o[j].z * inv, o[j].w * inv);
    }
    first += step;
  } while (WARPS == 1 && first < mine);
}

template <typename T, int D>
cudaError_t join(const ChunkArgs& a, const CacheArgs& prefix, const Slices& sl, cudaStream_t st) {
  const int each = 32 / (D / 4), qh = a.c.kvh * a.c.group;
  // Two rows a lane where that still leaves the SMs 16 warps each, four warps a row where there are at most
  // 8 rows an SM, eight where there are at most two (32 tokens of 32 heads: 76, 69 and 71 us a call with
  // one, four and eight, four tokens: 18.7, 16.6 and 15.0).
  const int64_t all = int64_t(a.c.total_q) * qh / each, sms = device_sm_count();
  const bool many = all >= sms * 16 * kRowsALane, few = all <= sms * 8, least = all <= sms * 2;
  const int rows = each * (many ? 8 * kRowsALane : (least ? 1 : (few ? 2 : 8)));
  cudaLaunchConfig_t cfg = {};
  // many rows: as many CTAs as fit, which take several rows one after the other
  const int64_t most = (int64_t(a.c.max_q) * qh + rows - 1) / rows;
  cfg.gridDim = dim3(unsigned(many ? std::min(most, std::max<int64_t>(1, kRounds * kResident * sms / a.c.batch)) : most), a.c.batch);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (many) return cudaLaunchKernelEx(&cfg, k_prefix_join<T, D, kRowsALane * (128 / D), 1>, a, prefix, sl);
  if (least) return cudaLaunchKernelEx(&cfg, k_prefix_join<T, D, 128 / D, 8>, a, prefix, sl);
  return few ? cudaLaunchKernelEx(&cfg, k_prefix_join<T, D, 128 / D, 4>, a, prefix, sl)
             : cudaLaunchKernelEx(&cfg, k_prefix_join<T, D, 128 / D, 1>, a, prefix, sl);
}

cudaError_t launch_join(const ChunkArgs& a, const CacheArgs& prefix, const Slices& sl, int dtype, cudaStream_t st) {
  if (dtype == MP_DTYPE_BF16)
    return a.c.d == 128 ? join<__nv_bfloat16, 128>(a, prefix, sl, st) : join<__nv_bfloat16, 64>(a, prefix, sl, st);
  return a.c.d == 128 ? join<float, 128>(a, prefix, sl, st) : join<float, 64>(a, prefix, sl, st);
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
  if (few || own <= 16) return {kFew, few ? kFew : (prefix_in_slices(p, total_q, max_group_q) ? kSlices : kTiles), rows, rows};
  return {kTiles, kTiles, 0, 0};
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
uint64_t pieces_bytes(const mp_cache_config* c, int total_q, int rows) { return align256(uint64_t(piece_keys(c, total_q, rows)) * c->kv_heads * 4); }
constexpr int kLeastRows = 4;  // of a block

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
  const uint64_t rows = slice_rows_most(cfg, total_q, max_q, max_kv, false) + slice_rows_most(prefix_cfg, total_q, max_group_q, max_prefix, true);
  *bytes = pieces_bytes(cfg, total_q, kLeastRows) + pieces_bytes(prefix_cfg, total_q, kLeastRows) + sums_bytes(cfg, rows) + ml_bytes(cfg, rows) +
           (cfg->dtype == MP_DTYPE_BF16 ? both_tc_workspace(cfg, max_q, max_kv, prefix_cfg, max_group_q, max_prefix) : 0);
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
  const uint64_t rows = uint64_t(own_slices + slices) * total_q, sums = sums_bytes(cfg, rows), ml = ml_bytes(cfg, rows),
                 own_pieces = plan.own_rows ? pieces_bytes(cfg, total_q, plan.own_rows) : 0,
                 pre_pieces = plan.pre_rows ? pieces_bytes(prefix_cfg, total_q, plan.pre_rows) : 0;
  const bool own_tiles = plan.own == kTiles, shared_tiles = plan.shared == kTiles;
  uint64_t need = own_pieces + pre_pieces + sums + ml;
  if (own_tiles || shared_tiles)
    need += both_tc_workspace(own_tiles ? cfg : nullptr, max_q, max_kv, shared_tiles ? prefix_cfg : nullptr, max_group_q, max_prefix);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return MP_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MP_ERR_SCRATCH;
  if (injected("prefix")) return MP_ERR_INJECTED;

  char* ws = static_cast<char*>(workspace);
  Slices sl = {slices, own_slices, nullptr, nullptr, 0, 0, plan.pre_rows, plan.own_rows};
  if (!own_tiles) {
    sl.own_pieces = reinterpret_cast<int32_t*>(ws);
    sl.own_keys = int(piece_keys(cfg, total_q, plan.own_rows));
  }
  if (!shared_tiles) {
    sl.pre_pieces = reinterpret_cast<int32_t*>(ws + own_pieces);
    if (plan.shared != kSlices) sl.pre_keys = int(piece_keys(prefix_cfg, total_q, plan.pre_rows));
  }
  ws += own_pieces + pre_pieces;
  void* tiles = ws + sums + ml;
  ChunkArgs p, a;
  a.c = cache_args(cfg, page_table, cu_q, kv_len, total_q, max_q, max_kv, status);
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
  p.c = cache_args(prefix_cfg, prefix_table, cu_q, prefix_len, total_q, max_group_q, max_prefix, status);
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
    ChunkArgs both = a;
    both.state = p.part;
    both.state_ml = p.ml;
    both.own_slice = slices * slice;
    ProfScope ps(st, K_PREFIX_ATTEND);
    if (launch_both_tc(both, own_tiles, shared_tiles ? &p : nullptr, tiles, st) != cudaSuccess) return MP_ERR_CUDA;
  }
  a.out = out;
  a.lse = lse;
  a.part = p.part;
  a.ml = p.ml;
  ProfScope ps(st, K_PREFIX_JOIN);
  return launch_join(a, p.c, sl, cfg->dtype, st) == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}

}  // extern "C"
