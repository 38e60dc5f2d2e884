// Host side of the cache operators: validation, workspace sizes and launches.
#include <algorithm>

#include "mp_cache_host.h"

namespace mp {

static StepPlan slices(const mp_cache_config* c, int total_q, int max_q, int max_kv) {
  StepPlan p = c->dtype == MP_DTYPE_BF16 ? chunk_step_plan(c, max_q, max_kv) : StepPlan{chunk_splits(c, max_q, max_kv), false};
  // with more rows than that, as many fewer slices
  if (!p.joined) p.splits = std::max(1, int(p.splits * part_rows(c, total_q, max_q) / total_q));
  return p;
}
static bool needs_join(const StepPlan& p) { return p.splits > 1 && !p.joined; }
static uint64_t part_bytes(const mp_cache_config* c, uint64_t rows, int splits) {
  return align256(uint64_t(splits) * rows * c->q_heads * c->head_dim * 4);
}
static uint64_t slices_bytes(const mp_cache_config* c, uint64_t rows, int splits) {
  return part_bytes(c, rows, splits) + align256(uint64_t(splits) * rows * c->q_heads * 2 * 4);
}
// What one call takes.
static uint64_t chunk_bytes(const mp_cache_config* c, int total_q, int max_q, int max_kv) {
  if (total_q == 0) return 0;
  max_q = std::min(max_q, total_q);
  if (chunk_on_tensor_cores(c, max_q)) return chunk_tc_workspace(c, max_q, max_kv);
  const StepPlan plan = slices(c, total_q, max_q, max_kv);
  return needs_join(plan) ? slices_bytes(c, total_q, plan.splits) : 0;
}
// What the calls take whose limits are at most these. One call's need falls where more rows or a
// shorter cache are cut into fewer slices, or into slices that join themselves, so this is the
// largest need over the smaller max_q, with slices that only grow with max_kv.
static uint64_t chunk_bytes_most(const mp_cache_config* c, int total_q, int max_q, int max_kv) {
  if (total_q == 0) return 0;
  max_q = std::min(max_q, total_q);
  const int group = c->q_heads / c->kv_heads;
  uint64_t most = 0;
  if (c->dtype == MP_DTYPE_BF16) {
    if (chunk_on_tensor_cores(c, max_q)) most = chunk_tc_workspace(c, max_q, max_kv);  // grows with both
    for (int q = 1; q <= max_q && chunk_is_step(group, q); ++q) {
      const int splits = chunk_step_most(c, q, max_kv);
      if (splits > 1) most = std::max(most, slices_bytes(c, part_rows(c, total_q, q), splits));
    }
    return most;
  }
  // the slices go by the number of row tiles: the largest max_q of each, until one slice is left
  for (int64_t rows = (int64_t(group) + kChunkRows - 1) / kChunkRows * kChunkRows;; rows += kChunkRows) {
    const int q = int(std::min<int64_t>(max_q, rows / group));
    const int splits = chunk_splits(c, q, max_kv);
    if (splits == 1) return most;
    most = std::max(most, slices_bytes(c, part_rows(c, total_q, q), splits));
    if (q == max_q) return most;
  }
}

// What the eviction writes against what it reads: its CTAs work in no order, so that a buffer that
// is both would be read after it was overwritten. dst_len may be kv_len (mp_evict.cu). Pages
// named by a table are the caller's business, a dense cache's are known.
static bool evict_overlaps(const mp_cache_config* c, const mp_cache_config* d, const void* keys, const void* values,
                           const void* table, const void* kv_len, const void* scores, int budget, const void* dst_keys,
                           const void* dst_values, const void* dst_table, const void* dst_scores, const void* dst_len,
                           const void* kept, const void* workspace) {
  const uint64_t units = uint64_t(c->batch) * c->kv_heads, row = uint64_t(c->head_dim) * (c->dtype == MP_DTYPE_BF16 ? 2 : 4);
  const uint64_t src_slots = uint64_t(c->max_pages) * c->page_size, dst_slots = uint64_t(d->max_pages) * d->page_size;
  const Range in[] = {{scores, units * src_slots * 4}, {table, uint64_t(c->batch) * c->max_pages * 4},
                      {dst_table, uint64_t(c->batch) * d->max_pages * 4}, {kv_len, uint64_t(c->batch) * 4}};
  const Range out[] = {{dst_scores, units * dst_slots * 4}, {kept, units * budget * 4}, {kept ? nullptr : workspace, units * budget * 4},
                       {dst_len, uint64_t(c->batch) * 4}};
  for (const Range& i : in)
    for (const Range& o : out)
      if (overlap(i, o) && !(i.p == kv_len && o.p == dst_len && kv_len == dst_len)) return true;
  if (table || dst_table) return false;
  const Range from[] = {{keys, units * src_slots * row}, {values, units * src_slots * row}};
  const Range to[] = {{dst_keys, units * dst_slots * row}, {dst_values, units * dst_slots * row}};
  for (const Range& i : from)
    for (const Range& o : to)
      if (overlap(i, o)) return true;
  return false;
}

static uint64_t evict_bytes(const mp_cache_config* c, int budget) {
  return align256(uint64_t(c->batch) * c->kv_heads * budget * 4);
}

}  // namespace mp

using namespace mp;

extern "C" {

int mp_cache_config_check(const mp_cache_config* cfg) { return check_cache(cfg); }

int mp_cache_append(const mp_cache_config* cfg, const mp_rotary* rotary, const void* q, int64_t q_stride, const void* k,
                    int64_t k_stride, const void* v, int64_t v_stride, const void* q_norm, const void* k_norm,
                    const double* inv_freq, const int32_t* positions, const int32_t* cu_q, const int32_t* kv_len,
                    int32_t total_q, void* keys, void* values, const int32_t* page_table, void* q_out,
                    uint32_t* status, void* stream) {
  int rc = check_cache(cfg);
  if (rc != MP_OK) return rc;
  if (rotary && rotary->rot_dim > 0 && !inv_freq) return MP_ERR_INVALID_ARG;
  if ((rc = check_rotary(rotary, cfg)) != MP_OK) return rc;
  const int vec = cfg->dtype == MP_DTYPE_BF16 ? 8 : 4;
  if ((rc = check_pages(cfg, page_table)) != MP_OK) return rc;
  if ((rc = check_limits(cfg, total_q, 1, 1)) != MP_OK) return rc;
  if (!cu_q || !kv_len || !keys || !values) return MP_ERR_INVALID_ARG;
  if (total_q == 0) return MP_OK;
  if (!q || !k || !v || !q_out) return MP_ERR_INVALID_ARG;
  const int64_t qw = int64_t(cfg->q_heads) * cfg->head_dim, kw = int64_t(cfg->kv_heads) * cfg->head_dim;
  if (q_stride < qw || k_stride < kw || v_stride < kw) return MP_ERR_INVALID_ARG;
  if (q_stride % vec || k_stride % vec || v_stride % vec) return MP_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, static_cast<const void*>(keys), static_cast<const void*>(values),
                        static_cast<const void*>(q_out), q_norm, k_norm})
    if (!aligned16(p)) return MP_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(positions), static_cast<const void*>(cu_q),
                        static_cast<const void*>(kv_len), static_cast<const void*>(page_table),
                        static_cast<const void*>(status)})
    if (!aligned4(p)) return MP_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(inv_freq) & 7u) return MP_ERR_INVALID_ARG;
  if (injected("append")) return MP_ERR_INJECTED;
  AppendArgs a;
  a.c = cache_args(cfg, page_table, cu_q, kv_len, total_q, total_q, INT_MAX, status);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.rot = rotary->rot_dim;
  a.interleaved = rotary->interleaved;
  a.eps = rotary->eps;
  a.keys = keys;
  a.values = values;
  a.q_out = q_out;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaGetLastError();  // clear a stale error so that it is not blamed on this call
  ProfScope ps(st, K_CACHE_APPEND);
  return launch_cache_append(a, cfg->dtype, st) == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}

int mp_chunk_workspace_bytes(const mp_cache_config* cfg, int32_t total_q, int32_t max_q, int32_t max_kv,
                             uint64_t* bytes) {
  int rc = check_cache(cfg);
  if (rc != MP_OK) return rc;
  if ((rc = check_limits(cfg, total_q, max_q, max_kv)) != MP_OK) return rc;
  if (!bytes) return MP_ERR_INVALID_ARG;
  *bytes = chunk_bytes_most(cfg, total_q, max_q, max_kv);
  return MP_OK;
}

int mp_chunk_attention(const mp_cache_config* cfg, const void* q, const int32_t* cu_q, const int32_t* kv_len,
                       int32_t total_q, int32_t max_q, int32_t max_kv, const void* keys, const void* values,
                       const int32_t* page_table, void* out, float* lse, void* workspace, size_t workspace_bytes,
                       uint32_t* status, void* stream) {
  int rc = check_cache(cfg);
  if (rc != MP_OK) return rc;
  if ((rc = check_pages(cfg, page_table)) != MP_OK) return rc;
  if ((rc = check_limits(cfg, total_q, max_q, max_kv)) != MP_OK) return rc;
  if (!cu_q || !kv_len || !keys || !values) return MP_ERR_INVALID_ARG;
  if (total_q == 0) return MP_OK;
  if (!q || !out) return MP_ERR_INVALID_ARG;
  for (const void* p : {q, keys, values, static_cast<const void*>(out)})
    if (!aligned16(p)) return MP_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(cu_q), static_cast<const void*>(kv_len),
                        static_cast<const void*>(page_table), static_cast<const void*>(lse),
                        static_cast<const void*>(status)})
    if (!aligned4(p)) return MP_ERR_INVALID_ARG;
  const uint64_t need = chunk_bytes(cfg, total_q, max_q, max_kv);
  if (need > 0) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return MP_ERR_INVALID_ARG;
    if (workspace_bytes < need) return MP_ERR_SCRATCH;
  }
  if (injected("chunk")) return MP_ERR_INJECTED;
  ChunkArgs a;
  a.c = cache_args(cfg, page_table, cu_q, kv_len, total_q, std::min(max_q, total_q), max_kv, status);
  a.q = q;
  a.keys = keys;
  a.values = values;
  a.out = out;
  a.lse = lse;
  a.splits = 1;
  a.joined = false;
  a.part = a.ml = nullptr;
#if MP_CHECK
  a.stall = injected("chunk_wait");
#endif
  a.cuts = nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaGetLastError();
  if (chunk_on_tensor_cores(cfg, a.c.max_q)) {
    ProfScope ps(st, K_CHUNK_ATTEND);
    return launch_chunk_tc(a, workspace, st) == cudaSuccess ? MP_OK : MP_ERR_CUDA;
  }
  const StepPlan plan = slices(cfg, total_q, a.c.max_q, max_kv);
  a.splits = plan.splits;
  a.joined = plan.joined;
  if (need > 0) {
    a.part = static_cast<float*>(workspace);
    a.ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + part_bytes(cfg, total_q, a.splits));
  }
  {
    ProfScope ps(st, K_CHUNK_ATTEND);
    const cudaError_t e = cfg->dtype == MP_DTYPE_BF16 ? launch_chunk_step(a, st) : launch_chunk_simt(a, st);
    if (e != cudaSuccess) return MP_ERR_CUDA;
  }
  if (needs_join(plan)) {
    ProfScope ps(st, K_CHUNK_JOIN);
    if (launch_chunk_join(a, cfg->dtype, st) != cudaSuccess) return MP_ERR_CUDA;
  }
  return MP_OK;
}

int mp_cache_weights(const mp_cache_config* cfg, const void* q, const float* lse, const int32_t* cu_q,
                     const int32_t* kv_len, int32_t total_q, int32_t max_q, int32_t max_kv, const void* keys,
                     const int32_t* page_table, float* scores, uint32_t* status, void* stream) {
  int rc = check_cache(cfg);
  if (rc != MP_OK) return rc;
  if ((rc = check_pages(cfg, page_table)) != MP_OK) return rc;
  if ((rc = check_limits(cfg, total_q, max_q, max_kv)) != MP_OK) return rc;
  if (!cu_q || !kv_len || !keys || !scores) return MP_ERR_INVALID_ARG;
  if (total_q == 0) return MP_OK;
  if (!q || !lse) return MP_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(keys)) return MP_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(cu_q), static_cast<const void*>(kv_len),
                        static_cast<const void*>(page_table), static_cast<const void*>(lse),
                        static_cast<const void*>(scores), static_cast<const void*>(status)})
    if (!aligned4(p)) return MP_ERR_INVALID_ARG;
  if (injected("weights")) return MP_ERR_INJECTED;
  WeightsArgs a;
  a.c = cache_args(cfg, page_table, cu_q, kv_len, total_q, max_q, max_kv, status);
  a.q = q;
  a.keys = keys;
  a.lse = lse;
  a.scores = scores;
#if MP_CHECK
  a.stall = injected("weights_wait");
#endif
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaGetLastError();
  ProfScope ps(st, K_CACHE_WEIGHTS);
  return launch_cache_weights(a, cfg->dtype, st) == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}

int mp_evict_workspace_bytes(const mp_cache_config* cfg, int32_t max_kv, int32_t budget, uint64_t* bytes) {
  int rc = check_cache(cfg);
  if (rc != MP_OK) return rc;
  if ((rc = check_limits(cfg, 0, 1, max_kv)) != MP_OK) return rc;
  if (!bytes || budget < 1) return MP_ERR_INVALID_ARG;
  *bytes = evict_bytes(cfg, budget);
  return MP_OK;
}

int mp_cache_evict(const mp_cache_config* cfg, const mp_cache_config* dst_cfg, const void* keys, const void* values,
                   const int32_t* page_table, const int32_t* kv_len, int32_t max_kv, const float* scores,
                   int32_t n_sink, int32_t window, int32_t budget, void* dst_keys, void* dst_values,
                   const int32_t* dst_page_table, float* dst_scores, int32_t* dst_len, int32_t* kept, void* workspace,
                   size_t workspace_bytes, uint32_t* status, void* stream) {
  int rc = check_cache(cfg);
  if (rc != MP_OK) return rc;
  if ((rc = check_cache(dst_cfg)) != MP_OK) return rc;
  if (dst_cfg->batch != cfg->batch || dst_cfg->kv_heads != cfg->kv_heads || dst_cfg->q_heads != cfg->q_heads ||
      dst_cfg->head_dim != cfg->head_dim || dst_cfg->dtype != cfg->dtype)
    return MP_ERR_INVALID_ARG;
  if ((rc = check_pages(cfg, page_table)) != MP_OK) return rc;
  if ((rc = check_pages(dst_cfg, dst_page_table)) != MP_OK) return rc;
  if ((rc = check_limits(cfg, 0, 1, max_kv)) != MP_OK) return rc;
  if (budget < 1 || n_sink < 0 || window < 0 || int64_t(n_sink) + window > budget) return MP_ERR_INVALID_ARG;
  if (int64_t(budget) > int64_t(dst_cfg->max_pages) * dst_cfg->page_size) return MP_ERR_CAPACITY;
  if (!keys || !values || !kv_len || !scores || !dst_keys || !dst_values || !dst_len) return MP_ERR_INVALID_ARG;
  for (const void* p : {keys, values, static_cast<const void*>(dst_keys), static_cast<const void*>(dst_values)})
    if (!aligned16(p)) return MP_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(page_table), static_cast<const void*>(kv_len),
                        static_cast<const void*>(scores), static_cast<const void*>(dst_page_table),
                        static_cast<const void*>(dst_scores), static_cast<const void*>(dst_len),
                        static_cast<const void*>(kept), static_cast<const void*>(status)})
    if (!aligned4(p)) return MP_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return MP_ERR_INVALID_ARG;
  if (workspace_bytes < evict_bytes(cfg, budget)) return MP_ERR_SCRATCH;
  if (injected("evict")) return MP_ERR_INJECTED;
  if (evict_overlaps(cfg, dst_cfg, keys, values, page_table, kv_len, scores, budget, dst_keys, dst_values, dst_page_table,
                     dst_scores, dst_len, kept, workspace))
    return MP_ERR_INVALID_ARG;
  EvictArgs a;
  a.c = cache_args(cfg, page_table, nullptr, kv_len, 0, 1, max_kv, status);
  a.keys = keys;
  a.values = values;
  a.scores = scores;
  a.n_sink = n_sink;
  a.window = window;
  a.budget = budget;
  a.dst_keys = dst_keys;
  a.dst_values = dst_values;
  a.dst_table = dst_page_table;
  a.dst_page_size = dst_cfg->page_size;
  a.dst_n_pages = dst_cfg->n_pages;
  a.dst_cols = dst_cfg->max_pages;
  a.dst_scores = dst_scores;
  a.dst_len = dst_len;
  a.kept = kept ? kept : static_cast<int32_t*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaGetLastError();
  {
    ProfScope ps(st, K_EVICT_SELECT);
    if (launch_evict_select(a, st) != cudaSuccess) return MP_ERR_CUDA;
  }
  ProfScope ps(st, K_EVICT_GATHER);
  return launch_evict_gather(a, cfg->dtype, st) == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}

}  // extern "C"
