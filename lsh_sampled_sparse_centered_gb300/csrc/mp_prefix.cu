// Attention of a batch whose sequences share prefixes (host side).
//
// The softmax over a row's prefix and its own slots is the join of two: every partial result is an
// unnormalised sum with its reference and its weights' sum (fp32), whatever slots it covers. So one pass
// goes over the prefixes, whose rows are those of all the sequences of a group: each prefix is read once,
// and the products have as many rows as the group has. The other goes over the sequences' own slots, as
// the attention of a chunk does. The last kernel joins both passes' slices.
#include "mp_cache_host.h"

namespace mp {
namespace {

// Slices of one pass over a cache, as (slice, packed row) pairs are kept for them.
int slices_of(const mp_cache_config* c, int total_q, int max_q, int max_kv) {
  if (chunk_on_tensor_cores(c, max_q)) return 1;
  const int s = c->dtype == MP_DTYPE_BF16 ? chunk_step_separate(c, max_q, max_kv) : chunk_splits(c, max_q, max_kv);
  // as many fewer where most packed rows belong to no sequence
  return std::max(1, int(s * part_rows(c, total_q, max_q) / total_q));
}
// The most that slices_of() * total_q comes to for limits that are at most these.
uint64_t slice_rows_most(const mp_cache_config* c, int total_q, int max_q, int max_kv) {
  const int group = c->q_heads / c->kv_heads;
  uint64_t most = uint64_t(total_q);
  if (c->dtype == MP_DTYPE_BF16) {
    for (int q = 1; q <= max_q && chunk_is_step(group, q); ++q)
      most = std::max(most, uint64_t(chunk_step_separate(c, q, max_kv)) * part_rows(c, total_q, q));
    return most;
  }
  // the slices go by the number of row tiles: the largest max_q of each, until one slice is left
  for (int64_t rows = (int64_t(group) + kChunkRows - 1) / kChunkRows * kChunkRows;; rows += kChunkRows) {
    const int q = int(std::min<int64_t>(max_q, rows / group)), s = chunk_splits(c, q, max_kv);
    most = std::max(most, uint64_t(s) * part_rows(c, total_q, q));
    if (s == 1 || q == max_q) return most;
  }
}
uint64_t tc_bytes(const mp_cache_config* c, int max_q, int max_kv) {
  return chunk_on_tensor_cores(c, max_q) ? chunk_tc_workspace(c, max_q, max_kv) : 0;
}
uint64_t sums_bytes(const mp_cache_config* c, uint64_t slice_rows) { return align256(slice_rows * c->q_heads * c->head_dim * 4); }
uint64_t ml_bytes(const mp_cache_config* c, uint64_t slice_rows) { return align256(slice_rows * c->q_heads * 2 * 4); }

int check(const mp_cache_config* c, const mp_cache_config* p, int total_q, int max_q, int max_kv, int max_group_q, int max_prefix) {
  int rc = check_cache(c);
  if (rc != MP_OK) return rc;
  if ((rc = check_cache(p)) != MP_OK) return rc;
  if (p->kv_heads != c->kv_heads || p->q_heads != c->q_heads || p->head_dim != c->head_dim || p->dtype != c->dtype) return MP_ERR_INVALID_ARG;
  if ((rc = check_limits(c, total_q, max_q, max_kv)) != MP_OK) return rc;
  return check_limits(p, total_q, max_group_q, max_prefix);
}

// One pass: its slices go to `part` and `ml`.
cudaError_t pass(ChunkArgs a, int dtype, bool tensor_cores, int slices, float* part, float* ml, void* pieces, cudaStream_t st) {
  a.out = nullptr;
  a.lse = nullptr;
  a.splits = slices;
  a.joined = false;
  a.cuts = nullptr;
  if (tensor_cores) {
    a.state = part;
    a.state_ml = ml;
    return launch_chunk_tc(a, pieces, st);
  }
  a.part = part;
  a.ml = ml;
  return dtype == MP_DTYPE_BF16 ? launch_chunk_step(a, st) : launch_chunk_simt(a, st);
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
  const uint64_t rows = slice_rows_most(cfg, total_q, max_q, max_kv) + slice_rows_most(prefix_cfg, total_q, max_group_q, max_prefix);
  *bytes = sums_bytes(cfg, rows) + ml_bytes(cfg, rows) +
           std::max(tc_bytes(cfg, max_q, max_kv), tc_bytes(prefix_cfg, max_group_q, max_prefix));
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
  const bool tc = chunk_on_tensor_cores(cfg, max_q), prefix_tc = chunk_on_tensor_cores(prefix_cfg, max_group_q);
  const int own = slices_of(cfg, total_q, max_q, max_kv), shared = slices_of(prefix_cfg, total_q, max_group_q, max_prefix);
  const uint64_t sums = sums_bytes(cfg, uint64_t(own + shared) * total_q), ml = ml_bytes(cfg, uint64_t(own + shared) * total_q);
  const uint64_t need = sums + ml + std::max(tc_bytes(cfg, max_q, max_kv), tc_bytes(prefix_cfg, max_group_q, max_prefix));
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return MP_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MP_ERR_SCRATCH;
  if (injected("prefix")) return MP_ERR_INJECTED;

  ChunkArgs a;
  a.c = cache_args(cfg, page_table, cu_q, kv_len, total_q, max_q, max_kv, status);
  a.q = q;
  a.keys = keys;
  a.values = values;
#if MP_CHECK
  a.stall = injected("prefix_wait");
#endif
  ChunkArgs p = a;
  p.c = cache_args(prefix_cfg, prefix_table, cu_q, prefix_len, total_q, max_group_q, max_prefix, status);
  p.c.cu_group = cu_group;
  p.c.sequences = cfg->batch;
  p.keys = prefix_keys;
  p.values = prefix_values;
  char* ws = static_cast<char*>(workspace);
  float *part0 = reinterpret_cast<float*>(ws), *ml0 = reinterpret_cast<float*>(ws + sums);
  void* pieces = ws + sums + ml;
  const int64_t slice = int64_t(total_q) * cfg->q_heads;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaGetLastError();
  {
    ProfScope ps(st, K_PREFIX_ATTEND);
    if (pass(p, cfg->dtype, prefix_tc, shared, part0, ml0, pieces, st) != cudaSuccess) return MP_ERR_CUDA;
  }
  {
    ProfScope ps(st, K_CHUNK_ATTEND);
    if (pass(a, cfg->dtype, tc, own, part0 + shared * slice * cfg->head_dim, ml0 + shared * slice * 2, pieces, st) != cudaSuccess)
      return MP_ERR_CUDA;
  }
  a.out = out;
  a.lse = lse;
  a.splits = shared + own;
  a.joined = false;
  a.part = part0;
  a.ml = ml0;
  ProfScope ps(st, K_PREFIX_JOIN);
  return launch_prefix_join(a, p.c, shared, cfg->dtype, st) == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}

}  // extern "C"
