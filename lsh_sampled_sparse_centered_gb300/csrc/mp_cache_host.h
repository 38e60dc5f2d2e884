// Host checks that the cache operators' entry points share.
#pragma once

#include <algorithm>
#include <climits>

#include "mp_cache.cuh"

namespace mp {

inline int check_cache(const mp_cache_config* c) {
  if (!c) return MP_ERR_INVALID_ARG;
  if (c->batch < 1 || c->kv_heads < 1 || c->q_heads < 1 || c->q_heads % c->kv_heads != 0) return MP_ERR_INVALID_ARG;
  if (c->page_size < 1 || c->n_pages < 1 || c->max_pages < 1) return MP_ERR_INVALID_ARG;
  if (c->dtype != MP_DTYPE_F32 && c->dtype != MP_DTYPE_BF16) return MP_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (c->reserved[i] != 0) return MP_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return MP_ERR_UNSUPPORTED;
  // grid limits: sequences and KV heads index blockIdx.z and blockIdx.y
  if (c->batch > 65535 || c->kv_heads > 65535) return MP_ERR_UNSUPPORTED;
  // slots of a sequence and rows of the pool (n_pages * kv_heads * page_size) are 32-bit
  if (int64_t(c->max_pages) * c->page_size > (int64_t(1) << 30)) return MP_ERR_UNSUPPORTED;
  if (int64_t(c->n_pages) * c->kv_heads > INT_MAX / c->page_size) return MP_ERR_UNSUPPORTED;
  return MP_OK;
}

// Without a table page b is sequence b's whole cache; with one, pages are whole 16-row boxes.
inline int check_pages(const mp_cache_config* c, const void* table) {
  if (table) return c->page_size % 16 == 0 ? MP_OK : MP_ERR_UNSUPPORTED;
  return c->max_pages == 1 && c->n_pages >= c->batch ? MP_OK : MP_ERR_INVALID_ARG;
}

inline int check_limits(const mp_cache_config* c, int total_q, int max_q, int max_kv) {
  if (total_q < 0 || max_q < 1 || max_kv < 1) return MP_ERR_INVALID_ARG;
  if (int64_t(max_kv) > int64_t(c->max_pages) * c->page_size) return MP_ERR_CAPACITY;
  // a chunk's query rows per KV head, and all rows, are 32-bit
  if (int64_t(max_q) * (c->q_heads / c->kv_heads) > (1 << 30)) return MP_ERR_UNSUPPORTED;
  if (int64_t(total_q) * c->q_heads > INT_MAX) return MP_ERR_UNSUPPORTED;
  return MP_OK;
}

inline int check_rotary(const mp_rotary* r, const mp_cache_config* c) {
  if (!r || r->reserved != 0) return MP_ERR_INVALID_ARG;
  if (r->rot_dim < 0 || r->rot_dim > c->head_dim || (r->rot_dim & 1)) return MP_ERR_INVALID_ARG;
  if (r->interleaved != 0 && r->interleaved != 1) return MP_ERR_INVALID_ARG;
  if (!(r->eps >= 0.f) || r->eps > 3e38f) return MP_ERR_INVALID_ARG;
  // vectors of 16 bytes hold whole halves of a rotation
  const int vec = c->dtype == MP_DTYPE_BF16 ? 8 : 4;
  if (!r->interleaved && r->rot_dim % (2 * vec) != 0) return MP_ERR_UNSUPPORTED;
  return MP_OK;
}

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// log2 of a power of two, else -1
inline int shift_of(int n) {
  for (int i = 0; i < 31; ++i)
    if (n == 1 << i) return i;
  return -1;
}

inline CacheCall cache_args(const mp_cache_config* c, const int32_t* table, const int32_t* cu_q, const int32_t* kv_len,
                            int total_q, int max_q, int max_kv, uint32_t* status) {
  CacheCall a;
  a.batch = c->batch;
  a.kvh = c->kv_heads;
  a.group = c->q_heads / c->kv_heads;
  a.d = c->head_dim;
  a.page_size = c->page_size;
  a.n_pages = c->n_pages;
  a.cols = c->max_pages;
  a.page_shift = shift_of(c->page_size);
  a.table = table;
  a.cu_q = cu_q;
  a.kv_len = kv_len;
  a.total_q = total_q;
  a.max_q = max_q;
  a.max_kv = max_kv;
  a.status = status;
  return a;
}

inline bool chunk_on_tensor_cores(const mp_cache_config* c, int max_q) {
  return c->dtype == MP_DTYPE_BF16 && !chunk_is_step(c->q_heads / c->kv_heads, max_q);
}
// Packed rows that partial results have to have a place for: all of them, unless most belong to no
// sequence. (A place for those alone cost the fp32 kernel, whose registers are full, 3 %.)
inline int64_t part_rows(const mp_cache_config* c, int total_q, int max_q) {
  return std::min(int64_t(total_q), 4 * int64_t(c->batch) * max_q);
}

// Memory that a call reads or writes (a null pointer is none).
struct Range {
  const void* p;
  uint64_t bytes;
};
inline bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && x < y + b.bytes && y < x + a.bytes;
}

}  // namespace mp
