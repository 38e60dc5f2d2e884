// What the cache operators' kernels share: the sequences of a packed batch, cut to the
// call's limits, and the address of a cache slot.
#pragma once

#include "mp_internal.h"

namespace mp {

// One layer's paged cache and the packed batch of a call (host-checked limits).
struct CacheArgs {
  int batch, kvh, group, d;      // group = q_heads / kv_heads
  int page_size, n_pages, cols;  // cols: columns of the page table
  int page_shift;                // log2(page_size) where it is a power of two, else -1
  const int32_t* table;          // nullptr: page b is sequence b's cache
  const int32_t* cu_q;           // nullptr: no packed rows (eviction)
  const int32_t* kv_len;
  int total_q, max_q, max_kv;
  uint32_t* status;              // may be nullptr
};

struct ChunkArgs {
  CacheArgs c;
  const void *q, *keys, *values;
  void* out;
  float* lse;   // may be nullptr
  // partial results in the workspace: slices [splits][total_q][q_heads], or (tensor cores)
  // slots of the pieces of tiles that are shared by CTAs
  int splits;   // slices of the keys per row tile
  bool joined;  // the slices are a cluster that joins itself
  float* part;  // [..][d]: unnormalised sums
  float* ml;    // [..][2]: their reference (log2) and sum
  void* cuts;   // shared tiles (tensor cores)
#if MP_CHECK
  bool stall;  // one CTA stops half way, so that the others' waits run out
#endif
};

struct WeightsArgs {
  CacheArgs c;
  const void *q, *keys;
  const float* lse;
  float* scores;
#if MP_CHECK
  bool stall;
#endif
};

struct AppendArgs {
  CacheArgs c;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const void *q_norm, *k_norm;
  const double* inv_freq;
  const int32_t* positions;
  int rot, interleaved;
  float eps;
  void *keys, *values, *q_out;
};

struct EvictArgs {
  CacheArgs c;
  const void *keys, *values;
  const float* scores;
  int n_sink, window, budget;
  void *dst_keys, *dst_values;
  const int32_t* dst_table;
  int dst_page_size, dst_n_pages, dst_cols;
  float* dst_scores;
  int32_t* dst_len;
  int32_t* kept;  // [batch][kv_heads][budget]
};

constexpr int kChunkRows = 64;  // query rows of a tile of the fp32 kernels

// What the limits alone fix, so that a workspace can be sized before the call: slices of the
// keys (fp32, and bf16 with few query rows), CTAs of the tensor-core kernel and its workspace.
int chunk_splits(const mp_cache_config* c, int max_q, int max_kv);
bool chunk_is_step(int group, int max_q);
struct StepPlan {
  int splits;
  bool joined;  // the slices join themselves
};
StepPlan chunk_step_plan(const mp_cache_config* c, int max_q, int max_kv);
int chunk_step_most(const mp_cache_config* c, int max_q, int max_kv);  // separate slices of any cache of up to max_kv slots
int chunk_tc_ctas(int batch, int kvh, int group, int max_q, int max_kv);
uint64_t chunk_tc_workspace(const mp_cache_config* c, int max_q, int max_kv);

// Rows of a TMA box of K or V: the most that divide a 128-key tile and never leave a page
// (16 at least: page sizes are multiples of 16). Without a table a box may run past the
// sequence's end into other rows of the pool, which are masked or zeroed.
inline int box_rows(const int32_t* table, int page_size) {
  int b = 128;
  while (table && page_size % b) b >>= 1;
  return b;
}

cudaError_t launch_cache_append(const AppendArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_chunk_simt(const ChunkArgs& a, cudaStream_t st);
cudaError_t launch_chunk_step(const ChunkArgs& a, cudaStream_t st);
cudaError_t launch_chunk_join(const ChunkArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_chunk_tc(const ChunkArgs& a, void* workspace, cudaStream_t st);
cudaError_t launch_cache_weights(const WeightsArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_weights_bf16(const WeightsArgs& a, cudaStream_t st);
cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t st);
cudaError_t launch_evict_gather(const EvictArgs& a, int dtype, cudaStream_t st);

#ifdef __CUDACC__
// The index arithmetic below also compiles for the host, where a test walks it over bad
// lengths and pages.
__host__ __device__ __forceinline__ void flag(uint32_t* status, uint32_t bit) {
  if (!status) return;
#ifdef __CUDA_ARCH__
  atomicOr(status, bit);
#else
  *status |= bit;
#endif
}

// Sequence b's packed rows [row0, row0 + m) and its n slots, cut to the call's limits, and the
// slot that row row0 stands in. That slot goes by the lengths as they are, so that a cut moves
// no token: row r is in slot kv_len - cu_q[b + 1] + r. Where every slot is behind (before) the
// cut ones, any value from n - 1 on (up to -m) says the same and `first` is that limit.
struct Seq {
  int row0, m, n, first;
  __host__ __device__ int seen() const { return max(0, min(n, first + m)); }  // slots that any row sees
};
__host__ __device__ __forceinline__ Seq seq_of(const CacheArgs& c, int b) {
  Seq s;
  const int64_t slots = int64_t(c.cols) * c.page_size;
  const int n = c.kv_len[b];
  s.n = max(0, min(n, int(min(int64_t(c.max_kv), slots))));
  bool cut = s.n != n;
  int r1 = 0;
  if (c.cu_q) {
    const int r0 = c.cu_q[b];
    r1 = c.cu_q[b + 1];
    s.row0 = max(0, min(r0, c.total_q));
    const int e = max(s.row0, min(r1, c.total_q));
    s.m = min(e - s.row0, c.max_q);
    cut = cut || s.row0 != r0 || s.row0 + s.m != r1;
  } else {
    s.row0 = 0;
    s.m = 0;
  }
  s.first = s.n - s.m;
  if (cut) {
    if (c.cu_q) s.first = int(max(int64_t(-s.m), min(int64_t(n) - r1 + s.row0, int64_t(s.n) - 1)));
    flag(c.status, MP_STATUS_BAD_LENGTH);
  }
  return s;
}

// Of numbers that are not negative; nearly always of 32 bits, where it costs a fraction.
__host__ __device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return uint64_t(a | b) >> 32 ? a / b : int64_t(uint32_t(a) / uint32_t(b));
}

// Sequence that packed row r belongs to, or -1: the last b with cu_q[b] <= r, if r is
// one of its rows. A table that decreases somewhere gives some sequence or none, never
// an index outside it.
__host__ __device__ __forceinline__ int seq_at(const CacheArgs& c, int r) {
  int lo = 0, hi = c.batch;  // cu_q[lo] <= r is kept where it holds for 0
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c.cu_q[mid] <= r) lo = mid;
    else hi = mid;
  }
  return (c.cu_q[lo] <= r && r < c.cu_q[lo + 1]) ? lo : -1;
}

#ifdef __CUDACC__
// The same for a whole warp that asks for one row: 32 boundaries are looked at at a time, so
// that up to 33 sequences take one round of loads and not five that wait for each other.
__device__ __forceinline__ int seq_at_warp(const CacheArgs& c, int r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = c.batch;  // cu_q[lo] <= r is kept where it holds for 0
  while (hi - lo > 1) {
    const int step = (hi - lo + 32) / 33, at = lo + (lane + 1) * step;
    const uint32_t below = __ballot_sync(0xffffffffu, at < hi && c.cu_q[min(at, hi - 1)] <= r);
    const int k = below == 0xffffffffu ? 32 : __ffs(~below) - 1;  // the first boundaries in a row
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return (c.cu_q[lo] <= r && r < c.cu_q[lo + 1]) ? lo : -1;
}
#endif

// Pool page of slot s (0 <= s < cols * page_size), or -1 when the table names none.
__host__ __device__ __forceinline__ int page_at(const int32_t* table, int cols, int n_pages, int b, int col, uint32_t* status) {
  if (!table) return b;
  const int p = table[int64_t(b) * cols + col];
  if (p < 0 || p >= n_pages) {
    flag(status, MP_STATUS_BAD_PAGE);
    return -1;
  }
  return p;
}

// Row of the pool that holds slot s of KV head h, for reading: a bad page reads page 0
// instead. The pool's rows are 32-bit (checked by the host).
__host__ __device__ __forceinline__ int slot_row(const CacheArgs& c, int b, int h, int s) {
  if (!c.table) return (b * c.kvh + h) * c.page_size + s;
  const int col = c.page_shift >= 0 ? s >> c.page_shift : s / c.page_size;
  const int p = max(0, page_at(c.table, c.cols, c.n_pages, b, col, c.status));
  return (p * c.kvh + h) * c.page_size + (s - col * c.page_size);
}
// Its element offset.
__host__ __device__ __forceinline__ int64_t slot_read(const CacheArgs& c, int b, int h, int s) {
  return int64_t(slot_row(c, b, h, s)) * c.d;
}
#endif

}  // namespace mp
