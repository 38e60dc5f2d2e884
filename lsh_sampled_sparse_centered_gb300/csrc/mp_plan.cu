// One step's lengths, pages and packed rows from how each sequence changes.
//
// Per sequence three running sums say everything: rows, pages taken and pages given back before it.
// The free pages with those given back behind them are one list e = 0, 1, ..., free + back - 1, of
// which the a-th page taken is entry free + back - 1 - a: where an entry lies (in the list as it was,
// or in the table of a sequence that shrinks) follows from the sums, so that no page has to be moved
// before another can be taken. What this reads (entries below n_free, pages of sequences that shrink) is
// written by no one, except lengths and n_free where they are updated in place: those are written behind
// a barrier, and so are the rows, which read their pages from the tables.
//
// Bound by latency: the sums are formed by every CTA for itself (a few reads a sequence) and rows and
// pages are shared out to one CTA, or a cluster of eight where there are many (64 single tokens 5.5 us a call,
// 1000 sequences with 29000 rows 12.4; an empty launch is 4).
#include <algorithm>

#include "mp_cache_host.h"
#include "mp_tc.cuh"

namespace mp {
namespace {

struct PlanArgs {
  int batch, page_size, page_shift, cols, n_pages, max_rows;
  const int32_t *change, *base, *kv_len, *n_free;
  int32_t *table, *free, *new_len, *new_free, *cu_q, *positions, *slots, *row_seq;
  uint32_t* status;
};

constexpr int kMostThreads = 1024;
constexpr int kCluster = 8;

// the last i in [0, n) with at[i] <= x, where at[0] = 0 <= x < at[n]
__device__ __forceinline__ int owner(const uint32_t* at, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <bool CLUSTER>
__global__ void __launch_bounds__(kMostThreads) k_cache_plan(const PlanArgs a) {
  extern __shared__ uint32_t sm[];
  __shared__ uint32_t sums[3][32];
  const int batch = a.batch, threads = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t* rows = sm;                    // [batch + 1], before each sequence
  uint32_t* taken = rows + batch + 1;     // [batch + 1] pages
  uint32_t* back = taken + batch + 1;     // [batch + 1] pages
  int* old_len = reinterpret_cast<int*>(back + batch + 1);  // [batch]
  int* left = old_len + batch;            // [batch]: of the old slots
  int* base = left + batch;               // [batch]
  const int rank = CLUSTER ? int(blockIdx.x) : 0, ctas = CLUSTER ? int(gridDim.x) : 1;
  auto pages = [&](int n) {
    const uint32_t up = uint32_t(n) + uint32_t(a.page_size) - 1u;
    return int(a.page_shift >= 0 ? up >> a.page_shift : up / uint32_t(a.page_size));
  };
  const int64_t cap = int64_t(a.cols) * a.page_size;
  uint32_t wrong = 0;

  const int given_free = a.table ? *a.n_free : 0;
  const int n_free = max(0, min(given_free, a.n_pages));
  if (a.table && n_free != given_free) wrong |= MP_STATUS_BAD_LENGTH;
  // Sums stop at a value that no comparison below tells from a larger one, so 32 bits hold them (rows and
  // pages are at most 2^30 each: a table's pages have 16 slots or more): min(a + b, top) is associative.
  const uint32_t top[3] = {uint32_t(a.max_rows) + 1, uint32_t(a.table ? a.n_pages : 0) + 1, uint32_t(a.table ? a.n_pages : 0) + 1};
  uint32_t carry[3] = {0, 0, 0};
  if (tid == 0) rows[0] = taken[0] = back[0] = 0;
  for (int b0 = 0; b0 < batch; b0 += threads) {
    const int b = b0 + tid;
    uint32_t v[3] = {0, 0, 0};
    if (b < batch) {
      const int given = a.kv_len[b], x = a.change[b];
      base[b] = a.base ? a.base[b] : 0;
      const int n = int(max(int64_t(0), min(int64_t(given), cap)));
      int grow = max(x, 0);
      if (n != given || int64_t(n) + grow > cap) wrong |= MP_STATUS_BAD_LENGTH;
      if (int64_t(n) + grow > cap) grow = 0;
      const int keep = int(max(int64_t(0), int64_t(n) + min(x, 0)));
      old_len[b] = n;
      left[b] = keep;
      v[0] = min(uint32_t(grow), top[0]);
      if (a.table) {
        v[1] = min(uint32_t(pages(n + grow) - pages(n)), top[1]);
        v[2] = min(uint32_t(pages(n) - pages(keep)), top[2]);
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, v[k], o);
        if (lane >= o) v[k] = min(v[k] + up, top[k]);
      }
    if (lane == 31)
#pragma unroll
      for (int k = 0; k < 3; ++k) sums[k][warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint32_t all = lane < threads / 32 ? sums[k][lane] : 0;  // of the warps up to this lane's
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all = min(all + up, top[k]);
      }
      const uint32_t pre = __shfl_sync(0xffffffffu, all, max(0, warp - 1));
      v[k] = min(carry[k] + min(v[k] + (warp ? pre : 0), top[k]), top[k]);
      carry[k] = min(carry[k] + __shfl_sync(0xffffffffu, all, 31), top[k]);
    }
    if (b < batch) {
      rows[b + 1] = v[0];
      taken[b + 1] = v[1];
      back[b + 1] = min(v[2], uint32_t(a.n_pages - n_free));
    }
    __syncthreads();
  }
  if (carry[2] > uint32_t(a.n_pages - n_free)) wrong |= MP_STATUS_BAD_LENGTH;
  const uint32_t list = uint32_t(n_free) + back[batch];  // free pages and those given back
  int served = 0;                                        // sequences before the first that has to wait
  for (int b0 = 0; b0 < batch; b0 += threads) {
    const int b = b0 + tid;
    served += __syncthreads_count(b < batch && rows[b + 1] <= uint32_t(a.max_rows) && taken[b + 1] <= list);
  }
  if (served < batch) wrong |= MP_STATUS_NO_ROOM;
  const uint32_t all_rows = rows[served], all_taken = taken[served];

  // where entry e of the list lies
  auto entry = [&](uint32_t e) -> const int32_t* {
    if (e < uint32_t(n_free)) return a.free + e;
    const int b = owner(back, batch, e - n_free), col = pages(left[b]) + int(e - n_free - back[b]);
    if (!inside(b >= 0 && b < batch && col >= 0 && col < a.cols && e < uint32_t(a.n_pages), a.status)) return a.table;
    return a.table + int64_t(b) * a.cols + col;
  };
  auto checked = [&](int p) {
    if (p < 0 || p >= a.n_pages) wrong |= MP_STATUS_BAD_PAGE;
    return p;
  };
  // What the loops over rows and pages given back wait for is a load per element, at a place that shared
  // memory gives: kAtOnce of them are in flight.
  constexpr int kAtOnce = 4;
  const uint32_t first = uint32_t(rank * threads + tid), step = uint32_t(ctas * threads);
  for (uint32_t i = first; i < all_taken; i += step) {
    const int b = owner(taken, served, i), col = pages(old_len[b]) + int(i - taken[b]);
    if (inside(b >= 0 && b < batch && col >= 0 && col < a.cols, a.status)) a.table[int64_t(b) * a.cols + col] = checked(*entry(list - 1 - i));
  }
  // pages given back and not taken again
  for (uint32_t e0 = uint32_t(n_free) + first; e0 + all_taken < list; e0 += kAtOnce * step) {
    int page[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const uint32_t e = e0 + k * step;
      page[k] = e + all_taken < list ? *entry(e) : 0;
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const uint32_t e = e0 + k * step;
      if (e + all_taken < list && inside(e < uint32_t(a.n_pages), a.status)) a.free[e] = checked(page[k]);
    }
  }
  // The pages taken are in the tables, and every CTA has read the lengths and n_free.
  if (CLUSTER) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  // kAtOnce rows from r0 on, `by` apart and before `end`; b_of says whose a row is
  auto write_rows = [&](uint32_t r0, uint32_t by, uint32_t end, auto b_of) {
    int b[kAtOnce], slot[kAtOnce], page[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const uint32_t r = r0 + k * by;
      if (r >= end) continue;
      b[k] = b_of(r);
      if (!inside(b[k] >= 0 && b[k] < batch && r < uint32_t(a.max_rows), a.status)) b[k] = 0;
      slot[k] = old_len[b[k]] + int(r - rows[b[k]]);
      page[k] = b[k];
      if (a.slots && a.table && inside(slot[k] >= 0 && slot[k] < cap, a.status)) page[k] = __ldcg(a.table + int64_t(b[k]) * a.cols + (pages(slot[k] + 1) - 1));
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const uint32_t r = r0 + k * by;
      if (r >= end || !inside(r < uint32_t(a.max_rows), a.status)) continue;
      if (a.positions) a.positions[r] = int(uint32_t(base[b[k]]) + uint32_t(slot[k]));
      if (a.row_seq) a.row_seq[r] = b[k];
      if (a.slots) {
        const int p = checked(page[k]), at = slot[k] - (pages(slot[k] + 1) - 1) * a.page_size;
        a.slots[r] = p >= 0 && p < a.n_pages ? p * a.page_size + at : -1;
      }
    }
  };
  const bool any_rows = a.positions || a.slots || a.row_seq;
  if (any_rows && !CLUSTER) {
    for (uint32_t r = first; r < all_rows; r += kAtOnce * step) write_rows(r, step, all_rows, [&](uint32_t at) { return owner(rows, served, at); });
  }
  if (any_rows && CLUSTER) {
    // Many rows: a search each is more than all the rest, so a tile's owners are marked where their rows
    // begin and carried on by a running maximum (31000 rows of 1000 sequences: 6 us of searches).
    uint32_t* own = reinterpret_cast<uint32_t*>(base + batch);  // [kAtOnce * threads]
    const uint32_t most = uint32_t(kAtOnce * threads), share = (all_rows + ctas - 1) / ctas, tile = min(most, max(1u, share));
    for (uint32_t begin = rank * tile; begin < all_rows; begin += ctas * tile) {
      const uint32_t end = min(all_rows, begin + tile);
      for (uint32_t i = tid; i < most; i += threads) own[i] = 0;
      __syncthreads();
      const int b0 = owner(rows, served, begin), b1 = owner(rows, served, end - 1);
      for (int b = b0 + tid; b <= b1; b += threads)
        if (rows[b + 1] > rows[b] && inside(max(rows[b], begin) - begin < most, a.status)) own[max(rows[b], begin) - begin] = uint32_t(b);
      __syncthreads();
      uint32_t v[kAtOnce], high = 0;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) v[k] = high = max(high, own[tid * kAtOnce + k]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, high, o);
        if (lane >= o) high = max(high, up);
      }
      if (lane == 31) sums[0][warp] = high;
      __syncthreads();
      uint32_t before = __reduce_max_sync(0xffffffffu, lane < warp ? sums[0][lane] : 0u);
      const uint32_t up = __shfl_up_sync(0xffffffffu, high, 1);
      if (lane > 0) before = max(before, up);
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) own[tid * kAtOnce + k] = max(v[k], before);
      __syncthreads();
      write_rows(begin + tid, threads, end, [&](uint32_t at) { return int(own[at - begin]); });
      __syncthreads();  // own and sums are written again
    }
  }
  for (int b = int(first); b < batch; b += int(step)) {
    a.new_len[b] = left[b] + (b < served ? int(rows[b + 1] - rows[b]) : 0);
    a.cu_q[b] = int(min(rows[b], all_rows));
  }
  if (first == 0) {
    a.cu_q[batch] = int(all_rows);
    if (a.table) *a.new_free = int(list - all_taken);
  }
  if (wrong) flag(a.status, wrong);
}

size_t plan_smem(int batch, int threads) { return (size_t(batch) * 6 + 3 + 4 * threads) * 4; }

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t st) {
  const bool many = std::max(a.batch, a.max_rows) > kMostThreads;
  const int threads = std::min(kMostThreads, (std::max(a.batch, std::min(a.max_rows, kMostThreads)) + 31) / 32 * 32);
  const size_t smem = plan_smem(a.batch, threads);
  if (smem > 40 * 1024) {  // 48 KB with the static part need no asking
    const cudaError_t e = many ? allow_smem<k_cache_plan<true>>() : allow_smem<k_cache_plan<false>>();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(many ? kCluster : 1);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = many ? 1 : 0;
  return many ? cudaLaunchKernelEx(&cfg, k_cache_plan<true>, a) : cudaLaunchKernelEx(&cfg, k_cache_plan<false>, a);
}

}  // namespace
}  // namespace mp

using namespace mp;

extern "C" int mp_cache_plan(const mp_cache_config* cfg, const int32_t* change, const int32_t* base, const int32_t* kv_len,
                             const int32_t* n_free, int32_t max_rows, int32_t* page_table, int32_t* free_pages,
                             int32_t* new_len, int32_t* new_free, int32_t* cu_q, int32_t* positions, int32_t* slots,
                             int32_t* row_seq, uint32_t* status, void* stream) {
  int rc = check_cache(cfg);
  if (rc != MP_OK) return rc;
  if ((rc = check_pages(cfg, page_table)) != MP_OK) return rc;
  if (max_rows < 0 || !change || !kv_len || !new_len || !cu_q) return MP_ERR_INVALID_ARG;
  if (page_table && (!n_free || !free_pages || !new_free)) return MP_ERR_INVALID_ARG;
  if (cfg->batch > MP_PLAN_SEQUENCES || max_rows > (1 << 30)) return MP_ERR_UNSUPPORTED;
  const uint64_t b = uint64_t(cfg->batch);
  const Range used[] = {{change, b * 4},
                        {base, b * 4},
                        {kv_len, b * 4},
                        {page_table ? n_free : nullptr, 4},
                        {page_table, b * cfg->max_pages * 4},
                        {page_table ? free_pages : nullptr, uint64_t(cfg->n_pages) * 4},
                        {new_len, b * 4},
                        {page_table ? new_free : nullptr, 4},
                        {cu_q, b * 4 + 4},
                        {positions, uint64_t(max_rows) * 4},
                        {slots, uint64_t(max_rows) * 4},
                        {row_seq, uint64_t(max_rows) * 4},
                        {status, 4}};
  constexpr int kUsed = sizeof(used) / sizeof(used[0]), kInputs = 4;  // inputs may overlap each other
  for (const Range& r : used)
    if (!aligned4(r.p)) return MP_ERR_INVALID_ARG;
  if (injected("plan")) return MP_ERR_INJECTED;
  for (int i = 0; i < kUsed; ++i)
    for (int j = std::max(i + 1, kInputs); j < kUsed; ++j)
      if (overlap(used[i], used[j]) && !(used[i].p == used[j].p && ((i == 2 && j == 6) || (i == 3 && j == 7))))  // updated in place
        return MP_ERR_INVALID_ARG;
  PlanArgs a;
  a.batch = cfg->batch;
  a.page_size = cfg->page_size;
  a.page_shift = shift_of(cfg->page_size);
  a.cols = cfg->max_pages;
  a.n_pages = cfg->n_pages;
  a.max_rows = max_rows;
  a.change = change;
  a.base = base;
  a.kv_len = kv_len;
  a.n_free = n_free;
  a.table = page_table;
  a.free = free_pages;
  a.new_len = new_len;
  a.new_free = new_free;
  a.cu_q = cu_q;
  a.positions = positions;
  a.slots = slots;
  a.row_seq = row_seq;
  a.status = status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaGetLastError();
  ProfScope ps(st, K_CACHE_PLAN);
  return launch_plan(a, st) == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}
