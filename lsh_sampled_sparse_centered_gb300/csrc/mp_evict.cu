// Cutting a cache to its budget: per (sequence, KV head) the slots to keep, and the copy
// of their rows of K and V into another cache.
//
// Selection orders the slots by their scores as unsigned keys (the order of the floats;
// both zeros alike, NaN lowest; sinks and window above all). The key of the budget-th
// highest slot is found by radix selection in digits of 12, 10 and 10 bits; slots above it
// stay, and of those equal to it the lowest ones that are still wanted. A cluster of up to
// eight CTAs shares a head: each holds the keys of its part of the slots in shared memory
// and counts their digits; the counts that are not zero are added to the first CTA's through
// distributed shared memory (all CTAs reading all counts took twice as long), which finds
// the digit and hands it back. The first digit has 12 bits (sign, exponent, three of the
// mantissa) so that scores of like size spread over many counters.
// The copy reads and writes the kept rows (and their scores) once, in 16-byte vectors,
// bound by memory.
#include <cooperative_groups.h>

#include <algorithm>

#include "mp_cache.cuh"

namespace mp {
namespace {

namespace cg = cooperative_groups;

constexpr int kSel = 1024, kWarps = kSel / 32;
constexpr int kStage = 32768;  // slots of a CTA that shared memory holds

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);  // -inf -> 0x007fffff > 0
}

struct alignas(16) SelectSmem {
  uint32_t hist[4096];             // of this CTA's keys, one digit
  uint32_t total[4096 + 1024 + 1024];  // of the cluster's (first CTA), one set per digit
  uint32_t warp_sum[kWarps];
  int2 warp_count[kWarps];  // slots above the threshold key and slots equal to it, of each warp
  int2 count;               // of the CTA
  uint32_t digit;           // handed out by the first CTA
  int left;
};

// The digit in which the want-th highest counted key lies, and how many are still wanted
// in it: a suffix sum over the counters, every thread with its own run of bins.
template <int BITS>
__device__ __forceinline__ void find_digit(SelectSmem& S, const uint32_t* total, cg::cluster_group& cluster, int want) {
  constexpr int BINS = 1 << BITS, PER = BINS / kSel;  // bins of a thread, 4 or 1
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int first = BINS - (tid + 1) * PER;  // the highest bins belong to thread 0
  uint32_t n[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) sum += n[i] = total[first + i];
  uint32_t pre = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += v;
  }
  if (lane == 31) S.warp_sum[warp] = pre;
  __syncthreads();
  uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? S.warp_sum[lane] : 0u) + pre - sum;
  // the thread whose run crosses `want` (there is one: at least `want` keys were counted)
  if (before < uint32_t(want) && before + sum >= uint32_t(want)) {
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) {
      if (before < uint32_t(want) && before + n[i] >= uint32_t(want)) {
        for (int r = 0; r < int(cluster.num_blocks()); ++r) {
          *cluster.map_shared_rank(&S.digit, r) = uint32_t(first + i);
          *cluster.map_shared_rank(&S.left, r) = want - int(before);
        }
      }
      before += n[i];
    }
  }
}

__global__ void __launch_bounds__(kSel, 1) k_evict_select(const EvictArgs a) {
  __shared__ SelectSmem S;
  extern __shared__ uint32_t stage[];
  cg::cluster_group cluster = cg::this_cluster();
  const CacheCall& c = a.c;
  const int ranks = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int h = blockIdx.x / ranks, b = blockIdx.y;
  const int n = seq_of(c, b).n;
  const int64_t unit = int64_t(b) * c.kvh + h;
  const float* sc = a.scores + unit * (int64_t(c.cols) * c.page_size);
  int32_t* kept = a.kept + unit * a.budget;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (n <= a.budget) {  // the same for the whole cluster
    for (int i = rank * kSel + tid; i < n; i += ranks * kSel) kept[i] = i;
    return;
  }
  const int lo = a.n_sink, hi = n - a.window;
  // this CTA's slots [p0, p1), a whole number of 32 per warp
  const int per = ((n + ranks * kWarps - 1) / (ranks * kWarps) + 31) & ~31;
  const int p0 = min(n, rank * kWarps * per), p1 = min(n, p0 + kWarps * per);
  const bool staged = p1 - p0 <= kStage;
  auto score_key = [&](int i) { return i < lo || i >= hi ? 0xffffffffu : order_key(sc[i]); };
  for (int i = tid; i < 4096; i += kSel) S.hist[i] = 0;
  for (int i = tid; i < 4096 + 1024 + 1024; i += kSel) S.total[i] = 0;
  if (staged) {
    for (int i = p0 + tid; i < p1; i += 8 * kSel) {  // eight loads in flight
      uint32_t k[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) k[u] = i + u * kSel < p1 ? score_key(i + u * kSel) : 0u;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i + u * kSel < p1) stage[i + u * kSel - p0] = k[u];
    }
  }
  auto key = [&](int i) { return staged ? stage[i - p0] : score_key(i); };
  if (ranks > 1) cluster.sync();  // every CTA's totals are zero
  else __syncthreads();
  int want = a.budget;
  uint32_t prefix = 0;
#pragma unroll
  for (int d = 0; d < 3; ++d) {
    const int bits = d == 0 ? 12 : 10, shift = d == 0 ? 20 : (d == 1 ? 10 : 0), bins = 1 << bits;
    uint32_t* total = S.total + (d == 0 ? 0 : (d == 1 ? 4096 : 4096 + 1024));
    const uint32_t mask = d == 0 ? 0u : 0xffffffffu << (shift + bits);
    uint32_t* hist = ranks > 1 ? S.hist : total;
#pragma unroll 4
    for (int i = p0 + tid; i < p1; i += kSel) {
      const uint32_t k = key(i);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & uint32_t(bins - 1)], 1u);
    }
    if (ranks > 1) {
      __syncthreads();
      uint32_t* to = cluster.map_shared_rank(total, 0);
      for (int i = tid; i < bins; i += kSel) {
        const uint32_t v = hist[i];
        if (v) {
          atomicAdd(&to[i], v);
          hist[i] = 0;
        }
      }
      cluster.sync();
    } else {
      __syncthreads();
    }
    if (rank == 0) {
      if (d == 0) find_digit<12>(S, total, cluster, want);
      else find_digit<10>(S, total, cluster, want);
    }
    if (ranks > 1) cluster.sync();
    else __syncthreads();
    prefix |= S.digit << shift;
    want = S.left;
  }
  // Each warp owns a run of slots: counts first, then the places. Slots above the threshold
  // all stay, the first `want` of those equal to it too.
  const int i0 = min(n, p0 + warp * per), i1 = min(n, i0 + per);
  int above_n = 0, tie_n = 0;
#pragma unroll 4
  for (int i = i0; i < i1; i += 32) {
    const uint32_t k = i + lane < i1 ? key(i + lane) : 0u;
    above_n += k > prefix;
    tie_n += i + lane < i1 && k == prefix;
  }
  above_n = __reduce_add_sync(0xffffffffu, above_n);
  tie_n = __reduce_add_sync(0xffffffffu, tie_n);
  if (lane == 0) S.warp_count[warp] = make_int2(above_n, tie_n);
  __syncthreads();
  if (warp == 0) {
    const int2 v = S.warp_count[lane];
    const int2 all = make_int2(__reduce_add_sync(0xffffffffu, v.x), __reduce_add_sync(0xffffffffu, v.y));
    if (lane == 0) S.count = all;
  }
  if (ranks > 1) cluster.sync();
  // what the warps and CTAs before this one hold
  int2 v = lane < warp ? S.warp_count[lane] : make_int2(0, 0);
  if (lane < rank) {
    const int2 o = *cluster.map_shared_rank(&S.count, lane);
    v.x += o.x;
    v.y += o.y;
  }
  int above_before = __reduce_add_sync(0xffffffffu, v.x), tie_before = __reduce_add_sync(0xffffffffu, v.y);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // k_evict_gather may be set up
  const uint32_t lower = (1u << lane) - 1u;
#pragma unroll 4
  for (int i = i0; i < i1; i += 32) {
    const bool live = i + lane < i1;
    const uint32_t k = live ? key(i + lane) : 0u;
    const bool above = k > prefix, tie = live && k == prefix;
    const uint32_t tb = __ballot_sync(0xffffffffu, tie), ab = __ballot_sync(0xffffffffu, above);
    const int t = tie_before + __popc(tb & lower);  // ties before this slot
    if (above || (tie && t < want)) kept[above_before + __popc(ab & lower) + min(t, want)] = i + lane;
    above_before += __popc(ab);
    tie_before += __popc(tb);
  }
  if (ranks > 1) cluster.sync();  // no CTA leaves while others read its counts
}

// ROW 16-byte vectors per row, one lane each, kRowsEach rows of K and V per lane so that
// enough loads are in flight.
constexpr int kRowsEach = 2, kResident = 8;  // CTAs of an SM: 32 registers

template <int ROW>
__global__ void __launch_bounds__(256, kResident) k_evict_gather(const EvictArgs a) {
  constexpr int GROUPS = 256 / ROW;
  const CacheCall& c = a.c;
  const int h = blockIdx.y, b = blockIdx.z;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // k_evict_select has written the kept slots
  const int m = min(seq_of(c, b).n, a.budget);
  const int j0 = blockIdx.x * (GROUPS * kRowsEach) + threadIdx.x / ROW, e = threadIdx.x % ROW;
  // Here and not by the selection, whose CTAs all read the old length: dst_len may be kv_len (both
  // lengths give this kernel the same m).
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) a.dst_len[b] = m;
  if (j0 >= m) return;
  const int64_t unit = int64_t(b) * c.kvh + h;
  const int32_t* kept = a.kept + unit * a.budget;
  const uint4 *keys = static_cast<const uint4*>(a.keys), *values = static_cast<const uint4*>(a.values);
  int64_t to[kRowsEach];
  uint4 k[kRowsEach], v[kRowsEach];
  float score[kRowsEach];
#pragma unroll
  for (int i = 0; i < kRowsEach; ++i) {
    const int j = j0 + i * GROUPS;
    to[i] = -1;
    if (j >= m) continue;
    const int col = j / a.dst_page_size;
    const int p = page_at(a.dst_table, a.dst_cols, a.dst_n_pages, b, col, c.status);
    const int64_t from = int64_t(slot_row(c, b, h, kept[j])) * ROW + e;
    k[i] = __ldcs(keys + from);
    v[i] = __ldcs(values + from);
    if (e == 0 && a.dst_scores) score[i] = a.scores[unit * (int64_t(c.cols) * c.page_size) + kept[j]];
    if (p >= 0) to[i] = ((int64_t(p) * c.kvh + h) * a.dst_page_size + (j - col * a.dst_page_size)) * ROW + e;
  }
  if (e == 0 && a.dst_scores)  // (a bad page takes no row, the slot's score stands all the same)
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i)
      if (j0 + i * GROUPS < m) a.dst_scores[unit * (int64_t(a.dst_cols) * a.dst_page_size) + j0 + i * GROUPS] = score[i];
#pragma unroll
  for (int i = 0; i < kRowsEach; ++i)
    if (to[i] >= 0) {
      static_cast<uint4*>(a.dst_keys)[to[i]] = k[i];
      static_cast<uint4*>(a.dst_values)[to[i]] = v[i];
    }
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t st) {
  // about 4096 slots per CTA; clusters of up to eight are always schedulable
  int ranks = 1;
  while (ranks < 8 && int64_t(ranks) * 4096 < a.c.max_kv) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.c.kvh * ranks, a.c.batch);
  cfg.blockDim = dim3(kSel);
  const int64_t part = ((int64_t(a.c.max_kv) + ranks * kWarps - 1) / (ranks * kWarps) + 31) / 32 * 32 * kWarps;
  cfg.dynamicSmemBytes = size_t(std::min<int64_t>(part, kStage)) * 4;
  cudaError_t e = cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, kStage * 4);
  if (e != cudaSuccess) return e;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_evict_select, a);
}

cudaError_t launch_evict_gather(const EvictArgs& a, int dtype, cudaStream_t st) {
  const int row = a.c.d * (dtype == MP_DTYPE_BF16 ? 2 : 4) / 16;
  const int most = a.budget < a.c.max_kv ? a.budget : a.c.max_kv;
  const int per = 256 / row * kRowsEach;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((most + per - 1) / per, a.c.kvh, a.c.batch);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return row == 8    ? cudaLaunchKernelEx(&cfg, k_evict_gather<8>, a)
         : row == 16 ? cudaLaunchKernelEx(&cfg, k_evict_gather<16>, a)
                     : cudaLaunchKernelEx(&cfg, k_evict_gather<32>, a);
}

}  // namespace mp
