// Cutting a cache to its budget: per (sequence, KV head) the slots to keep, and the copy
// of their rows of K and V into another cache.
//
// Selection orders the slots between the sinks and the window by their scores as unsigned
// keys (the order of the floats; both zeros alike, NaN lowest). The key of the want-th
// highest score is found by radix selection, four passes of 8 bits over the scores; slots
// above it stay, and of those equal to it the lowest ones that are still wanted.
// The copy reads and writes the kept rows once, in 16-byte vectors.
#include "mp_cache.cuh"

namespace mp {
namespace {

constexpr int kSel = 1024;

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);  // -inf -> 0x007fffff > 0
}

__global__ void __launch_bounds__(kSel) k_evict_select(const EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ int warp_sum[2][32];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_want;
  const CacheArgs& c = a.c;
  const int h = blockIdx.x, b = blockIdx.y;
  const int n = seq_of(c, b).n;
  const int64_t unit = int64_t(b) * c.kvh + h;
  const float* sc = a.scores + unit * (int64_t(c.cols) * c.page_size);
  int32_t* kept = a.kept + unit * a.budget;
  float* ds = a.dst_scores ? a.dst_scores + unit * (int64_t(a.dst_cols) * a.dst_page_size) : nullptr;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (h == 0 && tid == 0) a.dst_len[b] = min(n, a.budget);
  if (n <= a.budget) {
    for (int i = tid; i < n; i += kSel) {
      kept[i] = i;
      if (ds) ds[i] = sc[i];
    }
    return;
  }
  const int lo = a.n_sink, hi = n - a.window;
  int want = a.budget - a.n_sink - a.window;  // < hi - lo
  uint32_t prefix = 0;
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int i = lo + tid; i < hi; i += kSel) {
        const uint32_t k = order_key(sc[i]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        int left = want;
        int bin = 255;
        while (bin > 0 && int(hist[bin]) < left) left -= int(hist[bin--]);
        sh_prefix = prefix | (uint32_t(bin) << shift);
        sh_want = left;
      }
      __syncthreads();
      prefix = sh_prefix;
      want = sh_want;
      __syncthreads();
    }
  }
  // keep: every key above `prefix` and the first `want` keys equal to it (none at all when
  // nothing is wanted between the sinks and the window)
  const bool any = a.budget > a.n_sink + a.window;
  int base = 0, ties = 0;  // kept and tied slots before this round
  for (int i0 = 0; i0 < n; i0 += kSel) {
    const int i = i0 + tid;
    bool keep = false, tie = false;
    float x = 0.f;
    if (i < n) {
      x = sc[i];
      if (i < lo || i >= hi) keep = true;
      else if (any) {
        const uint32_t k = order_key(x);
        keep = k > prefix;
        tie = k == prefix;
      }
    }
    const uint32_t tb = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) warp_sum[0][warp] = __popc(tb);
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
      before += w < warp ? warp_sum[0][w] : 0;
      all += warp_sum[0][w];
    }
    if (tie && ties + before + __popc(tb & ((1u << lane) - 1u)) < want) keep = true;
    ties += all;
    const uint32_t kb = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) warp_sum[1][warp] = __popc(kb);
    __syncthreads();
    before = 0;
    all = 0;
    for (int w = 0; w < 32; ++w) {
      before += w < warp ? warp_sum[1][w] : 0;
      all += warp_sum[1][w];
    }
    if (keep) {
      const int at = base + before + __popc(kb & ((1u << lane) - 1u));
      kept[at] = i;
      if (ds) ds[at] = x;
    }
    base += all;
  }
}

// One 16-byte vector of K and of V per thread; rows of a (sequence, KV head) in order.
template <int ROW>  // vectors per row
__global__ void __launch_bounds__(256) k_evict_gather(const EvictArgs a) {
  const CacheArgs& c = a.c;
  const int h = blockIdx.y, b = blockIdx.z;
  const int m = min(seq_of(c, b).n, a.budget);
  const int j = blockIdx.x * (256 / ROW) + threadIdx.x / ROW, e = threadIdx.x % ROW;
  if (j >= m) return;
  const int32_t src = a.kept[(int64_t(b) * c.kvh + h) * a.budget + j];
  const int col = j / a.dst_page_size;
  const int p = page_at(a.dst_table, a.dst_cols, a.dst_n_pages, b, col, c.status);
  if (p < 0) return;
  const int64_t from = slot_read(c, b, h, src) / c.d * ROW + e;
  const int64_t to = ((int64_t(p) * c.kvh + h) * a.dst_page_size + (j - col * a.dst_page_size)) * ROW + e;
  static_cast<uint4*>(a.dst_keys)[to] = static_cast<const uint4*>(a.keys)[from];
  static_cast<uint4*>(a.dst_values)[to] = static_cast<const uint4*>(a.values)[from];
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t st) {
  k_evict_select<<<dim3(a.c.kvh, a.c.batch), kSel, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_evict_gather(const EvictArgs& a, int dtype, cudaStream_t st) {
  const int row = a.c.d * (dtype == MP_DTYPE_BF16 ? 2 : 4) / 16;
  const int most = a.budget < a.c.max_kv ? a.budget : a.c.max_kv;
  const dim3 grid((most + 256 / row - 1) / (256 / row), a.c.kvh, a.c.batch);
  if (row == 8) k_evict_gather<8><<<grid, 256, 0, st>>>(a);
  else if (row == 16) k_evict_gather<16><<<grid, 256, 0, st>>>(a);
  else k_evict_gather<32><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace mp
