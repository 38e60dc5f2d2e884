// Exact attention of few query rows per KV head (single tokens, a handful of draft tokens),
// bf16: bound by one pass over K and V.
//
// At most 16 rows (tokens x heads of the group) per KV head. The slots are cut into slices,
// one CTA each, 16 slots per warp and round. K and V go from global memory straight into
// the fragments of warp-level products, so that nothing but registers holds them:
//   S[row][key]: the sum over d has no order to keep, so lane t of a key's four takes the
//     16-byte chunks t, t + 4, ... and feeds their halves to two products.
//   O^T[d][row] += V^T P^T: lane (g, t) holds chunk g of V of the keys 2t, 2t + 1, 2t + 8
//     and 2t + 9; element i of the chunks makes the 16 x 16 tile of the d that are i modulo 8.
//     The accumulators of S are P^T's fragments as they stand.
// Loads of the next round are issued as soon as their registers are free. The reference of
// a row's softmax is raised only when a logit passes it by more than 8 (log2). P enters the
// second product as the sum of two bf16 terms (2^-17 relative per weight): the products are
// a few percent of the time, and one term would double the result's error.
#include <cooperative_groups.h>

#include <atomic>

#include "mp_cache.cuh"
#include "mp_tc.cuh"

namespace mp {
namespace {

namespace cg = cooperative_groups;

constexpr int kRound = 16;  // slots of a warp and round
__host__ __device__ constexpr int warps_of(bool joined) { return joined ? 8 : 4; }
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.0f;
// Slots of a cache, and of a slice, up to which the slices may be a cluster that joins itself
constexpr int kShort = 4096, kSlice = 1024;

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w)); }
// element e (0..7) of the 16-byte chunks a and b as one pair
__device__ __forceinline__ uint32_t pair(const uint4& a, const uint4& b, int e) {
  return __byte_perm(word(a, e >> 1), word(b, e >> 1), (e & 1) ? 0x7632 : 0x5410);
}

// NT: query rows in eights. JOINED: the slices of a KV head are a cluster and join through
// distributed shared memory (no second kernel, no workspace).
template <int D, int NT, bool JOINED>
__global__ void __launch_bounds__(warps_of(JOINED) * 32) k_chunk_step(const ChunkArgs a) {
  constexpr int kWarps = warps_of(JOINED);
  constexpr int KC = D / 32;      // chunks of a K row per lane
  constexpr int VC = D / 64;      // chunks of a V row per lane
  constexpr int TILES = D / 16;   // 16-row tiles of O^T
  __shared__ float so[kWarps][NT * 8][D + 4];
  __shared__ float sm[kWarps][NT * 8], sl[kWarps][NT * 8];
  const CacheCall& c = a.c;
  const int b = blockIdx.z, h = blockIdx.y, split = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Seq s = seq_of(c, b);
  const int rows = s.m * c.group, first = s.first, qh = c.kvh * c.group;
  // A cluster goes through its barriers without new tokens too: were the length written meanwhile
  // (a caller that does not wait for its own copy), a CTA that had left would be read by the
  // others, which faults.
  if (!JOINED && rows == 0) return;
  // this CTA's slots, a whole number of rounds of all warps
  const int per = ((s.n + a.splits - 1) / a.splits + kWarps * kRound - 1) / (kWarps * kRound) * (kWarps * kRound);
  const int k0 = int(min(int64_t(s.n), int64_t(split) * per)), k1 = rows == 0 ? k0 : min(s.n, k0 + per);

  // Q: row r of the tile is token r / group, head r % group; rows behind the last are zero
  uint4 q[NT][KC];
  int see[NT];  // the lane's row (8 u + g) sees the slots below this
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int r = u * 8 + g;
    see[u] = r < rows ? min(s.n, first + r / c.group + 1) : 0;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                               (int64_t(s.row0 + r / c.group) * qh + h * c.group + r % c.group) * D + t * 8;
#pragma unroll
    for (int i = 0; i < KC; ++i)
      q[u][i] = r < rows ? *reinterpret_cast<const uint4*>(src + i * 32) : make_uint4(0, 0, 0, 0);
  }
  const float scale = kLog2e * rsqrtf(float(D));
  float o[NT][TILES][4], m[NT], l[NT];
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    m[u] = -INFINITY;
    l[u] = 0.f;
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[u][i][j] = 0.f;
  }
  const __nv_bfloat16 *keys = static_cast<const __nv_bfloat16*>(a.keys), *values = static_cast<const __nv_bfloat16*>(a.values);
  uint4 k[2][KC], v[4][VC];
  // Rows of the pool for a round's slots, looked up a round ahead of their loads. Slots behind
  // the last are read as the last: their weights are zero.
  int rk[2], rv[4];
  auto find_k = [&](int n0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) rk[i] = slot_row(c, b, h, min(n0 + g + 8 * i, s.n - 1));
  };
  auto find_v = [&](int n0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) rv[i] = slot_row(c, b, h, min(n0 + 2 * t + (i & 1) + 8 * (i >> 1), s.n - 1));
  };
  auto load_k = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __nv_bfloat16* src = keys + int64_t(rk[i]) * D + t * 8;
#pragma unroll
      for (int j = 0; j < KC; ++j) k[i][j] = __ldcs(reinterpret_cast<const uint4*>(src + j * 32));
    }
  };
  auto load_v = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat16* src = values + int64_t(rv[i]) * D + g * 8;
#pragma unroll
      for (int j = 0; j < VC; ++j) v[i][j] = __ldcs(reinterpret_cast<const uint4*>(src + j * 64));
    }
  };
  int n0 = k0 + warp * kRound;
  if (n0 < k1) {
    find_k(n0);
    load_k();
    find_v(n0);
    load_v();
    find_k(n0 + kWarps * kRound);
    find_v(n0 + kWarps * kRound);
  }
  for (; n0 < k1; n0 += kWarps * kRound) {
    const int next = n0 + kWarps * kRound;
    // S: x[u][key half][..]: rows g (and 8 + g), keys 2t, 2t + 1 of each half
    float x[NT][2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        mma_16816(d, q[0][j].x, NT > 1 ? q[NT - 1][j].x : 0u, q[0][j].y, NT > 1 ? q[NT - 1][j].y : 0u, k[i][j].x, k[i][j].y);
        mma_16816(d, q[0][j].z, NT > 1 ? q[NT - 1][j].z : 0u, q[0][j].w, NT > 1 ? q[NT - 1][j].w : 0u, k[i][j].z, k[i][j].w);
      }
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          x[u][i][j] = n0 + 8 * i + 2 * t + j < see[u] ? d[2 * u + j] * scale : -INFINITY;
    }
    if (next < k1) {
      load_k();
      find_k(next + kWarps * kRound);
    }
    uint32_t p[NT][2], rest[NT][2];  // P and what its rounding leaves
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      float top = fmaxf(fmaxf(x[u][0][0], x[u][0][1]), fmaxf(x[u][1][0], x[u][1][1]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const bool raise = top > m[u] + kRaise || (m[u] == -INFINITY && top > m[u]);
      if (__any_sync(0xffffffffu, raise)) {
        const float by = raise ? exp2f(m[u] - top) : 1.f;  // 0 for the first reference
        if (raise) m[u] = top;
        l[u] *= by;
        const float b0 = __shfl_sync(0xffffffffu, by, 8 * t), b1 = __shfl_sync(0xffffffffu, by, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
          o[u][i][0] *= b0;
          o[u][i][1] *= b1;
          o[u][i][2] *= b0;
          o[u][i][3] *= b1;
        }
      }
      const float ref = m[u] == -INFINITY ? 0.f : m[u];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float e0 = ex2(x[u][i][0] - ref), e1 = ex2(x[u][i][1] - ref);
        l[u] += e0 + e1;
        p[u][i] = bf2(e0, e1);
        rest[u][i] = bf2(e0 - __uint_as_float(p[u][i] << 16), e1 - __uint_as_float(p[u][i] & 0xffff0000u));
      }
    }
    // O^T: tile i holds the d that are i modulo 8 (of both 64-element halves; d = 64: i and i + 4)
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const int e1 = D == 128 ? i : i + 4, c1 = D == 128 ? VC - 1 : 0;
      const uint32_t a0 = pair(v[0][0], v[1][0], i), a1 = pair(v[0][c1], v[1][c1], e1);
      const uint32_t a2 = pair(v[2][0], v[3][0], i), a3 = pair(v[2][c1], v[3][c1], e1);
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        mma_16816(o[u][i], a0, a1, a2, a3, p[u][0], p[u][1]);
        mma_16816(o[u][i], a0, a1, a2, a3, rest[u][0], rest[u][1]);
      }
    }
    if (next < k1) {
      load_v();
      find_v(next + kWarps * kRound);
    }
  }
  if (!JOINED) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // k_chunk_join may be set up
  // the warps' parts, in their order
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
    if (t == 0) {
      sm[warp][u * 8 + g] = m[u];
      sl[warp][u * 8 + g] = l[u];
    }
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const int d0 = 8 * g + i, d1 = D == 128 ? d0 + 64 : d0 + 4;
      so[warp][u * 8 + 2 * t][d0] = o[u][i][0];
      so[warp][u * 8 + 2 * t + 1][d0] = o[u][i][1];
      so[warp][u * 8 + 2 * t][d1] = o[u][i][2];
      so[warp][u * 8 + 2 * t + 1][d1] = o[u][i][3];
    }
  }
  __syncthreads();
  for (int r = warp; r < rows; r += kWarps) {
    float top = sm[0][r], sum = 0.f, by[kWarps];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm[w][r]);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      by[w] = ex2(sm[w][r] - ref);
      sum = fmaf(sl[w][r], by[w], sum);
    }
    const int64_t row = int64_t(s.row0 + r / c.group) * qh + h * c.group + r % c.group;
    const int64_t at = int64_t(split) * c.total_q * qh + row;
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    if (lane == 0 && !JOINED) {
      if (a.splits > 1) *reinterpret_cast<float2*>(a.ml + at * 2) = make_float2(top, sum);
      else if (a.lse) a.lse[row] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
    }
    for (int d = lane * 4; d < D; d += 128) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(&so[w][r][d]);
        y.x = fmaf(z.x, by[w], y.x);
        y.y = fmaf(z.y, by[w], y.y);
        y.z = fmaf(z.z, by[w], y.z);
        y.w = fmaf(z.w, by[w], y.w);
      }
      if (JOINED)
        *reinterpret_cast<float4*>(&so[0][r][d]) = y;  // this row's own place, read above
      else if (a.splits > 1)
        *reinterpret_cast<float4*>(a.part + at * D + d) = y;
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * D + d) =
            make_uint2(bf2(y.x * inv, y.y * inv), bf2(y.z * inv, y.w * inv));
    }
    if (JOINED) {
      __syncwarp();
      if (lane == 0) {
        sm[0][r] = top;
        sl[0][r] = sum;
      }
    }
  }
  if (!JOINED) return;
  // the slices' sums, in their order: CTA i of the cluster joins the rows i, i + size, ...
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  constexpr int kMost = 8;
  for (int r = split + warp * a.splits; r < rows; r += kWarps * a.splits) {
    float part_m[kMost], part_l[kMost], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      part_m[i] = i < a.splits ? *cluster.map_shared_rank(&sm[0][r], i) : -INFINITY;
      part_l[i] = i < a.splits ? *cluster.map_shared_rank(&sl[0][r], i) : 0.f;
      top = fmaxf(top, part_m[i]);
    }
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      part_m[i] = ex2(part_m[i] - ref);
      sum = fmaf(part_l[i], part_m[i], sum);
    }
    const int64_t row = int64_t(s.row0 + r / c.group) * qh + h * c.group + r % c.group;
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    if (lane == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
    for (int d = lane * 4; d < D; d += 128) {
      float4 z[kMost], y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kMost; ++i)
        z[i] = i < a.splits ? *reinterpret_cast<const float4*>(cluster.map_shared_rank(&so[0][r][d], i)) : y;
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        y.x = fmaf(z[i].x, part_m[i], y.x);
        y.y = fmaf(z[i].y, part_m[i], y.y);
        y.z = fmaf(z[i].z, part_m[i], y.z);
        y.w = fmaf(z[i].w, part_m[i], y.w);
      }
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * D + d) =
          make_uint2(bf2(y.x * inv, y.y * inv), bf2(y.z * inv, y.w * inv));
    }
  }
  cluster.sync();  // no CTA leaves while others read its sums
}

template <int D>
cudaError_t launch(const ChunkArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.splits, a.c.kvh, a.c.batch);
  cfg.blockDim = dim3(warps_of(a.joined) * 32);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = a.splits;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  const bool one = int64_t(a.c.max_q) * a.c.group <= 8;
  if (a.joined) {
    cfg.numAttrs = 1;
    return one ? cudaLaunchKernelEx(&cfg, k_chunk_step<D, 1, true>, a) : cudaLaunchKernelEx(&cfg, k_chunk_step<D, 2, true>, a);
  }
  return one ? cudaLaunchKernelEx(&cfg, k_chunk_step<D, 1, false>, a) : cudaLaunchKernelEx(&cfg, k_chunk_step<D, 2, false>, a);
}

}  // namespace

bool chunk_is_step(int group, int max_q) { return int64_t(max_q) * group <= 16; }

// Clusters of `size` CTAs that run at once on the current device (kept per device; without one, a
// low guess, so that sizes can be asked for).
static int clusters_at_once(int d, bool one, int size) {
  static std::atomic<int> cache[64][2][2][3];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 76 / size;
  }
  std::atomic<int>& kept = cache[dev][d == 128][one][size == 8 ? 2 : (size == 4 ? 1 : 0)];
  int n = kept.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size, 65535);
    cfg.blockDim = dim3(warps_of(true) * 32);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = size;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    auto ask = [&](auto kernel) { return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg); };
    const cudaError_t e = d == 128 ? (one ? ask(k_chunk_step<128, 1, true>) : ask(k_chunk_step<128, 2, true>))
                                   : (one ? ask(k_chunk_step<64, 1, true>) : ask(k_chunk_step<64, 2, true>));
    if (e != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = 76 / size;
    }
    kept.store(n, std::memory_order_relaxed);
  }
  return n;
}

// CTAs of a separate slice that an SM of the current device holds (the same way).
static int ctas_per_sm(int d, bool one) {
  static std::atomic<int> cache[64][2][2];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return one ? 3 : 2;
  }
  std::atomic<int>& kept = cache[dev][d == 128][one];
  int n = kept.load(std::memory_order_relaxed);
  if (n == 0) {
    auto ask = [&](auto kernel) { return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, warps_of(false) * 32, 0); };
    const cudaError_t e = d == 128 ? (one ? ask(k_chunk_step<128, 1, false>) : ask(k_chunk_step<128, 2, false>))
                                   : (one ? ask(k_chunk_step<64, 1, false>) : ask(k_chunk_step<64, 2, false>));
    if (e != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = one ? 3 : 2;
    }
    kept.store(n, std::memory_order_relaxed);
  }
  return n;
}

// Slices of at least 128 slots: one wave of the CTAs that fit (d = 128: three per SM with up to
// eight rows, two with more; d = 64: four. One less, d = 64, 98304 slots of 32 KV heads: 143 us
// instead of 127, one more 137), or two waves where a slice then still has 2048 slots (98304 slots
// of eight KV heads: 66.8 us in one wave, 71.0 in two; four times that: 222 and 217 us).
static int separate_slices(const mp_cache_config* c, bool one, int max_kv) {
  const int64_t units = int64_t(c->batch) * c->kv_heads, most = (int64_t(max_kv) + 127) / 128;
  const int64_t fit = int64_t(device_sm_count()) * ctas_per_sm(c->head_dim, one), wave = fit / units, two = 2 * fit / units;
  const int64_t fill = two * 2048 <= max_kv ? two : wave, s = fill < most ? fill : most;
  return int(s < 1 ? 1 : s);
}

// Short caches take a cluster of slices that joins itself instead (no second kernel, no
// workspace), the largest of 8, 4 and 2 whose clusters all run at once: its CTAs have twice the
// warps and need an SM each (half of one with d = 64 and up to eight rows), and a second round of
// them costs more than the join. One token, d = 128, four heads per KV head, us in one cluster of
// 8, 4 or 2 per KV head and as separate slices:
//   8 KV heads x 1024 slots    6.5   7.3   9.2    8.7
//   16 (15 clusters of 8 fit) 12.2   8.0  10.2    9.4
//   32 x 4096 slots           30.9  17.6  25.0   18.4
//   64 x 1024                 30.4  16.4  11.7   13.8
//   56 x 4096                 42.4  32.8  27.9   25.9
//   8 x 8192                  15.8  24.1  41.4   14.0
//   56 x 30000               176.8 166.3 159.1  132.2
StepPlan chunk_step_plan(const mp_cache_config* c, int max_q, int max_kv) {
  const int64_t rows = int64_t(max_q) * (c->q_heads / c->kv_heads), units = int64_t(c->batch) * c->kv_heads;
  const int64_t most = (int64_t(max_kv) + 127) / 128;
  for (int size = 8; max_kv <= kShort && size > 1; size /= 2)
    if (size < 2 * most && max_kv <= size * kSlice && units <= clusters_at_once(c->head_dim, rows <= 8, size)) return {size, true};
  return {separate_slices(c, rows <= 8, max_kv), false};
}
// (separate_slices only grows with max_kv; caches of up to max_kv slots all join themselves where
// the longest of them do in fours, or up to two slices' slots in twos)
int chunk_step_most(const mp_cache_config* c, int max_q, int max_kv) {
  const bool one = int64_t(max_q) * (c->q_heads / c->kv_heads) <= 8;
  const int64_t units = int64_t(c->batch) * c->kv_heads;
  if (max_kv <= kShort && units <= clusters_at_once(c->head_dim, one, 2) &&
      (max_kv <= 2 * kSlice || units <= clusters_at_once(c->head_dim, one, 4)))
    return 1;
  return separate_slices(c, one, max_kv);
}

cudaError_t launch_chunk_step(const ChunkArgs& a, cudaStream_t st) {
  return a.c.d == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace mp
