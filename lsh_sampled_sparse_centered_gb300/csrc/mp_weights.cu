// The attention that a chunk's tokens paid to every cached key, bf16.
//
// A key's weight is the sum over query rows of 2^(x - z), x = q k log2(e) / sqrt(d) and z
// the row's log-sum-exp in log2. Nothing but K, Q and z is read; each key's sum is written by
// one thread, its parts joined in a fixed order without atomics.
//
// Long chunks: k_weights_tc, keys as the M dimension of tcgen05 products (256 keys of a
// CTA, as two halves, against 96 query rows at a time), so that a thread owns a key and
// sums along its accumulator row. -z enters through one more K step, after the others: a
// column (1, 1, 1, 0, ...) of the keys times the split of -z sqrt(d) into three bf16 terms
// (exact to fp32), so that the threads neither load nor add it. K is copied into tensor
// memory first: from shared memory both operands of a 128 x 128 product need all of its
// bandwidth (16384 slots, 1000 tokens of 32 heads: 124 us so, 117 us from tensor
// memory). Beside it there is room for four accumulators of 96 columns, two for each half,
// each with a warpgroup that reads it, so that products and exponentials of both halves run
// at once. A step of 96 rows costs an SM 864 clocks of products and 768 of exponentials.
// A CTA stays for several blocks of keys and loads the next ones while it works. The CTAs go
// in clusters of two that share the last block of an odd number, half of the rows each: whole
// blocks for each CTA alone leave most SMs without work in the last round (512 blocks for 152
// SMs, 1000 tokens over 16384 slots: 117 us so, 107 us now, 111 among other calls; over 2048 slots
// 33 and 25 us; where a CTA has one block at most either way, the search for it costs: 300 over
// 4096, 19 and 21 us).
// Q loaded once for both by multicast was slower, 35 us a round of 152 blocks against 28.
//
// Few rows: k_weights_step, one pass over K from global memory straight into the fragments
// of warp-level products, bound by that read.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "mp_cache.cuh"
#include "mp_tc.cuh"

namespace mp {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kHalf = 128, kKeys = 256, kCols = 96;  // keys of a product and of a CTA, query rows of a step
constexpr int kThreads = 640;  // four warpgroups of sums, a warp each of loads and z, two of products
constexpr int kGroup = 512;    // sequences of a launch

// Keys of one KV head against the blocks of query rows that see any of them.
struct Item {
  Seq s;
  int b, h, n0;   // sequence, KV head, first slot
  int halves;     // of 128 keys
  int i0, steps;  // first block of rows, blocks; no steps: the CTA's work has ended
  int share;      // of an item that two CTAs share: 1 gets the other's sums, 2 gives its own
};

template <int D>
struct WSmem {
  static constexpr int kSub = D / 64;
  static constexpr int kStages = D == 128 ? 5 : 8;
  __nv_bfloat16 k[2][kSub][kHalf * 64];
  __nv_bfloat16 q[kStages][kSub][kCols * 64];
  __nv_bfloat16 z[kStages][kCols * 16];  // (hi, mid, lo, 0, ...) of the step's rows (32-byte swizzle)
  __nv_bfloat16 ones[kHalf * 16];        // rows (1, 1, 1, 0, ...) (32-byte swizzle)
  float sums[kKeys];                     // of the odd steps
  uint64_t k_full, k_ready[2], k_free[2], q_full[kStages], q_empty[kStages], s_full[2][2], s_empty[2][2], drain[2];
  uint64_t item_full[2], item_empty[2], sums_full[2], sums_empty[2];
  Item item[2];
  uint64_t other_full[2];
  float other[kKeys];    // the other CTA's sums of an item that two share
  int64_t past[kGroup];  // key blocks of a KV head, up to and with each sequence
  Seq seqs[kGroup];
  uint32_t loaded[3];    // phase of the last keys; the ring's next place and its phase
  uint32_t steps[2];     // of the ring: loads issued, z given
  uint32_t tmem_base;
  uint32_t abort;
};

// Query rows in blocks of at most 96: whole tokens of `group` rows, or, with more than
// 96 heads in a group, runs of 96 heads of one token.
struct Blocks {
  int group, heads, per, runs;  // rows of a token in a block, tokens of a block, blocks of a token
  int n;
};
__host__ __device__ __forceinline__ Blocks blocks_of(int group, int m) {
  Blocks b;
  b.group = group;
  b.heads = group < kCols ? group : kCols;
  b.per = kCols / b.heads;
  b.runs = (group + kCols - 1) / kCols;
  b.n = group <= kCols ? (m + b.per - 1) / b.per : m * b.runs;
  return b;
}
struct Block {
  int t0, h0, cols;
};
__device__ __forceinline__ Block block_at(const Blocks& b, int i, int m) {
  Block x;
  if (b.runs == 1) {
    x.t0 = i * b.per;
    x.h0 = 0;
    x.cols = min(b.per, m - x.t0) * b.group;
  } else {
    x.t0 = i / b.runs;
    x.h0 = (i - x.t0 * b.runs) * kCols;
    x.cols = min(kCols, b.group - x.h0);
  }
  return x;
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_weights_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ, const WeightsArgs a,
                 const int box, const int b_begin, const int b_end) {
  extern __shared__ __align__(1024) unsigned char smraw[];
  const uint32_t base = saddr(smraw);
  WSmem<D>& S = *reinterpret_cast<WSmem<D>*>(smraw + ((1024 - (base & 1023)) & 1023));
  constexpr int kSub = WSmem<D>::kSub, kStages = WSmem<D>::kStages;
  // 128-byte swizzle: tiles from 1024-byte boundaries, 32-byte swizzle: from 256-byte ones
  static_assert(offsetof(WSmem<D>, k) % 1024 == 0 && offsetof(WSmem<D>, q) % 1024 == 0 && sizeof(S.k[0][0]) % 1024 == 0 &&
                sizeof(S.q[0][0]) % 1024 == 0 && offsetof(WSmem<D>, z) % 256 == 0 && offsetof(WSmem<D>, ones) % 256 == 0 &&
                sizeof(S.z[0]) % 256 == 0);
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.x & 1;
  volatile uint32_t* abort = &S.abort;
  const int qh = c.kvh * c.group;
  const Blocks bl = blocks_of(c.group, 0);  // all but n, which is a sequence's own

  // rows of a block that no load fills stay zero, and so does all but the first three elements
  // of z and ones
  constexpr int kZero = kThreads / 2;  // threads that do this, the others look at the lengths
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int z0 = int(threadIdx.x) < kZero ? int(threadIdx.x) : INT_MAX / 2;
  for (int i = z0; i < int(sizeof(S.z) / 16); i += kZero) reinterpret_cast<uint4*>(&S.z[0][0])[i] = zero;
  const int filled = bl.heads * bl.per;  // rows of a full load
  for (int i = z0; i < (kCols - filled) * 8 * kSub * kStages; i += kZero)
    reinterpret_cast<uint4*>(&S.q[0][0][0])[(i / ((kCols - filled) * 8)) * (kCols * 8) + filled * 8 + i % ((kCols - filled) * 8)] = zero;
  for (int r = z0; r < kHalf; r += kZero) {
    uint4* row = reinterpret_cast<uint4*>(&S.ones[r * 16]);  // 16-byte chunk i of row r at i ^ (r / 4 % 2)
    row[(r >> 2) & 1] = make_uint4(0x3f803f80u, 0x00003f80u, 0, 0);
    row[1 - ((r >> 2) & 1)] = zero;
  }
  for (int i = int(threadIdx.x) - kZero; i >= 0 && i < b_end - b_begin; i += kThreads - kZero) {
    const Seq s = seq_of(c, b_begin + i);
    S.seqs[i] = s;
    S.past[i] = s.m == 0 ? 0 : (s.seen() + kKeys - 1) / kKeys;
  }
  fence_async();
  if (threadIdx.x == kThreads - 32) {
    mbar_init(&S.k_full, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&S.q_full[i], 2);  // the load and z
      mbar_init(&S.q_empty[i], 2);  // both halves' products
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_ready[i], 8);
      mbar_init(&S.drain[i], 1);
      mbar_init(&S.k_free[i], 1);
      mbar_init(&S.item_full[i], 1);
      mbar_init(&S.item_empty[i], 19);  // z, two of products, 16 of sums
      mbar_init(&S.sums_full[i], 4);
      mbar_init(&S.sums_empty[i], 4);
      mbar_init(&S.other_full[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&S.s_full[i >> 1][i & 1], 1);
      mbar_init(&S.s_empty[i >> 1][i & 1], 4);
    }
    S.abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 17) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&S.tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  cluster_arrive();
  bool met = false;  // waited for the other CTA's arrival
  fence_after();
  const uint32_t tmem = S.tmem_base;
  const uint32_t t_k = tmem + 4 * kCols;  // K: d / 2 columns of each half behind the accumulators

  if (warp == 16) {
    // ---------------- the CTA's items: the keys once, then blocks of query rows ----------------
    int64_t all = 0;
    for (int i0 = 0; i0 < b_end - b_begin; i0 += 32) {  // sums up to each sequence, by this warp alone
      const int64_t mine = i0 + lane < b_end - b_begin ? S.past[i0 + lane] : 0;
      int64_t pre = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += v;
      }
      if (i0 + lane < b_end - b_begin) S.past[i0 + lane] = all + pre;
      all += __shfl_sync(0xffffffffu, pre, 31);
    }
    __syncwarp();
    const int64_t blocks = all * c.kvh;
    bool ok = true;
    int st = 0;
    uint32_t ph = 1, items = 0, keys = 0, issued = 0;
    // The pairs of CTAs take blocks of keys in turn and their CTAs every other one of these. Where
    // that leaves a last one over, they share it, half of the rows each: the second CTA first
    // of all, the first at its end, so that it finds the other's sums there.
    const int64_t pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    const int64_t mine = blocks > pair ? quotient(blocks - pair + pairs - 1, pairs) : 0;  // of the pair
    const int shared = int(mine & 1);
    const int64_t turns = (mine >> 1) + shared;
    for (int64_t i = 0; ok; ++i) {
      Item it;
      it.steps = 0;
      it.share = shared && i == (rank ? 0 : turns - 1) ? 1 + rank : 0;
      const int64_t block = pair + pairs * (it.share ? mine - 1 : rank ? 2 * (i - shared) + 1 : 2 * i);
      if (i < turns) {
        // block = (blocks of the sequences before b) * kvh + h * (blocks of b) + its own
        int lo = 0, hi = b_end - b_begin - 1;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (S.past[mid] * c.kvh > block) hi = mid;
          else lo = mid + 1;
        }
        const int64_t before = lo > 0 ? S.past[lo - 1] : 0, per = S.past[lo] - before, in = block - before * c.kvh;
        it.b = b_begin + lo;
        it.h = int(quotient(in, per));
        it.s = S.seqs[lo];
        it.n0 = int(in - it.h * per) * kKeys;
        const Blocks own = blocks_of(c.group, it.s.m);
        // tokens before slot n0 see none of these keys
        const int t_start = max(0, it.n0 - it.s.first);
        it.i0 = own.runs == 1 ? t_start / own.per : t_start * own.runs;
        it.halves = it.s.n - it.n0 > kHalf ? 2 : 1;
        it.steps = own.n - it.i0;  // at least one: n0 < seen()
        if (it.share && it.steps == 1) {
          if (rank) continue;  // nothing to share
          it.share = 0;
        }
        if (it.share) {
          const int first = (it.steps + 1) / 2;
          if (rank) it.i0 += first;
          it.steps = rank ? it.steps - first : first;
        }
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&S.item_empty[items & 1], ((items >> 1) & 1) ^ 1, abort));
      if (!ok) break;
      if (lane == 0) {
        S.item[items & 1] = it;
        mbar_arrive(&S.item_full[items & 1]);
      }
      __syncwarp();
      ++items;
      if (it.steps == 0) break;
      // the last item's keys have gone to tensor memory
      if (items > 1) ok = __all_sync(0xffffffffu, mbar_wait(&S.k_ready[items & 1], ((items - 2) >> 1) & 1, abort));
      if (!ok) break;
      const int live = max(0, min(kKeys, it.s.n - it.n0)), boxes = (live + box - 1) / box;
      if (lane == 0) mbar_expect_tx(&S.k_full, uint32_t(boxes) * box * 128 * kSub);
      __syncwarp();
      for (int i = lane; i < boxes; i += 32) {
        const int row = slot_row(c, it.b, it.h, it.n0 + i * box);
#pragma unroll
        for (int u = 0; u < kSub; ++u)
          tma_load_2d(&S.k[i * box / kHalf][u][i * box % kHalf * 64], &tmK, u * 64, row, &S.k_full);
      }
      __syncwarp();
      ++keys;
      for (int j = 0; j < it.steps; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(&S.q_empty[st], ph, abort));
        if (!ok) break;
        if (lane == 0) {
          const Block x = block_at(bl, it.i0 + j, it.s.m);
          mbar_expect_tx(&S.q_full[st], uint32_t(bl.heads) * bl.per * 128 * kSub);
#pragma unroll
          for (int u = 0; u < kSub; ++u)
            tma_load_3d(&S.q[st][u][0], &tmQ, u * 64, it.h * c.group + x.h0, it.s.row0 + x.t0, &S.q_full[st]);
        }
        __syncwarp();
        ++issued;
        if (++st == kStages) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (lane == 0) {
      S.loaded[0] = (keys & 1) ^ 1;
      S.loaded[1] = st;
      S.loaded[2] = ph;
      S.steps[0] = issued;
    }
  } else if (warp == 18) {
    // ---------------- -z of the rows, the next step's loads in flight ----------------
    constexpr int kPer = kCols / 32;
    int tok[kPer], head[kPer];  // of this lane's columns within a block
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int col = u * 32 + lane;
      tok[u] = bl.runs == 1 ? col / bl.group : 0;
      head[u] = col - tok[u] * bl.group;
    }
    const float root = sqrtf(float(D));
    bool ok = true;
    int st = 0;
    uint32_t ph = 1, given = 0;
    for (uint32_t n = 0; ok; ++n) {
      ok = __all_sync(0xffffffffu, mbar_wait(&S.item_full[n & 1], (n >> 1) & 1, abort));
      if (!ok) break;
      const Item it = S.item[n & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.item_empty[n & 1]);
      if (it.steps == 0) break;
      auto load_z = [&](int j, float (&z)[kPer]) {
        const Block x = block_at(bl, it.i0 + min(j, it.steps - 1), it.s.m);
#pragma unroll
        for (int u = 0; u < kPer; ++u)
          z[u] = u * 32 + lane < x.cols ? a.lse[int64_t(it.s.row0 + x.t0 + tok[u]) * qh + it.h * c.group + x.h0 + head[u]]
                                        : INFINITY;  // columns without a row: 2^-inf
      };
      float z0[kPer], z1[kPer];
      auto put = [&](const float (&z)[kPer]) {
        ok = __all_sync(0xffffffffu, mbar_wait(&S.q_empty[st], ph, abort));
        if (!ok) return;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
          const int r = u * 32 + lane;
          const float v = -z[u] * root;
          const __nv_bfloat16 hi = __float2bfloat16(v);
          const float rest = isinf(v) ? 0.f : v - __bfloat162float(hi);
          const __nv_bfloat16 mid = __float2bfloat16(rest);
          const float low = rest - __bfloat162float(mid);
          *reinterpret_cast<uint2*>(&S.z[st][r * 16 + ((r >> 2) & 1) * 8]) =
              make_uint2(uint32_t(__bfloat16_as_ushort(hi)) | uint32_t(__bfloat16_as_ushort(mid)) << 16, bf2(low, 0.f));
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.q_full[st]);
        ++given;
        if (++st == kStages) {
          st = 0;
          ph ^= 1;
        }
      };
      load_z(0, z0);
      for (int j = 0; j < it.steps && ok; j += 2) {
#if MP_CHECK
        if (a.stall && blockIdx.x == 0 && given == 2) {  // z is given no more: the waits run out
          ok = false;
          break;
        }
#endif
        load_z(j + 1, z1);
        put(z0);
        if (j + 1 >= it.steps || !ok) break;
        load_z(j + 2, z0);
        put(z1);
      }
    }
    if (lane == 0) S.steps[1] = given;
  } else if (warp >= 16) {
    // ---------------- products S[key][row]: warp 17 for the first half of the keys, 19 for the
    // second, so that one's products run while the other waits ----------------
    const int half = warp == 17 ? 0 : 1;
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kCols >> 3) << 17) | (uint32_t(kHalf >> 4) << 24);
    const uint64_t dq = sw128_desc(saddr(&S.q[0][0][0]));
    const uint64_t d1 = sw32_desc(saddr(&S.ones[0])), dz = sw32_desc(saddr(&S.z[0][0]));
    constexpr uint32_t kTile = kCols * D * 2 / 16, kSlabQ = kCols * 128 / 16, kTileZ = kCols * 32 / 16;
    bool ok = true;
    int st = 0;
    uint32_t ph = 0, g = 0;  // g: this half's steps so far
    for (uint32_t n = 0; ok; ++n) {
      ok = mbar_wait_warp(&S.item_full[n & 1], (n >> 1) & 1, abort);
      if (!ok) break;
      const int steps = __reduce_max_sync(0xffffffffu, S.item[n & 1].steps);
      const bool active = __reduce_max_sync(0xffffffffu, S.item[n & 1].halves) > half;
      if (steps == 0) break;
      ok = mbar_wait_warp(&S.k_ready[n & 1], (n >> 1) & 1, abort);
      if (elect_one()) mbar_arrive(&S.item_empty[n & 1]);  // after the wait: k_ready's next phase is of item n + 2
      __syncwarp();
      for (int j = 0; j < steps && ok; ++j) {
        ok = mbar_wait_warp(&S.q_full[st], ph, abort);
        if (!active) {  // the block of rows passes this half by
          if (ok && elect_one()) mbar_arrive(&S.q_empty[st]);
        } else {
          ok = ok && mbar_wait_warp(&S.s_empty[half][g & 1], ((g >> 1) & 1) ^ 1, abort);
          if (!ok) break;
          fence_after();
          if (elect_one()) {
            const uint32_t ts = tmem + uint32_t((half * 2 + (g & 1)) * kCols);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ta(ts, t_k + uint32_t(half * (D / 2) + kk * 8), dq + st * kTile + (kk >> 2) * kSlabQ + (kk & 3) * 2,
                          idesc, kk > 0 ? 1u : 0u);
            mma_bf16(ts, d1, dz + st * kTileZ, idesc, 1u);
            mma_commit(&S.s_full[half][g & 1]);
            mma_commit(&S.q_empty[st]);
            if (j == steps - 1) mma_commit(&S.k_free[half]);
          }
          ++g;
        }
        __syncwarp();
        if (++st == kStages) {
          st = 0;
          ph ^= 1;
        }
      }
      if (ok && !active && elect_one()) mbar_arrive(&S.k_free[half]);
      __syncwarp();
    }
    if (!ok) {
      if (elect_one()) mma_commit(&S.drain[half]);
      __syncwarp();
      if (lane == 0) mbar_drain(&S.drain[half], 0);
      __syncwarp();
    }
  } else {
    // ---------------- one thread per key and every other step ----------------
    const int half = warp >> 3, odd = (warp >> 2) & 1, key = (warp & 3) * 32 + lane;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const float scale = kLog2e * rsqrtf(float(D));
    const uint64_t sc2 = pk2(scale, scale);
    const uint32_t ts = tmem + lanes + uint32_t((half * 2 + odd) * kCols);
    uint32_t g = 0, joined = 0;  // this half's steps and items so far
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      ok = __all_sync(0xffffffffu, mbar_wait(&S.item_full[n & 1], (n >> 1) & 1, abort));
      if (!ok) break;
      const Item& it = S.item[n & 1];
      const int steps = it.steps;
      if (steps == 0) break;
      const bool active = half < it.halves;
      const int slot = it.n0 + half * kHalf + key, m = it.s.m, i0 = it.i0, first = it.s.first;
      const bool mine = active && slot < it.s.n;
      const int share = it.share;
      float* const score = a.scores + (int64_t(it.b) * c.kvh + it.h) * (int64_t(c.cols) * c.page_size) + slot;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.item_empty[n & 1]);
      const float old = mine && odd == 0 && share != 2 ? *score : 0.f;
      if (odd == 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&S.k_full, n & 1, abort) && mbar_wait(&S.k_free[half], (n & 1) ^ 1, abort));
        if (!ok) break;
        if (active) {
          fence_after();
          // this thread's key into tensor memory (16-byte chunk i of row k lies at i ^ (k % 8))
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 v = *reinterpret_cast<const uint4*>(&S.k[half][u][key * 64 + ((i ^ (key & 7)) << 3)]);
              w[4 * i] = v.x;
              w[4 * i + 1] = v.y;
              w[4 * i + 2] = v.z;
              w[4 * i + 3] = v.w;
            }
            tmem_st32(t_k + lanes + uint32_t(half * (D / 2) + u * 32), w);
          }
          tmem_wait_st();
          fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.k_ready[n & 1]);
      }
      if (!active) continue;
      float sum = 0.f;
      for (int j = (g ^ odd) & 1; j < steps; j += 2) {
        ok = __all_sync(0xffffffffu, mbar_wait(&S.s_full[half][odd], ((g + j) >> 1) & 1, abort));
        if (!ok) break;
        fence_after();
        const Block x = block_at(bl, i0 + j, m);
        // columns [low, x.cols) see this thread's key
        const int dt = min(slot - first - x.t0, bl.per);
        const int low = dt <= 0 ? 0 : (bl.runs == 1 ? dt * bl.group : kCols);
        const bool last = bl.runs == 1 ? x.cols < bl.per * bl.group : x.cols < bl.heads;
        const bool plain = !__any_sync(0xffffffffu, low > 0) && !last;
        uint64_t l0 = 0, l1 = 0;  // a step's own sums: two levels keep long chunks' sums exact
        auto weigh = [&](const uint32_t (&v)[32], int col) {
          if (plain) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const uint64_t y0 = mul2(pk2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), sc2);
              const uint64_t y1 = mul2(pk2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), sc2);
              l0 = add2(l0, pk2(ex2(lo2(y0)), ex2(hi2(y0))));
              l1 = add2(l1, pk2(ex2(lo2(y1)), ex2(hi2(y1))));
            }
          } else {
            // rows outside the sequence may hold anything: selected away, not multiplied
            float l = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float e = ex2(__uint_as_float(v[i]) * scale);
              l += col + i >= low && col + i < x.cols ? e : 0.f;
            }
            l0 = add2(l0, pk2(l, 0.f));
          }
        };
        uint32_t v0[32], v1[32];
        tmem_ld32(ts, v0);
        tmem_wait_ld(v0);
        tmem_ld32(ts + 32, v1);
        weigh(v0, 0);
        tmem_wait_ld(v1);
        tmem_ld32(ts + 64, v0);
        weigh(v1, 32);
        tmem_wait_ld(v0);
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.s_empty[half][odd]);
        weigh(v0, 64);
        sum += (lo2(l0) + hi2(l0)) + (lo2(l1) + hi2(l1));
      }
      if (!ok) break;
      g += uint32_t(steps);
      // the odd steps' sums join the even ones'
      if (odd == 1) {
        ok = __all_sync(0xffffffffu, mbar_wait(&S.sums_empty[half], (joined & 1) ^ 1, abort));
        if (!ok) break;
        S.sums[half * kHalf + key] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.sums_full[half]);
      } else {
        ok = __all_sync(0xffffffffu, mbar_wait(&S.sums_full[half], joined & 1, abort));
        if (!ok) break;
        sum += S.sums[half * kHalf + key];
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.sums_empty[half]);
        if (share == 2) {
          if (!met) cluster_wait();
          met = true;
          put_remote(&S.other[half * kHalf + key], 0, sum);
          __syncwarp();
          if (lane == 0) {
            fence_cluster();
            mbar_arrive_remote(&S.other_full[half], 0);
          }
        } else {
          if (share == 1) {
            ok = __all_sync(0xffffffffu, mbar_wait(&S.other_full[half], 0, abort));
            if (!ok) break;
            fence_cluster();
            sum += S.other[half * kHalf + key];
          }
          if (mine) *score = old + sum;
        }
      }
      ++joined;
    }
  }
  fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && S.abort) {
    mbar_drain(&S.k_full, S.loaded[0]);
    // a load whose z was not given completes its barrier with this
    for (uint32_t i = S.steps[1]; i < S.steps[0]; ++i) mbar_arrive(&S.q_full[i % kStages]);
    for (int i = 0; i < kStages; ++i) mbar_drain(&S.q_full[i], i < int(S.loaded[1]) ? S.loaded[2] ^ 1 : S.loaded[2]);
    flag(c.status, MP_STATUS_WAIT_TIMEOUT);
  }
  if (warp == 17) {
    __syncwarp();
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  if (!met) cluster_wait();
  cluster_arrive();
  cluster_wait();  // the other CTA's sums come here
}

// ---- few query rows ----

constexpr int kStepWarps = 4, kRound = 16;  // keys of a warp and round

// 16 keys (M) x 8 NT query rows (N) per warp and round. The sum over d has no order to
// keep, so lane t of a row's four takes the 16-byte chunks t, t + 4, ... and feeds their
// halves to two products: the loads are whole vectors and need no shared memory. The next
// round's keys are loaded as soon as their registers are free, their places looked up a
// round before that.
template <int D, int NT>
__global__ void __launch_bounds__(kStepWarps * 32) k_weights_step(const WeightsArgs a) {
  constexpr int KC = D / 32;  // 16-byte chunks of a row per lane
  const CacheArgs& c = a.c;
  const int b = blockIdx.z, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Seq s = seq_of(c, b);
  constexpr int kAll = kStepWarps * kRound;
  const int per = ((s.n + int(gridDim.x) - 1) / int(gridDim.x) + kAll - 1) / kAll * kAll;
  const int64_t p0 = int64_t(blockIdx.x) * per;
  if (p0 >= s.n || s.m == 0) return;
  const int p1 = min(s.n, int(p0) + per);
  const int first = s.first, qh = c.kvh * c.group, rows = s.m * c.group;
  const float root = rsqrtf(float(D));
  float* scores = a.scores + (int64_t(b) * c.kvh + h) * (int64_t(c.cols) * c.page_size);
  const __nv_bfloat16* keys = static_cast<const __nv_bfloat16*>(a.keys);
  uint4 k[2][KC];
  int row[2];
  float old[2];
  auto find = [&](int n0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) row[i] = slot_row(c, b, h, min(n0 + g + 8 * i, s.n - 1));
  };
  auto load = [&](int n0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __nv_bfloat16* src = keys + int64_t(row[i]) * D + t * 8;
#pragma unroll
      for (int j = 0; j < KC; ++j) k[i][j] = __ldcs(reinterpret_cast<const uint4*>(src + j * 32));
      old[i] = t == 0 ? scores[min(n0 + g + 8 * i, s.n - 1)] : 0.f;
    }
  };
  int n0 = int(p0) + warp * kRound;
  if (n0 >= p1) return;
  find(n0);
  load(n0);
  find(n0 + kAll);
  uint4 q[NT][KC];
  float nz[NT][2];
  int see[NT][2];  // the thread's columns see the slots below this
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int r = u * 8 + g;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                               (int64_t(s.row0 + r / c.group) * qh + h * c.group + r % c.group) * D + t * 8;
#pragma unroll
    for (int i = 0; i < KC; ++i)
      q[u][i] = r < rows ? *reinterpret_cast<const uint4*>(src + i * 32) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rc = u * 8 + 2 * t + i;
      see[u][i] = rc < rows ? first + rc / c.group + 1 : 0;
      nz[u][i] = rc < rows ? -a.lse[int64_t(s.row0 + rc / c.group) * qh + h * c.group + rc % c.group] : 0.f;
    }
  }
  for (; n0 < p1; n0 += kAll) {
    const int next = n0 + kAll;
    float x[NT][4];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[u][i] = 0.f;
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        mma_16816(x[u], k[0][j].x, k[1][j].x, k[0][j].y, k[1][j].y, q[u][j].x, q[u][j].y);
        mma_16816(x[u], k[0][j].z, k[1][j].z, k[0][j].w, k[1][j].w, q[u][j].z, q[u][j].w);
      }
    }
    const float was[2] = {old[0], old[1]};
    if (next < p1) {
      load(next);
      find(next + kAll);
    }
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n0 + g + 8 * (i >> 1) < see[u][i & 1])  // z taken off before the change to log2: its rounding there would count
          sum[i >> 1] += ex2(kLog2e * fmaf(x[u][i], root, nz[u][i & 1]));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
      const int slot = n0 + g + 8 * i;
      if (t == 0 && slot < s.n) scores[slot] = was[i] + sum[i];
    }
  }
}

// CTAs of k_weights_step that an SM of the current device holds, for up to 8, 16 or 32 rows (kept
// per device).
template <int D>
int step_ctas_per_sm(int kind) {
  static std::atomic<int> cache[64][3];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 4;
  n = cache[dev][kind].load(std::memory_order_relaxed);
  if (n == 0) {
    auto ask = [&](auto kernel) { return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kStepWarps * 32, 0); };
    const cudaError_t e = kind == 0 ? ask(k_weights_step<D, 1>) : (kind == 1 ? ask(k_weights_step<D, 2>) : ask(k_weights_step<D, 4>));
    if (e != cudaSuccess || n < 1) return 4;  // the launch will say what is wrong
    cache[dev][kind].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int D>
cudaError_t launch(const WeightsArgs& a, cudaStream_t st) {
  const CacheArgs& c = a.c;
  const int64_t rows = int64_t(c.max_q) * c.group;
  if (rows <= 32) {
    // Slices of at least four rounds, one wave of the CTAs that fit (one more per SM than fit: 16
    // rows, 65536 slots of 32 KV heads 106 us instead of 84; half of them: 111).
    const int kind = rows <= 8 ? 0 : (rows <= 16 ? 1 : 2);
    const int64_t fit = int64_t(device_sm_count()) * step_ctas_per_sm<D>(kind) / (int64_t(c.kvh) * c.batch);
    const int64_t most = (c.max_kv + 4 * kStepWarps * kRound - 1) / (4 * kStepWarps * kRound);
    const dim3 grid(unsigned(std::max<int64_t>(1, std::min(fit, most))), c.kvh, c.batch);
    if (kind == 0) k_weights_step<D, 1><<<grid, kStepWarps * 32, 0, st>>>(a);
    else if (kind == 1) k_weights_step<D, 2><<<grid, kStepWarps * 32, 0, st>>>(a);
    else k_weights_step<D, 4><<<grid, kStepWarps * 32, 0, st>>>(a);
    return cudaGetLastError();
  }
  CUtensorMap mk, mq;
  const int box = box_rows(c.table, c.page_size);
  const Blocks bl = blocks_of(c.group, 1);
  if (!make_map(&mk, a.keys, D, uint64_t(c.n_pages) * c.kvh * c.page_size, 64, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map3(&mq, a.q, D, uint64_t(c.kvh) * c.group, c.total_q, 64, bl.heads, bl.per))
    return cudaErrorInvalidValue;
  const size_t smem = sizeof(WSmem<D>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(k_weights_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  // A pair of CTAs per pair of SMs, or fewer when the limits leave fewer blocks than pairs.
  for (int b = 0; b < c.batch; b += kGroup) {
    const int n = std::min(kGroup, c.batch - b);
    const int64_t most = int64_t(n) * c.kvh * ((int64_t(c.max_kv) + kKeys - 1) / kKeys);
    const int ctas = 2 * int(std::min<int64_t>(device_sm_count() / 2, most));
    if (ctas == 0) continue;
    k_weights_tc<D><<<ctas, kThreads, smem, st>>>(mk, mq, a, box, b, b + n);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_weights_bf16(const WeightsArgs& a, cudaStream_t st) {
  return a.c.d == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace mp
