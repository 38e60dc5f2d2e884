// Exact attention of a chunk of new tokens over the paged cache, and the attention
// weights that its keys received, on the CUDA cores: the fp32 forms.
//
// A tile is 64 query rows of one KV head (row = token * group + head of the group, so the
// heads of a group share every key they load) against 64 keys at a time. The softmax is
// online: per row the running maximum m and sum l of 2^(x - m), x = q k log2(e) / sqrt(d),
// and the unnormalised sum of 2^(x - m) v; keys past a row's own slot enter as -infinity.
// The slots can be split over several CTAs; each then stores (m, l, sum) and k_chunk_join
// combines them.
#include <algorithm>
#include <type_traits>

#include "mp_cache.cuh"
#include "mp_prefix_few.cuh"

namespace mp {
namespace {

constexpr int kBM = kChunkRows, kBN = 64, kThr = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// 64 rows into shared memory as [d][64] (row index fastest): thread t takes row t % 64 and
// every other group of 8 elements; p(row) is the row's address or nullptr (zeros).
template <int D, typename P>
__device__ __forceinline__ void load_transposed(float* dst, P p) {
  const int row = threadIdx.x & 63;
  const float* src = p(row);
#pragma unroll 4
  for (int e = (threadIdx.x >> 6) * 8; e < D; e += 16) {
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (src) load8(src + e, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[(e + i) * 64 + row] = x[i];
  }
}
// S[8][4] of rows ty*8.. and keys tx*4.. from [d][64] tiles
template <int D>
__device__ __forceinline__ void dot_tile(const float* qt, const float* kt, int ty, int tx, float (&s)[8][4]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int e = 0; e < D; ++e) {
    const float4 a0 = *reinterpret_cast<const float4*>(qt + e * 64 + ty * 8);
    const float4 a1 = *reinterpret_cast<const float4*>(qt + e * 64 + ty * 8 + 4);
    const float4 b0 = *reinterpret_cast<const float4*>(kt + e * 64 + tx * 4);
    const float a[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w}, b[4] = {b0.x, b0.y, b0.z, b0.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = fmaf(a[i], b[j], s[i][j]);
  }
}

// 16 bytes of global memory into shared memory in the background, zeros where !live
__device__ __forceinline__ void copy16(float* dst, const float* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A CTA's tiles where the work of all is cut into runs; `sm` is free afterwards.
__device__ __forceinline__ auto walk_of(const PrefixFew& a, float* sm) {
  using Cut = few::Cutting<kBM, kBN, 1, 1, 2048>;
  __shared__ int64_t totals[kThr / 32];
  __shared__ int leasts[kThr / 32];
  int2* kept = reinterpret_cast<int2*>(sm);
  int64_t total = 0;
  int least = 0;
  few::survey<Cut>(a, kept, threadIdx.x, kThr, &total, &least);
  if ((threadIdx.x & 31) == 0) {
    totals[threadIdx.x >> 5] = total;
    leasts[threadIdx.x >> 5] = least;
  }
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < kThr / 32; ++i) {
    total += totals[i] * a.own.c.kvh;
    least = max(least, leasts[i]);
  }
  few::Walk<Cut> walk(a, kept, total, least, blockIdx.x, gridDim.x);
  __syncthreads();  // `kept` lies where the tiles go
  return walk;
}
// A sequence and a split of its slots for each CTA, which has one tile.
struct OneTile {
  bool there = true;
  __device__ __forceinline__ bool open(few::Piece*) { return there; }
  __device__ __forceinline__ void advance() { there = false; }
};

// Thread (ty, tx) holds S of rows 8 ty .. + 8 and keys tx, tx + 16, ..., and O of the same rows
// and the columns 4 tx .. + 4 of each 64. The vectors that a warp reads or writes at once fall on
// all banks of shared memory: with d = 64 by rows padded by four floats, with d = 128, where
// padding leaves room for one CTA on an SM instead of two (512 tokens over 8192 slots, 32/8
// heads: 2988 against 2098 us), by keeping the 16-byte chunk i of a row at i ^ x, x = key % 8 for K,
// row / 8 % 2 for Q, key % 16 for P, 0 for V (with d = 64 3 % slower than padding).
// Products run as packed pairs, over pairs of d for S and of rows for O. V arrives under S and
// the softmax, the next K under the product with V.
//
// RUNS: groups over their prefixes and sequences over their own slots. The tiles of all, a step for every 64
// slots, are laid end to end and cut into equal runs, one a CTA, as the warps of the kernels of few rows have them
// (mp_prefix_few.cuh). Slices of one length for all took longer where lengths differ, us a call:
//   drafts of 1 to 9 tokens of 33 sequences, 6/2 heads, prefixes of 614, 20978 and 47562 slots, d = 64   836   140
//   of 29 sequences, 12/1 heads, five prefixes of 1 to 14768, d = 128                                   1190   160
//   of 14 sequences, 28/4 heads, prefixes of 26434 and 11304, d = 64                                     552   408
// and less where they do not (five chunks, 101 rows over 2000 slots, eight heads: 37 and 38).
// One function for both: with the tile in a function of its own, which the compiler inlined, the kernel without runs
// took ten registers more and 2 % of its time (512 tokens over 8192 slots, 32/8 heads: 1937 us, in one function 1907,
// alone 1896), and the one with runs with d = 64 9 % (five chunks, 101 rows over 2000 slots, eight heads, in a graph:
// 39.1 and 35.5 us).
template <int D, bool RUNS>
__global__ void __launch_bounds__(kThr, D == 64 ? 3 : 2) k_chunk_simt(const __grid_constant__ std::conditional_t<RUNS, PrefixFew, ChunkArgs> args) {
  constexpr bool kPad = D == 64;
  constexpr int kRow = D + kPad * 4, kPt = kBM + kPad * 4;
  auto place = [](int at, int x) { return kPad ? at : at ^ (x * 4); };  // of a chunk's first float
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;                // [64][kRow]
  float* ks = qs + kBM * kRow;   // [64][kRow]
  float* vs = ks + kBN * kRow;   // [64][kRow]
  float* pt = vs + kBN * kRow;   // [64 keys][kPt]
  auto walk = [&] {
    if constexpr (RUNS) return walk_of(args, sm);
    else return OneTile();
  }();
  few::Piece p = {};
  for (; walk.open(&p); walk.advance()) {
    const auto& a = [&]() -> const auto& {
      if constexpr (RUNS) return p.own ? args.own : args.pre;
      else return args;
    }();
    const CacheCall& c = a.c;
    const int b = RUNS ? p.b : int(blockIdx.z), h = RUNS ? p.h : int(blockIdx.y);
    const int split = RUNS ? p.slice : int(blockIdx.x % a.splits);  // the slice for the tile's sums, where there are slices
    const Seq s = [&] {
      if constexpr (RUNS) return walk.s;
      else return seq_of(c, b);
    }();
    const int rows = s.m * c.group, r0 = RUNS ? p.r0 : int(blockIdx.x / a.splits) * kBM;
    if (!RUNS && r0 >= rows) return;
    const int qh = c.kvh * c.group;
    const int first = s.first;                                       // slot of token 0
    const int last = first + min(r0 + kBM - 1, rows - 1) / c.group;   // slot of the tile's last token
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    // the tile's keys: a piece of a run, or this split's run of 64-key tiles of the sequence
    const int tiles = (s.n + kBN - 1) / kBN, per = RUNS ? 0 : (tiles + a.splits - 1) / a.splits;
    const int k0 = min(s.n, (RUNS ? p.u0 : split * per) * kBN), k1 = min(min(s.n, last + 1), (RUNS ? p.u1 : (split + 1) * per) * kBN);
    const bool slices = RUNS || a.splits > 1;
    constexpr int kVec = D / 4, kStep = kThr / kVec;  // vectors of a row, rows that the CTA copies at a time
    const int cr = threadIdx.x / kVec, ce = threadIdx.x % kVec * 4;
    auto copy_tile = [&](float* dst, const void* base, int n0, int swizzle) {
#pragma unroll 4
      for (int i = cr; i < kBN; i += kStep) {
        const bool live = n0 + i < k1;
        const float* src = static_cast<const float*>(base) + (live ? slot_read(c, b, h, n0 + i) + ce : 0);
        copy16(dst + i * kRow + place(ce, i & swizzle), src, live);
      }
      copy_commit();
    };
    // Q's copies are of K's group, so that there are none where no slot is seen: nothing would wait for them, and
    // they could land on the rows of the CTA's next tile.
    if (k0 < k1) {
      for (int i = cr; i < kBM; i += kStep) {
        const int r = r0 + i;
        const bool live = r < rows;
        const float* src = static_cast<const float*>(a.q);
        if (live) src += (int64_t(s.row0 + r / c.group) * qh + h * c.group + r % c.group) * D + ce;
        copy16(qs + i * kRow + place(ce, (i >> 3) & 1), src, live);
      }
      copy_tile(ks, a.keys, k0, 7);
      copy_tile(vs, a.values, k0, 0);
    }
    float m[8], l[8];
    uint64_t o[4][D / 16];  // rows 2 i and 2 i + 1 of a column
    int see[8];             // a row sees the slots below this
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      see[i] = first + (r0 + ty * 8 + i) / c.group + 1;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[i / 2][j] = 0;
    }
    const float scale = kLog2e * rsqrtf(float(D));
    for (int n0 = k0; n0 < k1; n0 += kBN) {
      copy_wait<1>();  // K is there, V may still come
      __syncthreads();
      uint64_t x2[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x2[i][j] = 0;
#pragma unroll(D == 64 ? 1 : 2)
      for (int e = 0; e < D; e += 4) {
        const int ek = place(e, tx & 7), eq = place(e, ty & 1);
        uint64_t kv[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(ks + (tx + 16 * j) * kRow + ek);
          kv[j][0] = v.x;
          kv[j][1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(qs + (ty * 8 + i) * kRow + eq);
#pragma unroll
          for (int j = 0; j < 4; ++j) x2[i][j] = fma2(q.y, kv[j][1], fma2(q.x, kv[j][0], x2[i][j]));
        }
      }
      float x[8][4], by[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int slot = n0 + tx + 16 * j;
          x[i][j] = slot < see[i] && slot < k1 ? (lo2(x2[i][j]) + hi2(x2[i][j])) * scale : -INFINITY;
          top = fmaxf(top, x[i][j]);
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        const float mn = fmaxf(m[i], top);
        const float ref = mn == -INFINITY ? 0.f : mn;
        by[i] = exp2f(m[i] - ref);
        m[i] = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[i][j] = exp2f(x[i][j] - ref);
          sum += x[i][j];
        }
        l[i] = l[i] * by[i] + sum;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < D / 16; ++j) o[i][j] = mul2(o[i][j], pk2(by[2 * i], by[2 * i + 1]));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        *reinterpret_cast<float4*>(pt + (tx + 16 * j) * kPt + place(ty * 8, tx)) = make_float4(x[0][j], x[1][j], x[2][j], x[3][j]);
        *reinterpret_cast<float4*>(pt + (tx + 16 * j) * kPt + place(ty * 8 + 4, tx)) = make_float4(x[4][j], x[5][j], x[6][j], x[7][j]);
      }
      __syncthreads();  // K has been read, P is written
      const bool more = n0 + kBN < k1;
      if (more) {
        copy_tile(ks, a.keys, n0 + kBN, 7);
        copy_wait<1>();
      } else {
        copy_wait<0>();
      }
      __syncthreads();  // V is there
#pragma unroll 4
      for (int k = 0; k < kBN; ++k) {
        const ulonglong2 p0 = *reinterpret_cast<const ulonglong2*>(pt + k * kPt + place(ty * 8, k & 15));
        const ulonglong2 p1 = *reinterpret_cast<const ulonglong2*>(pt + k * kPt + place(ty * 8 + 4, k & 15));
        const uint64_t p[4] = {p0.x, p0.y, p1.x, p1.y};
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
          const float4 v4 = *reinterpret_cast<const float4*>(vs + k * kRow + g * 64 + tx * 4);
          const uint64_t v[4] = {pk2(v4.x, v4.x), pk2(v4.y, v4.y), pk2(v4.z, v4.z), pk2(v4.w, v4.w)};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][g * 4 + j] = fma2(p[i], v[j], o[i][g * 4 + j]);
        }
      }
      __syncthreads();  // V and P have been read
      if (more) copy_tile(vs, a.values, n0 + kBN, 0);
    }
    copy_wait<0>();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be set up
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float sum = l[i];
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      const int r = r0 + ty * 8 + i;
      if (r >= rows) continue;
      const int64_t row = int64_t(s.row0 + r / c.group) * qh + h * c.group + r % c.group;
      const int64_t at = int64_t(split) * c.total_q * qh + row;
      const float inv = slices ? 1.f : (sum > 0.f ? 1.0f / sum : sum);
      if (tx == 0) {
        if (slices) *reinterpret_cast<float2*>(a.ml + at * 2) = make_float2(m[i], sum);
        else if (a.lse) a.lse[row] = sum == 0.f ? -INFINITY : m[i] * kLn2 + logf(sum);
      }
      float* out = slices ? a.part + at * D : static_cast<float*>(a.out) + row * D;
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = (i & 1 ? hi2(o[i / 2][g * 4 + j]) : lo2(o[i / 2][g * 4 + j])) * inv;
        *reinterpret_cast<float4*>(out + g * 64 + tx * 4) = make_float4(y[0], y[1], y[2], y[3]);
      }
    }
  }
}

// Joins the splits' (m, l, sum) of a query row, in an order that is fixed by their number:
// WARPS warps per row (8 where there are many splits, so that their loads overlap) take
// eight splits at a time each. Started while the slices still run (its launch costs as much
// as its work); it waits for them first.
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(256) k_chunk_join(const ChunkArgs a) {
  constexpr int PER = D / 32;
  __shared__ float so[8][D], sl[8];
  const CacheCall& c = a.c;
  const int qh = c.kvh * c.group;
  const int64_t rows = int64_t(c.total_q) * qh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * (8 / WARPS) + warp / WARPS;
  const int part = warp % WARPS;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= rows) return;
  const int t = int(row / qh), b = seq_at_warp(c, t);
  if (b < 0) return;
  const Seq s = seq_of(c, b);
  if (t < s.row0 || t >= s.row0 + s.m) return;
  const float2* ml = reinterpret_cast<const float2*>(a.ml) + row;
  float m = -INFINITY;
  for (int i = lane; i < a.splits; i += 32) m = fmaxf(m, ml[i * rows].x);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f, o[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) o[j] = 0.f;
  for (int i = part * 8; i < a.splits; i += WARPS * 8) {
    float x[8][PER], f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 v = i + k < a.splits ? ml[(i + k) * rows] : make_float2(-INFINITY, 0.f);
      f[k] = v.y == 0.f ? 0.f : exp2f(v.x - ref);
      l = fmaf(v.y, f[k], l);
      const bool live = v.y != 0.f;  // an empty slice has written no sum
      const float* p = a.part + ((i + k) * rows + row) * D + lane * PER;
#pragma unroll
      for (int j = 0; j < PER; ++j) x[k][j] = live ? p[j] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < PER; ++j) o[j] = fmaf(x[k][j], f[k], o[j]);
  }
  if (WARPS > 1) {  // one row per CTA: no warp has left
#pragma unroll
    for (int j = 0; j < PER; ++j) so[warp][lane * PER + j] = o[j];
    if (lane == 0) sl[warp] = l;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      l += sl[w];
#pragma unroll
      for (int j = 0; j < PER; ++j) o[j] += so[w][lane * PER + j];
    }
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
#pragma unroll
  for (int j = 0; j < PER; ++j) static_cast<T*>(a.out)[row * D + lane * PER + j] = T(o[j] * inv);
}

// Attention weights: one CTA owns 64 slots of one KV head and walks the chunk's query
// rows in order, so every slot's sum has one owner and a fixed order.
template <int D>
__global__ void __launch_bounds__(kThr) k_weights_simt(const WeightsArgs a) {
  extern __shared__ float sm[];
  float* qt = sm;            // [D][64]
  float* kt = qt + D * kBM;  // [D][64]
  float* col = kt + D * kBN; // [8][64] partial column sums
  const CacheCall& c = a.c;
  const int b = blockIdx.z, h = blockIdx.y, n0 = blockIdx.x * kBN;
  const Seq s = seq_of(c, b);
  if (n0 >= s.seen() || s.m == 0) return;
  const int rows = s.m * c.group, first = s.first, qh = c.kvh * c.group;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  load_transposed<D>(kt, [&](int i) -> const float* {
    return n0 + i < s.n ? static_cast<const float*>(a.keys) + slot_read(c, b, h, n0 + i) : nullptr;
  });
  const float root = rsqrtf(float(D));
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  // rows before token n0 - first see none of these slots
  const int start = max(0, n0 - first) * c.group / kBM * kBM;
  for (int r0 = start; r0 < rows; r0 += kBM) {
    __syncthreads();
    load_transposed<D>(qt, [&](int i) -> const float* {
      const int r = r0 + i;
      return r < rows ? static_cast<const float*>(a.q) + (int64_t(s.row0 + r / c.group) * qh + h * c.group + r % c.group) * D
                      : nullptr;
    });
    __syncthreads();
    float x[8][4];
    dot_tile<D>(qt, kt, ty, tx, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + ty * 8 + i;
      if (r >= rows) continue;
      const int t = r / c.group;
      const float z = a.lse[int64_t(s.row0 + t) * qh + h * c.group + r % c.group];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n0 + tx * 4 + j <= first + t) acc[j] += exp2f(kLog2e * fmaf(x[i][j], root, -z));
    }
  }
  *reinterpret_cast<float4*>(col + ty * 64 + tx * 4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  const int k = threadIdx.x;
  if (k < kBN && n0 + k < s.n) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += col[i * 64 + k];
    float* to = a.scores + (int64_t(b) * c.kvh + h) * (int64_t(c.cols) * c.page_size) + n0 + k;
    *to += sum;
  }
}

constexpr int simt_smem(int d) { return (3 * 64 * (d + (d == 64 ? 4 : 0)) + 64 * (64 + (d == 64 ? 4 : 0))) * 4; }
template <int D>
cudaError_t chunk_simt(const ChunkArgs& a, cudaStream_t st) {
  constexpr int smem = simt_smem(D);
  cudaError_t e = cudaFuncSetAttribute(k_chunk_simt<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t(a.c.max_q) * a.c.group + kBM - 1) / kBM;
  k_chunk_simt<D, false><<<dim3(unsigned(tiles * a.splits), a.c.kvh, a.c.batch), kThr, smem, st>>>(a);
  return cudaGetLastError();
}
template <int D>
cudaError_t prefix_simt(const PrefixFew& a, cudaStream_t st) {
  constexpr int smem = simt_smem(D);
  static_assert(2048 * sizeof(int2) <= smem);
  cudaError_t e = cudaFuncSetAttribute(k_chunk_simt<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  double steps = 0;
  for (const PrefixArgs* x : {&a.pre, &a.own}) {
    const int units = x == &a.pre ? a.groups : (a.own_units ? x->c.batch : 0);
    steps += double(units) * x->c.kvh * ((int64_t(x->c.max_q) * x->c.group + kBM - 1) / kBM) * ((x->c.max_kv + kBN - 1) / kBN + 1);
  }
  const int ctas = int(std::max(1.0, std::min((D == 64 ? 3.0 : 2.0) * device_sm_count(), steps)));
  k_chunk_simt<D, true><<<ctas, kThr, smem, st>>>(a);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t join(const ChunkArgs& a, cudaStream_t st) {
  const int64_t rows = int64_t(a.c.total_q) * a.c.kvh * a.c.group;
  cudaLaunchConfig_t cfg = {};
  const bool wide = a.splits > 8;
  cfg.gridDim = dim3(unsigned(wide ? rows : (rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&cfg, k_chunk_join<T, D, 8>, a) : cudaLaunchKernelEx(&cfg, k_chunk_join<T, D, 1>, a);
}
template <int D>
cudaError_t weights_simt(const WeightsArgs& a, cudaStream_t st) {
  constexpr int smem = (2 * D * 64 + 8 * 64) * 4;
  cudaError_t e = cudaFuncSetAttribute(k_weights_simt<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  k_weights_simt<D><<<dim3((a.c.max_kv + kBN - 1) / kBN, a.c.kvh, a.c.batch), kThr, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

// Slices of the keys: as many as the CTAs that fit leave room for, each of at least 256 slots.
int chunk_splits(const mp_cache_config* c, int max_q, int max_kv) {
  const int64_t group = c->q_heads / c->kv_heads;
  const int64_t ctas = (max_q * group + kBM - 1) / kBM * c->kv_heads * c->batch;
  const int64_t fill = (c->head_dim == 64 ? 3 : 2) * int64_t(device_sm_count()) / ctas, most = (int64_t(max_kv) + 255) / 256;
  const int64_t s = fill < most ? fill : most;
  return int(s < 1 ? 1 : (s > 64 ? 64 : s));
}

cudaError_t launch_chunk_simt(const ChunkArgs& a, cudaStream_t st) {
  return a.c.d == 128 ? chunk_simt<128>(a, st) : chunk_simt<64>(a, st);
}
cudaError_t launch_prefix_simt(const PrefixFew& a, cudaStream_t st) { return a.own.c.d == 128 ? prefix_simt<128>(a, st) : prefix_simt<64>(a, st); }
cudaError_t launch_chunk_join(const ChunkArgs& a, int dtype, cudaStream_t st) {
  if (dtype == MP_DTYPE_BF16) return a.c.d == 128 ? join<__nv_bfloat16, 128>(a, st) : join<__nv_bfloat16, 64>(a, st);
  return a.c.d == 128 ? join<float, 128>(a, st) : join<float, 64>(a, st);
}
cudaError_t launch_cache_weights(const WeightsArgs& a, int dtype, cudaStream_t st) {
  if (dtype == MP_DTYPE_BF16) return launch_weights_bf16(a, st);
  return a.c.d == 128 ? weights_simt<128>(a, st) : weights_simt<64>(a, st);
}

}  // namespace mp
