// Attention with shared prefixes in fp32, units with up to 16 query rows per KV head (tokens x heads of
// the group). Runs and slices as in mp_prefix_few.cuh, a warp each.
//
// A lane holds four elements of d: of every query row, and of K and V of each slot (d = 64: the halves of
// a warp take every other slot). It forms its part of the logits of 32 (slot, row) pairs; a butterfly that
// halves the values it passes on leaves each lane the whole logit of one pair, so that the softmax costs
// one exponential a lane.
//
// Bound by one pass over K and V with up to 4 rows, by the products and exchanges with more. Against the
// tiles of 64 rows (mp_chunk.cu), which are mostly empty, us a call with the join, d = 128:
//   128 single tokens of 40 heads without grouping, ~700 own slots   543 (6.8 TB/s)   2919
//   32 single tokens, ~3450 own slots of 8 KV heads, 4 rows each     141 (6.4 TB/s)   1075
//                                                    8 rows each     193 (4.7 TB/s)   1076
//   32 single tokens, ~8450 own slots of 1 KV head, 16 rows each     131              297
//   one token, 100000 shared slots of 8 KV heads, 4 rows each        135 (6.1 TB/s)   790
#include <algorithm>

#include "mp_cache_host.h"
#include "mp_prefix_few.cuh"

namespace mp {
namespace {

using namespace few;

constexpr int kWarps = 4;
constexpr int resident(int rows) { return rows <= 8 ? 3 : 2; }  // CTAs of an SM

// R: query rows, 4, 8 or 16.
template <int D, int R>
__global__ void __launch_bounds__(kWarps * 32, resident(R)) k_prefix_few32(const __grid_constant__ PrefixFew a) {
  constexpr int L = D / 4, HALVES = 32 / L;  // lanes of a row of K; rows of a load
  constexpr int SL = L / R;                  // slots of a round of each half
  constexpr int SR = SL * HALVES, kRounds = kStep / SR;
  using Cut = Cutting<R, kStep, kLead, kMinRun, 2048>;
  __shared__ int2 kept[Cut::kKept];
  __shared__ int64_t totals[kWarps];
  __shared__ int leasts[kWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane % L, half = lane / L, own_row = lane % R;
  const CacheCall& co = a.own.c;
  const int group = co.group, qh = co.kvh * group;
  int64_t total = 0;
  int least = 0;
  survey<Cut>(a, kept, threadIdx.x, kWarps * 32, &total, &least);
  if (lane == 0) {
    totals[warp] = total;
    leasts[warp] = least;
  }
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    total += totals[i] * co.kvh;
    least = max(least, leasts[i]);
  }
  Walk<Cut> walk(a, kept, total, least, int64_t(blockIdx.x) * kWarps + warp, int64_t(gridDim.x) * kWarps);
  const float scale = kLog2e * rsqrtf(float(D));
  Piece p = {};
  for (; walk.open(&p); walk.advance()) {
    const CacheCall& c = p.own ? co : a.pre.c;
    const PrefixArgs& side = p.own ? a.own : a.pre;
    const float *keys = static_cast<const float*>(side.keys) + part * 4, *values = static_cast<const float*>(side.values) + part * 4;
    auto row_of = [&](int r) { return int64_t(p.row0 + r / group) * qh + p.h * group + r % group; };
    float4 q[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
      q[r] = r < p.rows ? *reinterpret_cast<const float4*>(static_cast<const float*>(a.own.q) + row_of(r) * D + part * 4)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    const int see = own_row < p.rows ? min(p.n, p.first + own_row / group + 1) : 0;  // this lane's row sees the slots below
    float4 o[R];
#pragma unroll
    for (int r = 0; r < R; ++r) o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;  // of this lane's row; l of its own pairs
    const int n0 = p.u0 * kStep, rounds = (p.u1 - p.u0) * kRounds;
    // a step's first row of the pool, looked up a step ahead
    int at = slot_row(c, p.b, p.h, n0), next = p.u0 + 1 < p.u1 ? slot_row(c, p.b, p.h, n0 + kStep) : 0;
    // slots behind the last are read as the last: their weights are zero
    auto element = [&](int round, int i, int first) {
      const int slot = round % kRounds * SR + i * HALVES + half, step = n0 + round / kRounds * kStep;
      return int64_t(first + min(slot, p.n - 1 - step)) * D;
    };
    float4 k[SL], v[SL];
#pragma unroll
    for (int i = 0; i < SL; ++i) k[i] = __ldcs(reinterpret_cast<const float4*>(keys + element(0, i, at)));
#pragma unroll
    for (int i = 0; i < SL; ++i) v[i] = __ldcs(reinterpret_cast<const float4*>(values + element(0, i, at)));
    for (int j = 0; j < rounds; ++j) {
      // value s R + r: this lane's part of the logit of slot s (of its half) and row r
      float x[L];
#pragma unroll
      for (int i = 0; i < SL; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) x[i * R + r] = fmaf(q[r].w, k[i].w, fmaf(q[r].z, k[i].z, fmaf(q[r].y, k[i].y, q[r].x * k[i].x)));
      const bool turn = (j + 1) % kRounds == 0;
      const int ahead = turn ? next : at;
      if (j + 1 < rounds) {
#pragma unroll
        for (int i = 0; i < SL; ++i) k[i] = __ldcs(reinterpret_cast<const float4*>(keys + element(j + 1, i, ahead)));
      }
#pragma unroll
      for (int w = L / 2; w >= 1; w /= 2) {
        const bool high = lane & w;
#pragma unroll
        for (int i = 0; i < w; ++i) {
          const float got = __shfl_xor_sync(0xffffffffu, high ? x[i] : x[i + w], w);
          x[i] = (high ? x[i + w] : x[i]) + got;
        }
      }
      // the lane's pair: row lane % R, slot part / R of its half
      const int slot = n0 + j * SR + part / R * HALVES + half;
      const float logit = slot < see ? x[0] * scale : -INFINITY;
      float top = logit;
#pragma unroll
      for (int w = R; w < 32; w *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const bool raise = top > m + kRaise || (m == -INFINITY && top > m);
      if (__any_sync(0xffffffffu, raise)) {
        const float by = raise ? exp2f(m - top) : 1.f;  // 0 for the first reference
        if (raise) m = top;
        l *= by;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float f = __shfl_sync(0xffffffffu, by, r);
          o[r].x *= f;
          o[r].y *= f;
          o[r].z *= f;
          o[r].w *= f;
        }
      }
      const float weight = exp2f(logit - (m == -INFINITY ? 0.f : m));
      l += weight;
#pragma unroll
      for (int i = 0; i < SL; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float f = __shfl_sync(0xffffffffu, weight, half * L + i * R + r);
          o[r].x = fmaf(f, v[i].x, o[r].x);
          o[r].y = fmaf(f, v[i].y, o[r].y);
          o[r].z = fmaf(f, v[i].z, o[r].z);
          o[r].w = fmaf(f, v[i].w, o[r].w);
        }
      if (j + 1 < rounds) {
#pragma unroll
        for (int i = 0; i < SL; ++i) v[i] = __ldcs(reinterpret_cast<const float4*>(values + element(j + 1, i, ahead)));
      }
      if (turn) {
        at = next;
        const int step = p.u0 + (j + 1) / kRounds + 1;
        next = step < p.u1 ? slot_row(c, p.b, p.h, step * kStep) : 0;
      }
    }
    // the piece's sums to its slice
#pragma unroll
    for (int w = R; w < 32; w *= 2) l += __shfl_xor_sync(0xffffffffu, l, w);
    if (!inside(p.slice >= 0 && p.slice < (p.own ? a.most_own : a.most_shared) && p.row0 + (p.rows - 1) / group < co.total_q, co.status)) continue;
    const int64_t slice = int64_t(p.slice) * co.total_q * qh;
    if (lane < R && lane < p.rows) *reinterpret_cast<float2*>(side.ml + (slice + row_of(lane)) * 2) = make_float2(m, l);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (HALVES == 2) {
        o[r].x += __shfl_xor_sync(0xffffffffu, o[r].x, 16);
        o[r].y += __shfl_xor_sync(0xffffffffu, o[r].y, 16);
        o[r].z += __shfl_xor_sync(0xffffffffu, o[r].z, 16);
        o[r].w += __shfl_xor_sync(0xffffffffu, o[r].w, 16);
      }
      if (half == 0 && r < p.rows) *reinterpret_cast<float4*>(side.part + (slice + row_of(r)) * D + part * 4) = o[r];
    }
  }
}

template <int D>
cudaError_t launch(const PrefixFew& a, int rows, int ctas, cudaStream_t st) {
  if (rows <= 4) k_prefix_few32<D, 4><<<ctas, kWarps * 32, 0, st>>>(a);
  else if (rows <= 8) k_prefix_few32<D, 8><<<ctas, kWarps * 32, 0, st>>>(a);
  else k_prefix_few32<D, 16><<<ctas, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix_few32(const PrefixFew& a, int rows, cudaStream_t st) {
  const int ctas = device_sm_count() * resident(rows);
  return a.own.c.d == 128 ? launch<128>(a, rows, ctas, st) : launch<64>(a, rows, ctas, st);
}

}  // namespace mp
