// Attention with shared prefixes, with few query rows per KV head (tokens x heads of the group): the own
// slots of sequences with up to 16 rows (d = 64: 32), and the prefixes of groups with as few, or with more
// over short prefixes, as many of them at a time. bf16, bound by one pass over K and V (467 MB of own slots
// of 128 tokens: 88 us, 5.3 TB/s).
//
// Many sequences with a few hundred slots each are many short streams, and what a stream costs besides
// its bytes (lengths, pages, Q, the sums' way out) is as much as they are. So every warp works for itself,
// without a barrier of its CTA: the steps of all (sequence, KV head) units, 16 slots each, are laid end to
// end and cut into equal runs, one a warp. A warp's TMA copies run ahead of its products by a ring of
// three steps (d = 64: six), across the ends of units. A unit that is cut lies in several slices: warp w
// writes slice w - (first warp of the unit), k_prefix_join joins them.
//
// S and O^T are warp-level products, with the fragments of the few-row attention (mp_chunk_step.cu):
// lane (g, t) takes the 16-byte chunks t, t + 4, ... of the keys g and g + 8, and chunk g of V of the
// keys 2t, 2t + 1, 2t + 8 and 2t + 9. P enters the second product as the sum of two bf16 terms.
#pragma once

#include "mp_cache.cuh"
#include "mp_prefix.h"
#include "mp_tc.cuh"

namespace mp {
namespace few {

constexpr int kStep = 16;     // slots
constexpr int kLead = 3;      // steps that starting and ending a unit counts as
constexpr int kMinRun = 4;    // steps of a warp at least
constexpr int kKept = 8192;   // units' lengths that the planning keeps
// How work is cut: blocks of so many query rows, and the four above.
template <int ROWS, int STEP = kStep, int LEAD = kLead, int MIN_RUN = kMinRun, int KEPT = kKept>
struct Cutting {
  static constexpr int kRows = ROWS, kStep = STEP, kLead = LEAD, kMinRun = MIN_RUN, kKept = KEPT;
};
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRaise = 8.0f;

struct Maps {
  CUtensorMap k[2], v[2];  // of the prefixes, of the own slots
};
struct Piece {
  int own, b;  // 0: of a prefix; group or sequence
  int row0, r0, rows, first, n, h, u0, u1, slice;  // rows [r0, rows) of those that start in packed row row0
};
// A warp's tiles (from a 1024-byte boundary: copies are swizzled) and the rest of its shared memory.
template <int D, int STAGES>
struct Ring {
  static constexpr int kSub = D / 64;
  __nv_bfloat16 tile[STAGES][2][kSub][kStep * 64];
};
template <int STAGES>
struct State {
  static_assert(STAGES <= 6);  // and so at most eight pieces in `piece`
  uint64_t full[STAGES];
  Piece piece[8];  // from the one that is worked on to the one that is fetched
  uint32_t abort;
};

bool few_maps(const PrefixFew& a, Maps* maps);  // false when the driver refuses

#ifdef __CUDACC__
__device__ __forceinline__ Seq unit_of(const PrefixFew& a, int v) {
  return v < a.groups ? group_of(a.pre.c, v) : seq_of(a.own.c, v - a.groups);
}
template <typename C>
__device__ __forceinline__ void note_pieces(const PrefixFew& a, int v, const Seq& s, int h, int block, int pieces) {
  const bool own = v >= a.groups;
  const int key = piece_key(s.row0, a.own.c.group, C::kRows, block, own ? v - a.groups : v), keys = own ? a.own_keys : a.pre_keys;
  if (!inside(key >= 0 && key < keys && pieces >= 0 && pieces <= (own ? a.most_own : a.most_shared), a.own.c.status)) return;
  (own ? a.own_pieces : a.pre_pieces)[int64_t(h) * keys + key] = pieces;
}
template <typename C>
__device__ __forceinline__ int steps_in(const Seq& s) { return s.m > 0 ? (s.n + C::kStep - 1) / C::kStep : 0; }
template <typename C>
__device__ __forceinline__ int blocks_in(const Seq& s, int group) { return (s.m * group + C::kRows - 1) / C::kRows; }

// Lengths and blocks of the units of this thread, of `threads`: their steps, summed and with kLead each (of
// one KV head), and the least steps of a run for which no unit is cut into more pieces than it may. Units
// without a slot have no piece.
template <typename C>
__device__ __forceinline__ void survey(const PrefixFew& a, int2* kept, int thread, int threads, int64_t* sum, int* at_least) {
  const CacheCall& co = a.own.c;
  const int kvh = co.kvh, group = co.group;
  const int units = a.groups + (a.own_units ? co.batch : 0);
  int64_t total = 0;
  int64_t least = C::kMinRun;  // as long as a unit's steps by one less than its most pieces
  for (int v = thread; v < units; v += threads) {
    const Seq s = unit_of(a, v);
    const int n = steps_in<C>(s), blocks = blocks_in<C>(s, group);
    if (v < C::kKept) kept[v] = make_int2(n, blocks);
    total += n ? int64_t(n + C::kLead) * blocks : 0;
    const int most = v < a.groups ? a.most_shared : a.most_own;
    least = max(least, int64_t((n + most - 2) / (most - 1)));
    if (n == 0 && v % gridDim.x == blockIdx.x)
      for (int h = 0; h < kvh; ++h)
        for (int i = 0; i < blocks; ++i) note_pieces<C>(a, v, s, h, i, 0);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  *sum = total;
  *at_least = __reduce_max_sync(0xffffffffu, int(least));
}

// A worker's run, `worker` of `workers`, of `total` steps in all: its pieces in order. All lanes hold the same.
template <typename C>
struct Walk {
  static constexpr int kLead = C::kLead;
  const PrefixFew& a;
  int64_t run, r0, r1, at = 0;  // at: the first step of the unit (kLead of them before its slots) among all
  int units, v = 0, i = 0, steps = 0, blocks = 1;  // i: KV head and block of rows, the blocks next to each other
  Seq s = {0, 0, 0, 0};

  __device__ __forceinline__ Walk(const PrefixFew& few, const int2* kept, int64_t total, int64_t least, int64_t worker, int64_t workers) : a(few) {
    const int lane = threadIdx.x & 31, kvh = a.own.c.kvh, group = a.own.c.group;
    units = a.groups + (a.own_units ? a.own.c.batch : 0);
    run = max(least, quotient(total + workers - 1, workers));
    r0 = worker * run;
    r1 = min(total, r0 + run);
    if (r0 >= total) {
      at = r1;  // nothing is left
      return;
    }
    int64_t in = r0;  // into what is left
    for (int v0 = 0; v0 < units; v0 += 32) {
      int2 k = make_int2(0, 1);
      if (v0 + lane < units) {
        if (v0 + lane < C::kKept) {
          k = kept[v0 + lane];
        } else {
          const Seq u = unit_of(a, v0 + lane);
          k = make_int2(steps_in<C>(u), blocks_in<C>(u, group));
        }
      }
      const int64_t mine = k.x ? int64_t(k.x + kLead) * kvh * k.y : 0;
      int64_t pre = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, pre > in);
      if (past) {
        const int l = __ffs(past) - 1;
        in -= __shfl_sync(0xffffffffu, pre - mine, l);
        v = v0 + l;
        steps = __shfl_sync(0xffffffffu, k.x, l);
        blocks = __shfl_sync(0xffffffffu, k.y, l);
        break;
      }
      in -= __shfl_sync(0xffffffffu, pre, 31);
    }
    i = int(quotient(in, int64_t(steps + kLead)));
    at = r0 - (in - int64_t(i) * (steps + kLead));
    s = unit_of(a, v);
  }
  __device__ __forceinline__ void advance() {  // to the next unit
    at += steps + kLead;
    if (++i < a.own.c.kvh * blocks) return;
    i = 0;
    steps = 0;
    while (at < r1 && ++v < units) {
      s = unit_of(a, v);
      steps = steps_in<C>(s);
      blocks = blocks_in<C>(s, a.own.c.group);
      if (steps) break;
    }
    if (steps == 0) at = r1;
  }
  // The piece of the unit that the walk is at, or of the first behind it that has one; false where the run
  // has ended. The warp that starts a unit notes its number of pieces.
  __device__ __forceinline__ bool open(Piece* p) {
    for (; at + kLead < r1; advance()) {
      const int64_t lead = at + kLead;
      const int u0 = int(max(int64_t(0), r0 - lead)), u1 = int(min(int64_t(steps), r1 - lead));
      if (u1 <= u0) continue;
      const int64_t first = quotient(lead, run);  // the warp that has the unit's first step
      const int h = i / blocks, block = i - h * blocks;
      p->own = v >= a.groups;
      p->b = v >= a.groups ? v - a.groups : v;
      p->row0 = s.row0;
      p->r0 = block * C::kRows;
      p->rows = s.m * a.own.c.group;
      p->first = s.first;
      p->n = s.n;
      p->h = h;
      p->u0 = u0;
      p->u1 = u1;
      p->slice = int(quotient(r0, run) - first);
      if (u0 == 0 && (threadIdx.x & 31) == 0) note_pieces<C>(a, v, s, h, block, int(quotient(lead + steps - 1, run) - first) + 1);
      return true;
    }
    return false;
  }
};

// One warp's run: `worker` of `workers`, of `total` steps in all. `found` is called by all warps of the CTA
// between the last look at `kept` and the first copy into the rings.
template <int D, int NT, int STAGES, typename F>
__device__ __forceinline__ void work(const Maps& maps, const PrefixFew& a, Ring<D, STAGES>& ring, State<STAGES>& S, const int2* kept, const int64_t total,
                                     const int64_t least, const int64_t worker, const int64_t workers, F found) {
  constexpr int kStages = STAGES, kSub = Ring<D, STAGES>::kSub;
  static_assert(sizeof(ring.tile[0][0][0]) % 1024 == 0);
  constexpr int KC = D / 32, VC = D / 64, TILES = D / 16;
  constexpr int kSets = (NT + 1) / 2;  // 16-row sets of Q
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const CacheCall& co = a.own.c;
  const int kvh = co.kvh, group = co.group, qh = kvh * group;
  Walk<Cutting<NT * 8>> walk(a, kept, total, least, worker, workers);
  found();
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&S.full[i], 1);
    S.abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
  }
  __syncwarp();

  // ---- fetching: pieces in order, a step a call ----
  uint32_t fetched = 0, pushed = 0;
  int fu = 0, f_base = 0, f_row = 0;
  Piece next = {};  // the piece that is fetched
  auto look = [&]() {  // the next 32 steps' rows of the pool, one a lane
    f_base = fu;
    const CacheCall& c = next.own ? co : a.pre.c;
    f_row = fu + lane < next.u1 ? slot_row(c, next.b, next.h, (fu + lane) * kStep) : 0;
  };
  auto open = [&]() {
    if (!walk.open(&next)) return false;
    if (lane == 0) S.piece[pushed & 7] = next;
    ++pushed;
    fu = next.u0;
    look();
    return true;
  };
  bool more = open();
  auto fetch = [&]() {
    if (!more) return;
    const int st = int(fetched % kStages);
    if (fu - f_base == 32) look();
    const int row = __shfl_sync(0xffffffffu, f_row, fu - f_base);
    uint32_t bytes = kStep * D * 2 * 2;
#if MP_CHECK
    if (a.stall && worker == 0 && fetched == 0) bytes += 16;  // that never come: the wait for them runs out
#endif
    if (lane == 0) mbar_expect_tx(&S.full[st], bytes);
    __syncwarp();
    if (lane < 2 * kSub) {
      const int kv = lane / kSub, sub = lane % kSub, which = next.own;
      tma_load_2d(&ring.tile[st][kv][sub][0], kv ? &maps.v[which] : &maps.k[which], sub * 64, row, &S.full[st]);
    }
    ++fetched;
    if (++fu == next.u1) {
      walk.advance();
      more = open();
    }
  };
  for (int i = 0; i < kStages; ++i) fetch();

  // ---- the pieces ----
  uint32_t used = 0;
  bool ok = true;
  const float scale = kLog2e * rsqrtf(float(D));
  for (uint32_t i = 0; i < pushed && ok; ++i) {
    __syncwarp();
    const Piece p = S.piece[i & 7];
    uint4 q[NT][KC];
    int see[NT];  // the lane's row (8 u + g) sees the slots below this
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int r = p.r0 + u * 8 + g;
      see[u] = r < p.rows ? min(p.n, p.first + r / group + 1) : 0;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.own.q) +
                                 (int64_t(p.row0 + r / group) * qh + p.h * group + r % group) * D + t * 8;
#pragma unroll
      for (int j = 0; j < KC; ++j) q[u][j] = r < p.rows ? *reinterpret_cast<const uint4*>(src + j * 32) : make_uint4(0, 0, 0, 0);
    }
    float o[NT][TILES][4], m[NT], l[NT];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      m[u] = -INFINITY;
      l[u] = 0.f;
#pragma unroll
      for (int j = 0; j < TILES; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[u][j][k] = 0.f;
    }
    for (int u16 = p.u0; u16 < p.u1; ++u16) {
      const int st = int(used % kStages), n0 = u16 * kStep;
      ok = mbar_wait_warp(&S.full[st], (used / kStages) & 1, &S.abort);
      if (!ok) break;
      const char* const ks = reinterpret_cast<const char*>(&ring.tile[st][0][0][0]);
      char* const vs = reinterpret_cast<char*>(&ring.tile[st][1][0][0]);
      if (n0 + kStep > p.n) {
        // rows of V behind the last slot may hold anything, and 0 * NaN is NaN (in S they are masked)
        const int live = p.n - n0;
#pragma unroll
        for (int j = 0; j < kSub; ++j)
          for (int k = live * 8 + lane; k < kStep * 8; k += 32) *reinterpret_cast<uint4*>(vs + j * (kStep * 128) + k * 16) = make_uint4(0, 0, 0, 0);
        fence_async();  // before the next copy into this place
        __syncwarp();
      }
      // 16-byte chunk c of row r of a tile lies at c ^ (r % 8)
      float x[NT][2][2];
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2) {
        float d[kSets][4];
#pragma unroll
        for (int s = 0; s < kSets; ++s) d[s][0] = d[s][1] = d[s][2] = d[s][3] = 0.f;
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          const int c = t + 4 * j, r = g + 8 * i2;
          const uint4 k = *reinterpret_cast<const uint4*>(ks + (c >> 3) * (kStep * 128) + r * 128 + (((c & 7) ^ g) << 4));
#pragma unroll
          for (int s = 0; s < kSets; ++s) {
            const uint4 lo = q[2 * s][j], hi = 2 * s + 1 < NT ? q[2 * s + 1 < NT ? 2 * s + 1 : 0][j] : make_uint4(0, 0, 0, 0);
            mma_16816(d[s], lo.x, hi.x, lo.y, hi.y, k.x, k.y);
            mma_16816(d[s], lo.z, hi.z, lo.w, hi.w, k.z, k.w);
          }
        }
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            x[u][i2][j] = n0 + 8 * i2 + 2 * t + j < see[u] ? d[u / 2][2 * (u & 1) + j] * scale : -INFINITY;
      }
      uint4 v[4][VC];
      auto load_v = [&]() {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = 2 * t + (k & 1) + 8 * (k >> 1);
#pragma unroll
          for (int j = 0; j < VC; ++j) v[k][j] = *reinterpret_cast<const uint4*>(vs + j * (kStep * 128) + r * 128 + ((g ^ (r & 7)) << 4));
        }
        __syncwarp();  // K and V have been read
        ++used;
        fetch();
      };
      if (NT < 4) load_v();  // else when the softmax needs its registers no more
      uint32_t w[NT][2], rest[NT][2];  // P and what its rounding leaves
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
          for (int j = 0; j < TILES; ++j) {
            o[u][j][0] *= b0;
            o[u][j][1] *= b1;
            o[u][j][2] *= b0;
            o[u][j][3] *= b1;
          }
        }
        const float ref = m[u] == -INFINITY ? 0.f : m[u];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float e0 = ex2(x[u][j][0] - ref), e1 = ex2(x[u][j][1] - ref);
          l[u] += e0 + e1;
          w[u][j] = bf2(e0, e1);
          rest[u][j] = bf2(e0 - __uint_as_float(w[u][j] << 16), e1 - __uint_as_float(w[u][j] & 0xffff0000u));
        }
      }
      if (NT == 4) load_v();
      auto word = [](const uint4& y, int k) { return k == 0 ? y.x : (k == 1 ? y.y : (k == 2 ? y.z : y.w)); };
      auto pair = [&](const uint4& y, const uint4& z, int e) { return __byte_perm(word(y, e >> 1), word(z, e >> 1), (e & 1) ? 0x7632 : 0x5410); };
#pragma unroll
      for (int j = 0; j < TILES; ++j) {
        const int e1 = D == 128 ? j : j + 4, c1 = D == 128 ? VC - 1 : 0;
        const uint32_t a0 = pair(v[0][0], v[1][0], j), a1 = pair(v[0][c1], v[1][c1], e1);
        const uint32_t a2 = pair(v[2][0], v[3][0], j), a3 = pair(v[2][c1], v[3][c1], e1);
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          mma_16816(o[u][j], a0, a1, a2, a3, w[u][0], w[u][1]);
          mma_16816(o[u][j], a0, a1, a2, a3, rest[u][0], rest[u][1]);
        }
      }
    }
    if (!ok) break;
    // The piece's sums to its slice. Lane (g, t) has the rows 2t and 2t + 1 of every eight, of them the
    // elements 8 g .. 8 g + 7 (d = 128: and those 64 further on).
    const PrefixArgs& to = p.own ? a.own : a.pre;
    if (!inside(p.slice >= 0 && p.slice < (p.own ? a.most_own : a.most_shared) && p.row0 + (p.rows - 1) / group < co.total_q, co.status)) continue;
    const int64_t slice = int64_t(p.slice) * co.total_q * qh;
    auto row_at = [&](int r) { return slice + int64_t(p.row0 + r / group) * qh + p.h * group + r % group; };
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
      if (t == 0 && p.r0 + u * 8 + g < p.rows) *reinterpret_cast<float2*>(to.ml + row_at(p.r0 + u * 8 + g) * 2) = make_float2(m[u], l[u]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = p.r0 + u * 8 + 2 * t + k;
        if (r >= p.rows) continue;
        float4* dst = reinterpret_cast<float4*>(to.part + row_at(r) * D + 8 * g);
        dst[0] = make_float4(o[u][0][k], o[u][1][k], o[u][2][k], o[u][3][k]);
        if constexpr (D == 128) {
          dst[1] = make_float4(o[u][4][k], o[u][5][k], o[u][6][k], o[u][7][k]);
          dst[16] = make_float4(o[u][0][2 + k], o[u][1][2 + k], o[u][2][2 + k], o[u][3][2 + k]);
          dst[17] = make_float4(o[u][4][2 + k], o[u][5][2 + k], o[u][6][2 + k], o[u][7][2 + k]);
        } else {
          dst[1] = make_float4(o[u][0][2 + k], o[u][1][2 + k], o[u][2][2 + k], o[u][3][2 + k]);
        }
      }
    }
  }
  if (!ok && lane == 0) {
    for (; used != fetched; ++used) mbar_drain(&S.full[used % kStages], (used / kStages) & 1);
    flag(co.status, MP_STATUS_WAIT_TIMEOUT);
  }
}
#endif

}  // namespace few
}  // namespace mp
