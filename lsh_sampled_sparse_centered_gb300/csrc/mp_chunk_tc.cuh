// Exact attention of a chunk of new tokens on the 5th-generation tensor cores (bf16), and of the rows of
// groups over the prefixes that their sequences share (see Mode).
//
// A CTA works on 256 query rows of one KV head (row = token * group + head of the group),
// as two halves of 128 rows, against 128 keys at a time:
//   S = Q K^T   (128 x 128 x d, both operands in shared memory, fp32 in tensor memory)
//   P = 2^(S log2(e) / sqrt(d) - m)   one thread per row, P as bf16 over S's columns
//   O += P V    (128 x d x 128, P from tensor memory, V from shared memory)
// While the softmax warps of one half work, the tensor cores work for the other half.
// Warps 0-3 and 4-7 are the softmax of the halves, warp 8 streams K and V by TMA into a
// ring of shared-memory tiles, warps 9 and 11 issue the halves' products, warp 10 walks the
// CTA's work.
//
// The reference m of a row is raised only when a logit passes it by more than 8 (in log2),
// so that O is rescaled in few steps; P then is at most 2^8, which costs a float nothing.
// P enters the second product as bf16 (2^-8 relative per weight); the sum of the weights
// is taken before that rounding. Everything else is fp32.
//
// Tensor memory: S of the halves in columns 0 and 128, O in 256 and 256 + d. With d = 128
// that fills it and P overlays its S, so that the next S waits for the product with P. With
// d = 64 P has columns of its own (384 and 448): the next S is formed while the softmax of
// this one still runs.
//
// With d = 128 the halves take turns: one reads its S and weighs three quarters of it, then
// the other may. Left alone they may fall into step, both in the softmax and then both
// waiting for products, and stay there (2048 tokens over 32768 slots, 32/8 heads, short runs: 700
// to 770 us by how they started, 670 us with turns, 750 in long runs under the power cap; 1024 over
// 8192: 117 and 104 us). With d = 64, where S is formed ahead, turns cost a quarter (540 against
// 680 us).
#pragma once

#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

#include "mp_cache.cuh"
#include "mp_prefix_few.cuh"
#include "mp_tc.cuh"

namespace mp {
namespace {

constexpr int kRows = kTileRows;  // query rows of a CTA
constexpr int kKeys = 128;   // keys of a step
constexpr int kThreads = 384;  // 12 warps: two of softmax for each lane quarter, TMA, work, two of products
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.0f;
constexpr int kGroup = 1024;  // sequences of a launch
// Units that starting and ending a tile costs: 5.5 us, a step 1.1 us with d = 64 and 1.5 with
// d = 128, of which some runs under the neighbouring tiles. Where there are tiles for every
// CTA, d = 128 counts more (8192 tokens over as many slots: 429 us with 3, 404 with 4, 398 with
// 5, 394 with 6); where tiles are cut in many pieces, less (300 over 2000: 27.3 and 29.5 us).
constexpr int kLead = 3, kLeadWhole = 5;
// The same for a piece of a cut, whose sums are written and joined besides: its start is Q behind the first
// copies of K and V (1 and 2 pieces a CTA, 512 rows over 98304 slots: 139 and 150 us).
constexpr int kLeadPiece = 7;
// And where every tile's sums are written and joined (six chunks of 33 to 517 tokens over 16384 shared
// slots, 32/8 heads: 302 us with 5, 277 with 8, 280 with 11, 286 with 14).
constexpr int kLeadBoth = 8;
constexpr int kMinRun = 2;    // units of a CTA at least
constexpr int kCut = 10;      // units that cutting the tiles costs: a second piece for most CTAs, and the join

// One piece of work: the steps [u0, u1) of a tile, as every role of the CTA sees it.
struct Piece {
  int b, h, row0, n, lead;  // sequence, KV head, first packed row, slots, slot of that row
  int r0, rows;             // the tile's first row, and the rows of the whole chunk
  int u0, u1;               // u0 == u1: the run has ended
  int whole, slot;          // all of its tile's units; else where its partial result goes (in slices: the slice)
};

static_assert(kKeys / 16 <= 8, "boxes of 16 rows at least");

// What a launch works on, and where its sums go. P is one bf16 term in all of them, for single tokens over prefixes
// too, which mp_chunk_step gives two: a second is a second product and its conversions in the softmax warps, whose
// chain a step waits for, and with d = 64 tensor memory has no place for it. (Error of the output against 64 bits
// 0.0023, of rounding it alone 0.0017.)
enum Mode {
  kChunk,  // chunks over their sequences' slots: out and lse
  kBoth,   // groups' rows over the prefixes that their sequences share, and chunks over their own slots: sums to a.state
  kCuts,   // groups over their prefixes in slices: every tile of a group is cut into as many pieces of its keys
  kPairs,  // the same with at most 128 rows a group: the halves share them and take every other step
};

// The prefixes of kBoth: its units are the groups, and behind them the sequences of `a`.
struct Prefixes {
  CacheArgs c;
  int box, groups;
  int64_t own_slice;  // where the own slots' sums begin, in rows of a.state
  int first_slot;     // of this launch's cut tiles
  int pre_keys, own_keys;
  int2 *pre_pieces, *own_pieces;  // [KV head][keys], at piece_key() of kRows: pieces of a tile, and the slot of the first if it is cut
};

template <int D>
struct Smem {
  static constexpr int kSub = D / 64;
  static constexpr bool kOwnP = D == 64;  // P beside S
  static constexpr int kStages = D == 128 ? 5 : 8;
  __nv_bfloat16 q[2][kSub][128 * 64];
  __nv_bfloat16 kv[kStages][kSub][kKeys * 64];
  uint64_t full[kStages], empty[kStages], tail;
  uint64_t q_full[2], s_full[2], s_free[2], p_full[2][2], o_full[2];
  uint64_t piece_full[2], piece_empty[2], drain[2], turn[2];
  Piece piece[2];
  int64_t left, run;
  int lead;      // units that a tile counts besides its steps
  int start[4];  // sequence, KV head, tile, unit
  Seq first;     // that sequence
  int longest[12];  // steps of a tile, of each warp's sequences
  uint64_t pair_full, pair_done, q_asked;
  int64_t own_total[12], tile_steps, tiles;  // slices: each warp's own steps, all tiles' steps of a KV head
  int own_least[12];
  uint8_t filled[kStages];  // phase in which each tile of the ring was last filled (1: never)
  uint32_t tmem_base;
  uint32_t abort;
};

__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return r;
}
// MN-major operand (V: rows are keys, d contiguous) in 128B-swizzled boxes of 64 elements
// x 128 keys: 8-key groups 1024 B apart, 64-element groups 128 rows apart.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t addr) {
  uint64_t d = 0;
  d |= uint64_t((addr & 0x3FFFFu) >> 4);
  d |= uint64_t((kKeys * 128) >> 4) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}
// Work is counted in units: one 256-row tile of a KV head against 128 keys (a tile that
// sees nothing counts one, so that its rows are written), and `lead` more for starting a
// tile. The units of all tiles, in the order (sequence, KV head, tile, lead, keys), are cut
// into equal runs, one per CTA, whatever the lengths: a CTA's run covers the end of one
// tile, whole tiles, and the start of another.
// Whole tiles are written out; of a tile that is cut every piece stores its unnormalised
// sum, and k_chunk_tc_join puts the pieces together. A CTA has two such pieces at most: the
// one that starts its run (slot 2 cta) and the one that ends it (slot 2 cta + 1). With prefixes (kBoth) whole
// tiles are sums too, pieces lie [slot][row][d] and k_prefix_join finds them; the first is in an odd slot and
// the others in the even ones of the CTAs behind.
__device__ __forceinline__ int tiles_of(const Seq& s, int group) {
  return int((int64_t(s.m) * group + kRows - 1) / kRows);
}
// steps of tile t: 128 keys each, up to the last slot that its last token sees
__device__ __forceinline__ int steps_of(const Seq& s, int group, int t) {
  const int64_t last = min(int64_t(t + 1) * kRows, int64_t(s.m) * group) - 1;
  const int see = min(s.n, s.first + int(last / group) + 1);
  return max(1, (see + kKeys - 1) / kKeys);
}

// What k_chunk_tc_join needs of a tile that CTA `cta` began and did not end.
struct Cut {
  int64_t row;     // packed row of the tile's first token, as a row of (token, query head)
  int pieces;      // CTAs that share the tile (0: nothing to join)
  int slot;        // slot of the first piece; the others are slots 2 (cta + i)
  int r0, rows;    // the tile's first row and its rows
};

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Pieces of a tile of `steps` steps, so that none is longer than `longest`; piece i of n starts at its
// step i steps / n.
__device__ __forceinline__ int pieces_of(int steps, int longest) { return (steps + longest - 1) / longest; }
// Steps of a prefix (0: none).
__device__ __forceinline__ int prefix_steps(const Seq& s) { return (s.n + kKeys - 1) / kKeys; }

// The cut of kCuts and kPairs. Tiles that share a prefix are cut at the same keys and worked on side by
// side, so that K and V come from HBM once whatever the number of tiles (512 rows over 98304 slots of
// eight KV heads in equal runs of units, whose tiles meet a key 400 MB apart: twice). Pieces are at most
// L steps long: short enough that there are no more than r for every CTA, for the r that ends first. With
// U steps and T tiles in all, L steps give U / L to U / L + T pieces: for each r that leaves L between two
// limits, of which the upper one is short enough; up to 32 groups are counted for four values, one a lane.
// Called by a warp. get(g, &steps, &tiles) says a group's steps and tiles (of a KV head); it is called by
// all lanes at once, with one group each in `own` and with the same one otherwise.
template <typename Own, typename Get>
__device__ __forceinline__ int longest_piece(Own own, Get get, int groups, int kvh, int ctas, int most_pieces) {
  const int lane = threadIdx.x & 31;
  int top = 1;
  int64_t all = 0, all_tiles = 0;
  for (int g = lane; g < groups; g += 32) {
    int steps, tiles;
    own(g, &steps, &tiles);
    if (tiles) top = max(top, steps);
    all += int64_t(tiles) * steps;
    all_tiles += steps ? tiles : 0;
  }
  top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    all_tiles += __shfl_xor_sync(0xffffffffu, all_tiles, o);
  }
  all *= kvh;
  all_tiles *= kvh;
  const int64_t r = 1 + lane / 4, room = r * ctas - all_tiles;
  const bool counted = groups <= 32;
  uint32_t cost = UINT32_MAX;
  int length = top, high = top;
  if (room > 0) {
    const int low = int(quotient(all + r * ctas - 1, r * ctas));
    high = int(min(int64_t(top), quotient(all + room - 1, room)));
    length = max(max(1, (top + most_pieces - 1) / most_pieces), min(top, counted ? low + (high - low) * (lane & 3) / 3 : high));
  }
  int64_t n = 0;
  for (int g = 0; counted && g < groups; ++g) {
    int steps, tiles;
    get(g, &steps, &tiles);
    n += int64_t(tiles) * pieces_of(steps, length);
  }
  if (room > 0 && (length >= high || (counted && n * kvh <= r * ctas))) cost = uint32_t(min(r * (length + kLeadPiece), int64_t(INT32_MAX)));
  const uint32_t best = __reduce_min_sync(0xffffffffu, cost);
  if (best == UINT32_MAX) return top;
  return __shfl_sync(0xffffffffu, length, __ffs(__ballot_sync(0xffffffffu, cost == best)) - 1);
}

// What the modes take besides: kBoth the prefixes, the slices the own slots, which some CTAs go over meanwhile.
template <Mode MODE>
struct Extra {};
template <>
struct Extra<kBoth> {
  CUtensorMap k, v;
  Prefixes pre;
};
struct OwnSide {
  few::Maps maps;
  PrefixFew few;
};
template <>
struct Extra<kCuts> : OwnSide {};
template <>
struct Extra<kPairs> : OwnSide {};
template <Mode MODE>
using ArgsOf = std::conditional_t<MODE == kChunk, ChunkArgs, PrefixArgs>;

// CTAs of `ctas` that take the own slots (the last of the grid), so that both kinds end together. Times in
// 0.1 us: a step of large tiles takes an SM 1.5 us with two halves (d = 64: 1.1) and about 1.0 for 128 rows
// on alternate steps (0.6), with 12 us at the start and the end; 16 own slots 0.13 us (0.07), and 4. Where a
// group of SMs that load through one port (20 of them, in the order of the grid) has both kinds, the
// tiles there wait for a third of the time that the own slots take: 32 tokens over 32768 shared slots take
// 56 us with 40 own CTAs, 63 with 48; the kinds spread over each other (in pairs of SMs) 60, and 128 tokens
// over 98304 210 and 233. Tried with the tiles' steps or the own slots a third shorter and two fifths longer, and the own
// slots twice as long, on twelve batches (d = 64 and 128; 16/4, 32/8, 64/8, 16/2, 8/1, 40/40 heads; 16 to 128 tokens
// over 16384 to 98304 shared and 256 to 1500 own slots): none is more than 6 % better in any, and each is 14 to 59 %
// worse in some. Called by a warp; each lane tries one split.
template <int D, bool PAIR>
__device__ __forceinline__ int own_ctas(int64_t tile_steps, int64_t tiles, int64_t own_steps, int ctas) {
  if (own_steps == 0) return 0;
  if (tile_steps == 0) return ctas;
  constexpr int kPort = 20;
  const float step = D == 128 ? (PAIR ? 10.f : 15.f) : (PAIR ? 6.f : 11.f), own = D == 128 ? 1.3f : 0.7f;
  const int lane = threadIdx.x & 31, most = int(quotient(ctas, tiles));  // pieces that each tile can have at once
  // whole ports, or what whole numbers of pieces leave, or even parts
  int n = lane < 7 ? (lane + 1) * kPort : (most >= 2 ? ctas - (most - (lane - 7)) * int(tiles) : (lane - 6) * ctas / 26);
  const bool fits = n <= ctas - 1 && (lane < 7 || most < 2 || most - (lane - 7) >= 1);
  n = max(1, min(ctas - 1, n));
  const int64_t pieces = quotient(ctas - n, tiles);
  const float tile_time = 120.f + step * (pieces >= 1 ? ceilf(float(tile_steps) / float(pieces * tiles)) : float(tile_steps) / float(ctas - n));
  const float own_time = 40.f + float(own_steps) * own / float(n);
  const float time = fits ? fmaxf(tile_time + (n % kPort ? own_time / 3.f : 0.f), own_time) : INFINITY;
  float best = time;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, o));
  return __shfl_sync(0xffffffffu, n, __ffs(__ballot_sync(0xffffffffu, time == best)) - 1);
}

// NT: rows in eights of the own side's units (slices).
template <int D, Mode MODE, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    k_chunk_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const ArgsOf<MODE> a,
               const int box, const int b_begin, const int b_end, const int slot_rows,
               const __grid_constant__ Extra<MODE> extra) {
  constexpr bool BOTH = MODE == kBoth;
  constexpr bool PAIR = MODE == kPairs, CUT = MODE == kCuts || PAIR;
  extern __shared__ __align__(1024) unsigned char smraw[];
  const uint32_t base = saddr(smraw);
  Smem<D>& S = *reinterpret_cast<Smem<D>*>(smraw + ((1024 - (base & 1023)) & 1023));
  constexpr int kSub = Smem<D>::kSub, kStages = Smem<D>::kStages;
  // 128-byte swizzle: copies and products take the tiles from 1024-byte boundaries (members in
  // front of them would move them off, and the copies then fault)
  static_assert(offsetof(Smem<D>, q) % 1024 == 0 && offsetof(Smem<D>, kv) % 1024 == 0 && sizeof(S.q[0][0]) % 1024 == 0 &&
                sizeof(S.kv[0][0]) % 1024 == 0);
  constexpr uint32_t kRowBytes = 128;
  const auto& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile uint32_t* abort = &S.abort;
  const int qh = c.kvh * c.group;
  auto rows_at = [&](int b) {
    if constexpr (BOTH) return b < extra.pre.groups ? group_of(extra.pre.c, b) : seq_of(c, b - extra.pre.groups);
    else return rows_of<CUT>(c, b);
  };

  if (threadIdx.x == 320) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 2);  // both halves' products
      S.filled[i] = 1;
    }
    mbar_init(&S.tail, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.q_full[i], 4);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.s_free[i], 4);
      mbar_init(&S.p_full[i][0], 4);
      mbar_init(&S.p_full[i][1], 4);
      mbar_init(&S.piece_full[i], 1);
      mbar_init(&S.piece_empty[i], 11);  // the TMA warp, two of products, eight of softmax
      mbar_init(&S.o_full[i], 1);
      mbar_init(&S.drain[i], 1);
      mbar_init(&S.turn[i], 4);
    }
    mbar_init(&S.pair_full, 8);
    mbar_init(&S.pair_done, 8);
    mbar_init(&S.q_asked, 4);
    S.abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (CUT) {  // Q, which is not much here, is asked for while the pieces are planned: it came 2 us later otherwise
    const int64_t bytes = int64_t(c.total_q) * qh * D * 2;
    for (int64_t at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 128; at < bytes; at += int64_t(gridDim.x) * kThreads * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(a.q) + at));
  }
  if (MODE != kChunk && threadIdx.x == 256) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmV)) : "memory");
    if constexpr (BOTH) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&extra.k)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&extra.v)) : "memory");
    }
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&S.tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // ---- where this CTA's run starts ----
  int64_t* units = reinterpret_cast<int64_t*>(&S.kv[0][0][0]);  // of each sequence and KV head; the ring is not yet in use
  int* counts = reinterpret_cast<int*>(&S.kv[1][0][0]);                  // tiles of each sequence and KV head
  Seq* seqs = reinterpret_cast<Seq*>(&S.kv[2][0][0]);
  int* steps = reinterpret_cast<int*>(seqs);  // of each prefix (kCuts, kPairs)
  static_assert(kGroup * sizeof(Seq) <= kKeys * 128, "one tile of the ring");
  int longest = 0;  // steps of a tile
  const bool by_warp = CUT && b_end - b_begin <= 32;  // then the warp that walks the pieces plans alone
  for (int b = by_warp ? b_end : b_begin + warp; b < b_end; b += kThreads / 32) {
    const Seq s = rows_at(b);
    const int tiles = tiles_of(s, c.group);
    if (CUT) {
      if (lane == 0) {
        steps[b - b_begin] = prefix_steps(s);
        counts[b - b_begin] = tiles;
      }
      continue;
    }
    int64_t u = 0;
    for (int t = lane; t < tiles; t += 32) {
      const int mine = steps_of(s, c.group, t);
      u += mine;
      longest = max(longest, mine);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    if (lane == 0) {  // of one KV head
      seqs[b - b_begin] = s;
      units[b - b_begin] = u;
      counts[b - b_begin] = tiles;
    }
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) S.longest[warp] = longest;
  Seq early = {0, 0, 0, 0};  // the first groups, a lane each, for the warp that walks the pieces
  int tile_ctas = gridDim.x;  // the others go over the own slots
  int64_t own_total = 0;
  int own_least = 0;
  int2* own_kept = reinterpret_cast<int2*>(&S.kv[kStages == 5 ? 3 : 4][0][0]);
  if constexpr (CUT) {
    static_assert(few::kKept * sizeof(int2) <= 2 * sizeof(S.kv[0]) || kStages == 8);
    int64_t sum;
    int least;
    if (warp == 10 && by_warp) early = b_begin + lane < b_end ? group_of(c, b_begin + lane) : early;
    few::survey<few::Cutting<NT * 8>>(extra.few, own_kept, threadIdx.x, kThreads, &sum, &least);
    if (lane == 0) {
      S.own_total[warp] = sum;
      S.own_least[warp] = least;
    }
    if (warp == 10 && by_warp) {
      const int tiles = tiles_of(early, c.group), steps1 = prefix_steps(early);
      const int64_t mine = warp_sum(int64_t(tiles) * steps1), all = warp_sum(steps1 ? tiles : 0);
      if (lane == 0) {
        S.tile_steps = mine;
        S.tiles = all;
      }
    }
  }
  if (CUT || !by_warp) __syncthreads();
  if constexpr (CUT) {
    const int groups = b_end - b_begin;
    int64_t tile_steps = by_warp ? S.tile_steps : 0, tiles = by_warp ? S.tiles : 0;
    if (!by_warp) {
      if (warp == 10 && b_begin + lane < b_end) early = group_of(c, b_begin + lane);
      for (int g = lane; g < groups; g += 32) {
        tile_steps += int64_t(counts[g]) * steps[g];
        tiles += steps[g] ? counts[g] : 0;
      }
      tile_steps = warp_sum(tile_steps);
      tiles = warp_sum(tiles);
    }
    for (int i = 0; i < kThreads / 32; ++i) {
      own_total += S.own_total[i] * c.kvh;
      own_least = max(own_least, S.own_least[i]);
    }
    tile_ctas -= own_ctas<D, PAIR>(tile_steps * c.kvh, max(int64_t(1), tiles * c.kvh), own_total, gridDim.x);
    int length = 0;
    if (by_warp && warp == 10) {
      const int steps1 = prefix_steps(early), tiles1 = tiles_of(early, c.group);
      length = longest_piece(
          [&](int, int* st, int* ti) {
            *st = steps1;
            *ti = tiles1;
          },
          [&](int g, int* st, int* ti) {
            *st = __shfl_sync(0xffffffffu, steps1, g);
            *ti = __shfl_sync(0xffffffffu, tiles1, g);
          },
          groups, c.kvh, max(1, tile_ctas), a.splits);
      if (blockIdx.x == 0)
        for (int g = 0; g < groups; ++g) {
          const int n = pieces_of(__shfl_sync(0xffffffffu, steps1, g), length);
          for (int h = lane; h < c.kvh; h += 32) a.pieces[int64_t(b_begin + g) * c.kvh + h] = n;
        }
    }
    if (!by_warp && warp == 0) {
      auto at = [&](int g, int* st, int* ti) {
        *st = steps[g];
        *ti = counts[g];
      };
      length = longest_piece(at, at, groups, c.kvh, max(1, tile_ctas), a.splits);
      if (blockIdx.x == 0)
        for (int i = lane; i < groups * c.kvh; i += 32) a.pieces[int64_t(b_begin) * c.kvh + i] = pieces_of(steps[i / c.kvh], length);
      fence_async();
    }
    if (length > 0 && lane == 0) S.lead = length;
  } else if (warp == 0) {
    int64_t all = 0, all_tiles = 0;
    for (int b = lane; b < b_end - b_begin; b += 32) {
      all += units[b] * c.kvh;
      all_tiles += int64_t(counts[b]) * c.kvh;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      all_tiles += __shfl_xor_sync(0xffffffffu, all_tiles, o);
    }
    longest = __reduce_max_sync(0xffffffffu, lane < kThreads / 32 ? S.longest[lane] : 0);
    const int lead = BOTH ? kLeadBoth : D == 128 && all_tiles >= gridDim.x ? kLeadWhole : kLead;
    all += lead * all_tiles;
    longest += lead;
    auto units_of = [&](int b) { return units[b - b_begin] + int64_t(lead) * counts[b - b_begin]; };
    const int64_t run = max(int64_t(kMinRun), quotient(all + gridDim.x - 1, gridDim.x));
    // Equal runs cut tiles; where a CTA for each tile takes little longer, none is cut (1024
    // tokens, 32/8 heads, 128 tiles: over 2048 slots 47 against 51 us; over 8192, where the rule
    // cuts, 107 against 104).
    const bool by_tile = all_tiles <= gridDim.x && longest <= run + kCut;
    int64_t at = by_tile ? blockIdx.x : blockIdx.x * run;  // into the tiles, or their units
    int64_t left = max(int64_t(0), by_tile ? min(int64_t(1), all_tiles - at) : min(run, all - at));
    if (left > 0) {
      // the sequence, by prefix sums of 32 at a time
      int b = b_begin;
      bool found = false;
      for (; b < b_end; b += 32) {
        const int64_t mine =
            b + lane < b_end ? (by_tile ? counts[b + lane - b_begin] : units_of(b + lane)) * c.kvh : 0;
        int64_t pre = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, pre, o);
          if (lane >= o) pre += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, pre > at);
        if (past) {
          const int i = __ffs(past) - 1;
          at -= __shfl_sync(0xffffffffu, pre - mine, i);
          b += i;
          found = true;
          break;
        }
        at -= __shfl_sync(0xffffffffu, pre, 31);
      }
      const int64_t per = !found ? 1 : by_tile ? counts[b - b_begin] : units_of(b);
      const int h = int(quotient(at, per));
      at -= h * per;
      const Seq s = found ? seqs[b - b_begin] : Seq{0, 0, 0, 0};
      const int tiles = tiles_of(s, c.group);
      int t = 0;
      if (by_tile) {
        t = int(at);
        at = 0;
        found = t < tiles;
        if (found) left = lead + steps_of(s, c.group, t);
      }
      for (; !by_tile && t < tiles; t += 32) {
        const int64_t mine = t + lane < tiles ? lead + steps_of(s, c.group, t + lane) : 0;
        int64_t pre = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, pre, o);
          if (lane >= o) pre += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, pre > at);
        if (past) {
          const int i = __ffs(past) - 1;
          at -= __shfl_sync(0xffffffffu, pre - mine, i);
          t += i;
          found = true;
          break;
        }
        at -= __shfl_sync(0xffffffffu, pre, 31);
      }
      if (!found) left = 0;
      if (lane == 0) {
        S.start[0] = b;
        S.start[1] = h;
        S.start[2] = t;
        S.start[3] = int(at);
        S.first = s;
      }
    }
    if (lane == 0) {
      S.left = left;
      S.run = run;
      S.lead = lead;
    }
    fence_async();
  }

  if (CUT) fence_async();  // what lies in the ring has been read
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = S.tmem_base;
  const bool own_side = CUT && int(blockIdx.x) >= tile_ctas;

  // registers: 8 x 208 + 4 x 80 a lane, within the 12 x 168 of the launch
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (own_side) {
      // nothing to do
    } else if (warp == 10 && CUT) {
      // ---------------- the CTA's pieces: numbers cta, cta + ctas, ... of (group, KV head, piece, tile) ----------------
      const int length = S.lead;
      int64_t item = blockIdx.x, base = 0;  // base: pieces of the groups before these 32
      int g0 = b_begin;
      Seq s = early;
      int tiles = 0, pieces = 0;
      int64_t mine = 0, pre = 0;
      auto look = [&]() {  // a group per lane
        if (g0 != b_begin) s = g0 + lane < b_end ? rows_of<CUT>(c, g0 + lane) : Seq{0, 0, 0, 0};
        tiles = tiles_of(s, c.group);
        pieces = pieces_of(prefix_steps(s), length);
        pre = mine = int64_t(tiles) * pieces * c.kvh;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, pre, o);
          if (lane >= o) pre += v;
        }
      };
      look();
      bool ok = true;
      for (uint32_t i = 0; ok; ++i, item += tile_ctas) {
        uint32_t past = 0;
        while (g0 < b_end) {
          past = __ballot_sync(0xffffffffu, base + pre > item);
          if (past) break;
          base += __shfl_sync(0xffffffffu, pre, 31);
          g0 += 32;
          look();
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&S.piece_empty[i & 1], ((i >> 1) & 1) ^ 1, abort));
        if (!ok) break;
        Piece& p = S.piece[i & 1];
        if (!past) {
          if (lane == 0) {
            p.u0 = p.u1 = 0;
            mbar_arrive(&S.piece_full[i & 1]);
          }
          break;
        }
        if (lane == __ffs(past) - 1) {
          int64_t at = item - base - (pre - mine);
          const int64_t per = int64_t(tiles) * pieces;
          p.b = g0 + lane;
          p.h = int(quotient(at, per));
          at -= p.h * per;
          p.slot = int(quotient(at, tiles));
          p.r0 = int(at - int64_t(p.slot) * tiles) * kRows;
          p.row0 = s.row0;
          p.n = s.n;
          p.lead = s.first;
          p.rows = s.m * c.group;
          p.whole = 0;
          const int64_t steps = prefix_steps(s);
          p.u0 = int(quotient(p.slot * steps, pieces));
          p.u1 = int(quotient((p.slot + 1) * steps, pieces));
          mbar_arrive(&S.piece_full[i & 1]);
        }
        __syncwarp();
      }
    } else if (warp == 10) {
      // ---------------- the run's pieces, two of them ahead ----------------
      if (lane == 0) {
        Cut cut;
        cut.pieces = 0;
        int64_t left = S.left;
        const int lead = S.lead;
        const int64_t run = S.run, end = blockIdx.x * run + left;
        int b = S.start[0], h = S.start[1], t = S.start[2], at = S.start[3];  // at: units into the tile
        Seq s = {0, 0, 0, 0};
        int tiles = 0;
        if (left > 0) {
          s = S.first;
          tiles = tiles_of(s, c.group);
        }
        for (uint32_t i = 0;;) {
          const int k = i & 1;
          if (!mbar_wait(&S.piece_empty[k], ((i >> 1) & 1) ^ 1, abort)) break;
          Piece& p = S.piece[k];
          if (left <= 0) {
            p.u0 = p.u1 = 0;
            mbar_arrive(&S.piece_full[k]);
            break;
          }
          const int steps = steps_of(s, c.group, t);
          const int to = int(min(int64_t(lead + steps), at + left));
          const int u0 = max(0, at - lead), u1 = max(0, to - lead);
          if (u1 > u0) {  // a run that ends within the lead leaves the tile to the next
            p.b = b;
            p.h = h;
            p.row0 = s.row0;
            p.n = s.n;
            p.lead = s.first;
            p.r0 = t * kRows;
            p.rows = s.m * c.group;
            p.u0 = u0;
            p.u1 = u1;
            const bool whole = u0 == 0 && u1 == steps;
            int slot = 2 * int(blockIdx.x) + (i == 0 ? 0 : 1);
            if constexpr (BOTH) slot = extra.pre.first_slot + 2 * int(blockIdx.x) + (u0 == 0 ? 1 : 0);
            p.whole = whole;
            p.slot = slot;
            mbar_arrive(&S.piece_full[k]);
            if (u0 == 0 && (BOTH || !whole)) {
              // this CTA begins the tile; the CTAs of the units up to the tile's last go on with it
              const int pieces = whole ? 1 : int(quotient(end - left - at + lead + steps - 1, run)) - int(blockIdx.x) + 1;
              if constexpr (BOTH) {
                const Prefixes& pre = extra.pre;
                const bool own = b >= pre.groups;
                (own ? pre.own_pieces : pre.pre_pieces)[int64_t(h) * (own ? pre.own_keys : pre.pre_keys) +
                                                       piece_key(s.row0, c.group, kRows, t, own ? b - pre.groups : b)] = make_int2(pieces, slot);
              } else {
                cut.row = int64_t(s.row0) * qh + h * c.group;
                cut.slot = slot;
                cut.r0 = t * kRows;
                cut.rows = min(kRows, s.m * c.group - t * kRows);
                cut.pieces = pieces;
              }
            }
            ++i;
          }
          left -= to - at;
          at = 0;
          if (++t < tiles) continue;
          t = 0;
          if (++h < c.kvh) continue;
          h = 0;
          do {
            if (++b >= b_end) {
              left = 0;
              break;
            }
            s = rows_at(b);
            tiles = tiles_of(s, c.group);
          } while (tiles == 0);
        }
        if (!BOTH) static_cast<Cut*>(a.cuts)[blockIdx.x] = cut;
      }
      __syncwarp();
    } else if (warp == 8) {
      // ---------------- K and V tiles ----------------
      int st = 0;
      uint32_t ph = 0, tails = 0;  // ring phase, tail tiles so far
      bool ok = true;
      for (uint32_t i = 0; ok; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(&S.piece_full[i & 1], (i >> 1) & 1, abort));
        if (!ok) break;
        const Piece pc = S.piece[i & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.piece_empty[i & 1]);
        if (pc.u0 == pc.u1) break;
        // Where the boxes of a tile lie (eight at most), for four steps at a time and one such round
        // ahead: a page looked up when its box is due cost every tile that wait (a ragged batch over
        // pages of 16: 2 us a step).
        const CacheCall* cache = &c;
        const CUtensorMap *map_k = &tmK, *map_v = &tmV;
        int cb = pc.b, rows_of_box = box;
        if constexpr (BOTH) {
          if (pc.b < extra.pre.groups) {
            cache = &extra.pre.c;
            map_k = &extra.k;
            map_v = &extra.v;
            rows_of_box = extra.pre.box;
          } else {
            cb -= extra.pre.groups;
          }
        }
        auto look = [&](int u) {
          const int n = u * kKeys + (lane >> 3) * kKeys + (lane & 7) * rows_of_box;
          const bool any = u + (lane >> 3) < pc.u1 && (lane & 7) * rows_of_box < kKeys && n < pc.n;
          return any ? slot_row(*cache, cb, pc.h, n) : 0;
        };
        int rows = 0, ahead = look(pc.u0);
        for (int u = pc.u0; u < pc.u1 && ok; ++u) {
          if (((u - pc.u0) & 3) == 0) {
            rows = ahead;
            ahead = look(u + 4);
          }
          const int row = __shfl_sync(0xffffffffu, rows, ((u - pc.u0) & 3) * 8 + (lane & 7));
          const int n0 = u * kKeys;
          const int live = max(0, min(kKeys, pc.n - n0));  // rows that hold slots of the sequence
          const int boxes = (live + rows_of_box - 1) / rows_of_box;
          for (int kv = 0; kv < 2; ++kv) {
            // Q behind five tiles in the memory's queue came 7 us late, so its loads go before all but the first
            if (MODE != kChunk && i == 0 && u == pc.u0 && kv == 1) {
              ok = __all_sync(0xffffffffu, mbar_wait(&S.q_asked, 0, abort));
              if (!ok) break;
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&S.empty[st], ph ^ 1, abort));
            if (!ok) break;
            // rows of V behind the last slot are zeroed before the products see the tile: they may
            // hold anything, and 0 * NaN is NaN (in S such columns are masked)
            const bool patch = kv == 1 && live < kKeys;
            uint64_t* bar = patch ? &S.tail : &S.full[st];
            if (lane == 0) {
              mbar_expect_tx(bar, uint32_t(boxes) * rows_of_box * kRowBytes * kSub);
              S.filled[st] = uint8_t(ph);
            }
            __syncwarp();
            if (lane < boxes) {
#pragma unroll
              for (int s = 0; s < kSub; ++s)
                tma_load_2d(&S.kv[st][s][lane * rows_of_box * 64], kv ? map_v : map_k, s * 64, row, bar);
            }
            if (patch) {
              ok = __all_sync(0xffffffffu, mbar_wait(&S.tail, tails & 1, abort));
              if (!ok) {
                if (lane == 0) {  // this copy is nobody else's to wait for
                  mbar_drain(&S.tail, tails & 1);
                  S.filled[st] = uint8_t(ph ^ 1);
                }
                break;
              }
              ++tails;
              const uint4 z = make_uint4(0, 0, 0, 0);
              for (int s = 0; s < kSub; ++s) {
                uint4* p = reinterpret_cast<uint4*>(&S.kv[st][s][0]);
                for (int j = live * 8 + lane; j < kKeys * 8; j += 32) p[j] = z;
              }
              fence_async();
              __syncwarp();
              if (lane == 0) mbar_arrive(&S.full[st]);
            }
            if (++st == kStages) {
              st = 0;
              ph ^= 1;
            }
          }
        }
      }
    } else {
      // ---------------- products: warp 9 for the first half, 11 for the second ----------------
      // Each runs as one warp and an elected lane issues. A warp's own products follow each
      // other (P overlays S), the other's fill the tensor cores while it waits for its P.
      const int half = warp == 9 ? 0 : 1;
      const uint32_t id_s = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kKeys >> 3) << 17) | (uint32_t(128 >> 4) << 24);
      const uint32_t id_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (uint32_t(D >> 3) << 17) |
                            (uint32_t(128 >> 4) << 24);
      const uint64_t dq = sw128_desc(saddr(&S.q[half][0][0])), dk = sw128_desc(saddr(&S.kv[0][0][0])),
                     dv = sw128_desc_mn(saddr(&S.kv[0][0][0]));
      constexpr uint32_t kTile = kKeys * D * 2 / 16, kSlab = kKeys * 128 / 16;  // in descriptor units of 16 bytes
      constexpr bool kOwnP = Smem<D>::kOwnP;
      const uint32_t t_s = tmem + uint32_t(half * 128), t_o = tmem + uint32_t(256 + half * D);
      const uint32_t t_p = kOwnP ? tmem + uint32_t(384 + half * 64) : t_s;
      // The ring holds K and V tiles in turn. They are used in that order where P overlays S:
      // one cursor (two cost 6 percent there). With P beside S a K tile is used before the V
      // tile that precedes it: a cursor each.
      int st = 0, v_st = 1;
      uint32_t ph = 0, v_ph = 0, ph_q = 0, ph_p = 0, ph_f = 0;
      auto advance = [&]() {  // st, ph: the next tile, or the next K tile
        if ((st += kOwnP ? 2 : 1) >= kStages) {
          st -= kStages;
          ph ^= 1;
        }
      };
      auto advance_v = [&]() {
        if (!kOwnP) return advance();
        if ((v_st += 2) >= kStages) {
          v_st -= kStages;
          v_ph ^= 1;
        }
      };
      auto product_s = [&]() {
        fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kSlab + (kk & 3) * 2;
            mma_bf16(t_s, dq + off, dk + st * kTile + off, id_s, kk > 0 ? 1u : 0u);
          }
          mma_commit(&S.s_full[half]);
          mma_commit(&S.empty[st]);
        }
        __syncwarp();
        advance();
      };
      bool ok = true;
      for (uint32_t i = 0; ok; ++i) {
        ok = mbar_wait_warp(&S.piece_full[i & 1], (i >> 1) & 1, abort);
        if (!ok) break;
        const Piece& pc = S.piece[i & 1];
        const int steps = __reduce_max_sync(0xffffffffu, pc.u1 - pc.u0);
        const bool active = __reduce_max_sync(0xffffffffu, pc.rows - pc.r0) > half * 128;
        if (elect_one()) mbar_arrive(&S.piece_empty[i & 1]);
        __syncwarp();
        if (steps == 0) break;
        if (PAIR) {
          // Steps half, half + 2, ... of the piece. The ring's tiles in between are the other half's, but are
          // waited for and given back here too: a half that passed one unseen could take a barrier's phase for
          // the one before it (copies do not land in order), and one that did not give it back could miss a phase.
          int k_at = 0, v_at = 0;  // steps whose tiles the cursors have come to (one cursor: v_at)
          auto pass = [&](int stage, uint32_t phase) {
            ok = ok && mbar_wait_warp(&S.full[stage], phase, abort);
            if (ok && elect_one()) mbar_arrive(&S.empty[stage]);
            __syncwarp();
          };
          auto to_k = [&](int u) {
            for (int& at = kOwnP ? k_at : v_at; ok && at < u; ++at) {
              pass(st, ph);
              advance();
              if (!kOwnP) {
                pass(st, ph);
                advance();
              }
            }
          };
          auto to_v = [&](int u) {
            if (kOwnP)
              for (; ok && v_at < u; ++v_at) {
                pass(v_st, v_ph);
                advance_v();
              }
          };
          auto form_s = [&](int u) {
            to_k(u);
            ok = ok && mbar_wait_warp(&S.full[st], ph, abort);
            if (ok) product_s();
            ++k_at;
          };
          if (half < steps) {
            ok = mbar_wait_warp(&S.q_full[half], ph_q, abort);
            ph_q ^= 1;
            if (ok) form_s(half);
          }
          for (int u = half; ok && u < steps; u += 2) {
            if (kOwnP) {
              ok = mbar_wait_warp(&S.s_free[half], ph_f, abort);
              if (!ok) break;
              ph_f ^= 1;
              if (u + 2 < steps) form_s(u + 2);
              to_v(u);
              if (!ok) break;
            }
            const int at = kOwnP ? v_st : st;
            ok = mbar_wait_warp(&S.full[at], kOwnP ? v_ph : ph, abort);
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              ok = ok && mbar_wait_warp(&S.p_full[half][part], ph_p, abort);
              if (!ok) break;
              fence_after();
              if (elect_one()) {
#pragma unroll
                for (int kk = part * 4; kk < part * 4 + 4; ++kk)
                  mma_bf16_ta(t_o, t_p + uint32_t(kk * 8), dv + at * kTile + kk * 128, id_o, (u > half || kk > 0) ? 1u : 0u);
                if (part == 1) {
                  mma_commit(&S.o_full[half]);
                  mma_commit(&S.empty[at]);
                }
              }
              __syncwarp();
            }
            if (!ok) break;
            ph_p ^= 1;
            advance_v();
            ++v_at;
            if (!kOwnP && u + 2 < steps) form_s(u + 2);
          }
          to_k(steps);
          to_v(steps);
          continue;
        }
        if (!active) {  // the ring's tiles pass this half by
          for (int j = 0; j < steps && ok; ++j) {
            ok = mbar_wait_warp(&S.full[st], ph, abort);
            if (ok && elect_one()) mbar_arrive(&S.empty[st]);
            __syncwarp();
            advance();
            ok = ok && mbar_wait_warp(&S.full[kOwnP ? v_st : st], kOwnP ? v_ph : ph, abort);
            if (ok && elect_one()) mbar_arrive(&S.empty[kOwnP ? v_st : st]);
            __syncwarp();
            advance_v();
          }
          continue;
        }
        ok = mbar_wait_warp(&S.full[st], ph, abort) && mbar_wait_warp(&S.q_full[half], ph_q, abort);
        ph_q ^= 1;
        if (!ok) break;
        product_s();
        for (int j = 0; j < steps; ++j) {
          if (kOwnP) {
            // S is free once the softmax has it in registers
            ok = mbar_wait_warp(&S.s_free[half], ph_f, abort);
            if (!ok) break;
            ph_f ^= 1;
            if (j + 1 < steps) {
              ok = mbar_wait_warp(&S.full[st], ph, abort);
              if (!ok) break;
              product_s();
            }
          }
          ok = mbar_wait_warp(&S.full[kOwnP ? v_st : st], kOwnP ? v_ph : ph, abort);
          // P arrives in two parts of 64 keys: the product starts on the first
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            ok = ok && mbar_wait_warp(&S.p_full[half][part], ph_p, abort);
            if (!ok) break;
            fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = part * 4; kk < part * 4 + 4; ++kk)
                mma_bf16_ta(t_o, t_p + uint32_t(kk * 8), dv + (kOwnP ? v_st : st) * kTile + kk * 128, id_o, (j > 0 || kk > 0) ? 1u : 0u);
              if (part == 1) {
                mma_commit(&S.o_full[half]);
                mma_commit(&S.empty[kOwnP ? v_st : st]);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          ph_p ^= 1;
          advance_v();
          if (!kOwnP && j + 1 < steps) {
            ok = mbar_wait_warp(&S.full[st], ph, abort);
            if (!ok) break;
            product_s();
          }
        }
      }
      if (!ok) {
        if (elect_one()) mma_commit(&S.drain[half]);
        __syncwarp();
        if (lane == 0) mbar_drain(&S.drain[half], 0);
        __syncwarp();
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    if constexpr (CUT) {
      if (own_side) {  // eight rings from Q's place on, the rest behind them
        constexpr int kOwnStages = D == 128 ? 3 : 4;
        auto* rings = reinterpret_cast<few::Ring<D, kOwnStages>*>(&S.q[0][0][0]);
        auto* states = reinterpret_cast<few::State<kOwnStages>*>(rings + 8);
        static_assert(8 * (sizeof(*rings) + sizeof(*states)) <= sizeof(S.q) + sizeof(S.kv) && offsetof(Smem<D>, kv) == sizeof(S.q));
        few::work<D, NT, kOwnStages>(extra.maps, extra.few, rings[warp], states[warp], own_kept, own_total, own_least,
                         int64_t(blockIdx.x - tile_ctas) * 8 + warp, int64_t(gridDim.x - tile_ctas) * 8, [] {
                           fence_async();
                           asm volatile("bar.sync 1, 256;" ::: "memory");
                         });
      }
    }
    // ---------------- softmax: one thread per row ----------------
    const int half = warp >> 2, quarter = warp & 3;
    const uint32_t ts = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(half * 128);
    const uint32_t to = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(256 + half * D);
    constexpr bool kOwnP = Smem<D>::kOwnP;
    const uint32_t tp = kOwnP ? tmem + (uint32_t(quarter * 32) << 16) + uint32_t(384 + half * 64) : ts;
    const float scale = kLog2e * rsqrtf(float(D));
    uint32_t ph_s = 0, ph_o = 0;  // phases of s_full, and of o_full's next completion
    uint32_t ph_t = half == 0;    // of turn; the first turn is half 0's
    bool first_piece = true;
    bool ok = true;
    for (uint32_t i = 0; ok && !own_side; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait(&S.piece_full[i & 1], (i >> 1) & 1, abort));
      if (!ok) break;
      const Piece& pc = S.piece[i & 1];
      const int r0 = pc.r0 + (PAIR ? 0 : half * 128), rows = pc.rows;
      if (pc.u0 == pc.u1) break;
      if (PAIR && i > 0) {  // the other half has read this half's sums of the piece before
        ok = __all_sync(0xffffffffu, mbar_wait(&S.pair_done, (i & 1) ^ 1, abort));
        if (!ok) break;
      }
      if (r0 < rows) {
        const int64_t head = int64_t(pc.row0) * qh + pc.h * c.group;  // row of token 0's first head
        const int r = r0 + quarter * 32 + lane;
        const int64_t row = head + int64_t(r / c.group) * qh + r % c.group;
        const int steps = PAIR ? (pc.u1 - pc.u0 - half + 1) / 2 : pc.u1 - pc.u0;
        // the warp's rows of Q into their swizzled places (16-byte chunk i of row k at i ^ (k % 8)),
        // 512 contiguous bytes a load (none for a half without a step: its sums take that place at once)
        if (!PAIR || steps > 0) {
          constexpr int kChunks = D / 8, kAtOnce = 32 / kChunks;
          const int i = lane % kChunks, own = lane / kChunks;
          uint4 v[kChunks];
#pragma unroll
          for (int j = 0; j < kChunks; ++j) {
            const int k = j * kAtOnce + own;
            const int64_t from = __shfl_sync(0xffffffffu, row, k);
            v[j] = make_uint4(0, 0, 0, 0);
            if (r - lane + k < rows)
              v[j] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + from * D)[i];
          }
          if (MODE != kChunk && half == 0 && first_piece) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.q_asked);
            first_piece = false;
          }
#pragma unroll
          for (int j = 0; j < kChunks; ++j) {
            const int k = quarter * 32 + j * kAtOnce + own;
            *reinterpret_cast<uint4*>(&S.q[half][i >> 3][k * 64 + (((i & 7) ^ (k & 7)) << 3)]) = v[j];
          }
          fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.q_full[half]);
        }
        // slots below this, counted from the piece's first, are seen
        constexpr int kStride = PAIR ? 2 * kKeys : kKeys;  // from one of this half's steps to the next
        int see = r < rows ? min(pc.n, pc.lead + r / c.group + 1) - (pc.u0 + (PAIR ? half : 0)) * kKeys : 0;
        // the lowest limit of this warp's rows decides whether a step needs the mask at all
        int see_low = __reduce_min_sync(0xffffffffu, r < rows ? see : INT32_MAX);
        float m = -INFINITY;  // the row's reference, in log2
        uint64_t l0 = 0, l1 = 0;
        const bool turns = !PAIR && !kOwnP && rows - pc.r0 > 128;  // both halves have rows
        for (int j = 0; j < steps; ++j) {
          ok = __all_sync(0xffffffffu, mbar_wait(&S.s_full[half], ph_s, abort));
          ph_s ^= 1;
          if (!ok) break;
          if (turns) {
            ok = __all_sync(0xffffffffu, mbar_wait(&S.turn[half], ph_t, abort));
            ph_t ^= 1;
            if (!ok) break;
          }
          fence_after();
          uint32_t x0[32], x1[32], x2[32], x3[32];
          tmem_ld32(ts, x0);
          tmem_ld32(ts + 32, x1);
          tmem_ld32(ts + 64, x2);
          tmem_ld32(ts + 96, x3);
          tmem_wait_ld(x0);
          tmem_tie(x1);
          tmem_tie(x2);
          tmem_tie(x3);
          if (kOwnP) {
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.s_free[half]);
          }
          if (see_low < kKeys) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (i >= see) x0[i] = 0xff800000u;
              if (i + 32 >= see) x1[i] = 0xff800000u;
              if (i + 64 >= see) x2[i] = 0xff800000u;
              if (i + 96 >= see) x3[i] = 0xff800000u;
            }
          }
          see -= kStride;
          see_low -= kStride;
          float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            t0 = max3(t0, x0[i], x0[i + 1]);
            t1 = max3(t1, x1[i], x1[i + 1]);
            t2 = max3(t2, x2[i], x2[i + 1]);
            t3 = max3(t3, x3[i], x3[i + 1]);
          }
          const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * scale;
          const bool raise = top > m + kRaise || (m == -INFINITY && top > m);
          if (__any_sync(0xffffffffu, raise)) {
            const float by = raise ? exp2f(m - top) : 1.0f;  // 0 for the first reference
            if (raise) m = top;
            const uint64_t by2 = pk2(by, by);
            l0 = mul2(l0, by2);
            l1 = mul2(l1, by2);
            if (j > 0) {
              ok = __all_sync(0xffffffffu, mbar_wait(&S.o_full[half], ph_o ^ 1, abort));
              if (!ok) break;
              fence_after();
#pragma unroll
              for (int g = 0; g < D / 32; ++g) {
                uint32_t o[32];
                tmem_ld32(to + g * 32, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
                tmem_st32(to + g * 32, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;
          const uint64_t sc2 = pk2(scale, scale), ref2 = pk2(-ref, -ref);
          uint32_t p[32];
          auto weigh = [&](const uint32_t (&x)[32], int at) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const uint64_t y0 = fma2(pk2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), sc2, ref2);
              const uint64_t y1 = fma2(pk2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), sc2, ref2);
              const float e0 = ex2(lo2(y0)), e1 = ex2(hi2(y0)), e2 = ex2(lo2(y1)), e3 = ex2(hi2(y1));
              l0 = add2(l0, pk2(e0, e1));
              l1 = add2(l1, pk2(e2, e3));
              p[at + i / 2] = bf2(e0, e1);
              p[at + i / 2 + 1] = bf2(e2, e3);
            }
          };
          auto hand = [&](int part) {
            tmem_st32(tp + part * 32, p);
            tmem_wait_st();
            fence_before();
            __syncwarp();
#if MP_CHECK
            if (a.stall && blockIdx.x == 0 && half == 0 && j == 1) return;  // never handed over: the waits run out
#endif
            if (lane == 0) mbar_arrive(&S.p_full[half][part]);
          };
          weigh(x0, 0);
          weigh(x1, 16);
          if (kOwnP && j > 0) {  // the last step's product has read P
            ok = __all_sync(0xffffffffu, mbar_wait(&S.o_full[half], ph_o ^ 1, abort));
            if (!ok) break;
            fence_after();
          }
          hand(0);
          weigh(x2, 0);
          if (turns) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.turn[half ^ 1]);
          }
          weigh(x3, 16);
          hand(1);
          ph_o ^= 1;  // past this step's second product
        }
        if (!ok) break;
        if (!PAIR || steps > 0) ok = __all_sync(0xffffffffu, mbar_wait(&S.o_full[half], ph_o ^ 1, abort));
        if (!ok) break;
        fence_after();
        const float sum = lo2(l0) + hi2(l0) + lo2(l1) + hi2(l1);
        if constexpr (CUT || BOTH) {
          // the sums of this piece: a slice of its rows, or (kBoth, cut) its slot's
          int64_t place = int64_t(pc.slot) * c.total_q * qh + row;
          float *to_ml = a.ml, *to_part = a.part;
          if constexpr (BOTH) {
            place = int64_t(pc.slot) * slot_rows + (r - pc.r0);
            if (pc.whole) {
              place = (pc.b < extra.pre.groups ? 0 : extra.pre.own_slice) + row;
              to_ml = a.state_ml;
              to_part = a.state;
            }
          }
          const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16) + 256;
          float by0 = 1.f, by1 = 0.f, top = m, all_sum = sum;
          if (PAIR) {
            // both halves' sums over these rows: each half takes half of the columns of both
            const int own = quarter * 32 + lane;
            float2* const ml = reinterpret_cast<float2*>(&S.q[0][0][0]);  // in the place of Q, which has been read
            float2* const ml1 = reinterpret_cast<float2*>(&S.q[1][0][0]);
            (half ? ml1 : ml)[own] = make_float2(m, sum);
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.pair_full);
            ok = __all_sync(0xffffffffu, mbar_wait(&S.pair_full, i & 1, abort));
            if (!ok) break;
            fence_after();
            const float2 a0 = ml[own], a1 = ml1[own];
            top = fmaxf(a0.x, a1.x);
            by0 = a0.y == 0.f ? 0.f : exp2f(a0.x - top);
            by1 = a1.y == 0.f ? 0.f : exp2f(a1.x - top);
            all_sum = fmaf(a0.y, by0, a1.y * by1);
          }
          if (r < rows && (!PAIR || half == 0)) *reinterpret_cast<float2*>(to_ml + place * 2) = make_float2(top, all_sum);
          constexpr int kBlocks = PAIR ? D / 64 : D / 32;  // of 32 columns
          const int g0 = PAIR ? half * kBlocks : 0;
          uint32_t mine[kBlocks][32], others[PAIR ? kBlocks : 1][32];
#pragma unroll
          for (int g = 0; g < kBlocks; ++g) {
            tmem_ld32(lanes + (PAIR ? 0 : half * D) + (g0 + g) * 32, mine[g]);
            if (PAIR) tmem_ld32(lanes + D + (g0 + g) * 32, others[g]);
          }
          tmem_wait_ld(mine[0]);
#pragma unroll
          for (int g = 0; g < kBlocks; ++g) {
            if (g > 0) tmem_tie(mine[g]);
            if (PAIR) tmem_tie(others[g]);
          }
          if (PAIR) {
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.pair_done);
          }
#pragma unroll
          for (int g = 0; g < kBlocks; ++g) {
            float v[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              v[k] = __uint_as_float(mine[g][k]);
              if (PAIR) {  // a half without a step has written nothing
                v[k] = by0 == 0.f ? 0.f : v[k] * by0;
                v[k] = by1 == 0.f ? v[k] : fmaf(__uint_as_float(others[g][k]), by1, v[k]);
              }
            }
            // four lanes swap their rows' 32-byte parts, so that they write 128 bytes of a row together
#pragma unroll
            for (int bit = 1; bit <= 2; bit *= 2) {
              const bool high = lane & bit;
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                if (k & (8 * bit)) continue;
                const float got = __shfl_xor_sync(0xffffffffu, high ? v[k] : v[k + 8 * bit], bit);
                if (high) v[k] = got;
                else v[k + 8 * bit] = got;
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int64_t to_row = __shfl_sync(0xffffffffu, place, (lane & ~3) + k);
              if (r - (lane & 3) + k < rows) {
                float4* dst = reinterpret_cast<float4*>(to_part + to_row * D + (g0 + g) * 32 + (lane & 3) * 8);
                dst[0] = make_float4(v[8 * k], v[8 * k + 1], v[8 * k + 2], v[8 * k + 3]);
                dst[1] = make_float4(v[8 * k + 4], v[8 * k + 5], v[8 * k + 6], v[8 * k + 7]);
              }
            }
          }
        } else {
          const float inv = sum > 0.f ? 1.0f / sum : sum;
          const bool real = r < rows, whole = pc.whole;
          const int64_t at = int64_t(pc.slot) * slot_rows + (r - pc.r0);
          if (real) {
            if (!whole) *reinterpret_cast<float2*>(a.ml + at * 2) = make_float2(m, sum);
            else if (a.lse) a.lse[row] = sum == 0.f ? -INFINITY : m * kLn2 + logf(sum);
          }
          uint32_t all[D / 32][32];
#pragma unroll
          for (int g = 0; g < D / 32; ++g) tmem_ld32(to + g * 32, all[g]);
          tmem_wait_ld(all[0]);
#pragma unroll
          for (int g = 1; g < D / 32; ++g) tmem_tie(all[g]);
#pragma unroll
          for (int g = 0; g < D / 32; ++g) {
            uint32_t (&o)[32] = all[g];
            if (!whole) {
              if (real && sum > 0.f) {
                float4* dst = reinterpret_cast<float4*>(a.part) +
                              (int64_t(pc.slot) * (D / 4) + g * 8) * slot_rows + (r - pc.r0);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  dst[i * slot_rows] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                   __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
              }
            } else {
              // Four lanes swap their rows' 16-byte parts, so that each store writes 64 bytes of a row.
              uint32_t v[16];
#pragma unroll
              for (int k = 0; k < 16; ++k)
                v[k] = bf2(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
#pragma unroll
              for (int bit = 1; bit <= 2; bit *= 2) {
                const bool high = lane & bit;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  if (k & (4 * bit)) continue;
                  const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? v[k] : v[k + 4 * bit], bit);
                  if (high) v[k] = got;
                  else v[k + 4 * bit] = got;
                }
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int64_t to_row = __shfl_sync(0xffffffffu, row, (lane & ~3) + i);
                if (r - (lane & 3) + i < rows)
                  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + to_row * D + g * 32 + (lane & 3) * 8) =
                      make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.piece_empty[i & 1]);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  if (threadIdx.x == 0 && S.abort) {
    for (int i = 0; i < kStages; ++i) mbar_drain(&S.full[i], S.filled[i]);
    flag(c.status, MP_STATUS_WAIT_TIMEOUT);
  }
}

// Joins the pieces' (m, l, sum) of the tiles that were cut, in their order: a warp takes 32
// rows, a lane each, and 8 columns. Partial sums lie [slot][column / 4][row][4], so that
// the threads that own rows (in the kernel above and here) write and read whole lines. Set up
// while k_chunk_tc still runs; it waits for it first.
template <int D>
__global__ void __launch_bounds__(256) k_chunk_tc_join(const ChunkArgs a, const int slot_rows) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Cut cut = static_cast<const Cut*>(a.cuts)[blockIdx.x];
  const int task = blockIdx.y * 8 + (threadIdx.x >> 5), columns = task % (D / 8);
  const int i = task / (D / 8) * 32 + (threadIdx.x & 31);
  if (i >= cut.rows || cut.pieces == 0) return;
  auto slot = [&](int p) { return int64_t(p == 0 ? cut.slot : 2 * (int(blockIdx.x) + p)); };
  const float2* ml = reinterpret_cast<const float2*>(a.ml) + i;
  const float4* part = reinterpret_cast<const float4*>(a.part) + int64_t(columns) * 2 * slot_rows + i;
  float m = -INFINITY, l = 0.f;
  float4 o[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kAtOnce = 4;  // pieces whose loads are in flight together
  for (int p0 = 0; p0 < cut.pieces; p0 += kAtOnce) {
    float2 v[kAtOnce];
    float4 x[kAtOnce][2];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      v[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int j = 0; j < 2; ++j) x[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p0 + k >= cut.pieces) continue;
      const int64_t at = slot(p0 + k);
      v[k] = ml[at * slot_rows];
#pragma unroll
      for (int j = 0; j < 2; ++j) x[k][j] = part[(at * (D / 4) + j) * slot_rows];
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, v[k].x);
    const float ref = top == -INFINITY ? 0.f : top;
    const float before = exp2f(m - ref);  // 0 while nothing was seen
    m = top;
    l *= before;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      o[j].x *= before;
      o[j].y *= before;
      o[j].z *= before;
      o[j].w *= before;
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const bool live = v[k].y != 0.f;  // a piece that saw nothing has written no sum
      const float by = live ? exp2f(v[k].x - ref) : 0.f;
      l = fmaf(v[k].y, by, l);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        o[j].x = live ? fmaf(x[k][j].x, by, o[j].x) : o[j].x;
        o[j].y = live ? fmaf(x[k][j].y, by, o[j].y) : o[j].y;
        o[j].z = live ? fmaf(x[k][j].z, by, o[j].z) : o[j].z;
        o[j].w = live ? fmaf(x[k][j].w, by, o[j].w) : o[j].w;
      }
    }
  }
  const int group = a.c.group, r = cut.r0 + i;
  const int64_t row = cut.row + int64_t(r / group) * (a.c.kvh * group) + r % group;
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  if (a.lse && columns == 0) a.lse[row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
  uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * D + columns * 8);
  out[0] = make_uint4(bf2(o[0].x * inv, o[0].y * inv), bf2(o[0].z * inv, o[0].w * inv),
                        bf2(o[1].x * inv, o[1].y * inv), bf2(o[1].z * inv, o[1].w * inv));
}

int slot_rows_of(int group, int max_q) { return int(std::min<int64_t>(kRows, int64_t(max_q) * group)); }

template <int D, Mode MODE, int NT>
cudaError_t launch(ArgsOf<MODE> a, Extra<MODE> extra, int units, int ctas, int slot_rows, void* workspace, cudaStream_t st) {
  const CacheCall& c = a.c;
  CUtensorMap mk, mv;
  const int box = box_rows(c.table, c.page_size);
  const uint64_t rows = uint64_t(c.n_pages) * c.kvh * c.page_size;
  if (!make_map(&mk, a.keys, D, rows, 64, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&mv, a.values, D, rows, 64, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const size_t smem = sizeof(Smem<D>) + 1024;
  static_assert(sizeof(Smem<D>) + 1024 <= 227 * 1024);
  cudaError_t e = cudaFuncSetAttribute(k_chunk_tc<D, MODE, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  if (MODE == kChunk) {
    char* ws = static_cast<char*>(workspace);
    a.cuts = ws;
    ws += align256(uint64_t(ctas) * sizeof(Cut));
    a.ml = reinterpret_cast<float*>(ws);
    ws += align256(uint64_t(2 * ctas) * slot_rows * 8);
    a.part = reinterpret_cast<float*>(ws);
  }
  for (int b = 0; b < units; b += kGroup) {
    k_chunk_tc<D, MODE, NT><<<ctas, kThreads, smem, st>>>(mk, mv, a, box, b, std::min(units, b + kGroup), slot_rows, extra);
    if constexpr (MODE == kBoth) {
      extra.pre.first_slot += 2 * ctas;
    } else if constexpr (MODE != kChunk) {
      extra.few.own_units = false;  // the first launch has done them
    } else {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(ctas, ((slot_rows + 31) / 32 * (D / 8) + 7) / 8);
      cfg.blockDim = dim3(256);
      cfg.stream = st;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      if ((e = cudaLaunchKernelEx(&cfg, k_chunk_tc_join<D>, ChunkArgs(a), int(slot_rows))) != cudaSuccess) return e;
    }
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace mp
