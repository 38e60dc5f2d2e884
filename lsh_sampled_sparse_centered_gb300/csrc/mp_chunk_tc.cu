// Exact attention of a chunk of new tokens on the 5th-generation tensor cores (bf16).
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
#include <cudaTypedefs.h>

#include <algorithm>

#include "mp_cache.cuh"
#include "mp_tc.cuh"

namespace mp {
namespace {

constexpr int kRows = 256;   // query rows of a CTA
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
constexpr int kMinRun = 2;    // units of a CTA at least
constexpr int kCut = 10;      // units that cutting the tiles costs: a second piece for most CTAs, and the join

// One piece of work: the steps [u0, u1) of a tile, as every role of the CTA sees it.
struct Piece {
  int b, h, row0, n, lead;  // sequence, KV head, first packed row, slots, slot of that row
  int r0, rows;             // the tile's first row, and the rows of the whole chunk
  int u0, u1;               // u0 == u1: the run has ended
  int whole, slot;          // all of its tile's units; else where its partial result goes
};

static_assert(kKeys / 16 <= 8, "boxes of 16 rows at least");

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
// one that starts its run (slot 2 cta) and the one that ends it (slot 2 cta + 1).
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_chunk_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const ChunkArgs a,
               const int box, const int b_begin, const int b_end, const int slot_rows) {
  extern __shared__ __align__(1024) unsigned char smraw[];
  const uint32_t base = saddr(smraw);
  Smem<D>& S = *reinterpret_cast<Smem<D>*>(smraw + ((1024 - (base & 1023)) & 1023));
  constexpr int kSub = Smem<D>::kSub, kStages = Smem<D>::kStages;
  // 128-byte swizzle: copies and products take the tiles from 1024-byte boundaries (members in
  // front of them would move them off, and the copies then fault)
  static_assert(offsetof(Smem<D>, q) % 1024 == 0 && offsetof(Smem<D>, kv) % 1024 == 0 && sizeof(S.q[0][0]) % 1024 == 0 &&
                sizeof(S.kv[0][0]) % 1024 == 0);
  constexpr uint32_t kRowBytes = 128;
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile uint32_t* abort = &S.abort;
  const int qh = c.kvh * c.group;

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
    S.abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
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
  static_assert(kGroup * sizeof(Seq) <= kKeys * 128, "one tile of the ring");
  int longest = 0;  // steps of a tile
  for (int b = b_begin + warp; b < b_end; b += kThreads / 32) {
    const Seq s = seq_of(c, b);
    const int tiles = tiles_of(s, c.group);
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
  __syncthreads();
  if (warp == 0) {
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
    const int lead = D == 128 && all_tiles >= gridDim.x ? kLeadWhole : kLead;
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

  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = S.tmem_base;

  // registers: 8 x 208 + 4 x 80 a lane, within the 12 x 168 of the launch
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 10) {
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
            const int slot = 2 * int(blockIdx.x) + (i == 0 ? 0 : 1);
            p.whole = whole;
            p.slot = slot;
            mbar_arrive(&S.piece_full[k]);
            if (u0 == 0 && !whole) {
              // this CTA begins the tile; the CTAs of the units up to the tile's last go on with it
              cut.row = int64_t(s.row0) * qh + h * c.group;
              cut.slot = slot;
              cut.r0 = t * kRows;
              cut.rows = min(kRows, s.m * c.group - t * kRows);
              cut.pieces = int(quotient(end - left - at + lead + steps - 1, run)) - int(blockIdx.x) + 1;
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
            s = seq_of(c, b);
            tiles = tiles_of(s, c.group);
          } while (tiles == 0);
        }
        static_cast<Cut*>(a.cuts)[blockIdx.x] = cut;
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
        auto look = [&](int u) {
          const int n = u * kKeys + (lane >> 3) * kKeys + (lane & 7) * box;
          const bool any = u + (lane >> 3) < pc.u1 && (lane & 7) * box < kKeys && n < pc.n;
          return any ? slot_row(c, pc.b, pc.h, n) : 0;
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
          const int boxes = (live + box - 1) / box;
          for (int kv = 0; kv < 2; ++kv) {
            ok = __all_sync(0xffffffffu, mbar_wait(&S.empty[st], ph ^ 1, abort));
            if (!ok) break;
            // rows of V behind the last slot are zeroed before the products see the tile: they may
            // hold anything, and 0 * NaN is NaN (in S such columns are masked)
            const bool patch = kv == 1 && live < kKeys;
            uint64_t* bar = patch ? &S.tail : &S.full[st];
            if (lane == 0) {
              mbar_expect_tx(bar, uint32_t(boxes) * box * kRowBytes * kSub);
              S.filled[st] = uint8_t(ph);
            }
            __syncwarp();
            if (lane < boxes) {
#pragma unroll
              for (int s = 0; s < kSub; ++s)
                tma_load_2d(&S.kv[st][s][lane * box * 64], kv ? &tmV : &tmK, s * 64, row, bar);
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
    // ---------------- softmax: one thread per row ----------------
    const int half = warp >> 2, quarter = warp & 3;
    const uint32_t ts = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(half * 128);
    const uint32_t to = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(256 + half * D);
    constexpr bool kOwnP = Smem<D>::kOwnP;
    const uint32_t tp = kOwnP ? tmem + (uint32_t(quarter * 32) << 16) + uint32_t(384 + half * 64) : ts;
    const float scale = kLog2e * rsqrtf(float(D));
    uint32_t ph_s = 0, ph_o = 0;  // phases of s_full, and of o_full's next completion
    uint32_t ph_t = half == 0;    // of turn; the first turn is half 0's
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait(&S.piece_full[i & 1], (i >> 1) & 1, abort));
      if (!ok) break;
      const Piece& pc = S.piece[i & 1];
      const int r0 = pc.r0 + half * 128, rows = pc.rows;
      if (pc.u0 == pc.u1) break;
      if (r0 < rows) {
        const int64_t head = int64_t(pc.row0) * qh + pc.h * c.group;  // row of token 0's first head
        const int r = r0 + quarter * 32 + lane;
        const int64_t row = head + int64_t(r / c.group) * qh + r % c.group;
        // the warp's rows of Q into their swizzled places (16-byte chunk i of row k at i ^ (k % 8)),
        // 512 contiguous bytes a load
        {
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
        int see = r < rows ? min(pc.n, pc.lead + r / c.group + 1) - pc.u0 * kKeys : 0;
        // the lowest limit of this warp's rows decides whether a step needs the mask at all
        int see_low = __reduce_min_sync(0xffffffffu, r < rows ? see : INT32_MAX);
        float m = -INFINITY;  // the row's reference, in log2
        uint64_t l0 = 0, l1 = 0;
        const int steps = pc.u1 - pc.u0;
        const bool turns = !kOwnP && rows - pc.r0 > 128;  // both halves have rows
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
          see -= kKeys;
          see_low -= kKeys;
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
        ok = __all_sync(0xffffffffu, mbar_wait(&S.o_full[half], ph_o ^ 1, abort));
        if (!ok) break;
        fence_after();
        const float sum = lo2(l0) + hi2(l0) + lo2(l1) + hi2(l1);
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

template <int D>
cudaError_t launch(ChunkArgs a, void* workspace, cudaStream_t st) {
  const CacheArgs& c = a.c;
  CUtensorMap mk, mv;
  const int box = box_rows(c.table, c.page_size);
  const uint64_t rows = uint64_t(c.n_pages) * c.kvh * c.page_size;
  if (!make_map(&mk, a.keys, D, rows, 64, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&mv, a.values, D, rows, 64, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const size_t smem = sizeof(Smem<D>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(k_chunk_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  const int ctas = chunk_tc_ctas(c.batch, c.kvh, c.group, c.max_q, c.max_kv);
  const int slot_rows = slot_rows_of(c.group, c.max_q);
  char* ws = static_cast<char*>(workspace);
  a.cuts = ws;
  ws += align256(uint64_t(ctas) * sizeof(Cut));
  a.ml = reinterpret_cast<float*>(ws);
  ws += align256(uint64_t(2 * ctas) * slot_rows * 8);
  a.part = reinterpret_cast<float*>(ws);
  for (int b = 0; b < c.batch; b += kGroup) {
    k_chunk_tc<D><<<ctas, kThreads, smem, st>>>(mk, mv, a, box, b, std::min(c.batch, b + kGroup), slot_rows);
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
  return cudaGetLastError();
}

}  // namespace

// One CTA per SM, or fewer when the limits leave fewer runs of units than that.
int chunk_tc_ctas(int batch, int kvh, int group, int max_q, int max_kv) {
  const int64_t tiles = (int64_t(max_q) * group + kRows - 1) / kRows;
  const double units = double(std::min(batch, kGroup)) * kvh * double(tiles) * ((max_kv + kKeys - 1) / kKeys);
  return int(std::max(1.0, std::min(double(device_sm_count()), units / kMinRun + 1.0)));
}

uint64_t chunk_tc_workspace(const mp_cache_config* c, int max_q, int max_kv) {
  const int group = c->q_heads / c->kv_heads, ctas = chunk_tc_ctas(c->batch, c->kv_heads, group, max_q, max_kv);
  const uint64_t rows = uint64_t(2 * ctas) * slot_rows_of(group, max_q);
  return align256(uint64_t(ctas) * sizeof(Cut)) + align256(rows * 8) + align256(rows * c->head_dim * 4);
}

cudaError_t launch_chunk_tc(const ChunkArgs& a, void* workspace, cudaStream_t st) {
  return a.c.d == 128 ? launch<128>(a, workspace, st) : launch<64>(a, workspace, st);
}

}  // namespace mp
