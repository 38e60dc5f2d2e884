// Exact attention of a chunk of new tokens on the 5th-generation tensor cores (bf16).
//
// A CTA works on 256 query rows of one KV head (row = token * group + head of the group),
// as two halves of 128 rows, against 128 keys at a time:
//   S = Q K^T   (128 x 128 x d, both operands in shared memory, fp32 in tensor memory)
//   P = 2^(S log2(e) / sqrt(d) - m)   one thread per row, P as bf16 over S's columns
//   O += P V    (128 x d x 128, P from tensor memory, V from shared memory)
// While the softmax warps of one half work, the tensor cores work for the other half.
// Warps 0-3 and 4-7 are the softmax of the halves, warp 8 streams K and V by TMA into a
// ring of shared-memory tiles, warp 9 issues the products.
//
// The reference m of a row is raised only when a logit passes it by more than 8 (in log2),
// so that O is rescaled in few steps; P then is at most 2^8, which costs a float nothing.
// P enters the second product as bf16 (2^-8 relative per weight); the sum of the weights
// is taken before that rounding. Everything else is fp32.
//
// Tensor memory: S/P of the halves in columns 0 and 128, O in 256 and 256 + d.
#include <cudaTypedefs.h>

#include "mp_cache.cuh"
#include "mp_tc.cuh"

namespace mp {
namespace {

constexpr int kRows = 256;   // query rows of a CTA
constexpr int kKeys = 128;   // keys of a step
constexpr int kThreads = 384;  // 12 warps: two of softmax for each lane quarter, TMA, products, two idle
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.0f;

template <int D>
struct Smem {
  static constexpr int kSub = D / 64;
  static constexpr int kStages = D == 128 ? 5 : 8;
  __nv_bfloat16 q[2][kSub][128 * 64];
  __nv_bfloat16 kv[kStages][kSub][kKeys * 64];
  uint64_t full[kStages], empty[kStages], tail;
  uint64_t q_full, s_full[2], p_full[2], o_full[2];
  uint32_t tmem_base;
  uint32_t abort;
};

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
// A from tensor memory
__device__ __forceinline__ void mma_bf16_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// One piece of work: rows [r0, r0 + 256) of KV head h of sequence b against the slots
// [k0, k1).
struct Item {
  Seq s;
  int b, h, r0, rows, first;
  int k0, k1, split;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_chunk_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const ChunkArgs a,
               const int box) {
  extern __shared__ __align__(1024) unsigned char smraw[];
  const uint32_t base = saddr(smraw);
  Smem<D>& S = *reinterpret_cast<Smem<D>*>(smraw + ((1024 - (base & 1023)) & 1023));
  constexpr int kSub = Smem<D>::kSub, kStages = Smem<D>::kStages;
  constexpr uint32_t kRowBytes = 128;
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile uint32_t* abort = &S.abort;

  Item it;
  it.b = blockIdx.z;
  it.h = blockIdx.y;
  it.split = blockIdx.x % a.splits;
  it.s = seq_of(c, it.b);
  it.rows = it.s.m * c.group;
  it.r0 = int(blockIdx.x / a.splits) * kRows;
  if (it.r0 >= it.rows) return;
  it.first = it.s.n - it.s.m;
  {
    const int last = it.first + min(it.r0 + kRows - 1, it.rows - 1) / c.group;
    const int tiles = (it.s.n + kKeys - 1) / kKeys, per = (tiles + a.splits - 1) / a.splits;
    it.k0 = it.split * per * kKeys;
    it.k1 = min(min(it.s.n, last + 1), (it.split + 1) * per * kKeys);
  }
  const int steps = it.k1 > it.k0 ? (it.k1 - it.k0 + kKeys - 1) / kKeys : 0;
  const int halves = it.rows - it.r0 > 128 ? 2 : 1;
  const int qh = c.kvh * c.group;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    mbar_init(&S.tail, 1);
    mbar_init(&S.q_full, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 4);
      mbar_init(&S.o_full[i], 1);
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
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = S.tmem_base;

  // registers: 8 x 208 + 4 x 80 a lane, within the 12 x 168 of the launch
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  if (warp == 8) {
    // ---------------- K and V tiles ----------------
    uint32_t cnt = 0;  // tiles issued: K of step 0, V of step 0, K of step 1, ...
    bool ok = true;
    for (int j = 0; j < steps && ok; ++j) {
      const int n0 = it.k0 + j * kKeys;
      const int live = min(kKeys, it.s.n - n0);          // rows that hold slots of the sequence
      const int boxes = (live + box - 1) / box;
      for (int kv = 0; kv < 2 && ok; ++kv, ++cnt) {
        const int st = cnt % kStages;
        ok = mbar_wait(&S.empty[st], ((cnt / kStages) & 1) ^ 1, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // rows of V behind the last slot are zeroed before the products see the tile: they may
        // hold anything, and 0 * NaN is NaN (in S such columns are masked)
        const bool patch = kv == 1 && live < kKeys;
        uint64_t* bar = patch ? &S.tail : &S.full[st];
        if (lane == 0) mbar_expect_tx(bar, uint32_t(boxes) * box * kRowBytes * kSub);
        __syncwarp();
        for (int i = lane; i < boxes; i += 32) {
          const int slot = n0 + i * box, col = slot / c.page_size;
          const int p = max(0, page_at(c.table, c.cols, c.n_pages, it.b, col, c.status));
          const int row = (p * c.kvh + it.h) * c.page_size + (slot - col * c.page_size);
#pragma unroll
          for (int s = 0; s < kSub; ++s)
            tma_load_2d(&S.kv[st][s][i * box * 64], kv ? &tmV : &tmK, s * 64, row, bar);
        }
        if (patch) {
          ok = __all_sync(0xffffffffu, mbar_wait(&S.tail, 0, abort));
          if (!ok) break;
          const uint4 z = make_uint4(0, 0, 0, 0);
          for (int s = 0; s < kSub; ++s) {
            uint4* p = reinterpret_cast<uint4*>(&S.kv[st][s][0]);
            for (int i = live * 8 + lane; i < kKeys * 8; i += 32) p[i] = z;
          }
          fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.full[st]);
        }
      }
    }
  } else if (warp == 9) {
    // ---------------- products ----------------
    if (lane == 0 && steps > 0) {
      const uint32_t id_s = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(kKeys >> 3) << 17) | (uint32_t(128 >> 4) << 24);
      const uint32_t id_o = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (uint32_t(D >> 3) << 17) |
                            (uint32_t(128 >> 4) << 24);
      auto product_s = [&](int half, int st) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int s = kk >> 2, off = (kk & 3) * 32;
          mma_bf16(tmem + uint32_t(half * 128), sw128_desc(saddr(&S.q[half][s][0]) + off),
                   sw128_desc(saddr(&S.kv[st][s][0]) + off), id_s, kk > 0 ? 1u : 0u);
        }
        mma_commit(&S.s_full[half]);
      };
      bool ok = mbar_wait(&S.q_full, 0, abort) && mbar_wait(&S.full[0], 0, abort);
      if (ok) {
        fence_after();
        for (int half = 0; half < halves; ++half) product_s(half, 0);
        mma_commit(&S.empty[0]);
      }
      for (int j = 0; j < steps && ok; ++j) {
        const uint32_t cv = 2 * j + 1, ck = 2 * j + 2;
        const int sv = cv % kStages, sk = ck % kStages;
        ok = mbar_wait(&S.full[sv], (cv / kStages) & 1, abort);
        for (int half = 0; half < halves && ok; ++half) {
          ok = mbar_wait(&S.p_full[half], j & 1, abort);
          if (!ok) break;
          fence_after();
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_bf16_ta(tmem + uint32_t(256 + half * D), tmem + uint32_t(half * 128 + kk * 8),
                        sw128_desc_mn(saddr(&S.kv[sv][0][0]) + kk * 2048), id_o, (j > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&S.o_full[half]);
          if (half == halves - 1) mma_commit(&S.empty[sv]);
          if (j + 1 < steps) {
            if (half == 0) {
              ok = mbar_wait(&S.full[sk], (ck / kStages) & 1, abort);
              if (!ok) break;
              fence_after();
            }
            product_s(half, sk);
            if (half == halves - 1) mma_commit(&S.empty[sk]);
          }
        }
      }
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---------------- softmax: one thread per row ----------------
    const int half = warp >> 2;
    // this thread's half of Q into its swizzled place (16-byte chunk c of row r at c ^ (r % 8))
    {
      const int t = threadIdx.x & 127;
      for (int i = t; i < 128 * (D / 8); i += 128) {
        const int r = i / (D / 8), ch = i % (D / 8), gr = it.r0 + half * 128 + r;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (gr < it.rows) {
          const int64_t at = (int64_t(it.s.row0 + gr / c.group) * qh + it.h * c.group + gr % c.group) * D + ch * 8;
          v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at);
        }
        *reinterpret_cast<uint4*>(&S.q[half][ch >> 3][r * 64 + (((ch & 7) ^ (r & 7)) << 3)]) = v;
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.q_full);
    }
    if (half < halves) {
      const int quarter = warp & 3;
      const int r = it.r0 + half * 128 + quarter * 32 + lane;
      const bool real = r < it.rows;
      const int see = real ? min(it.k1, it.first + r / c.group + 1) : 0;  // slots below this are seen
      // the lowest limit of this warp's rows decides whether a step needs the mask at all
      const int see_low = __reduce_min_sync(0xffffffffu, real ? see : INT32_MAX);
      const uint32_t ts = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(half * 128);
      const uint32_t to = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(256 + half * D);
      const float scale = kLog2e * rsqrtf(float(D));
      float m = -INFINITY;  // the row's reference, in log2
      uint64_t l0 = 0, l1 = 0;
      bool ok = true;
      for (int j = 0; j < steps; ++j) {
        const int n0 = it.k0 + j * kKeys;
        ok = __all_sync(0xffffffffu, mbar_wait(&S.s_full[half], j & 1, abort));
        if (!ok) break;
        fence_after();
        uint32_t x0[32], x1[32], x2[32], x3[32];
        tmem_ld32(ts, x0);
        tmem_ld32(ts + 32, x1);
        tmem_ld32(ts + 64, x2);
        tmem_ld32(ts + 96, x3);
        tmem_wait_ld();
        if (n0 + kKeys > see_low) {
          const int lim = see - n0;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (i >= lim) x0[i] = 0xff800000u;
            if (i + 32 >= lim) x1[i] = 0xff800000u;
            if (i + 64 >= lim) x2[i] = 0xff800000u;
            if (i + 96 >= lim) x3[i] = 0xff800000u;
          }
        }
        float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          t0 = fmaxf(t0, __uint_as_float(x0[i]));
          t1 = fmaxf(t1, __uint_as_float(x1[i]));
          t2 = fmaxf(t2, __uint_as_float(x2[i]));
          t3 = fmaxf(t3, __uint_as_float(x3[i]));
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
            ok = __all_sync(0xffffffffu, mbar_wait(&S.o_full[half], (j - 1) & 1, abort));
            if (!ok) break;
            fence_after();
#pragma unroll
            for (int g = 0; g < D / 32; ++g) {
              uint32_t o[32];
              tmem_ld32(to + g * 32, o);
              tmem_wait_ld();
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
        weigh(x0, 0);
        weigh(x1, 16);
        tmem_st32(ts, p);
        weigh(x2, 0);
        weigh(x3, 16);
        tmem_st32(ts + 32, p);
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full[half]);
      }
      if (ok && steps > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&S.o_full[half], (steps - 1) & 1, abort));
        fence_after();
      }
      if (ok) {
        const float sum = lo2(l0) + hi2(l0) + lo2(l1) + hi2(l1);
        const int64_t row = int64_t(it.s.row0 + r / c.group) * qh + it.h * c.group + r % c.group;
        const float inv = sum > 0.f ? 1.0f / sum : sum;
        const int64_t at = int64_t(it.split) * c.total_q * qh + row;
        if (real) {
          if (a.splits > 1) *reinterpret_cast<float2*>(a.ml + at * 2) = make_float2(m, sum);
          else if (a.lse) a.lse[row] = sum == 0.f ? -INFINITY : m * kLn2 + logf(sum);
        }
#pragma unroll
        for (int g = 0; g < D / 32; ++g) {
          uint32_t o[32];
          if (steps > 0) {
            tmem_ld32(to + g * 32, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          if (!real) {
          } else if (a.splits > 1) {
            if (sum > 0.f) {
              float4* dst = reinterpret_cast<float4*>(a.part + at * D + g * 32);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                dst[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                     __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
            }
          } else {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * D + g * 32);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = bf2(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
              dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  if (threadIdx.x == 0 && S.abort) flag(c.status, MP_STATUS_WAIT_TIMEOUT);
}

template <int D>
cudaError_t launch(const ChunkArgs& a, cudaStream_t st) {
  CUtensorMap mk, mv;
  const int box = box_rows(a.c.table, a.c.page_size);
  const uint64_t rows = uint64_t(a.c.n_pages) * a.c.kvh * a.c.page_size;
  if (!make_map(&mk, a.keys, D, rows, 64, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&mv, a.values, D, rows, 64, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const size_t smem = sizeof(Smem<D>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(k_chunk_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t(a.c.max_q) * a.c.group + kRows - 1) / kRows;
  k_chunk_tc<D><<<dim3(unsigned(tiles * a.splits), a.c.kvh, a.c.batch), kThreads, smem, st>>>(mk, mv, a, box);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk_tc(const ChunkArgs& a, cudaStream_t st) {
  return a.c.d == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace mp
