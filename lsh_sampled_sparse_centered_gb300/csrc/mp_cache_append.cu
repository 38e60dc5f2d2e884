// Norms and rotation of the new tokens' queries and keys, and the cache write.
//
// Per head x of d elements: y = x * rsqrt(mean(x^2) + eps) * w, then the pairs of the
// first rot elements turn by the angle position * inv_freq. The angle is reduced without
// rounding: inv_freq / 2 pi is held as a 64-bit fraction of a turn, its product with the
// integer position modulo 2^64 is the exact fraction of the turn that the angle leaves
// (error 2^-53 of a turn per position), so far positions cost no more than near ones.
//
// Memory bound: (q_heads + 2 kv_heads) * d values in and out per token. 16-byte vectors,
// d * size / 16 lanes per head; the sines and cosines are shared by a token's heads
// through shared memory (computing them per head would cost more than the traffic).
#include "mp_cache.cuh"

namespace mp {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
  x[0] = __uint_as_float(u.x);
  x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z);
  x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// TOK tokens of a CTA; kBatch vectors of a lane are in flight at a time, the first of them
// while the tokens' slots and angles are worked out.
constexpr int kBatch = 4;

template <typename T, int D, int TOK>
__global__ void __launch_bounds__(kThreads) k_cache_append(const AppendArgs a) {
  constexpr int V = Vec<T>::N, TPH = D / V, GROUPS = kThreads / TPH;
  __shared__ float2 cs[TOK][D / 2];  // cosine and sine of each pair's angle
  __shared__ int64_t dst[TOK];       // element offset of the slot's row of KV head 0, or -1
  __shared__ int64_t pos[TOK];       // where the token stands
  __shared__ int live[TOK];          // the row belongs to a sequence
  const CacheArgs& c = a.c;
  const int row0 = blockIdx.x * TOK, toks = min(TOK, c.total_q - row0);
  const int half = a.rot / 2;
  const int lane = threadIdx.x % TPH, e0 = lane * V, group = threadIdx.x / TPH;
  const int qh = c.kvh * c.group, heads = qh + 2 * c.kvh, items = toks * heads;

  auto source = [&](int i) -> const uint4* {
    const int tok = TOK == 1 ? 0 : i / heads, h = i - tok * heads;
    const int64_t r = row0 + tok;
    const T* p = h < qh ? static_cast<const T*>(a.q) + r * a.q_stride + int64_t(h) * D
                        : (h < qh + c.kvh ? static_cast<const T*>(a.k) + r * a.k_stride + int64_t(h - qh) * D
                                          : static_cast<const T*>(a.v) + r * a.v_stride + int64_t(h - qh - c.kvh) * D);
    return reinterpret_cast<const uint4*>(p + e0);
  };
  uint4 u[kBatch];
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    const int i = group + k * GROUPS;
    u[k] = i < items ? __ldcs(source(i)) : make_uint4(0, 0, 0, 0);
  }
  uint4 gq = make_uint4(0, 0, 0, 0), gk = gq;
  if (a.q_norm) gq = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q_norm) + e0);
  if (a.k_norm) gk = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k_norm) + e0);

  if (int(threadIdx.x) < toks) {
    const int t = threadIdx.x, r = row0 + t;
    const int b = seq_at(c, r);
    int64_t at = -1;
    int slot = -1;
    bool in = false;
    if (b >= 0) {
      const Seq s = seq_of(c, b);
      in = r >= s.row0 && r < s.row0 + s.m;
      slot = s.n - s.m + (r - s.row0);
      if (in && slot >= 0 && slot < int64_t(c.cols) * c.page_size) {
        const int col = slot / c.page_size;
        const int p = page_at(c.table, c.cols, c.n_pages, b, col, c.status);
        if (p >= 0) at = (int64_t(p) * c.kvh * c.page_size + (slot - col * c.page_size)) * D;
      } else if (in) {
        flag(c.status, MP_STATUS_BAD_LENGTH);
      }
    }
    dst[t] = at;
    live[t] = in;
    pos[t] = a.positions ? a.positions[r] : slot;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double turns = a.inv_freq[i] * 0.15915494309189533577;  // 1 / 2 pi
    const uint64_t step = static_cast<uint64_t>((turns - floor(turns)) * 18446744073709551616.0);
    for (int t = 0; t < toks; ++t) {
      const uint64_t phase = static_cast<uint64_t>(pos[t]) * step + 0x80000000ull;
      float sn, cn;
      sincospif(float(int32_t(uint32_t(phase >> 32))) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31 half turns
      cs[t][i] = make_float2(cn, sn);
    }
  }
  __syncthreads();

  const int64_t head_stride = int64_t(c.page_size) * D;
  // the partner half of a split rotation sits half / V lanes away
  const bool first = e0 < half, turns = e0 < a.rot;
  const int partner = (threadIdx.x & 31) + (a.interleaved || !turns ? 0 : (first ? half / V : -(half / V)));
  for (int base = group; base - group < items; base += kBatch * GROUPS) {
    if (base != group) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = base + k * GROUPS;
        u[k] = i < items ? __ldcs(source(i)) : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = base + k * GROUPS;
      const int tok = TOK == 1 ? 0 : min(i / heads, TOK - 1), h = i - tok * heads;
      const int kind = h < qh ? 0 : (h < qh + c.kvh ? 1 : 2);  // query, key, value
      float x[V], y[V];
      unpack(u[k], x);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
      for (int o = TPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (kind == 0 ? a.q_norm != nullptr : a.k_norm != nullptr) {
        const float rs = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
        float g[V];
        unpack(kind == 0 ? gq : gk, g);
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = x[j] * rs * g[j];
      }
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          if (e0 + j < a.rot) {
            const float2 t = cs[tok][(e0 + j) / 2];
            const float x0 = x[j], x1 = x[j + 1];
            x[j] = x0 * t.x - x1 * t.y;
            x[j + 1] = x1 * t.x + x0 * t.y;
          }
        }
      } else if (half > 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], partner);
        if (turns) {
          const float4* t4 = reinterpret_cast<const float4*>(&cs[tok][first ? e0 : e0 - half]);
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            const float4 t = t4[j / 2];
            x[j] = first ? x[j] * t.x - y[j] * t.y : x[j] * t.x + y[j] * t.y;
            x[j + 1] = first ? x[j + 1] * t.z - y[j + 1] * t.w : x[j + 1] * t.z + y[j + 1] * t.w;
          }
        }
      }
      if (i >= items || !live[tok]) continue;
      T* to;
      if (kind == 0) to = static_cast<T*>(a.q_out) + (int64_t(row0 + tok) * qh + h) * D;
      else if (dst[tok] < 0) continue;
      else to = static_cast<T*>(kind == 1 ? a.keys : a.values) + dst[tok] + (h - qh - (kind == 1 ? 0 : c.kvh)) * head_stride;
      *reinterpret_cast<uint4*>(to + e0) = kind == 2 ? u[k] : pack(x);
    }
  }
}

template <typename T, int D>
void launch(const AppendArgs& a, cudaStream_t st) {
  // several tokens share a CTA once there are enough to fill the SMs with CTAs of four
  if (a.c.total_q >= 8 * device_sm_count())
    k_cache_append<T, D, 4><<<(a.c.total_q + 3) / 4, kThreads, 0, st>>>(a);
  else
    k_cache_append<T, D, 1><<<a.c.total_q, kThreads, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, int dtype, cudaStream_t st) {
  if (dtype == MP_DTYPE_BF16) {
    if (a.c.d == 128) launch<__nv_bfloat16, 128>(a, st);
    else launch<__nv_bfloat16, 64>(a, st);
  } else {
    if (a.c.d == 128) launch<float, 128>(a, st);
    else launch<float, 64>(a, st);
  }
  return cudaGetLastError();
}

}  // namespace mp
