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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) k_cache_append(const AppendArgs a) {
  constexpr int V = Vec<T>::N, TPH = D / V, GROUPS = kThreads / TPH;
  __shared__ float2 cs[D / 2];  // cosine and sine of each pair's angle
  const CacheArgs& c = a.c;
  const int r = blockIdx.x;
  const int half = a.rot / 2;
  // the token's sequence and slot
  const int b = seq_at(c, r);
  int slot = -1;
  Seq s = {0, 0, 0};
  if (b >= 0) {
    s = seq_of(c, b);
    slot = s.n - s.m + (r - s.row0);
  }
  if (b < 0 || r < s.row0 || r >= s.row0 + s.m) return;  // a row outside every sequence
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double turns = a.inv_freq[i] * 0.15915494309189533577;  // 1 / 2 pi
    const uint64_t step = static_cast<uint64_t>((turns - floor(turns)) * 18446744073709551616.0);
    const int64_t pos = a.positions ? a.positions[r] : slot;
    const uint64_t phase = static_cast<uint64_t>(pos) * step + 0x80000000ull;
    float sn, cn;
    sincospif(float(int32_t(uint32_t(phase >> 32))) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31 half turns
    cs[i] = make_float2(cn, sn);
  }
  __syncthreads();

  int64_t dst = -1;  // element offset of the slot's row of KV head 0
  if (slot >= 0 && slot < int64_t(c.cols) * c.page_size) {
    const int col = slot / c.page_size;
    const int p = page_at(c.table, c.cols, c.n_pages, b, col, c.status);
    if (p >= 0) dst = (int64_t(p) * c.kvh * c.page_size + (slot - col * c.page_size)) * D;
  } else if (threadIdx.x == 0) {
    flag(c.status, MP_STATUS_BAD_LENGTH);
  }
  const int64_t head_stride = int64_t(c.page_size) * D;

  const int lane = threadIdx.x % TPH, e0 = lane * V;
  const int qh = c.kvh * c.group, heads = qh + 2 * c.kvh;
  for (int h0 = 0; h0 < heads; h0 += GROUPS) {
    const int h = h0 + threadIdx.x / TPH;
    const bool live = h < heads;
    const int kind = h < qh ? 0 : (h < qh + c.kvh ? 1 : 2);  // query, key, value
    const int hh = kind == 0 ? h : (kind == 1 ? h - qh : h - qh - c.kvh);
    uint4 u = make_uint4(0, 0, 0, 0);
    if (live) {
      const T* src = kind == 0 ? static_cast<const T*>(a.q) + r * a.q_stride
                               : (kind == 1 ? static_cast<const T*>(a.k) + r * a.k_stride
                                            : static_cast<const T*>(a.v) + r * a.v_stride);
      u = *reinterpret_cast<const uint4*>(src + int64_t(hh) * D + e0);
    }
    float x[V];
    unpack(u, x);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = TPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const T* w = static_cast<const T*>(kind == 0 ? a.q_norm : a.k_norm);
    if (kind < 2 && w) {
      const float rs = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
      float g[V];
      unpack(*reinterpret_cast<const uint4*>(w + e0), g);
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = x[i] * rs * g[i];
    }
    // the partner half of a split rotation sits half / V lanes away
    float y[V];
    const bool first = e0 < half;
    const int partner = first ? lane + half / V : lane - half / V;
    const int src_lane = (threadIdx.x & 31) - lane + (e0 < a.rot ? partner : lane);
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], src_lane & 31);
    if (kind < 2 && e0 < a.rot) {
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          if (e0 + i < a.rot) {
            const float2 t = cs[(e0 + i) / 2];
            const float x0 = x[i], x1 = x[i + 1];
            x[i] = x0 * t.x - x1 * t.y;
            x[i + 1] = x1 * t.x + x0 * t.y;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 t = cs[first ? e0 + i : e0 + i - half];
          x[i] = first ? x[i] * t.x - y[i] * t.y : x[i] * t.x + y[i] * t.y;
        }
      }
    }
    if (!live) continue;
    T* to;
    if (kind == 0) to = static_cast<T*>(a.q_out) + (int64_t(r) * qh + hh) * D;
    else if (dst < 0) continue;
    else to = static_cast<T*>(kind == 1 ? a.keys : a.values) + dst + hh * head_stride;
    *reinterpret_cast<uint4*>(to + e0) = kind == 2 ? u : pack(x);
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, int dtype, cudaStream_t st) {
  const dim3 grid(a.c.total_q);
  if (dtype == MP_DTYPE_BF16) {
    if (a.c.d == 128) k_cache_append<__nv_bfloat16, 128><<<grid, kThreads, 0, st>>>(a);
    else k_cache_append<__nv_bfloat16, 64><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (a.c.d == 128) k_cache_append<float, 128><<<grid, kThreads, 0, st>>>(a);
    else k_cache_append<float, 64><<<grid, kThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace mp
