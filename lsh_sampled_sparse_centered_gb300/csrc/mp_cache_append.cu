// Norms and rotation of the new tokens' queries and keys, and the cache write.
//
// Per head x of d elements: y = x * rsqrt(mean(x^2) + eps) * w, then the pairs of the
// first rot elements turn by the angle position * inv_freq. inv_freq / 2 pi, rounded to a double
// (2^-53 of a turn per position), is held as a 64-bit fraction of a turn; its product with the
// integer position modulo 2^64 is the fraction of the turn that the angle leaves, without a
// rounding of its own, so far positions cost no more than near ones. sincospif takes its
// upper 32 bits as a float.
//
// Memory bound: (q_heads + 2 kv_heads) * d values in and out per token. A warp takes whole
// heads of one token, d * size / 16 lanes with a 16-byte vector each per head. What it does
// once per token (slot, angles, the factors of its elements) costs about as many
// instructions as eight heads, so a warp takes all heads of its token where there are
// tokens enough, and a part of them where there are few.
#include "mp_cache.cuh"

namespace mp {
namespace {

constexpr int kWarps = 4;  // independent of each other
constexpr int kBatch = 2;  // vectors of a lane that are worked on, as many more are on their way
constexpr int kResident = 7;  // CTAs of an SM: left alone bf16 takes 80 registers, and six fit

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
__global__ void __launch_bounds__(kWarps * 32, kResident) k_cache_append(const AppendArgs a, const int parts) {
  constexpr int V = Vec<T>::N, TPH = D / V, HPW = 32 / TPH;  // heads of a warp at a time
  __shared__ alignas(16) float cosine[kWarps][D / 2], sine[kWarps][D / 2];  // of each pair's angle
  const CacheCall& c = a.c;
  const int warp = threadIdx.x >> 5, l32 = threadIdx.x & 31, lane = l32 % TPH, e0 = lane * V;
  const int64_t w = int64_t(blockIdx.x) * kWarps + warp;
  const int64_t r = w / parts;
  const int h0 = int(w - r * parts) * HPW + l32 / TPH, step = parts * HPW;  // this lane's heads
  if (r >= c.total_q) return;
  const int half = a.rot / 2;
  const int qh = c.kvh * c.group;

  // what does not wait for the token's sequence is on its way before that is looked up: the
  // first vectors of q, the frequencies and the position
  const T* q = static_cast<const T*>(a.q) + r * a.q_stride;
  uint4 early[kBatch];
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    const int h = h0 + k * step;
    early[k] = h < qh ? __ldcs(reinterpret_cast<const uint4*>(q + int64_t(h) * D + e0)) : make_uint4(0, 0, 0, 0);
  }
  double freq[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) freq[i] = i * 32 + l32 < half ? a.inv_freq[i * 32 + l32] : 0.0;
  const int64_t given = a.positions ? a.positions[r] : 0;

  const int b = seq_at_warp(c, int(r));
  if (b < 0) return;  // a row outside every sequence
  const Seq s = seq_of(c, b);
  if (r < s.row0 || r >= s.row0 + s.m) return;
  // from the lengths as they are: cut to the limits they would move the tokens to other slots
  const int64_t slot = int64_t(c.kv_len[b]) - c.cu_q[b + 1] + r;
  int64_t dst = -1;  // element offset of the slot's row of KV head 0
  if (slot >= 0 && slot < int64_t(c.cols) * c.page_size) {
    const int col = int(slot) / c.page_size;
    const int p = page_at(c.table, c.cols, c.n_pages, b, col, c.status);
    if (p >= 0) dst = (int64_t(p) * c.kvh * c.page_size + (slot - int64_t(col) * c.page_size)) * D;
  } else if (l32 == 0) {
    flag(c.status, MP_STATUS_BAD_LENGTH);
  }
  const int64_t pos = a.positions ? given : slot;
#pragma unroll
  for (int k = 0; k < D / 64; ++k) {
    const int i = k * 32 + l32;
    if (i >= half) break;
    const double turns = freq[k] * 0.15915494309189533577;  // 1 / 2 pi
    const uint64_t per = static_cast<uint64_t>((turns - floor(turns)) * 18446744073709551616.0);
    const uint64_t phase = static_cast<uint64_t>(pos) * per + 0x80000000ull;
    sincospif(float(int32_t(uint32_t(phase >> 32))) * 4.656612873077393e-10f, &sine[warp][i], &cosine[warp][i]);  // 2^-31 half turns
  }
  __syncwarp();

  // the partner half of a split rotation sits half / V lanes away
  const bool first = e0 < half, turns = e0 < a.rot;
  const int away = a.interleaved || !turns ? 0 : (first ? half / V : -(half / V));
  const int64_t head_stride = int64_t(c.page_size) * D;

  // A lane turns the same elements of every head, so norm and rotation of its elements are
  // one sum with the same factors for all query heads, and others for all key heads:
  //   y_i = r (x_i own_i + x_partner other_i), r the inverse root (1 without a norm),
  //   own_i = w_i cos, other_i = -+ w_partner sin.
  auto turn_heads = [&](const T* src, const void* norm, int heads, T* to, int64_t to_stride, const uint4* have) {
    float own[V], other[V];
    {
      float g[V], gp[V];
#pragma unroll
      for (int j = 0; j < V; ++j) g[j] = gp[j] = 1.f;
      if (norm) {
        unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(norm) + e0), g);
        unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(norm) + e0 + away * V), gp);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float cn = 1.f, sn = 0.f;
        if (a.interleaved ? e0 + j < a.rot : turns) {
          const int at = a.interleaved ? (e0 + j) / 2 : (first ? e0 + j : e0 + j - half);
          cn = cosine[warp][at];
          sn = (a.interleaved ? (j & 1) == 0 : first) ? -sine[warp][at] : sine[warp][at];
        }
        own[j] = g[j] * cn;
        other[j] = (a.interleaved ? g[j ^ 1] : gp[j]) * sn;
      }
    }
    uint4 u[kBatch], ahead[kBatch];  // a batch, and the next one on its way
    auto load = [&](int hb, uint4 (&v)[kBatch]) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int h = hb + k * step;
        v[k] = h < heads ? __ldcs(reinterpret_cast<const uint4*>(src + int64_t(h) * D + e0)) : make_uint4(0, 0, 0, 0);
      }
    };
    if (have) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) ahead[k] = have[k];
    } else {
      load(h0, ahead);
    }
    for (int hb = h0; hb - h0 < heads; hb += kBatch * step) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) u[k] = ahead[k];
      load(hb + kBatch * step, ahead);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int h = hb + k * step;
        if (h - h0 >= heads) break;  // the same for the whole warp
        float x[V], y[V], z[V];
        unpack(u[k], x);
        // An element that does not turn has no partner: an infinity next to it, or its own,
        // times the factor 0 would be NaN.
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < V; ++j) y[j] = e0 + (j & ~1) < a.rot ? x[j ^ 1] : 0.f;
        } else {
          uint4 o;
          o.x = __shfl_sync(0xffffffffu, u[k].x, l32 + away);
          o.y = __shfl_sync(0xffffffffu, u[k].y, l32 + away);
          o.z = __shfl_sync(0xffffffffu, u[k].z, l32 + away);
          o.w = __shfl_sync(0xffffffffu, u[k].w, l32 + away);
          if (!turns) o = make_uint4(0, 0, 0, 0);
          unpack(o, y);
        }
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int i = TPH / 2; i > 0; i >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, i);
        const float rs = norm ? rsqrtf(ss * (1.0f / D) + a.eps) : 1.f;
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] = rs * fmaf(x[j], own[j], y[j] * other[j]);
        if (h < heads) *reinterpret_cast<uint4*>(to + h * to_stride + e0) = pack(z);
      }
    }
  };
  turn_heads(q, a.q_norm, qh, static_cast<T*>(a.q_out) + r * qh * D, D, early);
  if (dst < 0) return;  // the same for the whole warp
  const T* v = static_cast<const T*>(a.v) + r * a.v_stride + e0;
  for (int hb = h0; hb < c.kvh; hb += 4 * step) {
    uint4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (hb + k * step < c.kvh) u[k] = __ldcs(reinterpret_cast<const uint4*>(v + int64_t(hb + k * step) * D));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (hb + k * step < c.kvh)
        *reinterpret_cast<uint4*>(static_cast<T*>(a.values) + dst + (hb + k * step) * head_stride + e0) = u[k];
  }
  turn_heads(static_cast<const T*>(a.k) + r * a.k_stride, a.k_norm, c.kvh, static_cast<T*>(a.keys) + dst, head_stride, nullptr);
}

template <typename T, int D>
void launch(const AppendArgs& a, cudaStream_t st) {
  constexpr int HPW = 32 / (D / Vec<T>::N);
  // as many warps per token as fill the SMs with about 32 warps each, at most one for every
  // round of heads
  const int64_t want = 32 * int64_t(device_sm_count()) / a.c.total_q, most = (a.c.kvh * a.c.group + HPW - 1) / HPW;
  const int parts = int(want < 1 ? 1 : (want < most ? want : most));
  const int64_t warps = int64_t(a.c.total_q) * parts;
  k_cache_append<T, D><<<unsigned((warps + kWarps - 1) / kWarps), kWarps * 32, 0, st>>>(a, parts);
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
