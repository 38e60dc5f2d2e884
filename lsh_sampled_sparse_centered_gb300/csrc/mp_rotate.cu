// Cached keys turned, in place, from the rotation that they have to another.
//
// A pair (a, b) of a key turns by t = to * to_freq - from * from_freq, and turns add up: the key that
// was rotated at `from` comes out as the one that is rotated at `to`. Angles are formed as in the append:
// frequency / 2 pi as a 64-bit fraction of a turn, times the integer position modulo 2^64; the upper
// 32 bits are the fraction of a turn that is left.
//
// Memory bound: the rotated elements of a key are read and written once. A lane holds both elements of
// 8 pairs (4 in fp32), two 16-byte vectors, so that nothing is exchanged between lanes; its frequencies
// stay in registers. Where a slot's heads stand at one position (no positions, or one for all heads) the
// lane turns all of them with one sine and cosine per pair; otherwise each head has its own.
#include <algorithm>
#include <cmath>

#include "mp_cache_host.h"

namespace mp {
namespace {

constexpr int kThr = 256;
constexpr int kAtOnce = 4;  // keys of a lane whose loads are in flight together

struct RotateArgs {
  CacheArgs c;
  void* keys;
  const double *from_freq, *to_freq;
  const int32_t *from, *to;  // [batch][position_heads][position_cols]; nullptr: the slot
  int position_heads, position_cols;
  int rot, interleaved, lanes;  // lanes of a key: a power of two
  float scale;
};

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  // The quarter of the turn is taken off first, so that the rest is small and its float exact enough.
  static __device__ __forceinline__ void turn(uint32_t phase, float* s, float* c) {
    const uint32_t quarter = (phase + 0x20000000u) >> 30;
    float s0, c0;
    sincospif(float(int32_t(phase - (quarter << 30))) * 4.656612873077393e-10f, &s0, &c0);  // 2^-31 half turns
    *s = quarter & 1 ? c0 : s0;
    *c = quarter & 1 ? s0 : c0;
    if (quarter & 2) *s = -*s;
    if (quarter == 1 || quarter == 2) *c = -*c;
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // off by 2^-21 in [-pi, pi], a 2^12th of what the result's rounding takes
  static __device__ __forceinline__ void turn(uint32_t phase, float* s, float* c) {
    const float x = float(int32_t(phase)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    *s = __sinf(x);
    *c = __cosf(x);
  }
};

// ONE: a slot's heads stand at one position. TWO: the new frequencies are others.
template <typename T, bool ONE, bool TWO>
__global__ void __launch_bounds__(kThr) k_cache_rotate(const RotateArgs a) {
  constexpr int V = Vec<T>::N;
  __shared__ uint64_t turns[2][64];  // a position's fraction of a turn
  const CacheArgs& c = a.c;
  const int half = a.rot / 2, b = blockIdx.z;
  for (int i = threadIdx.x; i < (TWO ? 2 : 1) * 64; i += kThr) {
    const int k = i >> 6, p = i & 63;
    if (p >= half) continue;
    const double t = (k ? a.to_freq : a.from_freq)[p] * 0.15915494309189533577;  // 1 / 2 pi
    turns[k][p] = static_cast<uint64_t>((t - floor(t)) * 18446744073709551616.0);
  }
  __syncthreads();
  const Seq s = seq_of(c, b);
  const int lane = threadIdx.x & (a.lanes - 1), own = threadIdx.x / a.lanes, per = kThr / a.lanes;
  const int p0 = lane * V;  // the lane's first pair
  if (p0 >= half) return;
  uint64_t from_turn[V], to_turn[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int p = min(p0 + j, half - 1);
    from_turn[j] = turns[0][p];
    to_turn[j] = turns[TWO ? 1 : 0][p];
  }
  const int e0 = a.interleaved ? 2 * p0 : p0, e1 = a.interleaved ? 2 * p0 + V : half + p0;  // its two vectors
  const bool whole = p0 + V <= half;
  const int64_t head_stride = int64_t(c.page_size) * c.d;
  T* keys = static_cast<T*>(a.keys);

  auto angles = [&](int slot, int h, float (&cs)[V], float (&sn)[V]) {
    const int64_t at = (int64_t(b) * a.position_heads + (ONE ? 0 : h)) * a.position_cols + slot;
    const int64_t from = a.from ? a.from[at] : slot, to = a.to ? a.to[at] : slot;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint64_t phase = TWO ? uint64_t(to) * to_turn[j] - uint64_t(from) * from_turn[j] : uint64_t(to - from) * from_turn[j];
      Vec<T>::turn(uint32_t((phase + 0x80000000ull) >> 32), &sn[j], &cs[j]);
      sn[j] *= a.scale;
      cs[j] *= a.scale;
    }
  };
  auto apply = [&](T* row, const uint4& u0, const uint4& u1, const float (&cs)[V], const float (&sn)[V]) {
    float x[V], y[V], x2[V], y2[V];
    Vec<T>::unpack(u0, x);
    Vec<T>::unpack(u1, y);
    if (a.interleaved) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float p = j < V / 2 ? x[2 * j % V] : y[2 * j % V], q = j < V / 2 ? x[2 * j % V + 1] : y[2 * j % V + 1];
        const bool live = whole || p0 + j < half;
        const float p2 = live ? p * cs[j] - q * sn[j] : p, q2 = live ? q * cs[j] + p * sn[j] : q;
        if (j < V / 2) {
          x2[2 * j % V] = p2;
          x2[2 * j % V + 1] = q2;
        } else {
          y2[2 * j % V] = p2;
          y2[2 * j % V + 1] = q2;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x2[j] = x[j] * cs[j] - y[j] * sn[j];
        y2[j] = y[j] * cs[j] + x[j] * sn[j];
      }
    }
    *reinterpret_cast<uint4*>(row + e0) = Vec<T>::pack(x2);
    *reinterpret_cast<uint4*>(row + e1) = Vec<T>::pack(y2);
  };
  // element offset of a slot's key of head h, or -1
  auto row_of = [&](int slot, int h) -> int64_t {
    const int col = c.page_shift >= 0 ? slot >> c.page_shift : slot / c.page_size;
    const int p = page_at(c.table, c.cols, c.n_pages, b, col, c.status);
    return p < 0 ? -1 : ((int64_t(p) * c.kvh + h) * c.page_size + (slot - col * c.page_size)) * c.d;
  };

  const int step = gridDim.x * per;
  if (ONE) {
    for (int slot = blockIdx.x * per + own; slot < s.n; slot += step) {
      const int64_t at = row_of(slot, 0);
      if (at < 0) continue;
      float cs[V], sn[V];
      angles(slot, 0, cs, sn);
      for (int h0 = 0; h0 < c.kvh; h0 += kAtOnce) {
        uint4 u[kAtOnce][2];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if (h0 + k < c.kvh) {
            const T* row = keys + at + (h0 + k) * head_stride;
            u[k][0] = *reinterpret_cast<const uint4*>(row + e0);
            u[k][1] = *reinterpret_cast<const uint4*>(row + e1);
          }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if (h0 + k < c.kvh) apply(keys + at + (h0 + k) * head_stride, u[k][0], u[k][1], cs, sn);
      }
    }
  } else {
    const int h = blockIdx.y;
    for (int slot = blockIdx.x * per + own; slot < s.n; slot += kAtOnce * step) {
      uint4 u[kAtOnce][2];
      int64_t at[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        at[k] = slot + int64_t(k) * step < s.n ? row_of(slot + k * step, h) : -1;
        if (at[k] < 0) continue;
        u[k][0] = *reinterpret_cast<const uint4*>(keys + at[k] + e0);
        u[k][1] = *reinterpret_cast<const uint4*>(keys + at[k] + e1);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        if (at[k] < 0) continue;
        float cs[V], sn[V];
        angles(slot + k * step, h, cs, sn);
        apply(keys + at[k], u[k][0], u[k][1], cs, sn);
      }
    }
  }
}

template <typename T>
cudaError_t launch(const RotateArgs& a, cudaStream_t st) {
  const bool one = a.position_heads == 1 || (!a.from && !a.to), two = a.to_freq != nullptr;
  const int heads = one ? 1 : a.c.kvh, per = kThr / a.lanes * (one ? 1 : kAtOnce);
  // CTAs that fit, and one more round of them: what a CTA sets up is paid once for all its slots
  const int64_t units = int64_t(a.c.batch) * heads, most = (int64_t(a.c.max_kv) + per - 1) / per;
  const int64_t fill = std::max<int64_t>(1, 8 * int64_t(device_sm_count()) / units);
  const dim3 grid(unsigned(std::min(most, fill)), unsigned(heads), unsigned(a.c.batch));
  if (one) {
    if (two) k_cache_rotate<T, true, true><<<grid, kThr, 0, st>>>(a);
    else k_cache_rotate<T, true, false><<<grid, kThr, 0, st>>>(a);
  } else {
    if (two) k_cache_rotate<T, false, true><<<grid, kThr, 0, st>>>(a);
    else k_cache_rotate<T, false, false><<<grid, kThr, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace mp

using namespace mp;

extern "C" int mp_cache_rotate(const mp_cache_config* cfg, const mp_rotary* rotary, void* keys, const int32_t* page_table,
                               const int32_t* kv_len, int32_t max_kv, const double* from_freq, const double* to_freq,
                               const int32_t* from_positions, const int32_t* to_positions, int32_t position_heads,
                               int32_t position_cols, float scale, uint32_t* status, void* stream) {
  int rc = check_cache(cfg);
  if (rc != MP_OK) return rc;
  if ((rc = check_rotary(rotary, cfg)) != MP_OK) return rc;
  if ((rc = check_pages(cfg, page_table)) != MP_OK) return rc;
  if ((rc = check_limits(cfg, 0, 1, max_kv)) != MP_OK) return rc;
  if (!keys || !kv_len || !std::isfinite(scale)) return MP_ERR_INVALID_ARG;
  if (rotary->rot_dim > 0 && !from_freq) return MP_ERR_INVALID_ARG;
  const bool positions = from_positions || to_positions;
  if (positions && ((position_heads != 1 && position_heads != cfg->kv_heads) || position_cols < max_kv)) return MP_ERR_INVALID_ARG;
  if (!aligned16(keys)) return MP_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(page_table), static_cast<const void*>(kv_len),
                        static_cast<const void*>(from_positions), static_cast<const void*>(to_positions),
                        static_cast<const void*>(status)})
    if (!aligned4(p)) return MP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(from_freq) | reinterpret_cast<uintptr_t>(to_freq)) & 7u) return MP_ERR_INVALID_ARG;
  if (injected("rotate")) return MP_ERR_INJECTED;
  if (rotary->rot_dim == 0) return MP_OK;
  RotateArgs a;
  a.c = cache_args(cfg, page_table, nullptr, kv_len, 0, 1, max_kv, status);
  a.keys = keys;
  a.from_freq = from_freq;
  a.to_freq = to_freq == from_freq ? nullptr : to_freq;
  a.from = from_positions;
  a.to = to_positions;
  a.position_heads = positions ? position_heads : 1;
  a.position_cols = positions ? position_cols : 0;
  a.rot = rotary->rot_dim;
  a.interleaved = rotary->interleaved;
  const int vec = cfg->dtype == MP_DTYPE_BF16 ? 8 : 4;
  a.lanes = 1;
  while (a.lanes * vec < a.rot / 2) a.lanes *= 2;
  a.scale = scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaGetLastError();
  ProfScope ps(st, K_CACHE_ROTATE);
  const cudaError_t e = cfg->dtype == MP_DTYPE_BF16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
  return e == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}
