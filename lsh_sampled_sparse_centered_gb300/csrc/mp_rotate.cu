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
constexpr int kOneAtOnce = 2, kOwnAtOnce = 1;  // keys of a lane that are worked on, as many more are on their way
// CTAs of an SM (98304 slots of eight heads, new frequencies: 68 us, 5.9 TB/s; four evicted caches of 12288 with a
// position for each head: 39 us, 5.2 TB/s, 45 with loads that nothing runs ahead of)
constexpr int kResident = 3;

struct RotateArgs {
  CacheCall c;
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
  static constexpr float kSign = 1.f;
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
  // The fraction's upper 23 bits as a mantissa, which takes no conversion (those go through the unit of the
  // sines): half a turn less than the angle, so that both come out with the other sign. The bits dropped are 0 to
  // 7.5e-7 of the angle; the floats next to 2 pi and 3 pi put 1.5e-7 to 3.3e-7 of that back in one multiply-add. Over all
  // 2^23 fractions, with all and none of the dropped bits set, sine and cosine are off by 2^-20.09 at most (2^-19.82
  // from a difference and a product), a 2^11th of what the result's rounding takes. (Half of what is dropped, added to
  // the phase, costs 2 % of the call's time.)
  static constexpr float kSign = -1.f;
  static __device__ __forceinline__ void turn(uint32_t phase, float* s, float* c) {
    const float x = fmaf(__uint_as_float(0x3f800000u | (phase >> 9)), 6.283185307179586f, -9.42477798461914f);
    *s = __sinf(x);
    *c = __cosf(x);
  }
};

// ONE: a slot's heads stand at one position. TWO: the new frequencies are others.
template <typename T, bool ONE, bool TWO>
__global__ void __launch_bounds__(kThr, kResident) k_cache_rotate(const RotateArgs a) {
  constexpr int V = Vec<T>::N, kAtOnce = ONE ? kOneAtOnce : kOwnAtOnce;
  __shared__ uint2 turns[TWO ? 2 : 1][64];  // a position's fraction of a turn (lower, upper half): pair j of lane i at j lanes + i
  const CacheCall& c = a.c;
  const int half = a.rot / 2, b = blockIdx.z;
  for (int i = threadIdx.x; i < (TWO ? 2 : 1) * 64; i += kThr) {
    const int k = i >> 6, p = i & 63;
    if (p >= a.lanes * V) continue;
    const double t = p < half ? (k ? a.to_freq : a.from_freq)[p] * 0.15915494309189533577 : 0.0;  // 1 / 2 pi
    const uint64_t per = static_cast<uint64_t>((t - floor(t)) * 18446744073709551616.0);
    turns[k][p % V * a.lanes + p / V] = make_uint2(uint32_t(per), uint32_t(per >> 32));
  }
  __syncthreads();
  const Seq s = seq_of(c, b);
  const int lane = threadIdx.x & (a.lanes - 1), own = threadIdx.x / a.lanes, per = kThr / a.lanes;
  const int p0 = lane * V;  // the lane's first pair
  if (p0 >= half) return;
  const int e0 = a.interleaved ? 2 * p0 : p0, e1 = a.interleaved ? 2 * p0 + V : half + p0;  // its two vectors
  const bool whole = p0 + V <= half;
  const int64_t head_stride = int64_t(c.page_size) * c.d;
  T* keys = static_cast<T*>(a.keys);

  const float scale = a.scale * Vec<T>::kSign;
  // upper half of position * turn modulo 2^64
  auto phase = [](int32_t position, uint2 turn) {
    return __umulhi(uint32_t(position), turn.x) + uint32_t(position) * turn.y - (position < 0 ? turn.x : 0u);
  };
  auto angles = [&](int32_t from, int32_t to, float (&cs)[V], float (&sn)[V]) {
    if (!TWO) {
      // by |to - from|, which fits 32 bits without a sign, and the other way round where it is less than 0
      const uint32_t by = to < from ? uint32_t(from) - uint32_t(to) : uint32_t(to) - uint32_t(from);
      const float back = to < from ? -scale : scale;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint2 turn = turns[0][j * a.lanes + lane];
        Vec<T>::turn(__umulhi(by, turn.x) + by * turn.y, &sn[j], &cs[j]);
        sn[j] *= back;
        cs[j] *= scale;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        Vec<T>::turn(phase(to, turns[TWO ? 1 : 0][j * a.lanes + lane]) - phase(from, turns[0][j * a.lanes + lane]), &sn[j], &cs[j]);
        sn[j] *= scale;
        cs[j] *= scale;
      }
    }
  };
  auto apply = [&](T* row, const uint4 (&u)[2], const float (&cs)[V], const float (&sn)[V]) {
    float x[V], y[V], x2[V], y2[V];
    Vec<T>::unpack(u[0], x);
    Vec<T>::unpack(u[1], y);
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
    uint4 w0 = Vec<T>::pack(x2), w1 = Vec<T>::pack(y2);
    if (V == 8 && !whole) {  // elements that do not turn keep their bits, whatever NaN they are
      const int live = half - p0;  // pairs, a 32-bit word each (only interleaved ones end inside a lane's vectors)
      w0 = make_uint4(w0.x, live > 1 ? w0.y : u[0].y, live > 2 ? w0.z : u[0].z, live > 3 ? w0.w : u[0].w);
      w1 = make_uint4(live > 4 ? w1.x : u[1].x, live > 5 ? w1.y : u[1].y, live > 6 ? w1.z : u[1].z, live > 7 ? w1.w : u[1].w);
    }
    __stcs(reinterpret_cast<uint4*>(row + e0), w0);
    __stcs(reinterpret_cast<uint4*>(row + e1), w1);
  };
  // the key of a slot and head 0 (ONE) or blockIdx.y, and where it stands; at < 0: none
  struct Key {
    int64_t at;
    int32_t from, to;
  };
  const int h = ONE ? 0 : blockIdx.y;
  auto find = [&](int64_t slot64) {
    Key k = {-1, 0, 0};
    if (slot64 >= s.n) return k;
    const int slot = int(slot64);
    const int64_t where = (int64_t(b) * a.position_heads + h) * a.position_cols + slot;
    if (!inside(!(a.from || a.to) || (slot < a.position_cols && h < a.position_heads), c.status)) return k;
    k.from = a.from ? a.from[where] : slot;
    k.to = a.to ? a.to[where] : slot;
    const int col = c.page_shift >= 0 ? slot >> c.page_shift : slot / c.page_size;
    const int p = page_at(c.table, c.cols, c.n_pages, b, col, c.status);
    if (p >= 0) k.at = ((int64_t(p) * c.kvh + h) * c.page_size + (slot - col * c.page_size)) * c.d;
    return k;
  };
  auto load = [&](int64_t at, uint4 (&u)[2]) {
    if (at < 0) return;
    u[0] = __ldcs(reinterpret_cast<const uint4*>(keys + at + e0));
    u[1] = __ldcs(reinterpret_cast<const uint4*>(keys + at + e1));
  };

  // A batch of keys is worked on while the next one's loads are in flight, and the one after that is looked up.
  const int64_t step = int64_t(gridDim.x) * per;
  int64_t slot = int64_t(blockIdx.x) * per + own;
  uint4 u[kAtOnce][2], ahead[kAtOnce][2];
  if (ONE) {
    Key now = find(slot), next = find(slot + step);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (k < c.kvh) load(now.at < 0 ? -1 : now.at + k * head_stride, ahead[k]);
    for (; slot < s.n; slot += step) {
      const Key later = find(slot + 2 * step);
      float cs[V], sn[V];
      angles(now.from, now.to, cs, sn);
      for (int h0 = 0; h0 < c.kvh; h0 += kAtOnce) {
        const bool last = h0 + kAtOnce >= c.kvh;
        const Key& k2 = last ? next : now;
        const int h2 = last ? 0 : h0 + kAtOnce;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          u[k][0] = ahead[k][0];
          u[k][1] = ahead[k][1];
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if (h2 + k < c.kvh) load(k2.at < 0 ? -1 : k2.at + (h2 + k) * head_stride, ahead[k]);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if (h0 + k < c.kvh && now.at >= 0) apply(keys + now.at + (h0 + k) * head_stride, u[k], cs, sn);
      }
      now = next;
      next = later;
    }
  } else {
    Key now[kAtOnce], next[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) now[k] = find(slot + k * step);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) load(now[k].at, ahead[k]);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) next[k] = find(slot + (kAtOnce + k) * step);
    for (; slot < s.n; slot += kAtOnce * step) {
      Key later[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        u[k][0] = ahead[k][0];
        u[k][1] = ahead[k][1];
        load(next[k].at, ahead[k]);
        later[k] = find(slot + (2 * kAtOnce + k) * step);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        if (now[k].at >= 0) {
          float cs[V], sn[V];
          angles(now[k].from, now[k].to, cs, sn);
          apply(keys + now[k].at, u[k], cs, sn);
        }
        now[k] = next[k];
        next[k] = later[k];
      }
    }
  }
}

template <typename T>
cudaError_t launch(const RotateArgs& a, cudaStream_t st) {
  const bool one = a.position_heads == 1 || (!a.from && !a.to), two = a.to_freq != nullptr;
  const int heads = one ? 1 : a.c.kvh, per = kThr / a.lanes * (one ? 1 : kOwnAtOnce);
  // CTAs that fit: what one sets up is paid once for all its slots (twice as many 39.5 us, four times 41)
  const int64_t units = int64_t(a.c.batch) * heads, most = (int64_t(a.c.max_kv) + per - 1) / per;
  const int64_t fill = std::max<int64_t>(1, kResident * int64_t(device_sm_count()) / units);
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
