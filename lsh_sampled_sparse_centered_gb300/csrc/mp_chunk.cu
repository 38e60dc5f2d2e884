// Exact attention of a chunk of new tokens over the paged cache, and the attention
// weights that its keys received, on the CUDA cores: the fp32 forms.
//
// A tile is 64 query rows of one KV head (row = token * group + head of the group, so the
// heads of a group share every key they load) against 64 keys at a time. The softmax is
// online: per row the running maximum m and sum l of 2^(x - m), x = q k log2(e) / sqrt(d),
// and the unnormalised sum of 2^(x - m) v; keys past a row's own slot enter as -infinity.
// The slots can be split over several CTAs; each then stores (m, l, sum) and k_chunk_join
// combines them.
#include "mp_cache.cuh"

namespace mp {
namespace {

constexpr int kBM = 64, kBN = 64, kThr = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// 64 rows into shared memory as [d][64] (row index fastest): thread t takes row t % 64 and
// every other group of 8 elements; p(row) is the row's address or nullptr (zeros).
template <int D, typename P>
__device__ __forceinline__ void load_transposed(float* dst, P p) {
  const int row = threadIdx.x & 63;
  const float* src = p(row);
#pragma unroll 4
  for (int e = (threadIdx.x >> 6) * 8; e < D; e += 16) {
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (src) load8(src + e, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[(e + i) * 64 + row] = x[i];
  }
}
template <int D, typename P>
__device__ __forceinline__ void load_rows(float* dst, P p) {
  for (int i = threadIdx.x; i < 64 * (D / 8); i += kThr) {
    const int row = i / (D / 8), e = (i % (D / 8)) * 8;
    const float* src = p(row);
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (src) load8(src + e, x);
    *reinterpret_cast<float4*>(dst + row * D + e) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(dst + row * D + e + 4) = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// S[8][4] of rows ty*8.. and keys tx*4.. from [d][64] tiles
template <int D>
__device__ __forceinline__ void dot_tile(const float* qt, const float* kt, int ty, int tx, float (&s)[8][4]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int e = 0; e < D; ++e) {
    const float4 a0 = *reinterpret_cast<const float4*>(qt + e * 64 + ty * 8);
    const float4 a1 = *reinterpret_cast<const float4*>(qt + e * 64 + ty * 8 + 4);
    const float4 b0 = *reinterpret_cast<const float4*>(kt + e * 64 + tx * 4);
    const float a[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w}, b[4] = {b0.x, b0.y, b0.z, b0.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = fmaf(a[i], b[j], s[i][j]);
  }
}

template <int D>
__global__ void __launch_bounds__(kThr) k_chunk_simt(const ChunkArgs a) {
  extern __shared__ float sm[];
  float* qt = sm;               // [D][64]
  float* kt = qt + D * kBM;     // [D][64]
  float* vs = kt + D * kBN;     // [64][D]
  float* pt = vs + D * kBN;     // [64 keys][64 rows]
  const CacheArgs& c = a.c;
  const int b = blockIdx.z, h = blockIdx.y;
  const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits;
  const Seq s = seq_of(c, b);
  const int rows = s.m * c.group, r0 = tile * kBM;
  if (r0 >= rows) return;
  const int qh = c.kvh * c.group;
  const int first = s.n - s.m;                                       // slot of token 0
  const int last = first + min(r0 + kBM - 1, rows - 1) / c.group;     // slot of the tile's last token
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  // this split's keys: a run of 64-key tiles of the sequence
  const int tiles = (s.n + kBN - 1) / kBN, per = (tiles + a.splits - 1) / a.splits;
  const int k0 = split * per * kBN, k1 = min(min(s.n, last + 1), (split + 1) * per * kBN);
  auto qrow = [&](int i) -> const float* {
    const int r = r0 + i;
    return r < rows ? static_cast<const float*>(a.q) + (int64_t(s.row0 + r / c.group) * qh + h * c.group + r % c.group) * D
                    : nullptr;
  };
  load_transposed<D>(qt, qrow);
  float m[8], l[8], o[8][D / 16];
  int see[8];  // a row sees the slots below this
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    see[i] = first + (r0 + ty * 8 + i) / c.group + 1;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[i][j] = 0.f;
  }
  const float scale = kLog2e * rsqrtf(float(D));
  for (int n0 = k0; n0 < k1; n0 += kBN) {
    __syncthreads();
    auto slot_ptr = [&](const void* base, int i) -> const float* {
      return n0 + i < k1 ? static_cast<const float*>(base) + slot_read(c, b, h, n0 + i) : nullptr;
    };
    load_transposed<D>(kt, [&](int i) { return slot_ptr(a.keys, i); });
    load_rows<D>(vs, [&](int i) { return slot_ptr(a.values, i); });
    __syncthreads();
    float x[8][4];
    dot_tile<D>(qt, kt, ty, tx, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int slot = n0 + tx * 4 + j;
        x[i][j] = slot < see[i] && slot < k1 ? x[i][j] * scale : -INFINITY;
        top = fmaxf(top, x[i][j]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const float mn = fmaxf(m[i], top);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float by = exp2f(m[i] - ref);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[i][j] = exp2f(x[i][j] - ref);
        sum += x[i][j];
      }
      l[i] = l[i] * by + sum;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[i][j] *= by;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      *reinterpret_cast<float4*>(pt + (tx * 4 + j) * 64 + ty * 8) = make_float4(x[0][j], x[1][j], x[2][j], x[3][j]);
      *reinterpret_cast<float4*>(pt + (tx * 4 + j) * 64 + ty * 8 + 4) =
          make_float4(x[4][j], x[5][j], x[6][j], x[7][j]);
    }
    __syncthreads();
#pragma unroll 2
    for (int k = 0; k < kBN; ++k) {
      const float4 a0 = *reinterpret_cast<const float4*>(pt + k * 64 + ty * 8);
      const float4 a1 = *reinterpret_cast<const float4*>(pt + k * 64 + ty * 8 + 4);
      const float p[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
      for (int g = 0; g < D / 64; ++g) {
        const float4 v4 = *reinterpret_cast<const float4*>(vs + k * D + g * 64 + tx * 4);
        const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][g * 4 + j] = fmaf(p[i], v[j], o[i][g * 4 + j]);
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // k_chunk_join may be set up
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float sum = l[i];
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    const int r = r0 + ty * 8 + i;
    if (r >= rows) continue;
    const int64_t row = int64_t(s.row0 + r / c.group) * qh + h * c.group + r % c.group;
    if (a.splits > 1) {
      const int64_t at = int64_t(split) * c.total_q * qh + row;
      if (tx == 0) *reinterpret_cast<float2*>(a.ml + at * 2) = make_float2(m[i], sum);
      if (sum > 0.f)
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
          *reinterpret_cast<float4*>(a.part + at * D + g * 64 + tx * 4) =
              make_float4(o[i][g * 4], o[i][g * 4 + 1], o[i][g * 4 + 2], o[i][g * 4 + 3]);
    } else {
      const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
      if (a.lse && tx == 0) a.lse[row] = sum == 0.f ? -INFINITY : m[i] * kLn2 + logf(sum);
      float* out = static_cast<float*>(a.out) + row * D;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) out[(j / 4) * 64 + tx * 4 + j % 4] = o[i][j] * inv;
    }
  }
}

// Joins the splits' (m, l, sum) of a query row, in an order that is fixed by their number:
// WARPS warps per row (8 where there are many splits, so that their loads overlap) take
// eight splits at a time each. Started while the slices still run (its launch costs as much
// as its work); it waits for them first.
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(256) k_chunk_join(const ChunkArgs a) {
  constexpr int PER = D / 32;
  __shared__ float so[8][D], sl[8];
  const CacheArgs& c = a.c;
  const int qh = c.kvh * c.group;
  const int64_t rows = int64_t(c.total_q) * qh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * (8 / WARPS) + warp / WARPS;
  const int part = warp % WARPS;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= rows) return;
  const int t = int(row / qh), b = seq_at(c, t);
  if (b < 0) return;
  const Seq s = seq_of(c, b);
  if (t < s.row0 || t >= s.row0 + s.m) return;
  const float2* ml = reinterpret_cast<const float2*>(a.ml) + row;
  float m = -INFINITY;
  for (int i = lane; i < a.splits; i += 32) m = fmaxf(m, ml[i * rows].x);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f, o[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) o[j] = 0.f;
  for (int i = part * 8; i < a.splits; i += WARPS * 8) {
    float x[8][PER], f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 v = i + k < a.splits ? ml[(i + k) * rows] : make_float2(-INFINITY, 0.f);
      f[k] = v.y == 0.f ? 0.f : exp2f(v.x - ref);
      l = fmaf(v.y, f[k], l);
      const bool live = v.y != 0.f;  // an empty slice has written no sum
      const float* p = a.part + ((i + k) * rows + row) * D + lane * PER;
#pragma unroll
      for (int j = 0; j < PER; ++j) x[k][j] = live ? p[j] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < PER; ++j) o[j] = fmaf(x[k][j], f[k], o[j]);
  }
  if (WARPS > 1) {  // one row per CTA: no warp has left
#pragma unroll
    for (int j = 0; j < PER; ++j) so[warp][lane * PER + j] = o[j];
    if (lane == 0) sl[warp] = l;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      l += sl[w];
#pragma unroll
      for (int j = 0; j < PER; ++j) o[j] += so[w][lane * PER + j];
    }
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
#pragma unroll
  for (int j = 0; j < PER; ++j) static_cast<T*>(a.out)[row * D + lane * PER + j] = T(o[j] * inv);
}

// Attention weights: one CTA owns 64 slots of one KV head and walks the chunk's query
// rows in order, so every slot's sum has one owner and a fixed order.
template <int D>
__global__ void __launch_bounds__(kThr) k_weights_simt(const WeightsArgs a) {
  extern __shared__ float sm[];
  float* qt = sm;            // [D][64]
  float* kt = qt + D * kBM;  // [D][64]
  float* col = kt + D * kBN; // [8][64] partial column sums
  const CacheArgs& c = a.c;
  const int b = blockIdx.z, h = blockIdx.y, n0 = blockIdx.x * kBN;
  const Seq s = seq_of(c, b);
  if (n0 >= s.n || s.m == 0) return;
  const int rows = s.m * c.group, first = s.n - s.m, qh = c.kvh * c.group;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  load_transposed<D>(kt, [&](int i) -> const float* {
    return n0 + i < s.n ? static_cast<const float*>(a.keys) + slot_read(c, b, h, n0 + i) : nullptr;
  });
  const float scale = kLog2e * rsqrtf(float(D));
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  // rows before token n0 - first see none of these slots
  const int start = max(0, n0 - first) * c.group / kBM * kBM;
  for (int r0 = start; r0 < rows; r0 += kBM) {
    __syncthreads();
    load_transposed<D>(qt, [&](int i) -> const float* {
      const int r = r0 + i;
      return r < rows ? static_cast<const float*>(a.q) + (int64_t(s.row0 + r / c.group) * qh + h * c.group + r % c.group) * D
                      : nullptr;
    });
    __syncthreads();
    float x[8][4];
    dot_tile<D>(qt, kt, ty, tx, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + ty * 8 + i;
      if (r >= rows) continue;
      const int t = r / c.group;
      const float z = a.lse[int64_t(s.row0 + t) * qh + h * c.group + r % c.group] * kLog2e;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n0 + tx * 4 + j <= first + t) acc[j] += exp2f(fmaf(x[i][j], scale, -z));
    }
  }
  *reinterpret_cast<float4*>(col + ty * 64 + tx * 4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  const int k = threadIdx.x;
  if (k < kBN && n0 + k < s.n) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += col[i * 64 + k];
    float* to = a.scores + (int64_t(b) * c.kvh + h) * (int64_t(c.cols) * c.page_size) + n0 + k;
    *to += sum;
  }
}

template <int D>
cudaError_t chunk_simt(const ChunkArgs& a, cudaStream_t st) {
  constexpr int smem = (3 * D * 64 + 64 * 64) * 4;
  cudaError_t e = cudaFuncSetAttribute(k_chunk_simt<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t(a.c.max_q) * a.c.group + kBM - 1) / kBM;
  k_chunk_simt<D><<<dim3(unsigned(tiles * a.splits), a.c.kvh, a.c.batch), kThr, smem, st>>>(a);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t join(const ChunkArgs& a, cudaStream_t st) {
  const int64_t rows = int64_t(a.c.total_q) * a.c.kvh * a.c.group;
  cudaLaunchConfig_t cfg = {};
  const bool wide = a.splits > 8;
  cfg.gridDim = dim3(unsigned(wide ? rows : (rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&cfg, k_chunk_join<T, D, 8>, a) : cudaLaunchKernelEx(&cfg, k_chunk_join<T, D, 1>, a);
}
template <int D>
cudaError_t weights_simt(const WeightsArgs& a, cudaStream_t st) {
  constexpr int smem = (2 * D * 64 + 8 * 64) * 4;
  cudaError_t e = cudaFuncSetAttribute(k_weights_simt<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  k_weights_simt<D><<<dim3((a.c.max_kv + kBN - 1) / kBN, a.c.kvh, a.c.batch), kThr, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

// Slices of the keys: as many as fill the SMs about twice, each of at least 256 slots.
int chunk_splits(const mp_cache_config* c, int max_q, int max_kv) {
  const int64_t group = c->q_heads / c->kv_heads;
  const int64_t ctas = (max_q * group + kBM - 1) / kBM * c->kv_heads * c->batch;
  const int64_t fill = 2 * int64_t(device_sm_count()) / ctas, most = (int64_t(max_kv) + 255) / 256;
  const int64_t s = fill < most ? fill : most;
  return int(s < 1 ? 1 : (s > 64 ? 64 : s));
}

cudaError_t launch_chunk_simt(const ChunkArgs& a, cudaStream_t st) {
  return a.c.d == 128 ? chunk_simt<128>(a, st) : chunk_simt<64>(a, st);
}
cudaError_t launch_chunk_join(const ChunkArgs& a, int dtype, cudaStream_t st) {
  if (dtype == MP_DTYPE_BF16) return a.c.d == 128 ? join<__nv_bfloat16, 128>(a, st) : join<__nv_bfloat16, 64>(a, st);
  return a.c.d == 128 ? join<float, 128>(a, st) : join<float, 64>(a, st);
}
cudaError_t launch_cache_weights(const WeightsArgs& a, int dtype, cudaStream_t st) {
  if (dtype == MP_DTYPE_BF16) return launch_weights_bf16(a, st);
  return a.c.d == 128 ? weights_simt<128>(a, st) : weights_simt<64>(a, st);
}

}  // namespace mp
