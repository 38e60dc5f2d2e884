// The kernel of mp_prefix_few.cuh alone, and its host side.
#include <algorithm>

#include "mp_cache_host.h"
#include "mp_prefix_few.cuh"

namespace mp {
namespace {

using namespace few;

constexpr int kWarps = 4, kCtas = 2;  // of a CTA; CTAs of an SM

template <int D>
struct Smem {
  static constexpr int kStages = 3 * (128 / D);
  Ring<D, kStages> ring[kWarps];
  State<kStages> state[kWarps];
  int64_t total[kWarps];
  int least[kWarps];
};

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, kCtas) k_prefix_few(const __grid_constant__ Maps maps, const __grid_constant__ PrefixFew a) {
  extern __shared__ __align__(1024) unsigned char smraw[];
  Smem<D>& S = *reinterpret_cast<Smem<D>*>(smraw + ((1024 - (saddr(smraw) & 1023)) & 1023));
  // the kernel behind this one needs nothing of it before its end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int2* kept = reinterpret_cast<int2*>(&S.ring[0]);
  static_assert(kKept * sizeof(int2) <= sizeof(S.ring));
  int64_t total = 0;
  int least = 0;
  survey<Cutting<NT * 8>>(a, kept, threadIdx.x, kWarps * 32, &total, &least);
  if (lane == 0) {
    S.total[warp] = total;
    S.least[warp] = least;
  }
  __syncthreads();
  total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    total += S.total[i] * a.own.c.kvh;
    least = max(least, S.least[i]);
  }
  work<D, NT, Smem<D>::kStages>(maps, a, S.ring[warp], S.state[warp], kept, total, least, int64_t(blockIdx.x) * kWarps + warp, int64_t(gridDim.x) * kWarps, [] {
    fence_async();
    __syncthreads();
  });
}

template <int D, int NT>
cudaError_t launch(const Maps& maps, const PrefixFew& a, int ctas, cudaStream_t st) {
  const size_t smem = sizeof(Smem<D>) + 1024;
  const cudaError_t e = cudaFuncSetAttribute(k_prefix_few<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  k_prefix_few<D, NT><<<ctas, kWarps * 32, smem, st>>>(maps, a);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_rows(const Maps& maps, const PrefixFew& a, int rows, int ctas, cudaStream_t st) {
  if (rows <= 8) return launch<D, 1>(maps, a, ctas, st);
  if constexpr (D == 64) {
    if (rows > 16) return launch<D, 4>(maps, a, ctas, st);
  }
  return launch<D, 2>(maps, a, ctas, st);
}

}  // namespace

bool few::few_maps(const PrefixFew& a, Maps* maps) {
  const PrefixArgs* both[2] = {&a.pre, &a.own};
  for (int i = 0; i < 2; ++i) {
    const CacheCall& c = both[i]->c;
    const uint64_t pool = uint64_t(c.n_pages) * c.kvh * c.page_size;
    if (!make_map(&maps->k[i], both[i]->keys, c.d, pool, 64, kStep, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&maps->v[i], both[i]->values, c.d, pool, 64, kStep, CU_TENSOR_MAP_SWIZZLE_128B))
      return false;
  }
  return true;
}

cudaError_t launch_prefix_few(const PrefixFew& a, int rows, cudaStream_t st) {
  Maps maps;
  if (!few_maps(a, &maps)) return cudaErrorInvalidValue;
  const PrefixArgs* both[2] = {&a.pre, &a.own};
  const int d = a.own.c.d;
  double steps = 0;
  for (int i = 0; i < 2; ++i) {
    const CacheCall& c = both[i]->c;
    const int units = i ? (a.own_units ? c.batch : 0) : a.groups;
    steps += double(units) * c.kvh * ((int64_t(c.max_q) * c.group + rows - 1) / rows) * ((c.max_kv + kStep - 1) / kStep + kLead);
  }
  const int ctas = int(std::min(double(kCtas) * device_sm_count(), steps / (kMinRun * kWarps) + 1));
  return d == 128 ? launch_rows<128>(maps, a, rows, ctas, st) : launch_rows<64>(maps, a, rows, ctas, st);
}

// K and V are read once for every `rows` rows, from L2 but for the first, and a step of 32 rows is 1 us of a
// warp. The large tiles do better, but a kernel of them starts 10 us later, and the more so the more own slots
// there are beside them. So it goes by the steps. us a call in a graph with blocks and with large tiles for the prefix,
// single tokens with 256 own slots, one group:
//                                      4096 steps     8192          16384         32768
//   d = 128, 32/8 heads,   64 rows     15.0  20.2     18.9  20.4    25.9  21.9    38.1  24.4
//                         128 rows     16.7  21.7     20.1  22.8    25.7  22.6    38.7  25.3
//                         512 rows                    35.5  62.7    39.7  70.0    50.7  52.1
//                        1024 rows                                  61.9  90.5    69.8  99.3
//            16/2 heads,  128 rows     13.8  18.1     17.5  19.7    23.7  21.7    35.5  22.7
//   d = 64,  16/4 heads,   64 rows     11.6  16.6     14.5  17.6    18.5  17.7    27.1  18.5
//                         128 rows     11.9  22.1     14.0  22.4    18.4  23.1    26.1  23.6
//                         512 rows     17.9  23.3     19.5  23.7    23.4  24.0    30.6  23.7
bool prefix_is_few(const mp_cache_config* c, int max_q, int max_kv, int rows) {
  const int64_t all = int64_t(max_q) * (c->q_heads / c->kv_heads), blocks = (all + rows - 1) / rows;
  const int64_t steps = int64_t(c->batch) * c->kv_heads * ((max_kv + kStep - 1) / kStep);
  return double(steps) * double(blocks) <= 16384;
}

// The most pieces that a unit is cut into: as many warps as there are for it, 32 at least, so that one long
// cache among many short ones is shared out too, and fewer where that takes more than 64 MB.
static int64_t pieces_wanted(const mp_cache_config* c, int max_kv) {
  const int64_t warps = int64_t(device_sm_count()) * kCtas * kWarps, steps = (max_kv + kStep - 1) / kStep;
  return std::min(std::max<int64_t>(32, 2 * warps / (int64_t(c->batch) * c->kv_heads) + 2), steps / kMinRun + 2);
}
static int64_t rows_at_most(const mp_cache_config* c) { return (int64_t(64) << 20) / (int64_t(c->q_heads) * c->head_dim * 4); }
int prefix_few_pieces(const mp_cache_config* c, int total_q, int max_kv) {
  return int(std::max<int64_t>(2, std::min(pieces_wanted(c, max_kv), rows_at_most(c) / total_q)));
}
int64_t prefix_few_rows_most(const mp_cache_config* c, int total_q, int max_kv) {
  return std::max<int64_t>(2 * int64_t(total_q), std::min(pieces_wanted(c, max_kv) * total_q, rows_at_most(c)));
}

}  // namespace mp
