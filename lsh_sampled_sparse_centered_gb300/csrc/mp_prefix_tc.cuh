// Prefixes in slices on large tiles, and beside them the own slots: one translation unit for each head size.
#pragma once

#include "mp_chunk_tc.cuh"

namespace mp {
namespace {

template <int D, Mode MODE>
cudaError_t launch_slices(const PrefixArgs& a, const OwnSide& own, int rows, cudaStream_t st) {
  Extra<MODE> x;
  static_cast<OwnSide&>(x) = own;
  const int ctas = device_sm_count();
  return rows <= 8 ? launch<D, MODE, 1>(a, x, a.c.batch, ctas, kRows, nullptr, st)
                   : launch<D, MODE, 2>(a, x, a.c.batch, ctas, kRows, nullptr, st);
}
template <int D>
cudaError_t launch_slices_of(const PrefixArgs& a, const PrefixFew& few, int rows, cudaStream_t st) {
  OwnSide own;
  own.few = few;
  if (!few::few_maps(few, &own.maps)) return cudaErrorInvalidValue;
  return int64_t(a.c.max_q) * a.c.group <= 128 ? launch_slices<D, kPairs>(a, own, rows, st) : launch_slices<D, kCuts>(a, own, rows, st);
}

}  // namespace
}  // namespace mp
