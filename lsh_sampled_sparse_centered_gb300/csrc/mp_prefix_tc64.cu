#include "mp_prefix_tc.cuh"

namespace mp {
cudaError_t launch_prefix_slices_64(const PrefixArgs& a, const PrefixFew& few, int rows, cudaStream_t st) {
  return launch_slices_of<64>(a, few, rows, st);
}
}  // namespace mp
