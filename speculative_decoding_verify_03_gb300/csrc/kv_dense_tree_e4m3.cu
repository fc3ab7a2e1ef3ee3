// Dense kernels (kv_dense.cuh) over the own tokens of trees, e4m3 cache.
#include "kv_dense.cuh"

namespace kv {
cudaError_t dense_tree_e4m3(const SpanParams &p, int D, int64_t tiles, int *grid, cudaStream_t s) {
  switch (D) {
    case 64: return dense_go<64, true, true>(p, tiles, grid, s);
    case 80: return dense_go<80, true, true>(p, tiles, grid, s);
    case 96: return dense_go<96, true, true>(p, tiles, grid, s);
    default: return dense_go<128, true, true>(p, tiles, grid, s);
  }
}
}  // namespace kv
