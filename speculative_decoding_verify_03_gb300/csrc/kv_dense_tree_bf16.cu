// Dense kernels (kv_dense.cuh) over the own tokens of trees, bf16 cache.
#include "kv_dense.cuh"

namespace kv {
cudaError_t dense_tree_bf16(const SpanParams &p, int D, int64_t tiles, int *grid, cudaStream_t s) {
  switch (D) {
    case 64: return dense_go<64, false, true>(p, tiles, grid, s);
    case 80: return dense_go<80, false, true>(p, tiles, grid, s);
    case 96: return dense_go<96, false, true>(p, tiles, grid, s);
    default: return dense_go<128, false, true>(p, tiles, grid, s);
  }
}
}  // namespace kv
