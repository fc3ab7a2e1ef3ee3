// Span kernels for trees (kv_span.cuh), e4m3 cache, heads of 64 and 80 elements.
#include "kv_span.cuh"

namespace kv {
cudaError_t tree_e4m3_64(const SpanParams &p, int wr, int64_t tiles, int *grid, cudaStream_t s) {
  return span_any<64, true, true>(p, wr, tiles, grid, s);
}
cudaError_t tree_e4m3_80(const SpanParams &p, int wr, int64_t tiles, int *grid, cudaStream_t s) {
  return span_any<80, true, true>(p, wr, tiles, grid, s);
}
}  // namespace kv
