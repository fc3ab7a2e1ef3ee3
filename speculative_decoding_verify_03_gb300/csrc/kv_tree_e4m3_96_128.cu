// Span kernels for trees (kv_span.cuh), e4m3 cache, heads of 96 and 128 elements.
#include "kv_span.cuh"

namespace kv {
cudaError_t tree_e4m3_96(const SpanParams &p, int wr, int64_t tiles, int *grid, cudaStream_t s) {
  return span_any<96, true, true>(p, wr, tiles, grid, s);
}
cudaError_t tree_e4m3_128(const SpanParams &p, int wr, int64_t tiles, int *grid, cudaStream_t s) {
  return span_any<128, true, true>(p, wr, tiles, grid, s);
}
}  // namespace kv
