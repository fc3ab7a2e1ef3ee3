// Span kernels (kv_span.cuh), e4m3 cache, heads of 96 and 128 elements.
#include "kv_span.cuh"

namespace kv {
cudaError_t span_e4m3_96(const SpanParams &p, int wr, int64_t tiles, int *grid, cudaStream_t s) {
  return span_any<96, true>(p, wr, tiles, grid, s);
}
cudaError_t span_e4m3_128(const SpanParams &p, int wr, int64_t tiles, int *grid, cudaStream_t s) {
  return span_any<128, true>(p, wr, tiles, grid, s);
}
}  // namespace kv
