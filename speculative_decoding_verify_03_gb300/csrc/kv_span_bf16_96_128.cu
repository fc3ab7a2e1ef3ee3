// Span kernels (kv_span.cuh), bf16 cache, heads of 96 and 128 elements.
#include "kv_span.cuh"

namespace kv {
cudaError_t span_bf16_96(const SpanParams &p, int wr, int64_t tiles, int *grid, cudaStream_t s) {
  return span_any<96, false>(p, wr, tiles, grid, s);
}
cudaError_t span_bf16_128(const SpanParams &p, int wr, int64_t tiles, int *grid, cudaStream_t s) {
  return span_any<128, false>(p, wr, tiles, grid, s);
}
}  // namespace kv
