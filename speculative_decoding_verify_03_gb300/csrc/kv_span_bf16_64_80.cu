// Span kernels (kv_span.cuh), bf16 cache, heads of 64 and 80 elements.
#include "kv_span.cuh"

namespace kv {
cudaError_t span_bf16_64(const SpanParams &p, int wr, int64_t tiles, int *grid, cudaStream_t s) {
  return span_any<64, false>(p, wr, tiles, grid, s);
}
cudaError_t span_bf16_80(const SpanParams &p, int wr, int64_t tiles, int *grid, cudaStream_t s) {
  return span_any<80, false>(p, wr, tiles, grid, s);
}
}  // namespace kv
