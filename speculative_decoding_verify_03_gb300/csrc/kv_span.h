// kv_span.h -- what the span kernels (kv_span.cuh) take, and the plan that
// they share with the merge kernel (kv_attend.cu).
//
// The attention is cut into items: one tile of RT query rows of one
// key/value head, over one list of pages.  Own items: the rows (i, g) of
// sequence b, r = i * G + g, over the sequence's own tokens.  Prefix items:
// rows of all sequences together, over the shared prefix.  The key tiles (64
// tokens) of all items, in item order, are numbered 0 .. W - 1; CTA c of C <= W
// works on tiles [W c / C, W (c + 1) / C) whatever the items' lengths, and
// leaves one partial result for each item that it touches in slot item + c
// (consecutive CTAs of one item: consecutive slots).
#pragma once

#include <atomic>

#include "kv_common.cuh"

namespace kv {

constexpr int kTile = 64;      // key tokens per tile
constexpr int kMaxGrid = 640;  // CTAs of a span kernel at most

struct Plan {            // device arrays of B + 1 words
  uint32_t *tiles;       // own: key tiles of the sequences before b
  uint32_t *items;       // own: items of the sequences before b
  uint32_t *rows;        // prefix: query rows (per key/value head) before b
  uint32_t *lost;        // prefix, per CTA: a wait gave up (null: no kernel with waits ran)
};

struct SpanParams {
  View w;
  const __nv_bfloat16 *q;
  int64_t qs0, qs1, qs2;  // strides in elements
  float *po, *pl;         // partial outputs [slot, RT, D], log2-sum-exps [slot, RT]
  Plan plan;
  float c;                // scale * log2 e
  int32_t G;              // query heads per key/value head
  int32_t prefix;         // 1: prefix items
  bool qvec;              // q rows are 4-byte aligned; 16-byte (dense kernel, 16 rows)
};

constexpr int kSmSmem = 228 * 1024;  // shared memory of an SM; 1 KB of it a CTA's own

// Multiprocessors and resident CTAs (at `smem` bytes) of one kernel, asked of
// the runtime once per device; sets the kernel's shared memory limit.
struct Slots {
  static constexpr int kDevices = 64;
  std::atomic<int> sms[kDevices] = {}, occ[kDevices] = {};
  cudaError_t get(const void *f, int threads, int smem, int most, int *n, int *per) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    *n = sms[dev].load(std::memory_order_acquire);
    if (*n == 0) {
      int s = 0, o = 0;
      if ((e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, most)) != cudaSuccess) return e;
      if ((e = cudaDeviceGetAttribute(&s, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
      if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o, f, threads, smem)) != cudaSuccess) return e;
      occ[dev].store(o > 0 ? o : 1, std::memory_order_relaxed);
      sms[dev].store(s, std::memory_order_release);
      *n = s;
    }
    *per = occ[dev].load(std::memory_order_relaxed);
    return cudaSuccess;
  }
};

// Launches the span kernel for RT = 16 * wr rows (wr 1 .. 4) on at most
// `tiles` CTAs; returns the CTAs used in *grid.
typedef cudaError_t (*span_launch_fn)(const SpanParams &p, int wr, int64_t tiles, int *grid,
                                      cudaStream_t s);
cudaError_t span_e4m3_64(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t span_e4m3_80(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t span_e4m3_96(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t span_e4m3_128(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t span_bf16_64(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t span_bf16_80(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t span_bf16_96(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t span_bf16_128(const SpanParams &, int, int64_t, int *, cudaStream_t);

// The dense kernel: prefix items of DN_ROWS rows, tiles of 128 tokens.
constexpr int DN_ROWS = 256;
constexpr int kMaxDense = 152;  // CTAs of the dense kernel at most: one on each multiprocessor
static_assert(kMaxDense <= kMaxGrid, "plan");
cudaError_t dense_e4m3(const SpanParams &, int D, int64_t tiles, int *grid, cudaStream_t);
cudaError_t dense_bf16(const SpanParams &, int D, int64_t tiles, int *grid, cudaStream_t);

// The CTA that works on tile x of W (C <= W CTAs): the largest c with W c / C <= x.
__host__ __device__ __forceinline__ uint32_t owner(uint32_t x, uint32_t W, uint32_t C) {
  if (W < (1u << 22)) return ((x + 1) * C - 1) / W;  // C <= 640: no overflow
  return static_cast<uint32_t>(((static_cast<uint64_t>(x) + 1) * C - 1) / W);
}

}  // namespace kv
