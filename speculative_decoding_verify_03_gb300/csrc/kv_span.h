// kv_span.h -- what the span kernels (kv_span.cuh) take, and the plan that
// they share with the merge kernel (kv_attend.cu).
//
// The attention is cut into items: one tile of RT query rows of one
// key/value head, over one list of pages.  Own items: the rows (i, g) of
// sequence b, r = i * G + g, over the sequence's own tokens.  Prefix items:
// rows of all sequences together, over the shared prefix.  The key tiles (64
// tokens; 128 in the dense kernel) of all items are set out in item order on
// places 0 .. W - 1: side by side, or, for the own items of trees, with a few
// places before each item's tiles for what it costs beside them (cost_of_item).
// CTA c of C <= W works on the tiles whose places are in [W c / C, W (c + 1) / C),
// whatever the items' lengths (where that is no tile, the CTA is idle), and
// leaves one partial result for each item that it touches in slot item + c
// (consecutive CTAs of one item: consecutive slots).  The tile at place x is
// worked on by CTA ((x + 1) C - 1) / W, the largest c with W c / C <= x.
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
  uint32_t *lost;        // per CTA of a dense launch: a wait gave up (null: none ran)
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
  const int32_t *mask;    // trees: [B, N, mask_words]
  bool behind;            // a kernel of the same call was launched before
  int32_t halves;         // dense kernel: 1 where no item has more than 128 rows, else 2
  int32_t mask_words;
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

// The same for trees (own items).
cudaError_t tree_e4m3_64(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t tree_e4m3_80(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t tree_e4m3_96(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t tree_e4m3_128(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t tree_bf16_64(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t tree_bf16_80(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t tree_bf16_96(const SpanParams &, int, int64_t, int *, cudaStream_t);
cudaError_t tree_bf16_128(const SpanParams &, int, int64_t, int *, cudaStream_t);

// Of 64 tokens from place `off` of the step on (below 0: before the step), those
// that a node sees: all before the step, and of the step's n those of its mask row.
__device__ __forceinline__ uint64_t seen_nodes(const int32_t *row, int words, int n, int off) {
  const int i = off >> 5;
  uint32_t x[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) x[k] = i + k < 0 ? ~0u : i + k < words ? static_cast<uint32_t>(__ldg(row + i + k)) : 0u;
  const uint64_t see = static_cast<uint64_t>(__funnelshift_r(x[1], x[2], off & 31)) << 32 | __funnelshift_r(x[0], x[1], off & 31);
  const int left = n - off;
  return left >= 64 ? see : left <= 0 ? 0 : see & ((1ull << left) - 1);
}

// Launches one of the attention kernels.  The second one of a call begins while the
// first still runs, on multiprocessors that are done with it: neither reads what the
// other writes.  It ends behind the first one's end (wait_for_first), so that
// whoever waits for the second waits for both.
template <class F>
cudaError_t launch(F *f, int grid, int threads, int smem, cudaStream_t s, const SpanParams &p) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = p.behind ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, f, p);
}
__device__ __forceinline__ void wait_for_first(const SpanParams &p) {
  if (p.behind) cudaGridDependencySynchronize();
}

// Trees: what an own item costs beside its tiles, in tiles, when work is shared out among
// the CTAs of the span kernel and of the dense one; nothing where every tile can have a
// CTA of its own, or all items are one sequence's and alike.  Measured, us for the call,
// with 0 / 1 / 2 / 3 (dense: / 4), 32 heads of 128 over 8 in e4m3: span kernel, 16 trees of 8
// nodes over 1..2000 tokens 41 / 31 / 28 / 29, 256 over 1..500 138 / 116 / 108 / 110, 8 of 16
// over 8000 87 / 85 / 85 / 88; dense kernel, 16 of 40 over 1..2000 80 / 47 / 43 / 42 / 44, 64
// of 40 over 1..500 104 / 84 / 76 / 76 / 78, 16 of 64 over 2000..8192 111 / 109 / 108 / 106 / 104.
constexpr uint32_t SP_ITEM = 2, DN_ITEM = 3;
__host__ __device__ __forceinline__ uint32_t cost_of_item(uint32_t tiles, uint32_t ctas, int B, uint32_t cost) {
  return tiles > ctas && B > 1 ? cost : 0;
}
// An item's places are its cost, then its tiles.  The first tile at or behind place x, with
// cum0 the tiles before each sequence and cum1 its items.
__device__ __forceinline__ uint32_t tile_at(const View &w, const uint32_t *cum0, const uint32_t *cum1, uint32_t cost, int tokens,
                                            uint32_t x) {
  if (x >= cum0[w.B] + cost * cum1[w.B]) return cum0[w.B];
  int b = 0, r = w.B;
  while (r - b > 1) {
    const int m = (b + r) >> 1;
    if (cum0[m] + cost * cum1[m] <= x) b = m;
    else r = m;
  }
  int own, n;
  row_shape(w, b, own, n);
  const uint32_t nt = (own + n + tokens - 1) / tokens;
  const uint32_t y = x - cum0[b] - cost * cum1[b], j = y / (nt + cost), t = y - j * (nt + cost);
  return cum0[b] + j * nt + (t > cost ? t - cost : 0);
}

// The dense kernel: items of DN_ROWS rows (of the prefix, or own ones of trees), tiles
// of 128 tokens.
constexpr int DN_ROWS = 256;
constexpr int kMaxDense = 152;  // CTAs of the dense kernel at most: one on each multiprocessor
static_assert(kMaxDense <= kMaxGrid, "plan");
cudaError_t dense_e4m3(const SpanParams &, int D, int64_t tiles, int *grid, cudaStream_t);
cudaError_t dense_bf16(const SpanParams &, int D, int64_t tiles, int *grid, cudaStream_t);
// The same over the own tokens of trees.
cudaError_t dense_tree_e4m3(const SpanParams &, int D, int64_t tiles, int *grid, cudaStream_t);
cudaError_t dense_tree_bf16(const SpanParams &, int D, int64_t tiles, int *grid, cudaStream_t);

}  // namespace kv
