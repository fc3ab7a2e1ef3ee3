// kv_common.cuh -- shared by the key/value-cache operators: argument checks
// of the cache and batch descriptors, the resolved (device-side) form of
// both, the opt-in for shared memory, and small device helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "spec_kv.h"

namespace kv {

constexpr int kMaxB = 4096;           // sequences per call
constexpr int kExpMin = -100, kExpMax = 119;

// Cache and batch as kernels take them.
struct View {
  const uint8_t *k, *v;        // pages
  const int8_t *ke, *ve;       // exponents (e4m3)
  int64_t kps, vps;            // page strides in bytes
  const int32_t *table, *ptable, *len, *gam;
  int64_t tstride;
  int32_t B, N, max_pages, prefix, n_pages, Hkv, ps_log2;
};

inline int log2_page(int p) { return p == 16 ? 4 : p == 32 ? 5 : p == 64 ? 6 : p == 128 ? 7 : -1; }

// Checks both descriptors; fills the view.  `step` is false for spec_kv_read
// (no step tokens).
inline spec_status make_view(const spec_kv_cache *c, const spec_kv_batch *b, bool step, View &w) {
  if (!c || !b) return SPEC_ERR_INVALID_ARG;
  if (c->format != SPEC_KV_BF16 && c->format != SPEC_KV_E4M3) return SPEC_ERR_INVALID_ARG;
  if (c->n_pages < 0 || c->n_kv_heads < 1 || c->head_dim < 1 || c->page_size < 1)
    return SPEC_ERR_INVALID_ARG;
  if (b->B < 0 || b->max_pages < 0 || b->prefix_len < 0 || (step && b->gamma_max < 0))
    return SPEC_ERR_INVALID_ARG;
  if (b->table_row_stride < b->max_pages) return SPEC_ERR_INVALID_ARG;
  const int lg = log2_page(c->page_size), D = c->head_dim;
  if (lg < 0 || (D != 64 && D != 80 && D != 96 && D != 128) || b->B > kMaxB)
    return SPEC_ERR_UNSUPPORTED;
  if (c->n_kv_heads > 1024 || (step && b->gamma_max >= (1 << 20)) ||
      static_cast<int64_t>(b->max_pages) * c->page_size > (1 << 30) || b->prefix_len > (1 << 30))
    return SPEC_ERR_UNSUPPORTED;
  const int64_t inner = static_cast<int64_t>(c->n_kv_heads) * c->page_size * D;
  if (c->k_page_stride < inner || c->v_page_stride < inner) return SPEC_ERR_INVALID_ARG;
  const int es = c->format == SPEC_KV_BF16 ? 2 : 1;
  if ((c->k_page_stride * es) % 16 || (c->v_page_stride * es) % 16) return SPEC_ERR_INVALID_ARG;
  if (b->B > 0) {
    if (!c->k_pages || !c->v_pages || !b->kv_len || (b->max_pages > 0 && !b->page_table) ||
        (b->prefix_len > 0 && !b->prefix_table))
      return SPEC_ERR_INVALID_ARG;
    if (es == 1 && (!c->k_exp || !c->v_exp)) return SPEC_ERR_INVALID_ARG;
    const uintptr_t all = reinterpret_cast<uintptr_t>(c->k_pages) |
                          reinterpret_cast<uintptr_t>(c->v_pages) |
                          (es == 1 ? reinterpret_cast<uintptr_t>(c->k_exp) |
                                         reinterpret_cast<uintptr_t>(c->v_exp)
                                   : 0);
    if (all & 15) return SPEC_ERR_INVALID_ARG;
  }
  w.k = static_cast<const uint8_t *>(c->k_pages);
  w.v = static_cast<const uint8_t *>(c->v_pages);
  w.ke = c->k_exp;
  w.ve = c->v_exp;
  w.kps = c->k_page_stride * es;
  w.vps = c->v_page_stride * es;
  w.table = b->page_table;
  w.ptable = b->prefix_table;
  w.len = b->kv_len;
  w.gam = b->gamma_per_row;
  w.tstride = b->table_row_stride;
  w.B = b->B;
  w.N = step ? b->gamma_max + 1 : 0;
  w.max_pages = b->max_pages;
  w.prefix = b->prefix_len;
  w.n_pages = c->n_pages;
  w.Hkv = c->n_kv_heads;
  w.ps_log2 = lg;
  return SPEC_OK;
}

constexpr int kDevices = 64;

// The kernel may use `most` bytes of dynamic shared memory: set once per device, whatever
// the launch at hand needs (beside static shared memory less than 48 KB may be too much
// without it).
inline bool allow_shared(const void *f, int most, std::atomic<bool> *ready) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return false;
  if (ready[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) return false;
  ready[dev].store(true, std::memory_order_release);
  return true;
}

// ------------------------------------------------------------------ device
__device__ __forceinline__ uint32_t s32(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16-byte asynchronous copy to shared memory; fills with zeros when !ok.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
  const int n = ok ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two e4m3 (the low or the high half of r) as two float16.
__device__ __forceinline__ uint32_t cvt_lo(uint32_t r) {
  uint32_t h;
  asm("{.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(h) : "r"(r));
  return h;
}
__device__ __forceinline__ uint32_t cvt_hi(uint32_t r) {
  uint32_t h;
  asm("{.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;}" : "=r"(h) : "r"(r));
  return h;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two floats as e4m3, to nearest even, saturating; stored2: an infinity (which
// e4m3 does not have) to NaN.
__device__ __forceinline__ uint32_t finite2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t stored2(float lo, float hi) {
  const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fffffff);
  return finite2(fabsf(lo) == inf ? nan : lo, fabsf(hi) == inf ? nan : hi);
}
// 2^e as a float, e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Row b of the batch: own tokens before the step, tokens in the step (none
// when N is 0: reading back); the status bits that its lengths give.
__device__ __forceinline__ int row_shape(const View &w, int b, int &own, int &n) {
  const int len = w.len[b];
  int st = 0;
  own = n = 0;
  if (w.N > 0) {
    const int g = w.gam ? w.gam[b] : w.N - 1;
    if (g < 0 || g > w.N - 1) st |= SPEC_ROW_BAD_GAMMA;
    else n = g + 1;
  }
  const int64_t cap = static_cast<int64_t>(w.max_pages) << w.ps_log2;
  if (len < w.prefix || static_cast<int64_t>(len) - w.prefix + n > cap) st |= SPEC_ROW_BAD_LENGTH;
  else own = len - w.prefix;
  if (st) own = n = 0;
  return st;
}

}  // namespace kv
