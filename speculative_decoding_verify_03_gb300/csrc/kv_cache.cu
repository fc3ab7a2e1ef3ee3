// kv_cache.cu -- write a step's keys and values to the paged cache (e4m3 with
// a power-of-two exponent for each token and head, or bfloat16) and read them
// back.
//
// Mathematics: e = least integer in [-100, 119] with max|x| <= 448 * 2^e, read
// off the bits of the row's largest finite magnitude; y = e4m3(x * 2^-e).
// The scale is a power of two, so x * 2^-e is exact and each value is rounded
// once; e4m3 is a floating format, so a finer scale would gain nothing but in
// its subnormals, 2^-15 and less of the row's maximum.
//
// Bound: memory.  One token and head (64 .. 128 elements) is a group of 8 or
// 16 lanes with 8 elements each: 16-byte loads of bfloat16, one shuffle
// reduction of 3 or 4 steps for the maximum, 8-byte stores of e4m3.  Keys and
// values go through the same thread, so that four independent loads are in
// flight before the first use.
#include <cuda_fp16.h>

#include <type_traits>

#include "kv_common.cuh"

namespace {

using kv::View;

constexpr int NT = 256;  // threads per CTA

struct Rows {  // a tensor [B, n, Hkv, D] with strides in elements
  const void *p;
  int64_t s0, s1, s2;
};

// Eight elements of a source row as they are; `vec`: 16-byte aligned.
template <bool F32>
struct Raw {
  uint4 q[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ void load8(const void *base, int64_t off, bool vec, Raw<F32> &r) {
  if constexpr (F32) {
    const float *p = static_cast<const float *>(base) + off;
    if (vec) {
      r.q[0] = __ldcs(reinterpret_cast<const uint4 *>(p));
      r.q[1] = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
    } else {
      const uint32_t *u = reinterpret_cast<const uint32_t *>(p);
      r.q[0] = make_uint4(u[0], u[1], u[2], u[3]);
      r.q[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
  } else {
    const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(base) + off;
    if (vec) {
      r.q[0] = __ldcs(reinterpret_cast<const uint4 *>(p));
    } else {
      const uint16_t *u = reinterpret_cast<const uint16_t *>(p);
      r.q[0] = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
    }
  }
}
template <bool F32>
__device__ __forceinline__ void values(const Raw<F32> &r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    const uint32_t u[4] = {r.q[i].x, r.q[i].y, r.q[i].z, r.q[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (F32) {
        x[4 * i + k] = __uint_as_float(u[k]);
      } else {
        x[2 * k] = __uint_as_float(u[k] << 16);
        x[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&t);
}

// Largest finite magnitude of the row as bits (the order of non-negative
// floats is that of their bits); lanes of a group of LPR hold 8 elements each.
template <int LPR>
__device__ __forceinline__ uint32_t row_max(const float (&x)[8], bool on) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(x[i]) & 0x7fffffffu;
    m = max(m, a < 0x7f800000u ? a : 0u);
  }
  if (!on) m = 0;
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

__device__ __forceinline__ int row_exp(uint32_t m) {
  const int k = static_cast<int>(m >> 23) - 127;  // m = 1.f * 2^k; 448 = 1.75 * 2^8
  const int e = k - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kv::kExpMin), kv::kExpMax);
}

struct AP {
  View w;
  Rows k, v;
  uint8_t *kp, *vp;
  int8_t *ke, *ve;
  int32_t *status;
  uint32_t total;  // rows: B * N * Hkv
  bool vec;
};

// U rows per group of lanes, whose loads come first: one where the call is
// small (latency), four (two of float32) where it streams.
template <int D, bool E4M3, bool F32, int U>
__global__ void __launch_bounds__(NT) append_kernel(const __grid_constant__ AP P) {
  constexpr int LPR = D == 64 ? 8 : 16;   // lanes per row
  constexpr int RPC = NT / LPR;           // rows per CTA and pass
  const View &w = P.w;
  const int lane = threadIdx.x % LPR;
  const bool on = lane * 8 < D;
  if (P.status) {  // one thread per sequence reports
    const uint32_t b = blockIdx.x * NT + threadIdx.x;
    if (b < static_cast<uint32_t>(w.B)) {
      int own, n;
      int st = kv::row_shape(w, b, own, n);
      const int32_t *t = w.table + b * w.tstride;
      if (n > 0)
        for (int p = own >> w.ps_log2; p <= (own + n - 1) >> w.ps_log2; ++p)
          if (static_cast<uint32_t>(t[p]) >= static_cast<uint32_t>(w.n_pages))
            st |= SPEC_ROW_BAD_PAGE;
      P.status[b] = st;
    }
  }
  const uint32_t r0 = blockIdx.x * (RPC * U) + threadIdx.x / LPR;
  if (blockIdx.x * static_cast<uint64_t>(RPC * U) >= P.total) return;  // a CTA for status only
  Raw<F32> k[U], v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = r0 + u * RPC;
    if (r < P.total && on) {
      const uint32_t h = r % w.Hkv, bt = r / w.Hkv, t = bt % w.N, b = bt / w.N;
      load8<F32>(P.k.p, b * P.k.s0 + t * P.k.s1 + h * P.k.s2 + lane * 8, P.vec, k[u]);
      load8<F32>(P.v.p, b * P.v.s0 + t * P.v.s1 + h * P.v.s2 + lane * 8, P.vec, v[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = r0 + u * RPC, h = r % w.Hkv, bt = r / w.Hkv, t = bt % w.N, b = bt / w.N;
    bool live = r < P.total;
    int own = 0, n = 0, page = -1;
    if (live) kv::row_shape(w, b, own, n);
    live = live && t < static_cast<uint32_t>(n);
    if (live) page = w.table[b * w.tstride + ((own + static_cast<int>(t)) >> w.ps_log2)];
    live = live && static_cast<uint32_t>(page) < static_cast<uint32_t>(w.n_pages);
    const int slot = (own + static_cast<int>(t)) & ((1 << w.ps_log2) - 1);
    const int64_t at = (static_cast<int64_t>(h) << w.ps_log2) + slot;  // row within the page
    float x[8], y[8];
    values<F32>(k[u], x);
    values<F32>(v[u], y);
    if constexpr (E4M3) {
      const int ek = row_exp(row_max<LPR>(x, live && on)), ev = row_exp(row_max<LPR>(y, live && on));
      if (!live) continue;
      if (on) {
        const float sk = kv::pow2i(-ek), sv = kv::pow2i(-ev);
        uint2 a, c;
        a.x = kv::stored2(x[0] * sk, x[1] * sk) | kv::stored2(x[2] * sk, x[3] * sk) << 16;
        a.y = kv::stored2(x[4] * sk, x[5] * sk) | kv::stored2(x[6] * sk, x[7] * sk) << 16;
        c.x = kv::stored2(y[0] * sv, y[1] * sv) | kv::stored2(y[2] * sv, y[3] * sv) << 16;
        c.y = kv::stored2(y[4] * sv, y[5] * sv) | kv::stored2(y[6] * sv, y[7] * sv) << 16;
        *reinterpret_cast<uint2 *>(P.kp + page * w.kps + at * D + lane * 8) = a;
        *reinterpret_cast<uint2 *>(P.vp + page * w.vps + at * D + lane * 8) = c;
      }
      if (lane == 0) {
        const int64_t s = ((static_cast<int64_t>(page) * w.Hkv) << w.ps_log2) + at;
        P.ke[s] = static_cast<int8_t>(ek);
        P.ve[s] = static_cast<int8_t>(ev);
      }
    } else {
      if (!live || !on) continue;
      *reinterpret_cast<uint4 *>(P.kp + page * w.kps + (at * D + lane * 8) * 2) =
          make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
      *reinterpret_cast<uint4 *>(P.vp + page * w.vps + (at * D + lane * 8) * 2) =
          make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
    }
  }
}

struct RP {
  View w;
  void *k, *v;
  int32_t *status;
  uint32_t total;  // rows: B * n * Hkv
  int32_t begin, n;
  bool vec;
};

template <bool E4M3>
__device__ __forceinline__ void fetch8(const uint8_t *p, float s, float (&x)[8]) {
  if constexpr (E4M3) {
    const uint2 a = __ldg(reinterpret_cast<const uint2 *>(p));
    const uint32_t u[2] = {a.x, a.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t two = static_cast<uint16_t>(u[i >> 1] >> ((i & 1) * 16));
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
      x[2 * i] = f.x * s;
      x[2 * i + 1] = f.y * s;
    }
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void *base, int64_t off, bool vec, const float (&x)[8]) {
  if constexpr (F32) {
    float *p = static_cast<float *>(base) + off;
    if (vec) {
      __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
      __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = x[i];
    }
  } else {
    __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(base) + off;
    if (vec) {
      __stcs(reinterpret_cast<uint4 *>(p),
             make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                        pack_bf16(x[6], x[7])));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = __float2bfloat16(x[i]);
    }
  }
}

template <int D, bool E4M3, bool F32>
__global__ void __launch_bounds__(NT) read_kernel(const __grid_constant__ RP P) {
  constexpr int LPR = D == 64 ? 8 : 16;
  constexpr int RPC = NT / LPR;
  constexpr int ES = E4M3 ? 1 : 2;
  const View &w = P.w;
  if (P.status) {
    const uint32_t b = blockIdx.x * NT + threadIdx.x;
    if (b < static_cast<uint32_t>(w.B)) {
      int own, n;
      int st = kv::row_shape(w, b, own, n);
      const uint32_t np = static_cast<uint32_t>(w.n_pages);
      const int last = st ? 0 : min(w.len[b], P.begin + P.n);  // positions begin .. last - 1
      for (int p = P.begin >> w.ps_log2; (p << w.ps_log2) < min(last, w.prefix); ++p)
        if (static_cast<uint32_t>(w.ptable[p]) >= np) st |= SPEC_ROW_BAD_PAGE;
      for (int p = max(P.begin - w.prefix, 0) >> w.ps_log2; (p << w.ps_log2) < last - w.prefix; ++p)
        if (static_cast<uint32_t>(w.table[b * w.tstride + p]) >= np) st |= SPEC_ROW_BAD_PAGE;
      P.status[b] = st;
    }
  }
  const int lane = threadIdx.x % LPR;
  const uint32_t r = blockIdx.x * RPC + threadIdx.x / LPR;
  if (lane * 8 >= D || r >= P.total) return;
  const uint32_t h = r % w.Hkv, bt = r / w.Hkv;
  const int t = static_cast<int>(bt % P.n) + P.begin;
  const uint32_t b = bt / P.n;
  float x[8] = {}, y[8] = {};
  int own, n;
  bool bad = kv::row_shape(w, b, own, n) != 0;
  if (!bad && t < w.len[b]) {
    const int p = t < w.prefix ? t : t - w.prefix;
    const int page =
        t < w.prefix ? w.ptable[p >> w.ps_log2] : w.table[b * w.tstride + (p >> w.ps_log2)];
    bad = static_cast<uint32_t>(page) >= static_cast<uint32_t>(w.n_pages);
    if (!bad) {
      const int64_t at = (static_cast<int64_t>(h) << w.ps_log2) + (p & ((1 << w.ps_log2) - 1));
      float sk = 1.0f, sv = 1.0f;
      if constexpr (E4M3) {
        const int64_t s = ((static_cast<int64_t>(page) * w.Hkv) << w.ps_log2) + at;
        sk = kv::pow2i(w.ke[s]);
        sv = kv::pow2i(w.ve[s]);
      }
      fetch8<E4M3>(w.k + page * w.kps + (at * D + lane * 8) * ES, sk, x);
      fetch8<E4M3>(w.v + page * w.vps + (at * D + lane * 8) * ES, sv, y);
    }
  }
  if (bad) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = __int_as_float(0x7fffffff);
  }
  const int64_t o = static_cast<int64_t>(r) * D + lane * 8;
  store8<F32>(P.k, o, P.vec, x);
  store8<F32>(P.v, o, P.vec, y);
}

// Calls f with the head size as a compile-time constant.
template <class F>
void by_head(int D, F f) {
  if (D == 64) f(std::integral_constant<int, 64>());
  else if (D == 80) f(std::integral_constant<int, 80>());
  else if (D == 96) f(std::integral_constant<int, 96>());
  else f(std::integral_constant<int, 128>());
}

// Rows per group of lanes: several once the call fills the machine twice over.
int rows_per_group(uint32_t rows, int D, int most) {
  return rows >= 2u * 152 * 8 * (NT / (D == 64 ? 8 : 16)) ? most : 1;
}

unsigned grid_of(uint32_t rows, int D, int B, bool status, int u) {
  const uint32_t rpc = NT / (D == 64 ? 8 : 16) * u;
  const uint32_t g = (rows + rpc - 1) / rpc, s = status ? (B + NT - 1) / NT : 0;
  return g > s ? g : s;
}

}  // namespace

extern "C" spec_status spec_kv_append(const spec_kv_cache *cache, const spec_kv_batch *batch,
                                      const void *k, const void *v, int32_t dtype,
                                      const int64_t *k_strides, const int64_t *v_strides,
                                      int32_t *row_status, void *stream) {
  AP P = {};
  const spec_status st = kv::make_view(cache, batch, true, P.w);
  if (st != SPEC_OK) return st;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (!k_strides || !v_strides) return SPEC_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (k_strides[i] < 0 || v_strides[i] < 0) return SPEC_ERR_INVALID_ARG;
  if (P.w.B == 0) return SPEC_OK;
  const uintptr_t es = dtype == SPEC_F32 ? 4 : 2;
  if (!k || !v || reinterpret_cast<uintptr_t>(k) % es || reinterpret_cast<uintptr_t>(v) % es)
    return SPEC_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(P.w.B) * P.w.N * P.w.Hkv;
  if (rows >= INT32_MAX) return SPEC_ERR_UNSUPPORTED;
  uintptr_t bits = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v);
  for (int i = 0; i < 3; ++i) bits |= static_cast<uintptr_t>(k_strides[i] | v_strides[i]) * es;
  P.vec = bits % 16 == 0;
  P.k = {k, k_strides[0], k_strides[1], k_strides[2]};
  P.v = {v, v_strides[0], v_strides[1], v_strides[2]};
  P.kp = static_cast<uint8_t *>(cache->k_pages);
  P.vp = static_cast<uint8_t *>(cache->v_pages);
  P.ke = cache->k_exp;
  P.ve = cache->v_exp;
  P.status = row_status;
  P.total = static_cast<uint32_t>(rows);
  const bool q = cache->format == SPEC_KV_E4M3, f = dtype == SPEC_F32;
  const int u = rows_per_group(P.total, cache->head_dim, f ? 2 : 4);
  const unsigned grid = grid_of(P.total, cache->head_dim, P.w.B, row_status != nullptr, u);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  by_head(cache->head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (q && f) u > 1 ? append_kernel<D, true, true, 2><<<grid, NT, 0, s>>>(P) : append_kernel<D, true, true, 1><<<grid, NT, 0, s>>>(P);
    else if (q) u > 1 ? append_kernel<D, true, false, 4><<<grid, NT, 0, s>>>(P) : append_kernel<D, true, false, 1><<<grid, NT, 0, s>>>(P);
    else if (f) u > 1 ? append_kernel<D, false, true, 2><<<grid, NT, 0, s>>>(P) : append_kernel<D, false, true, 1><<<grid, NT, 0, s>>>(P);
    else u > 1 ? append_kernel<D, false, false, 4><<<grid, NT, 0, s>>>(P) : append_kernel<D, false, false, 1><<<grid, NT, 0, s>>>(P);
  });
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

extern "C" spec_status spec_kv_read(const spec_kv_cache *cache, const spec_kv_batch *batch,
                                    int32_t begin, int32_t n, int32_t dtype, void *k_out,
                                    void *v_out, int32_t *row_status, void *stream) {
  RP P = {};
  const spec_status st = kv::make_view(cache, batch, false, P.w);
  if (st != SPEC_OK) return st;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (begin < 0 || n < 0 || static_cast<int64_t>(begin) + n > (1 << 30)) return SPEC_ERR_INVALID_ARG;
  if (P.w.B == 0 || n == 0) return SPEC_OK;
  const uintptr_t es = dtype == SPEC_F32 ? 4 : 2;
  if (!k_out || !v_out || reinterpret_cast<uintptr_t>(k_out) % es ||
      reinterpret_cast<uintptr_t>(v_out) % es)
    return SPEC_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(P.w.B) * n * P.w.Hkv;
  if (rows >= INT32_MAX) return SPEC_ERR_UNSUPPORTED;
  P.vec = (reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) % 16 == 0;
  P.k = k_out;
  P.v = v_out;
  P.status = row_status;
  P.total = static_cast<uint32_t>(rows);
  P.begin = begin;
  P.n = n;
  const unsigned grid = grid_of(P.total, cache->head_dim, P.w.B, row_status != nullptr, 1);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool q = cache->format == SPEC_KV_E4M3, f = dtype == SPEC_F32;
  by_head(cache->head_dim, [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (q && f) read_kernel<D, true, true><<<grid, NT, 0, s>>>(P);
    else if (q) read_kernel<D, true, false><<<grid, NT, 0, s>>>(P);
    else if (f) read_kernel<D, false, true><<<grid, NT, 0, s>>>(P);
    else read_kernel<D, false, false><<<grid, NT, 0, s>>>(P);
  });
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
