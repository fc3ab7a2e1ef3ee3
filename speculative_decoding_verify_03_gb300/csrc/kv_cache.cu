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
// Measured (replayed calls), 8 heads of 128: append 2 x 16384 tokens bfloat16 to
// e4m3 42.4 us (4.8 TB/s, 70 % of a copy's rate), to a bfloat16 cache 42.5 us (6.3
// TB/s, 93 %): as long for more bytes, so the e4m3 form is not held by them.  512 x
// 2..9 tokens float32 7.8 us, to bfloat16 6.5 us; it loads all 9 tokens of each
// sequence, 37.7 MB where 23.1 MB would do, from L2 when replayed.  One token
// 2.0 us.  Read 16 x 8192 tokens to bfloat16 from e4m3 142 us (5.6 TB/s, 83 %), from
// bfloat16 162 us (6.6 TB/s, 97 %).
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

// Largest magnitude of the lane's eight elements as float bits (the order of
// non-negative floats is that of their bits); `finite`: of the finite ones.
template <bool F32>
__device__ __forceinline__ uint32_t most8(const Raw<F32> &r, bool finite) {
  uint32_t m = 0;
  auto take = [&](uint32_t a) { m = max(m, finite && a >= 0x7f800000u ? 0u : a); };
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    const uint32_t u[4] = {r.q[i].x, r.q[i].y, r.q[i].z, r.q[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (F32) {
        take(u[k] & 0x7fffffffu);
      } else {
        take(u[k] & 0x7fff0000u);
        take(u[k] << 16 & 0x7fff0000u);
      }
    }
  }
  return m;
}
template <int LPR>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
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
  uint32_t total;  // rows of a sequence: N * Hkv
  bool vec;
};

// Eight elements times s as e4m3; `odd`: there may be infinities.
__device__ __forceinline__ uint2 store8(const float (&x)[8], float s, bool odd) {
  uint32_t t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    t[i] = odd ? kv::stored2(x[2 * i] * s, x[2 * i + 1] * s) : kv::finite2(x[2 * i] * s, x[2 * i + 1] * s);
  return make_uint2(t[0] | t[1] << 16, t[2] | t[3] << 16);
}

// Grid: rows (t, h) of a sequence, by sequences.  U rows per group of lanes,
// whose loads come first: one where the call is small (latency), four (two of
// float32) where it streams.
template <int D, bool E4M3, bool F32, int U>
__global__ void __launch_bounds__(NT) append_kernel(const __grid_constant__ AP P) {
  constexpr int LPR = D == 64 ? 8 : 16;   // lanes per row
  constexpr int RPC = NT / LPR;           // rows per CTA and pass
  const View &w = P.w;
  const int lane = threadIdx.x % LPR;
  const bool on = lane * 8 < D;
  const uint32_t b = blockIdx.y;
  const uint32_t r0 = blockIdx.x * (RPC * U) + threadIdx.x / LPR;
  Raw<F32> k[U] = {}, v[U] = {};
  uint32_t tok[U], head[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t r = r0 + u * RPC;
    tok[u] = r / w.Hkv;
    head[u] = r - tok[u] * w.Hkv;
    if (r < P.total && on) {
      load8<F32>(P.k.p, b * P.k.s0 + tok[u] * P.k.s1 + head[u] * P.k.s2 + lane * 8, P.vec, k[u]);
      load8<F32>(P.v.p, b * P.v.s0 + tok[u] * P.v.s1 + head[u] * P.v.s2 + lane * 8, P.vec, v[u]);
    }
  }
  int own, n;
  int st = kv::row_shape(w, b, own, n);
  const int32_t *ids = w.table + b * w.tstride;
  if (P.status && blockIdx.x == 0 && threadIdx.x == 0) {
    if (n > 0)
      for (int p = own >> w.ps_log2; p <= (own + n - 1) >> w.ps_log2; ++p)
        if (static_cast<uint32_t>(ids[p]) >= static_cast<uint32_t>(w.n_pages)) st |= SPEC_ROW_BAD_PAGE;
    P.status[b] = st;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int t = static_cast<int>(tok[u]);
    const bool live = r0 + u * RPC < P.total && t < n;
    const int id = live ? __ldg(ids + ((own + t) >> w.ps_log2)) : -1;
    const bool put = static_cast<uint32_t>(id) < static_cast<uint32_t>(w.n_pages);
    const uint32_t at = (head[u] << w.ps_log2) + ((own + t) & ((1 << w.ps_log2) - 1));  // row within the page
    float x[8], y[8];
    values<F32>(k[u], x);
    values<F32>(v[u], y);
    if constexpr (E4M3) {
      uint32_t mk = group_max<LPR>(most8<F32>(k[u], false)), mv = group_max<LPR>(most8<F32>(v[u], false));
      const bool odd = __any_sync(0xffffffffu, max(mk, mv) >= 0x7f800000u);
      if (odd) {  // rare: NaN or infinities among the warp's rows
        mk = group_max<LPR>(most8<F32>(k[u], true));
        mv = group_max<LPR>(most8<F32>(v[u], true));
      }
      const int ek = row_exp(mk), ev = row_exp(mv);
      if (!put) continue;
      if (on) {
        *reinterpret_cast<uint2 *>(P.kp + id * w.kps + at * D + lane * 8) = store8(x, kv::pow2i(-ek), odd);
        *reinterpret_cast<uint2 *>(P.vp + id * w.vps + at * D + lane * 8) = store8(y, kv::pow2i(-ev), odd);
      }
      if (lane == 0) {
        const int64_t s = ((static_cast<int64_t>(id) * w.Hkv) << w.ps_log2) + at;
        P.ke[s] = static_cast<int8_t>(ek);
        P.ve[s] = static_cast<int8_t>(ev);
      }
    } else {
      if (!put || !on) continue;
      *reinterpret_cast<uint4 *>(P.kp + id * w.kps + (at * D + lane * 8) * 2) =
          make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
      *reinterpret_cast<uint4 *>(P.vp + id * w.vps + (at * D + lane * 8) * 2) =
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

unsigned grid_of(uint32_t rows, int D, int B, bool status) {
  const uint32_t rpc = NT / (D == 64 ? 8 : 16);
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
  const int64_t rows = static_cast<int64_t>(P.w.N) * P.w.Hkv;
  if (rows >= INT32_MAX / 2) return SPEC_ERR_UNSUPPORTED;
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
  // Several rows per group of lanes once the call fills the machine twice over.
  const uint32_t rpc = NT / (cache->head_dim == 64 ? 8 : 16);
  const uint32_t u = rows * P.w.B >= 2ll * 152 * 8 * rpc ? (f ? 2 : 4) : 1;
  const dim3 grid((P.total + rpc * u - 1) / (rpc * u), P.w.B);
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
  const unsigned grid = grid_of(P.total, cache->head_dim, P.w.B, row_status != nullptr);
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
