// spec_adjust.cu -- penalties for repeated tokens, biases and a grammar's mask on
// the logits of a step.
//
// A CTA takes a slice of the vocabulary and some positions of one sequence.  It
// reads the sequence once and counts the slice's tokens in shared memory (integer
// atomics: the order does not matter), with a flag each for tokens of the prompt
// and of the drafts; the last entry of the bias list for a token is the largest
// index.  A bit per token then says whether anything is to be done at all, so that
// the stream over the logits looks up one bit each and is else a copy.  A draft
// counts at the positions that it comes before: tokens with the drafts' flag (a
// few per slice) go through the list of drafts and the position's mask.
//
// Bound: memory, the logits once in and once out.  The slice is a CTA's share of
// the vocabulary such that the grid fills the machine; each slice reads the whole
// sequence, from L2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "spec_kv.h"
#include "spec_tree.h"

namespace {

constexpr int AJ_NT = 256;         // threads per CTA
constexpr int AJ_SLICE = 8192;     // tokens of a slice at most
constexpr uint32_t kPrompt = 1u << 31, kDraft = 1u << 30, kCount = kDraft - 1;

struct JP {
  spec_adjust_params a;
  const void *in;
  void *out;
  int32_t *status;
  int32_t slice, slices;  // tokens of a slice (a multiple of 32), slices of the vocabulary
  int32_t npos, groups;   // positions of a CTA, groups of positions
  int32_t W;              // words of a tree mask's row
  bool same, vec;         // in place; rows of both equally far from 16 bytes
};

template <bool F32>
struct Elem;
template <>
struct Elem<true> {
  using T = uint32_t;
  static constexpr int VEC = 4;
  static constexpr uint32_t kNan = 0x7fffffffu, kMinf = 0xff800000u;
  static __device__ __forceinline__ float value(uint32_t x) { return __uint_as_float(x); }
  static __device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
};
template <>
struct Elem<false> {
  using T = uint16_t;
  static constexpr int VEC = 8;
  static constexpr uint16_t kNan = 0x7fffu, kMinf = 0xff80u;
  static __device__ __forceinline__ float value(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
  static __device__ __forceinline__ uint16_t bits(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};

// n bits from bit `at` of words (n <= 32, the last word is `last`).
__device__ __forceinline__ uint32_t bits_at(const uint32_t *w, int at, int last) {
  const int i = at >> 5;
  const uint32_t lo = w[i], hi = w[i < last ? i + 1 : i];
  return __funnelshift_r(lo, hi, at & 31);
}

// Shared memory: a word per token of the slice, a bit per token, then (with
// biases) half a word per token; the drafts.
template <bool F32>
__global__ void __launch_bounds__(AJ_NT) adjust_kernel(const __grid_constant__ JP P) {
  using E = Elem<F32>;
  using T = typename E::T;
  constexpr int VEC = E::VEC;
  extern __shared__ uint32_t sm[];
  const spec_adjust_params &a = P.a;
  const int tid = threadIdx.x;
  const int slice = blockIdx.x % P.slices, bg = blockIdx.x / P.slices;
  const int grp = bg % P.groups, b = bg / P.groups;
  const int v0 = slice * P.slice, n = min(P.slice, a.V - v0);
  const int N = a.gamma_max + 1, i0 = grp * P.npos, i1 = min(i0 + P.npos, N);
  uint32_t *count = sm, *touched = count + P.slice;
  uint32_t *bias = touched + P.slice / 32;  // 0: none, else entry + 1
  int32_t *drafts = reinterpret_cast<int32_t *>(bias + (a.n_bias ? P.slice : 0));

  const int g = a.gamma_per_row ? a.gamma_per_row[b] : a.gamma_max;
  const int len = a.seq_len[b], prompt = a.prompt_len ? a.prompt_len[b] : 0;
  const float r = a.repetition ? a.repetition[b] : 1.0f;
  const float f = a.frequency ? a.frequency[b] : 0.0f, p = a.presence ? a.presence[b] : 0.0f;
  int st = g < 0 || g > a.gamma_max ? SPEC_ROW_BAD_GAMMA : 0;
  if (len < 0 || len > a.capacity || prompt < 0 || prompt > len) st |= SPEC_ROW_BAD_LENGTH;
  if (!(r > 0.0f && r < INFINITY) || !(fabsf(f) < INFINITY) || !(fabsf(p) < INFINITY)) st |= SPEC_ROW_BAD_PENALTY;
  if (P.status && slice == 0 && grp == 0 && tid == 0) P.status[b] = st;
  const T *in = static_cast<const T *>(P.in) + b * a.logits_row_stride + v0;
  T *out = static_cast<T *>(P.out) + b * a.out_row_stride + v0;
  if (st) {
    for (int i = i0; i < i1; ++i)
      for (int x = tid; x < n; x += AJ_NT) out[i * a.out_pos_stride + x] = E::kNan;
    return;
  }

  // --- what the slice's tokens have behind them
  for (int x = tid; x < P.slice + P.slice / 32 + (a.n_bias ? P.slice : 0); x += AJ_NT) sm[x] = 0;
  __syncthreads();
  const bool counts = a.repetition || a.frequency || a.presence;
  if (counts) {
    const int32_t *seq = a.seq + b * a.seq_row_stride;
    for (int s0 = tid; s0 < len; s0 += 4 * AJ_NT) {
      int t[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) t[u] = s0 + u * AJ_NT < len ? __ldg(seq + s0 + u * AJ_NT) - v0 : -1;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (static_cast<uint32_t>(t[u]) < static_cast<uint32_t>(n)) {
          if (s0 + u * AJ_NT < prompt) atomicOr(count + t[u], kPrompt);
          else atomicAdd(count + t[u], 1u);
          atomicOr(touched + (t[u] >> 5), 1u << (t[u] & 31));
        }
    }
    for (int j = tid; j < g; j += AJ_NT) {
      const int t = __ldg(a.draft_tokens + static_cast<int64_t>(b) * a.gamma_max + j) - v0;
      drafts[j] = t;
      if (static_cast<uint32_t>(t) < static_cast<uint32_t>(n)) {
        atomicOr(count + t, kDraft);
        atomicOr(touched + (t >> 5), 1u << (t & 31));
      }
    }
  }
  for (int j = tid; j < a.n_bias; j += AJ_NT) {
    const int t = __ldg(a.bias_ids + static_cast<int64_t>(b) * a.n_bias + j) - v0;
    if (static_cast<uint32_t>(t) < static_cast<uint32_t>(n)) {
      atomicMax(bias + t, static_cast<uint32_t>(j + 1));
      atomicOr(touched + (t >> 5), 1u << (t & 31));
    }
  }
  __syncthreads();

  const float *bias_of = a.bias + static_cast<int64_t>(b) * a.n_bias - 1;
  // logit z of the slice's token x at position i
  auto change = [&](float z, int x, int i) {
    const uint32_t c = count[x];
    if (c) {
      uint32_t made = c & kCount;
      if (c & kDraft) {  // rare
        const int32_t *mask = a.tree_mask ? a.tree_mask + (static_cast<int64_t>(b) * N + i) * P.W : nullptr;
        for (int j = 0; j < (mask ? g : min(g, i)); ++j)
          if (drafts[j] == x && (!mask || (mask[(j + 1) >> 5] >> ((j + 1) & 31) & 1))) ++made;
      }
      if (made || (c & kPrompt)) z = z > 0.0f ? __fdiv_rn(z, r) : z * r;
      if (made) z = (z - f * static_cast<float>(made)) - p;
    }
    if (a.n_bias) {
      const uint32_t e = bias[x];
      if (e) z += bias_of[e];
    }
    return z;
  };

  const int last = (a.V - 1) >> 5, tlast = P.slice / 32 - 1;
  for (int i = i0; i < i1; ++i) {
    const T *src = in + i * a.logits_pos_stride;
    T *dst = out + i * a.out_pos_stride;
    const bool live = i <= g;
    if (!live && P.same) break;
    const uint32_t *allowed = a.allowed && live ? reinterpret_cast<const uint32_t *>(a.allowed) + b * a.allowed_row_stride + i * a.allowed_pos_stride : nullptr;
    auto one = [&](int x) {
      T e = src[x];
      if (live && (touched[x >> 5] >> (x & 31) & 1)) e = E::bits(change(E::value(e), x, i));
      if (allowed && !(allowed[(v0 + x) >> 5] >> ((v0 + x) & 31) & 1)) e = E::kMinf;
      dst[x] = e;
    };
    if (!P.vec) {
      for (int x = tid; x < n; x += AJ_NT) one(x);
      continue;
    }
    // up to the first multiple of 16 bytes, and behind the last
    const int head = min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / static_cast<int>(sizeof(T)), n);
    const int chunks = (n - head) / VEC, tail = head + chunks * VEC;
    if (tid < head) one(tid);
    if (tid < n - tail) one(tail + tid);
    for (int c0 = tid; c0 < chunks; c0 += 4 * AJ_NT) {
      uint4 q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c0 + u * AJ_NT < chunks) q[u] = __ldcs(reinterpret_cast<const uint4 *>(src + head) + c0 + u * AJ_NT);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = c0 + u * AJ_NT, x = head + c * VEC;
        if (c >= chunks) break;
        constexpr uint32_t all = (1u << VEC) - 1;
        const uint32_t t = live ? bits_at(touched, x, tlast) & all : 0;
        const uint32_t no = allowed ? ~bits_at(allowed, v0 + x, last) & all : 0;
        if (t | no) {
          T *e = reinterpret_cast<T *>(&q[u]);
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            if (t >> k & 1) e[k] = E::bits(change(E::value(e[k]), x + k, i));
            if (no >> k & 1) e[k] = E::kMinf;
          }
        } else if (P.same) {
          continue;
        }
        __stcs(reinterpret_cast<uint4 *>(dst + head) + c, q[u]);
      }
    }
  }
}

bool aligned(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

}  // namespace

extern "C" spec_status spec_adjust(const void *logits, const spec_adjust_params *params, void *out,
                                   int32_t *row_status, void *stream) {
  if (!params) return SPEC_ERR_INVALID_ARG;
  const spec_adjust_params &a = *params;
  if (a.B < 0 || a.gamma_max < 0 || a.V < 1 || a.V > 1 << 24 || a.capacity < 0 || a.n_bias < 0 ||
      (a.dtype != SPEC_F32 && a.dtype != SPEC_BF16))
    return SPEC_ERR_INVALID_ARG;
  if (a.logits_row_stride < 0 || a.logits_pos_stride < 0 || a.out_row_stride < 0 || a.out_pos_stride < 0 ||
      a.seq_row_stride < 0 || a.allowed_row_stride < 0 || a.allowed_pos_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  const int N = a.gamma_max + 1;
  if (a.gamma_max >= 1 << 20 || a.n_bias > 65534 || a.B > 1 << 20 || (a.tree_mask && N > SPEC_TREE_MAX) ||
      (a.gamma_max > 4096 && (a.repetition || a.presence || a.frequency)))
    return SPEC_ERR_UNSUPPORTED;
  if (a.B == 0) return SPEC_OK;
  const uintptr_t es = a.dtype == SPEC_F32 ? 4 : 2;
  const uintptr_t x = reinterpret_cast<uintptr_t>(logits), y = reinterpret_cast<uintptr_t>(out);
  if (!logits || !out || x % es || y % es || !a.seq_len || (a.capacity > 0 && !a.seq) ||
      (a.gamma_max > 0 && !a.draft_tokens) || (a.n_bias > 0 && (!a.bias_ids || !a.bias)))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(a.seq) || !aligned(a.seq_len) || !aligned(a.prompt_len) || !aligned(a.draft_tokens) ||
      !aligned(a.tree_mask) || !aligned(a.gamma_per_row) || !aligned(a.repetition) || !aligned(a.presence) ||
      !aligned(a.frequency) || !aligned(a.bias_ids) || !aligned(a.bias) || !aligned(a.allowed) || !aligned(row_status))
    return SPEC_ERR_INVALID_ARG;
  // rows of the output must not overlap, nor, in place, be read with other strides
  if ((a.gamma_max > 0 && a.out_pos_stride < a.V) || (a.B > 1 && a.out_row_stride < a.V)) return SPEC_ERR_INVALID_ARG;
  JP P = {};
  P.a = a;
  P.in = logits;
  P.out = out;
  P.status = row_status;
  P.same = x == y;
  if (P.same && ((a.B > 1 && a.logits_row_stride != a.out_row_stride) ||
                 (a.gamma_max > 0 && a.logits_pos_stride != a.out_pos_stride)))
    return SPEC_ERR_INVALID_ARG;
  P.W = (N + 31) / 32;
  const uintptr_t off = (x ^ y) | static_cast<uintptr_t>(a.B > 1 ? (a.logits_row_stride - a.out_row_stride) * static_cast<int64_t>(es) : 0) |
                        static_cast<uintptr_t>(a.gamma_max > 0 ? (a.logits_pos_stride - a.out_pos_stride) * static_cast<int64_t>(es) : 0);
  P.vec = off % 16 == 0;
  // Slices: as many as give the machine some 8 CTAs a multiprocessor, of 1024
  // tokens at least; then positions, down to one.
  const int64_t want = 152 * 8;
  int64_t slices = std::min<int64_t>((want + a.B - 1) / a.B, (a.V + 1023) / 1024);
  slices = std::max<int64_t>(slices, (a.V + AJ_SLICE - 1) / AJ_SLICE);
  P.slice = static_cast<int>(((a.V + slices - 1) / slices + 31) / 32 * 32);
  P.slices = (a.V + P.slice - 1) / P.slice;
  const int64_t have = static_cast<int64_t>(P.slices) * a.B;
  const int64_t groups = std::min<int64_t>(N, std::max<int64_t>(1, want / have));
  P.npos = static_cast<int>((N + groups - 1) / groups);
  P.groups = (N + P.npos - 1) / P.npos;
  const int64_t grid = have * P.groups;
  if (grid > INT32_MAX) return SPEC_ERR_UNSUPPORTED;
  const int smem = (P.slice + P.slice / 32 + (a.n_bias ? P.slice : 0) + std::min(a.gamma_max, 4096)) * 4;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto *k = a.dtype == SPEC_F32 ? adjust_kernel<true> : adjust_kernel<false>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024) != cudaSuccess)
    return SPEC_ERR_CUDA;
  k<<<static_cast<unsigned>(grid), AJ_NT, smem, s>>>(P);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
