// spec_adjust.cu -- penalties for repeated tokens, biases and a grammar's mask on
// the logits of a step.
//
// A CTA takes a slice of the vocabulary and some positions of one sequence.  It
// reads the sequence once and counts the slice's tokens in shared memory (integer
// atomics: the order does not matter), with a flag each for tokens of the prompt
// and of the drafts; the last entry of the bias list for a token is the largest
// index.  Tokens with any of these go on a list.  The stream over the logits is
// then a copy that knows the mask alone, and the listed tokens are changed behind
// it, one by one, from the logits as they were: their lines are still in L2, and no
// branch of the stream depends on the data.  In place
// there is no stream but the mask's.  A draft counts at the positions that it
// comes before: tokens with the drafts' flag (a few per slice) go through the list
// of drafts and the position's mask.
//
// Bound: memory, the logits once in and once out.  The slice is a CTA's share of
// the vocabulary such that the grid fills the machine; each slice reads the whole
// sequence, from L2.  Measured (replayed calls): 32 x 31 rows of 152064 in bfloat16 with
// penalties, biases and a mask for every row 114 us, 5.5 TB/s, 81 % of a copy's rate;
// 64 x 5 rows of 50304 in float32 29 us (a plain copy of them 22.6); one
// row of 50304 3.6 us.  More warps a multiprocessor (fewer registers) or wider slices
// lose: 123 to 170 us for the first.  That every slice reads the whole sequence shows where
// those are long: sequences of 200 / 2000 / 8000 / 65536 tokens, penalties alone, one row of
// 50304 3.7 / 4.4 / 7.5 / 19.6 us, 64 x 5 of 50304 26 / 27 / 40 / 111, 32 x 31 of 152064 106 / 140 /
// 180 / 341; the same in place 4.0 / 4.4 / 7.7 / 19.0, 15 / 20 / 32 / 86, 22 / 44 / 97 / 249.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kv_common.cuh"
#include "spec_tree.h"

namespace {

constexpr int AJ_NT = 256;           // threads per CTA
constexpr int AJ_SLICE = 8192;       // tokens of a slice at most
constexpr int AJ_DRAFTS = 4096;      // drafts of a sequence at most, where they are counted
constexpr int AJ_SMEM = AJ_SLICE * 10 + AJ_DRAFTS * 4;  // dynamic shared memory of a CTA at most
constexpr int AJ_COUNT = 128;        // of them counting, while the others begin with the stream;
constexpr int AJ_LONG = 16384;       // all of them for sequences of this length
constexpr int AJ_UNROLL = 4;         // loads of a thread in flight together: of the stream,
constexpr int AJ_SPARSE = 2;         // of a listed token (positions)
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

// The lanes of a 32-bit word that hold elements whose bits are set in `no`
// (VEC 4: one element, VEC 8: two).
template <bool F32>
__device__ __forceinline__ uint32_t masked(uint32_t x, uint32_t no) {
  if constexpr (F32) return no & 1 ? 0xff800000u : x;
  const uint32_t m = (no & 1 ? 0xffffu : 0u) | (no & 2 ? 0xffff0000u : 0u);
  return (x & ~m) | (0xff80ff80u & m);
}

// Shared memory: a word per token of the slice, (with biases) another one, a list
// of tokens, the drafts.
template <bool F32>
__global__ void __launch_bounds__(AJ_NT) adjust_kernel(const __grid_constant__ JP P) {
  using E = Elem<F32>;
  using T = typename E::T;
  constexpr int VEC = E::VEC, U = AJ_UNROLL, S = AJ_SPARSE;
  extern __shared__ __align__(16) uint32_t sm[];
  __shared__ uint32_t listed, next;  // tokens on the list; next part of the stream
  const spec_adjust_params &a = P.a;
  const int tid = threadIdx.x, lane = tid & 31;
  // the low tokens first: they are the frequent ones, and have the longest lists
  const int bg = blockIdx.x % (a.B * P.groups), slice = blockIdx.x / (a.B * P.groups);
  const int grp = bg % P.groups, b = bg / P.groups;
  const int v0 = slice * P.slice, n = min(P.slice, a.V - v0);
  const int N = a.gamma_max + 1, i0 = grp * P.npos, i1 = min(i0 + P.npos, N);
  uint32_t *count = sm, *bias = count + P.slice;  // bias: 0: none, else entry + 1
  uint16_t *list = reinterpret_cast<uint16_t *>(bias + (a.n_bias ? P.slice : 0));
  int32_t *drafts = reinterpret_cast<int32_t *>(list + P.slice);
  const bool counts = a.repetition || a.frequency || a.presence;

  if (tid == 0) listed = 0, next = 0;
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
  __syncthreads();

  // --- what the slice's tokens have behind them, by the first warps; the others
  // begin with the stream
  const int nc = len < AJ_LONG ? AJ_COUNT : AJ_NT;  // threads that count
  if (tid < nc && (counts || a.n_bias)) {
    auto meet = [&] { asm volatile("bar.sync 1, %0;" ::"r"(nc) : "memory"); };
    for (int x = tid; x < P.slice * (a.n_bias ? 2 : 1) / 4; x += nc)
      reinterpret_cast<uint4 *>(sm)[x] = make_uint4(0, 0, 0, 0);
    meet();
    if (counts) {
      const int32_t *seq = a.seq + b * a.seq_row_stride;
      auto see = [&](int t, int s) {  // token t of the sequence's place s
        const uint32_t x = static_cast<uint32_t>(t) - v0;
        if (x >= static_cast<uint32_t>(n)) return;
        if (s < prompt) atomicOr(count + x, kPrompt);
        else atomicAdd(count + x, 1u);
      };
      // four tokens at a time from the first multiple of 16 bytes on, four such loads in flight
      constexpr int K = 4;
      const int first = min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(seq) & 15)) & 15) / 4, len), quads = (len - first) / 4;
      for (int s = tid; s < first; s += nc) see(__ldg(seq + s), s);
      for (int s = first + 4 * quads + tid; s < len; s += nc) see(__ldg(seq + s), s);
      for (int q0 = tid; q0 < quads; q0 += K * nc) {
        int4 t[K];
#pragma unroll
        for (int u = 0; u < K; ++u)
          if (q0 + u * nc < quads) t[u] = __ldg(reinterpret_cast<const int4 *>(seq + first) + q0 + u * nc);
#pragma unroll
        for (int u = 0; u < K; ++u) {
          const int s = first + 4 * (q0 + u * nc);
          if (q0 + u * nc < quads) see(t[u].x, s), see(t[u].y, s + 1), see(t[u].z, s + 2), see(t[u].w, s + 3);
        }
      }
      for (int j = tid; j < g; j += nc) {
        const uint32_t t = static_cast<uint32_t>(__ldg(a.draft_tokens + static_cast<int64_t>(b) * a.gamma_max + j)) - v0;
        drafts[j] = static_cast<int32_t>(t);
        if (t < static_cast<uint32_t>(n)) atomicOr(count + t, kDraft);
      }
    }
    for (int j = tid; j < a.n_bias; j += nc) {
      const uint32_t t = static_cast<uint32_t>(__ldg(a.bias_ids + static_cast<int64_t>(b) * a.n_bias + j)) - v0;
      if (t < static_cast<uint32_t>(n)) atomicMax(bias + t, static_cast<uint32_t>(j + 1));
    }
    meet();
    for (int x0 = tid & ~31; x0 < n; x0 += nc) {  // 32 tokens' places side by side, so that their accesses are too
      const int x = x0 + lane;
      const bool on = x < n && (count[x] || (a.n_bias && bias[x]));
      const uint32_t all = __ballot_sync(~0u, on);
      uint32_t at = 0;
      if (lane == 0 && all) at = atomicAdd(&listed, __popc(all));
      at = __shfl_sync(~0u, at, 0);
      if (on) list[at + __popc(all & ((1u << lane) - 1))] = static_cast<uint16_t>(x);
    }
  }

  // --- the stream, in parts of 32 U x 16 bytes of a position, a warp each
  const uint32_t *allowed = a.allowed ? reinterpret_cast<const uint32_t *>(a.allowed) + b * a.allowed_row_stride : nullptr;
  const int last = (a.V - 1) >> 5;
  auto banned = [&](int i, int x) {  // token x of the slice at position i
    return allowed && i <= g && !(allowed[i * a.allowed_pos_stride + ((v0 + x) >> 5)] >> ((v0 + x) & 31) & 1);
  };
  const int end = P.same ? (allowed ? min(i1, g + 1) : i0) : i1;
  const int per = (n + 32 * U * VEC - 1) / (32 * U * VEC), parts = max(end - i0, 0) * per;
  for (;;) {
    int part = 0;
    if (lane == 0) part = atomicAdd(&next, 1u);
    part = __shfl_sync(~0u, part, 0);
    if (part >= parts) break;
    const int i = i0 + part / per, c0 = part % per * (32 * U);
    const T *src = in + i * a.logits_pos_stride;
    T *dst = out + i * a.out_pos_stride;
    auto one = [&](int x) {
      if (banned(i, x)) dst[x] = E::kMinf;
      else if (!P.same) dst[x] = src[x];
    };
    if (!P.vec) {
      for (int x = c0 * VEC + lane; x < min(n, (c0 + 32 * U) * VEC); x += 32) one(x);
      continue;
    }
    // elements before the first multiple of 16 bytes and behind the last one by one
    const int head = min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / static_cast<int>(sizeof(T)), n);
    const int chunks = (n - head) / VEC, behind = head + chunks * VEC;
    if (c0 == 0 && lane < head + n - behind) one(lane < head ? lane : behind + lane - head);
    const uint32_t *row = allowed && i <= g ? allowed + i * a.allowed_pos_stride : nullptr;
    uint4 q[U];
    uint32_t no[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + 32 * u + lane;
      no[u] = row && c < chunks ? ~bits_at(row, v0 + head + c * VEC, last) & ((1u << VEC) - 1) : 0;
      if (c < chunks && (!P.same || no[u])) q[u] = __ldcs(reinterpret_cast<const uint4 *>(src + head) + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + 32 * u + lane;
      if (c >= chunks || (P.same && !no[u])) continue;
      if (row) {
        constexpr int W = VEC / 4;  // elements of a word
        q[u].x = masked<F32>(q[u].x, no[u]), q[u].y = masked<F32>(q[u].y, no[u] >> W);
        q[u].z = masked<F32>(q[u].z, no[u] >> 2 * W), q[u].w = masked<F32>(q[u].w, no[u] >> 3 * W);
      }
      __stcs(reinterpret_cast<uint4 *>(dst + head) + c, q[u]);
    }
  }
  __syncthreads();  // the listed tokens' places are written again below

  // --- the tokens that something applies to, at the positions up to gamma_b
  const float *bias_of = a.bias + static_cast<int64_t>(b) * a.n_bias - 1;
  const int stop = min(i1, g + 1), blocks = stop > i0 ? (stop - i0 + S - 1) / S : 0;
  const int many = static_cast<int>(listed);
  for (int y = tid; y < many * blocks; y += AJ_NT) {
    const int ib = i0 + y / many * S, x = list[y % many];
    const uint32_t c = count[x], e = a.n_bias ? bias[x] : 0;
    const float more = e ? __ldg(bias_of + e) : 0.0f;
    T from[S];
    bool on[S];
#pragma unroll
    for (int u = 0; u < S; ++u) {
      on[u] = ib + u < stop && !banned(ib + u, x);  // banned: -inf already
      if (on[u]) from[u] = in[(ib + u) * a.logits_pos_stride + x];
    }
#pragma unroll
    for (int u = 0; u < S; ++u) {
      if (!on[u]) continue;
      const int i = ib + u;
      float z = E::value(from[u]);
      uint32_t made = c & kCount;
      if (c & kDraft) {  // rare
        const int32_t *mask = a.tree_mask ? a.tree_mask + (static_cast<int64_t>(b) * N + i) * P.W : nullptr;
        for (int j = 0; j < (mask ? g : min(g, i)); ++j)
          if (drafts[j] == x && (!mask || (mask[(j + 1) >> 5] >> ((j + 1) & 31) & 1))) ++made;
      }
      if (!made && !(c & kPrompt) && !e) continue;
      if (made || (c & kPrompt)) z = z > 0.0f ? __fdiv_rn(z, r) : z * r;
      if (made) z = (z - f * static_cast<float>(made)) - p;
      if (e) z += more;
      out[i * a.out_pos_stride + x] = E::bits(z);
    }
  }
}

bool aligned(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

// Rows of V elements that begin at p big + q small, p < nb, q < ns, and do not overlap: the
// ns inner ones are all within `big` elements.
struct Rows {
  int64_t big, nb, small, ns, V;
  // Whether a row that begins at t has an element in common with one of them (with
  // `both`, of those with negative p and q too): of p and of q only the two multiples
  // next to what is left of t can be.
  bool meet(int64_t t, bool both) const {
    auto next_to = [&](int64_t t, int64_t step, int64_t n, auto f) {
      if (n == 1) return f(0);
      const int64_t k = t / step - (t % step < 0);
      auto in = [&](int64_t k) { return k < n && k >= (both ? 1 - n : 0) && f(k); };
      return in(k) || in(k + 1);
    };
    return next_to(t, big, nb, [&](int64_t p) {
      const int64_t u = nb > 1 ? t - p * big : t;
      return next_to(u, small, ns, [&](int64_t q) {
        const int64_t d = ns > 1 ? u - q * small : u;
        return d < V && d > -V;
      });
    });
  }
};

// Whether some row of the logits has an element in common with some row of the output,
// which begins `at` elements behind them and whose rows do not overlap.
bool overlap(const spec_adjust_params &a, int64_t at) {
  const int64_t B = a.B, N = static_cast<int64_t>(a.gamma_max) + 1, V = a.V;
  const int64_t lr = B > 1 ? a.logits_row_stride : 0, lp = N > 1 ? a.logits_pos_stride : 0;
  const int64_t rs = B > 1 ? a.out_row_stride : 0, ps = N > 1 ? a.out_pos_stride : 0;
  if (at >= (B - 1) * lr + (N - 1) * lp + V || -at >= (B - 1) * rs + (N - 1) * ps + V) return false;
  const bool in_row = N == 1 || (B > 1 && rs >= (N - 1) * ps + V);  // positions within a row's stride
  const Rows out = in_row ? Rows{rs, B, ps, N, V} : Rows{ps, N, rs, B, V};
  if (lr == rs && lp == ps) return out.meet(-at, true);  // differences of two rows of the same kind
  for (int64_t b = 0; b < (lr ? B : 1); ++b)
    for (int64_t i = 0; i < (lp ? N : 1); ++i)
      if (out.meet(b * lr + i * lp - at, false)) return true;
  return false;
}

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
  if (a.gamma_max >= 1 << 20 || a.capacity >= 1 << 30 || a.n_bias > 65534 || a.B > 1 << 20 || (a.tree_mask && N > SPEC_TREE_MAX) ||
      (a.gamma_max > AJ_DRAFTS && (a.repetition || a.presence || a.frequency)))
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
  const int64_t rs = a.out_row_stride, ps = a.out_pos_stride;
  if ((a.gamma_max > 0 && ps < a.V) || (a.B > 1 && rs < a.V)) return SPEC_ERR_INVALID_ARG;
  if (a.gamma_max > 0 && a.B > 1 && rs < a.gamma_max * ps + a.V && ps < (a.B - 1) * rs + a.V) return SPEC_ERR_INVALID_ARG;
  JP P = {};
  P.a = a;
  P.in = logits;
  P.out = out;
  P.status = row_status;
  P.same = x == y;
  if (P.same && ((a.B > 1 && a.logits_row_stride != a.out_row_stride) ||
                 (a.gamma_max > 0 && a.logits_pos_stride != a.out_pos_stride)))
    return SPEC_ERR_INVALID_ARG;
  const int64_t apart = static_cast<int64_t>(y - x) / static_cast<int64_t>(es);
  if (!P.same && overlap(a, apart)) return SPEC_ERR_INVALID_ARG;
  P.W = (N + 31) / 32;
  const uintptr_t off = (x ^ y) | static_cast<uintptr_t>(a.B > 1 ? (a.logits_row_stride - a.out_row_stride) * static_cast<int64_t>(es) : 0) |
                        static_cast<uintptr_t>(a.gamma_max > 0 ? (a.logits_pos_stride - a.out_pos_stride) * static_cast<int64_t>(es) : 0);
  P.vec = off % 16 == 0;
  // Slices: as many as give the machine some 16 CTAs a multiprocessor, of 2048
  // tokens at least (each reads the whole sequence), of 512 where there would not be
  // one CTA a multiprocessor; then positions, down to one.  Measured, in us, 64 x 5 rows of
  // 50304 in float32 with 8 / 16 / 24 CTAs wanted: 30.5 / 29.1 / 42.9; of 1024
  // tokens at least: 30.4 / 33.6 / 37.0; 32 x 31 rows of 152064 in bfloat16: 123 / 114 / 114.
  // (152: a GB300's multiprocessors.)
  const int64_t want = 152 * 16;
  int64_t slices = std::min<int64_t>((want + a.B - 1) / a.B, (a.V + 2047) / 2048);
  if (slices * a.B < 152) slices = std::min<int64_t>((152 + a.B - 1) / a.B, (a.V + 511) / 512);
  slices = std::max<int64_t>(slices, (a.V + AJ_SLICE - 1) / AJ_SLICE);
  P.slice = static_cast<int>(((a.V + slices - 1) / slices + 31) / 32 * 32);
  P.slices = (a.V + P.slice - 1) / P.slice;
  const int64_t have = static_cast<int64_t>(P.slices) * a.B;
  const int64_t groups = std::min<int64_t>(N, std::max<int64_t>(1, want / have));
  P.npos = static_cast<int>((N + groups - 1) / groups);
  P.groups = (N + P.npos - 1) / P.npos;
  const int64_t grid = have * P.groups;
  if (grid > INT32_MAX) return SPEC_ERR_UNSUPPORTED;
  const int smem = P.slice * (a.n_bias ? 8 : 4) + P.slice * 2 + std::min(a.gamma_max, AJ_DRAFTS) * 4;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto *k = a.dtype == SPEC_F32 ? adjust_kernel<true> : adjust_kernel<false>;
  static std::atomic<bool> ready[2][kv::kDevices] = {};
  if (!kv::allow_shared(reinterpret_cast<const void *>(k), AJ_SMEM, ready[a.dtype == SPEC_F32])) return SPEC_ERR_CUDA;
  k<<<static_cast<unsigned>(grid), AJ_NT, smem, s>>>(P);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
