// kv_attend.cu -- spec_attend and spec_attend_tree: the plan of the span kernels' launches and the
// merge of their partial results.
//
// Merge: row (b, i, h) has one partial result (o_s, lse2_s) for every CTA that
// worked on its own item and, with a prefix, on its prefix item;
//   out = sum_s 2^(lse2_s - m) o_s / sum_s 2^(lse2_s - m),
//   lse = ln 2 (m + log2 sum_s 2^(lse2_s - m)),  m = max_s lse2_s,
// in the order of the slots (reproducible).  The partial results were written
// just before and are read from L2.  Where a row's results are, and its weights, take
// some hundred instructions: done by every lane for its warp's row they were 627 a row
// and 75 % of the issue slots.  Where there are many rows, a lane does them for a row of
// its own, and the warp then adds up rows, two at a time: 256 x 9 x 32 rows of 128, two to
// four results each, 28 us in place of 57.  Where there are few, a row's chain of loads
// counts: eight in flight, the first before the weights are known.
#include <algorithm>

#include "kv_span.h"
#include "spec_tree.h"

namespace {

using namespace kv;

constexpr int MG_NT = 256;
constexpr int MG_AHEAD = 8;  // partial results in flight

// n / d for n < 2^31: with 2^s < d <= 2^(s + 1) and mul = floor(2^(32 + s) / d) + 1 the
// high word of n mul, s bits down, is exact (n (mul d - 2^(32 + s)) < 2^(32 + s)).
struct Divisor {
  uint32_t mul = 0, shift = 0;  // mul 0: d is 1
  Divisor() = default;
  explicit Divisor(uint32_t d) {
    if (d == 1) return;
    while ((2ull << shift) < d) ++shift;
    mul = static_cast<uint32_t>((1ull << (32 + shift)) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return mul ? __umulhi(n, mul) >> shift : n; }
};

struct MP {
  View w;
  Plan plan;
  const float *po, *pl, *qo, *ql;  // partial results: own, prefix
  __nv_bfloat16 *out;
  float *lse;
  int32_t *status;
  int32_t G, Hq, D;
  int32_t rto, rtp, co, cp;        // rows per item and CTAs, own and prefix
  int32_t tp, ko_log2;             // key tiles of the prefix; tokens of an own tile
  uint32_t item;                   // trees: what an own item costs beside its tiles
  Divisor by_G, by_Hq, by_rto, by_rtp;
  const uint32_t *lost_own;          // as plan.lost, of the own items
};

// The CTAs c0 .. c0 + n - 1 that worked on the tiles at places x .. y of W (kv_span.h): CTA
// ((z + 1) C - 1) / W on the one at z, by an estimate that is off by one at most: C < 2^10, so
// the float's error is below 2^-11.
struct Owners {
  uint32_t c0, n;
};
__device__ __forceinline__ Owners owners(uint32_t x, uint32_t y, uint32_t W, uint32_t C) {
  static_assert(kMaxGrid < 1 << 10, "estimate");
  const float f = __fdividef(static_cast<float>(C), static_cast<float>(W));
  auto one = [&](uint32_t z) {
    uint32_t q = static_cast<uint32_t>(static_cast<float>(z + 1) * f);
    const int64_t r = static_cast<int64_t>(static_cast<uint64_t>(z + 1) * C - 1 - static_cast<uint64_t>(q) * W);
    return r < 0 ? q - 1 : r >= W ? q + 1 : q;
  };
  const uint32_t c0 = one(x);
  return {c0, one(y) - c0 + 1};
}

// LPR lanes per row, four elements each: 16 for heads of 64, else a warp.  They take RW
// rows; what the plan says of a row, and its weights, are worked out by a lane each, the
// weights where none of the rows has more than SOME partial results.
template <int LPR, int RW, int SOME>
__global__ void __launch_bounds__(MG_NT) merge_kernel(const __grid_constant__ MP P) {
  const View &w = P.w;
  const int b = blockIdx.y, lane = threadIdx.x % LPR;
  int own, n;
  int st = row_shape(w, b, own, n);
  int bad = 0;
  if (!st) {  // the page ids in use
    const uint32_t np = static_cast<uint32_t>(w.n_pages);
    const int pm = (1 << w.ps_log2) - 1;
    for (int p = threadIdx.x; p < (own + n + pm) >> w.ps_log2; p += MG_NT)
      bad |= static_cast<uint32_t>(__ldg(w.table + b * w.tstride + p)) >= np;
    for (int p = threadIdx.x; p < (w.prefix + pm) >> w.ps_log2; p += MG_NT)
      bad |= static_cast<uint32_t>(__ldg(w.ptable + p)) >= np;
  }
  cudaGridDependencySynchronize();  // from here on: the span kernels' results
  // what the plan says of the sequence, before the barriers wait for anything
  uint32_t prow = 0, rows = 0;
  if (w.prefix) prow = P.plan.rows[b], rows = P.plan.rows[w.B];
  const uint32_t item0 = P.plan.items[b], tiles = P.plan.tiles[w.B], cost = cost_of_item(tiles, P.co, w.B, P.item);
  const uint32_t Wo = tiles + cost * P.plan.items[w.B], tile0 = P.plan.tiles[b] + cost * item0;
  int lost = 0;
  if (P.plan.lost)
    for (int c = threadIdx.x; c < P.cp; c += MG_NT) lost |= P.plan.lost[c];
  if (P.lost_own)
    for (int c = threadIdx.x; c < P.co; c += MG_NT) lost |= P.lost_own[c];
  if (__syncthreads_or(bad)) st |= SPEC_ROW_BAD_PAGE;
  if (__syncthreads_or(lost)) st |= SPEC_ROW_WAIT_TIMEOUT;
  if (P.status && blockIdx.x == 0 && threadIdx.x == 0) P.status[b] = st;

  const int D = P.D, G = P.G;
  const int row0 = (blockIdx.x * (MG_NT / LPR) + threadIdx.x / LPR) * RW, row = row0 + lane % RW;
  // The lane's row has `all` partial results, np of them of the prefix item (places
  // ip, ip + rtp, ..), then those of the own item (io + np rto, ..).
  uint32_t np = 0, all = 0, ip = 0, io = 0;
  {
    const int i = P.by_Hq(row), h = row - i * P.Hq;
    const int head = P.by_G(h), r = i * G + h - head * G;
    if (!st && row < w.N * P.Hq && i < n) {
      if (w.prefix) {
        const uint32_t nj = P.by_rtp(rows + P.rtp - 1), W = nj * w.Hkv * P.tp;
        const uint32_t k = prow + r, y = P.by_rtp(k), item = head * nj + y;
        const Owners c = owners(item * P.tp, item * P.tp + P.tp - 1, W, min(static_cast<uint32_t>(P.cp), W));
        np = c.n;
        ip = (item + c.c0) * P.rtp + (k - y * P.rtp);
      }
      const int to = (own + n + (1 << P.ko_log2) - 1) >> P.ko_log2, nj = P.by_rto(n * G + P.rto - 1);
      const uint32_t y = P.by_rto(r), j = head * nj + y, x = tile0 + j * (to + cost) + cost;
      const Owners c = owners(x, x + to - 1, Wo, min(static_cast<uint32_t>(P.co), Wo));
      all = np + c.n;
      io = (item0 + j + c.c0 - np) * P.rto + (r - y * P.rto);
    }
  }
  const bool on = lane * 4 < D;
  auto of = [](uint32_t x, int r) { return RW == 1 ? x : __shfl_sync(~0u, x, r, LPR); };  // row r's
  auto lse_of = [&](uint32_t s, uint32_t np, uint32_t ip, uint32_t io) {  // of partial result s
    return s < np ? P.ql[ip + s * P.rtp] : P.pl[io + s * P.rto];
  };
  auto load = [&](uint32_t s, uint32_t np, uint32_t ip, uint32_t io) {
    const float *src = s < np ? P.qo + static_cast<uint64_t>(ip + s * P.rtp) * D : P.po + static_cast<uint64_t>(io + s * P.rto) * D;
    return __ldcg(reinterpret_cast<const float4 *>(src + lane * 4));
  };
  auto add = [](float4 &acc, float f, const float4 &x) {
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, x.z, acc.z);
    acc.w = fmaf(f, x.w, acc.w);
  };
  auto weight = [](float v, float m) { return v == -INFINITY ? 0.0f : ex2(v - m); };
  auto put = [&](int row, const float4 &acc, float f) {
    if (row >= w.N * P.Hq || !on) return;
    __nv_bfloat16 *to = P.out + (static_cast<int64_t>(b) * w.N * P.Hq + row) * D + lane * 4;
    *reinterpret_cast<__nv_bfloat162 *>(to) = __floats2bfloat162_rn(acc.x * f, acc.y * f);
    *reinterpret_cast<__nv_bfloat162 *>(to + 2) = __floats2bfloat162_rn(acc.z * f, acc.w * f);
  };
  auto put_lse = [&](int row, float m, float sum) {
    if (row >= w.N * P.Hq || !P.lse) return;
    const float l = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
    P.lse[static_cast<int64_t>(b) * w.N * P.Hq + row] = st ? __int_as_float(0x7fffffff) : l;
  };
  auto over = [&](float sum) { return st ? __int_as_float(0x7fffffff) : sum == 0.0f ? 0.0f : 1.0f / sum; };

  float4 x[MG_AHEAD];
  if (RW > 1 && !__any_sync(~0u, all > SOME)) {
    // a lane each for a row's weights, then the outputs of one row or two at a time
    float c[SOME], m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (uint32_t j = 0; j < SOME; ++j) c[j] = j < all ? lse_of(j, np, ip, io) : -INFINITY;
#pragma unroll
    for (int j = 0; j < SOME; ++j) m = fmaxf(m, c[j]);  // a NaN does not become the maximum
#pragma unroll
    for (int j = 0; j < SOME; ++j) sum += c[j] = weight(c[j], m);
    if (lane < RW) put_lse(row, m, sum);
    const float f = over(sum);
    constexpr int R = MG_AHEAD / SOME;
#pragma unroll 1
    for (int r0 = 0; r0 < RW; r0 += R) {
      uint32_t n[R];
#pragma unroll
      for (int u = 0; u < R; ++u) {
        const uint32_t p = of(np, r0 + u), q = of(ip, r0 + u), o = of(io, r0 + u), its = of(all, r0 + u);
        n[u] = on ? its : 0;
#pragma unroll
        for (uint32_t j = 0; j < SOME; ++j)
          if (j < n[u]) x[u * SOME + j] = load(j, p, q, o);
      }
#pragma unroll
      for (int u = 0; u < R; ++u) {
        float4 acc = {0, 0, 0, 0};
#pragma unroll
        for (uint32_t j = 0; j < SOME; ++j) {
          const float g = __shfl_sync(~0u, c[j], r0 + u, LPR);
          if (j < n[u]) add(acc, g, x[u * SOME + j]);
        }
        put(row0 + r0 + u, acc, __shfl_sync(~0u, f, r0 + u, LPR));
      }
    }
    return;
  }
  // LPR partial results of a row at a time: a lane each for the weights, then the
  // outputs, MG_AHEAD loads in flight together, the first of them before the weights.
#pragma unroll 1
  for (int rr = 0; rr < RW; ++rr) {
    const uint32_t p = of(np, rr), q = of(ip, rr), o = of(io, rr), its = of(all, rr);
    const uint32_t most = __reduce_max_sync(~0u, its);  // of the warp's rows
    float m = -INFINITY, sum = 0.0f;
    float4 acc = {0, 0, 0, 0};
    for (uint32_t s0 = 0; s0 < most; s0 += LPR) {
      const uint32_t s = s0 + lane, k = min(static_cast<uint32_t>(LPR), most - s0);
      auto ahead = [&](uint32_t j0) {  // four at a time
#pragma unroll
        for (uint32_t u = 0; u < MG_AHEAD; ++u) {
          if (u % 4 == 0 && j0 + u >= k) break;
          x[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (on && s0 + j0 + u < its) x[u] = load(s0 + j0 + u, p, q, o);
        }
      };
      const float v = s < its ? lse_of(s, p, q, o) : -INFINITY;
      ahead(0);
      float nm = v;
#pragma unroll
      for (int d = LPR / 2; d; d >>= 1) nm = fmaxf(nm, __shfl_xor_sync(~0u, nm, d));
      nm = fmaxf(nm, m);
      const float a = nm == -INFINITY ? 1.0f : ex2(m - nm), c = weight(v, nm);
      acc.x *= a, acc.y *= a, acc.z *= a, acc.w *= a;
      sum *= a;
      m = nm;
      for (uint32_t j0 = 0; j0 < k; j0 += MG_AHEAD) {
        if (j0) ahead(j0);
#pragma unroll
        for (uint32_t u = 0; u < MG_AHEAD; ++u) {
          if (j0 + u >= k) break;
          const float g = __shfl_sync(~0u, c, j0 + u, LPR);
          sum += g;
          add(acc, g, x[u]);
        }
      }
    }
    put(row0 + rr, acc, over(sum));
    if (lane == 0) put_lse(row0 + rr, m, sum);
  }
}

// Row warps (of 16 rows) of an item: an item costs its rows, padding included,
// and about 24 rows' time for what it does once for all of them.
int row_warps(int64_t rows) {
  int best = 1;
  int64_t least = INT64_MAX;
  for (int w = 1; w <= 4; ++w) {
    const int64_t cost = (rows + 16 * w - 1) / (16 * w) * (16 * w + 24);
    if (cost < least) least = cost, best = w;
  }
  return best;
}

// Query rows (of a key/value head) from which the prefix goes to the dense kernel:
// from the 65th on the span kernel reads the keys again.  Measured, 8 heads of 128
// in e4m3, replayed calls, span / dense kernel in us:
//   prefix   16 rows      64 rows      80 rows      320 rows
//      500   11.5 / 14.4  14.7 / 14.9  16.1 / 15.0  29.0 / 29.3
//     1000   13.1 / 14.8  22.0 / 15.5  18.0 / 15.6  35.3 / 30.7
//     2000   15.5 / 16.3  24.5 / 22.7  25.6 / 22.7  40.2 / 32.9
//     4096   24.4 / 22.3  30.8 / 24.7  29.5 / 24.5  50.4 / 39.8
//     8192   26.7 / 26.0  34.5 / 27.3  34.6 / 27.5  67.9 / 49.2
// Heads of 64 and bfloat16 caches cross over at 500 to 1000 tokens too.  So the
// prefix's length says more than the rows do; the rule is one of rows because the
// two kernels round differently (include/spec_kv.h).  It costs up to 7 us below 65
// rows, where the prefix is long, and 2 us at most above, where it is short.
constexpr int64_t kDenseRows = 65;

// Query rows of a sequence's key/value head from which a tree's own tokens go to the
// dense kernel: from the 65th on the span kernel reads the keys again.  Measured, 8
// key/value heads of 128 in e4m3, sequences x tokens, replayed calls, span / dense
// kernel in us:
//   rows   1 x 100   1 x 8000   8 x 500   8 x 4000   64 x 100   64 x 1000
//     48   12 / 13    30 / 23   17 / 19    41 / 42    29 / 39     83 / 87
//     64   12 / 13    29 / 23   23 / 23    50 / 44    32 / 39     96 / 88
//     80   12 / 13    32 / 23   27 / 24    66 / 45    39 / 41    141 / 92
//    128   12 / 14    35 / 23   29 / 24    85 / 45    62 / 55    185 / 108
//    256   12 / 17    49 / 27   39 / 28   148 / 52   116 / 85    359 / 144
// Heads of 64 cross over between 64 and 104 rows, bfloat16 caches as these do.  From
// here on the dense kernel loses 5 us at most, where the context is short.  Below, the
// span kernel loses up to 8 us where it is long; as with prefixes, the rule is one of rows
// because the two kernels round differently (include/spec_kv.h says from which on).
constexpr int64_t kDenseTreeRows = 65;
static_assert(2 * kMaxDense <= kMaxGrid, "plan: words for the CTAs of both dense launches");

struct Layout {
  int wo, wp;               // row warps of own and prefix items
  bool dense, dense_own;
  int ro, ko, rp, kp;       // rows and key tokens of a tile, own and prefix
  int64_t items_o, items_p; // items and key tiles at most
  int64_t tiles_o, tiles_p;
  size_t plan, po, pl, qo, ql, bytes;
};

// Where each part of the workspace begins; false if the problem is too large.
bool lay_out(const View &w, int D, int G, bool tree, Layout &L) {
  const auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const int64_t ro = static_cast<int64_t>(w.N) * G, rp = ro * w.B;
  if (rp > (1 << 30)) return false;
  L.wo = row_warps(ro);
  L.wp = row_warps(rp);
  L.dense = w.prefix > 0 && rp >= kDenseRows;
  L.rp = L.dense ? DN_ROWS : 16 * L.wp;
  L.kp = L.dense ? 128 : kTile;
  L.dense_own = tree && ro >= kDenseTreeRows;
  L.ro = L.dense_own ? DN_ROWS : 16 * L.wo;
  L.ko = L.dense_own ? 128 : kTile;
  const int64_t io = (ro + L.ro - 1) / L.ro * w.Hkv * w.B;
  const int64_t ip = w.prefix && rp ? (rp + L.rp - 1) / L.rp * w.Hkv : 0;
  const int64_t cap = (static_cast<int64_t>(w.max_pages) << w.ps_log2);
  L.tiles_o = io * ((cap + L.ko - 1) / L.ko);
  L.tiles_p = ip * ((w.prefix + static_cast<int64_t>(L.kp) - 1) / L.kp);
  if (io > INT32_MAX / 2 || ip > INT32_MAX / 2 || L.tiles_o + std::max<int64_t>(SP_ITEM, DN_ITEM) * io > INT32_MAX || L.tiles_p > INT32_MAX)
    return false;
  L.items_o = io, L.items_p = ip;
  const size_t so = static_cast<size_t>(io + (L.dense_own ? kMaxDense : kMaxGrid)) * L.ro;
  const size_t sp = ip ? static_cast<size_t>(ip + (L.dense ? kMaxDense : kMaxGrid)) * L.rp : 0;
  L.plan = 0;
  L.po = up(sizeof(uint32_t) * (3 * (w.B + 1) + kMaxGrid));
  L.pl = up(L.po + so * D * 4);
  L.qo = up(L.pl + so * 4);
  L.ql = up(L.qo + sp * D * 4);
  L.bytes = up(L.ql + sp * 4);
  return true;
}

span_launch_fn span_of(int format, int D, bool tree) {
  if (tree && format == SPEC_KV_E4M3)
    return D == 64 ? tree_e4m3_64 : D == 80 ? tree_e4m3_80 : D == 96 ? tree_e4m3_96 : tree_e4m3_128;
  if (tree) return D == 64 ? tree_bf16_64 : D == 80 ? tree_bf16_80 : D == 96 ? tree_bf16_96 : tree_bf16_128;
  if (format == SPEC_KV_E4M3)
    return D == 64 ? span_e4m3_64 : D == 80 ? span_e4m3_80 : D == 96 ? span_e4m3_96 : span_e4m3_128;
  return D == 64 ? span_bf16_64 : D == 80 ? span_bf16_80 : D == 96 ? span_bf16_96 : span_bf16_128;
}

size_t workspace_of(const spec_kv_cache *cache, const spec_kv_batch *batch, int32_t n_heads, bool tree) {
  View w;
  Layout L;
  if (!cache || !batch) return 0;
  spec_kv_cache c = *cache;  // the size goes by shapes: pointers may be unset
  spec_kv_batch s = *batch;
  c.k_pages = c.v_pages = reinterpret_cast<void *>(256);
  c.k_exp = c.v_exp = reinterpret_cast<int8_t *>(256);
  s.page_table = s.prefix_table = s.kv_len = reinterpret_cast<const int32_t *>(256);
  if (make_view(&c, &s, true, w) != SPEC_OK || n_heads < 1 || n_heads % w.Hkv) return 0;
  if (tree && w.N > SPEC_TREE_MAX) return 0;
  return lay_out(w, c.head_dim, n_heads / w.Hkv, tree, L) ? L.bytes : 0;
}

// mask: of a tree, or null.
spec_status attend(const spec_kv_cache *cache, const spec_kv_batch *batch, const int32_t *mask, bool tree,
                   const void *q, int32_t n_heads, const int64_t *q_strides, float scale, void *out,
                   float *lse, int32_t *row_status, void *workspace, size_t workspace_bytes, void *stream) {
  SpanParams P = {};
  const spec_status st = make_view(cache, batch, true, P.w);
  if (st != SPEC_OK) return st;
  if (tree && P.w.N > SPEC_TREE_MAX) return SPEC_ERR_UNSUPPORTED;
  if (n_heads < 1 || n_heads % P.w.Hkv || !q_strides || !(scale >= 0.0f) || !(scale < INFINITY))
    return SPEC_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (q_strides[i] < 0) return SPEC_ERR_INVALID_ARG;
  if (P.w.B == 0) return SPEC_OK;
  const uintptr_t qa = reinterpret_cast<uintptr_t>(q);
  if (!q || !out || qa % 2 || reinterpret_cast<uintptr_t>(out) % 4 ||
      reinterpret_cast<uintptr_t>(lse) % 4)
    return SPEC_ERR_INVALID_ARG;
  if (tree && (!mask || reinterpret_cast<uintptr_t>(mask) % 4)) return SPEC_ERR_INVALID_ARG;
  const int G = n_heads / P.w.Hkv, D = cache->head_dim;
  Layout L;
  if (!lay_out(P.w, D, G, tree, L)) return SPEC_ERR_UNSUPPORTED;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < L.bytes)
    return SPEC_ERR_WORKSPACE;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  P.plan.tiles = reinterpret_cast<uint32_t *>(ws + L.plan);
  P.plan.items = P.plan.tiles + P.w.B + 1;
  P.plan.rows = P.plan.items + P.w.B + 1;
  uint32_t *lost = P.plan.rows + P.w.B + 1;
  P.plan.lost = L.dense ? lost : nullptr;
  P.q = static_cast<const __nv_bfloat16 *>(q);
  P.qs0 = q_strides[0], P.qs1 = q_strides[1], P.qs2 = q_strides[2];
  const uintptr_t qbits = qa | static_cast<uintptr_t>((q_strides[0] | q_strides[1] | q_strides[2]) * 2);
  P.c = scale * 1.4426950408889634f;
  P.G = G;
  const span_launch_fn span = span_of(cache->format, D, false), own = span_of(cache->format, D, tree);
  MP m = {};
  m.w = P.w;
  m.plan = P.plan;
  m.G = G, m.Hq = n_heads, m.D = D, m.rto = L.ro, m.rtp = L.rp;
  m.by_G = Divisor(G), m.by_Hq = Divisor(n_heads), m.by_rto = Divisor(L.ro), m.by_rtp = Divisor(L.rp);
  m.tp = static_cast<int>((P.w.prefix + static_cast<int64_t>(L.kp) - 1) / L.kp);
  while (1 << m.ko_log2 < L.ko) ++m.ko_log2;
  m.item = !tree ? 0 : L.dense_own ? DN_ITEM : SP_ITEM;
  m.out = static_cast<__nv_bfloat16 *>(out);
  m.lse = lse;
  m.status = row_status;
  if (P.w.prefix) {
    P.prefix = 1;
    P.po = reinterpret_cast<float *>(ws + L.qo);
    P.pl = reinterpret_cast<float *>(ws + L.ql);
    m.qo = P.po, m.ql = P.pl;
    P.qvec = qbits % (L.dense || L.wp == 1 ? 16 : 4) == 0;
    P.halves = static_cast<int64_t>(P.w.N) * G * P.w.B <= DN_ROWS / 2 ? 1 : 2;
    const cudaError_t e = !L.dense ? span(P, L.wp, L.tiles_p, &m.cp, s)
                          : cache->format == SPEC_KV_E4M3 ? dense_e4m3(P, D, L.tiles_p, &m.cp, s)
                                                          : dense_bf16(P, D, L.tiles_p, &m.cp, s);
    if (e != cudaSuccess) return SPEC_ERR_CUDA;
  }
  P.behind = P.w.prefix > 0;
  P.halves = static_cast<int64_t>(P.w.N) * G <= DN_ROWS / 2 ? 1 : 2;
  P.prefix = 0;
  P.mask = mask;
  P.mask_words = (P.w.N + 31) / 32;
  P.qvec = qbits % (L.dense_own || L.wo == 1 ? 16 : 4) == 0;
  P.po = reinterpret_cast<float *>(ws + L.po);
  P.pl = reinterpret_cast<float *>(ws + L.pl);
  m.po = P.po, m.pl = P.pl;
  if (L.dense_own) {
    m.lost_own = P.plan.lost = lost + kMaxDense;
    const cudaError_t e = cache->format == SPEC_KV_E4M3 ? dense_tree_e4m3(P, D, L.tiles_o, &m.co, s)
                                                        : dense_tree_bf16(P, D, L.tiles_o, &m.co, s);
    if (e != cudaSuccess) return SPEC_ERR_CUDA;
  } else if (own(P, L.wo, L.tiles_o, &m.co, s) != cudaSuccess) {
    return SPEC_ERR_CUDA;
  }
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int64_t rows = static_cast<int64_t>(P.w.N) * n_heads;  // of a sequence
  const int64_t all = rows * P.w.B;
  // partial results of a row, about
  const int64_t some = (P.w.prefix ? 1 + m.cp / L.items_p : 0) + 1 + m.co / L.items_o;
  // Rows of a warp (of half a warp with heads of 64).  Measured, 32 heads of 128 over 8,
  // in us for the call, 1 / 4 / 8 rows: 4096 rows 17.6 / 17.6 / 17.6 (16 trees of 8
  // nodes, 300 tokens), 8192 26.5 / 24.2 / 24.7, 16384 35.4 / 28.0 / 30.2, 32768 110 /
  // 95.3 / 93.8 (1000 tokens); 16 heads of 64: 8192 20.8 / 19.7 / 21.2, 32768 160 / 154 /
  // 158.  With some five results a row, 1 / 4 rows of up to eight: 10240 rows behind a
  // prefix of 1000 62.1 / 59.1, 8192 rows of 4 trees over 4000 43.2 / 41.9.  (152: a GB300's
  // multiprocessors; on others the rule is right and measured for none.)
  const int rw = all <= 152 * 48 ? 1 : some > 4 || all <= 152 * 192 * (D == 64 ? 2 : 1) ? 4 : 8;
  const int per = MG_NT / (D == 64 ? 16 : 32) * rw;  // rows per CTA
  cfg.gridDim = dim3(static_cast<unsigned>((rows + per - 1) / per), P.w.B);
  cfg.blockDim = dim3(MG_NT);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto pick = [&](auto *one, auto *four, auto *four8, auto *eight) { return rw == 1 ? one : rw == 8 ? eight : some > 4 ? four8 : four; };
  auto *merge = D == 64 ? pick(merge_kernel<16, 1, 4>, merge_kernel<16, 4, 4>, merge_kernel<16, 4, 8>, merge_kernel<16, 8, 4>)
                        : pick(merge_kernel<32, 1, 4>, merge_kernel<32, 4, 4>, merge_kernel<32, 4, 8>, merge_kernel<32, 8, 4>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, merge, m);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

extern "C" size_t spec_attend_workspace_size(const spec_kv_cache *cache, const spec_kv_batch *batch,
                                             int32_t n_heads) {
  return workspace_of(cache, batch, n_heads, false);
}

extern "C" spec_status spec_attend(const spec_kv_cache *cache, const spec_kv_batch *batch,
                                   const void *q, int32_t n_heads, const int64_t *q_strides,
                                   float scale, void *out, float *lse, int32_t *row_status,
                                   void *workspace, size_t workspace_bytes, void *stream) {
  return attend(cache, batch, nullptr, false, q, n_heads, q_strides, scale, out, lse, row_status, workspace,
                workspace_bytes, stream);
}

extern "C" size_t spec_attend_tree_workspace_size(const spec_kv_cache *cache, const spec_kv_batch *batch,
                                                  int32_t n_heads) {
  return workspace_of(cache, batch, n_heads, true);
}

extern "C" spec_status spec_attend_tree(const spec_kv_cache *cache, const spec_kv_batch *batch,
                                        const int32_t *mask, const void *q, int32_t n_heads,
                                        const int64_t *q_strides, float scale, void *out, float *lse,
                                        int32_t *row_status, void *workspace, size_t workspace_bytes,
                                        void *stream) {
  return attend(cache, batch, mask, true, q, n_heads, q_strides, scale, out, lse, row_status, workspace,
                workspace_bytes, stream);
}
