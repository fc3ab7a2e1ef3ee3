// kv_attend.cu -- spec_attend: the plan of the span kernels' launches and the
// merge of their partial results.
//
// Merge: row (b, i, h) has one partial result (o_s, lse2_s) for every CTA that
// worked on its own item and, with a prefix, on its prefix item;
//   out = sum_s 2^(lse2_s - m) o_s / sum_s 2^(lse2_s - m),
//   lse = ln 2 (m + log2 sum_s 2^(lse2_s - m)),  m = max_s lse2_s,
// in the order of the slots (reproducible).  The partial results were written
// just before and are read from L2.  Measured: 256 x 9 x 32
// rows of 128, two results and more each, 56 us (the bytes alone from HBM: 14 us):
// the chain from a row's slots to its loads; every CTA also checks all page ids
// of its sequence.
#include "kv_span.h"

namespace {

using namespace kv;

constexpr int MG_NT = 256;

struct MP {
  View w;
  Plan plan;
  const float *po, *pl, *qo, *ql;  // partial results: own, prefix
  __nv_bfloat16 *out;
  float *lse;
  int32_t *status;
  int32_t G, Hq, D;
  int32_t rto, rtp, co, cp, kp;  // rows per item and CTAs, own and prefix; key tokens of a prefix tile
};

// LPR lanes per row, four elements each: 16 for heads of 64, else a warp.
template <int LPR>
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
  int lost = 0;
  if (P.plan.lost)
    for (int c = threadIdx.x; c < P.cp; c += MG_NT) lost |= P.plan.lost[c];
  if (__syncthreads_or(bad)) st |= SPEC_ROW_BAD_PAGE;
  if (__syncthreads_or(lost)) st |= SPEC_ROW_WAIT_TIMEOUT;
  if (P.status && blockIdx.x == 0 && threadIdx.x == 0) P.status[b] = st;

  const int D = P.D, G = P.G;
  const int row = blockIdx.x * (MG_NT / LPR) + threadIdx.x / LPR;
  const bool there = row < w.N * P.Hq;
  const int i = row / P.Hq, h = row - i * P.Hq;
  const int head = h / G, r = i * G + h - head * G;
  // Partial results: those of the prefix item, then those of the own item, at
  // lse index lo0 + s * rt (and D times that, the outputs).
  int np = 0, all = 0;
  int64_t lp = 0, lo = 0;
  if (!st && there && i < n) {
    if (w.prefix) {
      const int tp = (w.prefix + P.kp - 1) / P.kp;
      const int nj = (P.plan.rows[w.B] + P.rtp - 1) / P.rtp;
      const uint32_t W = static_cast<uint32_t>(nj) * w.Hkv * tp, C = min(static_cast<uint32_t>(P.cp), W);
      const uint32_t k = P.plan.rows[b] + r, y = k / P.rtp, item = head * nj + y;
      const uint32_t c0 = owner(item * tp, W, C);
      np = owner(item * tp + tp - 1, W, C) - c0 + 1;
      lp = static_cast<int64_t>(item + c0) * P.rtp + (k - y * P.rtp);
    }
    const int to = (own + n + kTile - 1) / kTile, nj = (n * G + P.rto - 1) / P.rto;
    const uint32_t W = P.plan.tiles[w.B], C = min(static_cast<uint32_t>(P.co), W);
    const int y = r / P.rto;
    const uint32_t j = head * nj + y, x = P.plan.tiles[b] + j * to;
    const uint32_t c0 = owner(x, W, C);
    all = np + owner(x + to - 1, W, C) - c0 + 1;
    lo = static_cast<int64_t>(P.plan.items[b] + j + c0) * P.rto + (r - y * P.rto);
  }
  const bool on = lane * 4 < D;
  const unsigned most = __reduce_max_sync(~0u, static_cast<unsigned>(all));  // of the warp's rows
  float m = -INFINITY, sum = 0.0f;
  float4 acc = {0, 0, 0, 0};
  // LPR of them at a time: a lane each for the weights, then the outputs, whose
  // loads do not depend on one another.
  for (int s0 = 0; s0 < static_cast<int>(most); s0 += LPR) {
    const int s = s0 + lane;
    float v = -INFINITY;
    if (s < all) v = s < np ? P.ql[lp + static_cast<int64_t>(s) * P.rtp] : P.pl[lo + static_cast<int64_t>(s - np) * P.rto];
    float nm = v;
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) nm = fmaxf(nm, __shfl_xor_sync(~0u, nm, o));
    nm = fmaxf(nm, m);  // a NaN does not become the maximum
    const float a = nm == -INFINITY ? 1.0f : ex2(m - nm), c = v == -INFINITY ? 0.0f : ex2(v - nm);
    acc.x *= a, acc.y *= a, acc.z *= a, acc.w *= a;
    sum *= a;
    m = nm;
    const int k = min(LPR, static_cast<int>(most) - s0);
#pragma unroll 2
    for (int j = 0; j < k; ++j) {
      const float f = __shfl_sync(~0u, c, j, LPR);
      const int t = s0 + j;
      float4 x = {0, 0, 0, 0};
      if (on && t < all) {
        const float *src = t < np ? P.qo + (lp + static_cast<int64_t>(t) * P.rtp) * D
                                  : P.po + (lo + static_cast<int64_t>(t - np) * P.rto) * D;
        x = __ldcg(reinterpret_cast<const float4 *>(src + lane * 4));
      }
      sum += f;
      acc.x = fmaf(f, x.x, acc.x);
      acc.y = fmaf(f, x.y, acc.y);
      acc.z = fmaf(f, x.z, acc.z);
      acc.w = fmaf(f, x.w, acc.w);
    }
  }
  if (!there) return;
  float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  float l = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
  if (st) f = l = __int_as_float(0x7fffffff);
  const int64_t at = static_cast<int64_t>(b) * w.N * P.Hq + row;
  if (on) {
    const __nv_bfloat162 lo2 = __floats2bfloat162_rn(acc.x * f, acc.y * f);
    const __nv_bfloat162 hi2 = __floats2bfloat162_rn(acc.z * f, acc.w * f);
    *reinterpret_cast<__nv_bfloat162 *>(P.out + at * D + lane * 4) = lo2;
    *reinterpret_cast<__nv_bfloat162 *>(P.out + at * D + lane * 4 + 2) = hi2;
  }
  if (lane == 0 && P.lse) P.lse[at] = l;
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
//      500   20.5 / 25.6  23.5 / 26.4  23.6 / 26.6  34.0 / 35.9
//     1000   24.1 / 27.0  27.0 / 28.0  27.7 / 28.0  40.8 / 37.8
//     2000   30.9 / 30.7  34.8 / 32.0  36.8 / 32.0  46.1 / 41.2
//     4096   43.3 / 34.7  49.0 / 36.2  43.3 / 36.5  56.0 / 50.6
//     8192   45.1 / 40.0  52.6 / 42.5  50.0 / 42.0  74.0 / 62.6
// Heads of 64 and bfloat16 caches cross over between 500 and 2000 tokens too.  So the
// prefix's length says more than the rows do: this rule costs up to 13 us below 65
// rows and up to 3 us from 65 rows on, where the prefix is short.
constexpr int64_t kDenseRows = 65;

struct Layout {
  int wo, wp;               // row warps of own and prefix items
  bool dense;
  int rp, kp;               // rows and key tokens of a prefix tile
  int64_t tiles_o, tiles_p; // key tiles at most
  size_t plan, po, pl, qo, ql, bytes;
};

// Where each part of the workspace begins; false if the problem is too large.
bool lay_out(const View &w, int D, int G, Layout &L) {
  const auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const int64_t ro = static_cast<int64_t>(w.N) * G, rp = ro * w.B;
  if (rp > (1 << 30)) return false;
  L.wo = row_warps(ro);
  L.wp = row_warps(rp);
  L.dense = w.prefix > 0 && rp >= kDenseRows;
  L.rp = L.dense ? DN_ROWS : 16 * L.wp;
  L.kp = L.dense ? 128 : kTile;
  const int64_t io = (ro + 16 * L.wo - 1) / (16 * L.wo) * w.Hkv * w.B;
  const int64_t ip = w.prefix && rp ? (rp + L.rp - 1) / L.rp * w.Hkv : 0;
  const int64_t cap = (static_cast<int64_t>(w.max_pages) << w.ps_log2);
  L.tiles_o = io * ((cap + kTile - 1) / kTile);
  L.tiles_p = ip * ((w.prefix + static_cast<int64_t>(L.kp) - 1) / L.kp);
  if (io > INT32_MAX / 2 || ip > INT32_MAX / 2 || L.tiles_o > INT32_MAX || L.tiles_p > INT32_MAX)
    return false;
  const size_t so = static_cast<size_t>(io + kMaxGrid) * 16 * L.wo;
  const size_t sp = ip ? static_cast<size_t>(ip + (L.dense ? kMaxDense : kMaxGrid)) * L.rp : 0;
  L.plan = 0;
  L.po = up(sizeof(uint32_t) * (3 * (w.B + 1) + kMaxGrid));
  L.pl = up(L.po + so * D * 4);
  L.qo = up(L.pl + so * 4);
  L.ql = up(L.qo + sp * D * 4);
  L.bytes = up(L.ql + sp * 4);
  return true;
}

span_launch_fn span_of(int format, int D) {
  if (format == SPEC_KV_E4M3)
    return D == 64 ? span_e4m3_64 : D == 80 ? span_e4m3_80 : D == 96 ? span_e4m3_96 : span_e4m3_128;
  return D == 64 ? span_bf16_64 : D == 80 ? span_bf16_80 : D == 96 ? span_bf16_96 : span_bf16_128;
}

}  // namespace

extern "C" size_t spec_attend_workspace_size(const spec_kv_cache *cache, const spec_kv_batch *batch,
                                             int32_t n_heads) {
  View w;
  Layout L;
  if (!cache || !batch) return 0;
  spec_kv_cache c = *cache;  // the size goes by shapes: pointers may be unset
  spec_kv_batch s = *batch;
  c.k_pages = c.v_pages = reinterpret_cast<void *>(256);
  c.k_exp = c.v_exp = reinterpret_cast<int8_t *>(256);
  s.page_table = s.prefix_table = s.kv_len = reinterpret_cast<const int32_t *>(256);
  if (make_view(&c, &s, true, w) != SPEC_OK || n_heads < 1 || n_heads % w.Hkv) return 0;
  return lay_out(w, c.head_dim, n_heads / w.Hkv, L) ? L.bytes : 0;
}

extern "C" spec_status spec_attend(const spec_kv_cache *cache, const spec_kv_batch *batch,
                                   const void *q, int32_t n_heads, const int64_t *q_strides,
                                   float scale, void *out, float *lse, int32_t *row_status,
                                   void *workspace, size_t workspace_bytes, void *stream) {
  SpanParams P = {};
  const spec_status st = make_view(cache, batch, true, P.w);
  if (st != SPEC_OK) return st;
  if (n_heads < 1 || n_heads % P.w.Hkv || !q_strides || !(scale >= 0.0f) || !(scale < INFINITY))
    return SPEC_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (q_strides[i] < 0) return SPEC_ERR_INVALID_ARG;
  if (P.w.B == 0) return SPEC_OK;
  const uintptr_t qa = reinterpret_cast<uintptr_t>(q);
  if (!q || !out || qa % 2 || reinterpret_cast<uintptr_t>(out) % 4 ||
      reinterpret_cast<uintptr_t>(lse) % 4)
    return SPEC_ERR_INVALID_ARG;
  const int G = n_heads / P.w.Hkv, D = cache->head_dim;
  Layout L;
  if (!lay_out(P.w, D, G, L)) return SPEC_ERR_UNSUPPORTED;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < L.bytes)
    return SPEC_ERR_WORKSPACE;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  P.plan.tiles = reinterpret_cast<uint32_t *>(ws + L.plan);
  P.plan.items = P.plan.tiles + P.w.B + 1;
  P.plan.rows = P.plan.items + P.w.B + 1;
  P.plan.lost = L.dense ? P.plan.rows + P.w.B + 1 : nullptr;
  P.q = static_cast<const __nv_bfloat16 *>(q);
  P.qs0 = q_strides[0], P.qs1 = q_strides[1], P.qs2 = q_strides[2];
  const uintptr_t qbits = qa | static_cast<uintptr_t>((q_strides[0] | q_strides[1] | q_strides[2]) * 2);
  P.c = scale * 1.4426950408889634f;
  P.G = G;
  const span_launch_fn span = span_of(cache->format, D);
  MP m = {};
  m.w = P.w;
  m.plan = P.plan;
  m.G = G, m.Hq = n_heads, m.D = D, m.rto = 16 * L.wo, m.rtp = L.rp, m.kp = L.kp;
  m.out = static_cast<__nv_bfloat16 *>(out);
  m.lse = lse;
  m.status = row_status;
  if (P.w.prefix) {
    P.prefix = 1;
    P.po = reinterpret_cast<float *>(ws + L.qo);
    P.pl = reinterpret_cast<float *>(ws + L.ql);
    m.qo = P.po, m.ql = P.pl;
    P.qvec = qbits % (L.dense || L.wp == 1 ? 16 : 4) == 0;
    const cudaError_t e = !L.dense ? span(P, L.wp, L.tiles_p, &m.cp, s)
                          : cache->format == SPEC_KV_E4M3 ? dense_e4m3(P, D, L.tiles_p, &m.cp, s)
                                                          : dense_bf16(P, D, L.tiles_p, &m.cp, s);
    if (e != cudaSuccess) return SPEC_ERR_CUDA;
  }
  P.prefix = 0;
  P.qvec = qbits % (L.wo == 1 ? 16 : 4) == 0;
  P.po = reinterpret_cast<float *>(ws + L.po);
  P.pl = reinterpret_cast<float *>(ws + L.pl);
  m.po = P.po, m.pl = P.pl;
  if (span(P, L.wo, L.tiles_o, &m.co, s) != cudaSuccess) return SPEC_ERR_CUDA;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int per = MG_NT / (D == 64 ? 16 : 32);  // rows per CTA
  cfg.gridDim = dim3((P.w.N * n_heads + per - 1) / per, P.w.B);
  cfg.blockDim = dim3(MG_NT);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = D == 64 ? cudaLaunchKernelEx(&cfg, merge_kernel<16>, m)
                                : cudaLaunchKernelEx(&cfg, merge_kernel<32>, m);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
