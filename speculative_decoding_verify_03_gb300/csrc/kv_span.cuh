// kv_span.cuh -- the span kernel of spec_attend: partial attention of a few
// query rows over a span of key tiles (see kv_span.h for the work's cut).
//
// Mathematics, in powers of two: z_j = scale log2(e) q.k_j and, with the
// stored exponents, k_j = 2^ek y_j, v_j = 2^ev u_j: the tensor cores form
// q.y_j, the column factor 2^ek is applied to the score, and the weight that
// multiplies u_j is P_j = 2^(z_j + ev_j - M), M the running maximum of
// z_j + ev_j.  So no exponent of v enters a 16-bit operand, and the sum of
// weights is l = sum_j P_j 2^-ev_j.  o = (sum_j P_j u_j) / l,
// lse2 = M + log2 l.  y and u are exact in float16 and q is scaled by a power
// of two into its range; P is biased by 2^8, so that weights down to 2^-33 of
// the largest survive.  bfloat16 caches: the same with ek = ev = 0 in
// bfloat16 operands.
//
// Layout: a CTA has WR x WT warps; a warp works on 16 rows and 64 / WT tokens
// of each tile with m16n8k16 products, and keeps its own running maximum, sum
// and output in registers; the WT warps of a row tile are joined at the end of
// an item.  K and V tiles come through a ring of asynchronous copies, rows
// padded to an odd multiple of 16 bytes (ldmatrix without bank conflicts).
// e4m3 bytes go through ldmatrix as pairs: a key row's four bytes per lane are
// the two halves of one k16 step (the order of d within a step is free as long
// as q has the same), and the transposed value pairs give two n8 tiles, even
// and odd d, after one byte permute.
#pragma once

#include <cuda_fp16.h>

#include "kv_span.h"

namespace kv {

__device__ __forceinline__ void ldm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldm2(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(a));
}
__device__ __forceinline__ void ldm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldm2t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(a));
}
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int D, bool E4M3, int WR, int WT>
struct SpanCfg {
  static constexpr int NT = 32 * WR * WT;
  static constexpr int RT = 16 * WR;
  static constexpr int DB = E4M3 ? D : 2 * D;        // bytes of a cached row
  static constexpr int CPR = DB / 16;                // 16-byte chunks of a row
  static constexpr int LD = (CPR | 1) * 16;          // row pitch in shared memory
  static constexpr int TILE = kTile * LD;            // bytes of a K or V tile
  static constexpr int STAGE = 2 * TILE + (E4M3 ? 2 * kTile : 0);
  static constexpr int ST = STAGE > 30000 ? 2 : 3;   // stages
  static constexpr int OLD = D + 4;                  // pitch of the joined output
  static constexpr int JOIN = WT > 1 ? (RT * OLD + 2 * WT * RT) * 4 : 0;
  static constexpr int FIXED = ST * STAGE + JOIN + 16;
  static constexpr int MIN_CTAS = WR <= 2 ? 3 : WR == 3 ? 3 : 2;
};

// A position in the tile sequence.
struct Cursor {
  uint32_t x;        // tile number
  int b, j, t;       // sequence, item within it, tile within the item
  int nt, nj;        // tiles of an item, items of the sequence
  int own, n;        // own tokens before the step, tokens in the step
};

template <int D, bool E4M3, int WR, int WT>
__global__ void __launch_bounds__(32 * WR *WT, SpanCfg<D, E4M3, WR, WT>::MIN_CTAS)
    span_kernel(const __grid_constant__ SpanParams P) {
  using C = SpanCfg<D, E4M3, WR, WT>;
  constexpr int NT = C::NT, RT = C::RT, LD = C::LD, ST = C::ST, CPR = C::CPR;
  constexpr int TPW = kTile / WT;   // tokens of a tile per warp
  constexpr int NG = TPW / 8;       // groups of 8 tokens
  constexpr int KS = D / 16;        // k16 steps of q.k
  constexpr float BIAS = E4M3 ? 8.0f : 0.0f;
  extern __shared__ __align__(128) uint8_t sm[];
  uint8_t *stages = sm;
  float *join = reinterpret_cast<float *>(sm + ST * C::STAGE);
  uint32_t *band = reinterpret_cast<uint32_t *>(sm + ST * C::STAGE + C::JOIN);  // 2 words
  uint32_t *wsum = band + 2;                                                    // 2 words
  uint32_t *cum0 = reinterpret_cast<uint32_t *>(sm + C::FIXED);  // B + 1: tiles or rows before b
  uint32_t *cum1 = cum0 + P.w.B + 1;                             // B + 1: items before b (own)

  const View &w = P.w;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wr = warp / WT, wt = warp % WT;
  const int g = lane >> 2, q4 = lane & 3;
  const int G = P.G, B = w.B;
  const bool pre = P.prefix != 0;

  // --- the plan: running sums over the sequences
  {
    const int per = (B + NT - 1) / NT;
    uint32_t a0 = 0, a1 = 0;
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) {
      int own, n;
      row_shape(w, b, own, n);
      const uint32_t rt = (n * G + RT - 1) / RT, nt = (own + n + kTile - 1) / kTile;
      cum0[b] = pre ? n * G : rt * w.Hkv * nt;
      cum1[b] = rt * w.Hkv;
      a0 += cum0[b];
      a1 += cum1[b];
    }
    uint32_t s0 = a0, s1 = a1;  // inclusive over the warp
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t0 = __shfl_up_sync(~0u, s0, o), t1 = __shfl_up_sync(~0u, s1, o);
      if (lane >= o) s0 += t0, s1 += t1;
    }
    if (tid < 2) wsum[tid] = 0, band[tid] = 0;
    uint32_t e0 = s0 - a0, e1 = s1 - a1;
    for (int v = 0; v < NT / 32; ++v) {  // warps in turn
      __syncthreads();
      if (warp == v) {
        e0 += wsum[0], e1 += wsum[1];
        const uint32_t t0 = __shfl_sync(~0u, s0, 31), t1 = __shfl_sync(~0u, s1, 31);
        __syncwarp();
        if (lane == 0) wsum[0] += t0, wsum[1] += t1;
      }
    }
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) {
      const uint32_t t0 = cum0[b], t1 = cum1[b];
      cum0[b] = e0, cum1[b] = e1;
      e0 += t0, e1 += t1;
    }
    __syncthreads();
    if (tid == 0) cum0[B] = wsum[0], cum1[B] = wsum[1];
    __syncthreads();
    if (blockIdx.x == 0)
      for (int b = tid; b <= B; b += NT) {
        if (pre) {
          P.plan.rows[b] = cum0[b];
        } else {
          P.plan.tiles[b] = cum0[b];
          P.plan.items[b] = cum1[b];
        }
      }
  }
  const uint32_t rows_all = cum0[B];  // prefix: query rows of a key/value head
  const int pnt = (w.prefix + kTile - 1) / kTile, pnj = (rows_all + RT - 1) / RT;
  const uint32_t W = pre ? static_cast<uint32_t>(pnt) * pnj * w.Hkv : cum0[B];
  const uint32_t ctas = min(gridDim.x, W);  // every one of them has a tile
  if (blockIdx.x >= ctas) return;
  const uint32_t lo = static_cast<uint32_t>(static_cast<uint64_t>(W) * blockIdx.x / ctas);
  const uint32_t hi = static_cast<uint32_t>(static_cast<uint64_t>(W) * (blockIdx.x + 1) / ctas);

  auto before = [&](uint32_t x) {  // largest b with cum0[b] <= x (x < cum0[B])
    int l = 0, r = B;
    while (r - l > 1) {
      const int m = (l + r) >> 1;
      if (cum0[m] <= x) l = m;
      else r = m;
    }
    return l;
  };
  auto enter = [&](Cursor &c) {  // shape of sequence c.b
    row_shape(w, c.b, c.own, c.n);
    c.nt = (c.own + c.n + kTile - 1) / kTile;
    c.nj = (c.n * G + RT - 1) / RT * w.Hkv;
  };
  auto seek = [&](Cursor &c, uint32_t x) {
    c.x = x;
    uint32_t y = x;
    if (pre) {
      c.b = 0, c.nt = pnt, c.nj = pnj * w.Hkv, c.own = w.prefix, c.n = 0;
    } else {
      c.b = before(x);
      y -= cum0[c.b];
      enter(c);
    }
    c.j = y / c.nt;
    c.t = y - c.j * c.nt;
  };
  auto step = [&](Cursor &c) {  // to the next tile; only while c.x + 1 < W
    ++c.x;
    if (++c.t < c.nt) return;
    c.t = 0;
    if (++c.j < c.nj || pre) return;
    c.j = 0;
    do ++c.b;
    while (cum0[c.b + 1] == cum0[c.b]);
    enter(c);
  };

  // --- copies of tile c into its stage
  auto fetch = [&](const Cursor &c) {
    uint8_t *s = stages + c.x % ST * C::STAGE;
    const uint32_t ks = s32(s), vs = ks + C::TILE;
    const int head = pre ? c.j / pnj : c.j / (c.nj / w.Hkv);
    const int32_t *ids = pre ? w.ptable : w.table + c.b * w.tstride;
    const int limit = c.own + c.n, t0 = c.t * kTile;
    const int lg = w.ps_log2, pm = (1 << lg) - 1;
#pragma unroll
    for (int i = tid; i < kTile * CPR; i += NT) {
      const int row = i / CPR, ch = i - row * CPR, tok = t0 + row;
      bool ok = tok < limit;
      const int id = ok ? __ldg(ids + (tok >> lg)) : -1;
      ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(w.n_pages);
      const int64_t at = ((static_cast<int64_t>(head) << lg) + (tok & pm)) * C::DB + ch * 16;
      cp16(ks + row * LD + ch * 16, ok ? w.k + id * w.kps + at : w.k, ok);
      cp16(vs + row * LD + ch * 16, ok ? w.v + id * w.vps + at : w.v, ok);
    }
    if constexpr (E4M3) {
      if (tid < 2 * kTile / 16) {  // exponents, 16 tokens at a time
        const int row = (tid >> 1) * 16, tok = t0 + row;
        bool ok = tok < limit;
        const int id = ok ? __ldg(ids + (tok >> lg)) : -1;
        ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(w.n_pages);
        const int64_t at = ((static_cast<int64_t>(id) * w.Hkv + head) << lg) + (tok & pm);
        const int8_t *e = tid & 1 ? w.ve : w.ke;
        cp16(ks + 2 * C::TILE + (tid & 1) * kTile + row, ok ? e + at : e, ok);
      }
    }
  };

  Cursor cur, ahead;
  seek(cur, lo);
  ahead = cur;
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) {
    if (lo + i < hi) {
      fetch(ahead);
      if (ahead.x + 1 < hi) step(ahead);
    }
    cp_commit();
  }

  uint32_t qf[KS][4];
  float o[D / 8][4];
  float M0, M1, l0, l1;
  float cq = P.c;             // score factor: scale log2 e 2^eq
  int lim0 = 0, lim1 = 0;     // tokens that rows g and g + 8 see
  int row0 = 0, rows = 0;     // first row of the item's tile, rows of the sequence
  int head = 0, free_to = 0;  // tokens that every row sees
  bool fresh = true;

  for (; cur.x < hi;) {
    if (fresh) {  // a new item: its rows' queries, in registers
      fresh = false;
      const int per = pre ? pnj : cur.nj / w.Hkv;
      head = cur.j / per;
      row0 = (cur.j - head * per) * RT;
      rows = pre ? rows_all : cur.n * G;
      free_to = pre ? w.prefix : cur.own + row0 / G + 1;
      const __nv_bfloat16 *src[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int r = row0 + wr * 16 + g + 8 * a;
        src[a] = nullptr;
        int lim = 0;
        if (r < rows) {
          const int b = pre ? before(r) : cur.b;
          const int rr = pre ? r - static_cast<int>(cum0[b]) : r;
          const int i = rr / G, gg = rr - i * G;
          src[a] = P.q + b * P.qs0 + i * P.qs1 + (head * G + gg) * P.qs2;
          lim = pre ? w.prefix : cur.own + i + 1;
        }
        (a ? lim1 : lim0) = lim;
      }
      auto word = [&](const __nv_bfloat16 *p, int d) -> uint32_t {  // elements d, d + 1
        if (!p) return 0;
        if (P.qvec) return __ldg(reinterpret_cast<const uint32_t *>(p + d));
        const uint32_t a = __ldg(reinterpret_cast<const uint16_t *>(p + d));
        const uint32_t b = __ldg(reinterpret_cast<const uint16_t *>(p + d + 1));
        return a | b << 16;
      };
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        // e4m3: the lane's four bytes of a key row are d = 16 k + 4 q4 + 0 .. 3
        const int d0 = E4M3 ? 16 * k + 4 * q4 : 16 * k + 2 * q4, d1 = E4M3 ? d0 + 2 : d0 + 8;
        qf[k][0] = word(src[0], d0);
        qf[k][1] = word(src[1], d0);
        qf[k][2] = word(src[0], d1);
        qf[k][3] = word(src[1], d1);
      }
      if constexpr (E4M3) {
        // bring the 16 rows' largest finite magnitude to [2^10, 2^11): exact
        // in float16 for all elements above 2^-28 of it
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a = qf[k][i] & 0x7fffu, b = qf[k][i] >> 16 & 0x7fffu;
            m = max(m, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
          }
        m = __reduce_max_sync(~0u, m);
        const int eq = max(static_cast<int>(m >> 7) - 127 - 10, -100);
        const float f = pow2i(-eq);
        cq = P.c * pow2i(eq);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            qf[k][i] = pack<true>(__uint_as_float(qf[k][i] << 16) * f,
                                  __uint_as_float(qf[k][i] & 0xffff0000u) * f);
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = 0.0f;
      M0 = M1 = -INFINITY;
      l0 = l1 = 0.0f;
    }

    cp_wait<ST - 2>();
    __syncthreads();
    if (cur.x + ST - 1 < hi) {
      fetch(ahead);
      if (ahead.x + 1 < hi) step(ahead);
    }
    cp_commit();

    uint8_t *stage = stages + cur.x % ST * C::STAGE;
    const uint32_t ks = s32(stage), vs = ks + C::TILE;
    const int8_t *ke = reinterpret_cast<const int8_t *>(stage + 2 * C::TILE), *ve = ke + kTile;
    const int t0 = cur.t * kTile;
    const bool edge = t0 + kTile > free_to;
    const int held = cur.own + cur.n;  // tokens present
    // Tokens that some row of the tile does not see but that are present: a
    // NaN or infinity among their values would reach every row through a zero
    // weight.  Take such elements out; add them below to the rows that see them.
    const bool banded = edge && !pre && held > free_to;
    uint32_t hot[2] = {0, 0};
    if (banded) {
      const int first = max(free_to - t0, 0), last = min(held - t0, kTile);
      for (int i = first * CPR + tid; i < last * CPR; i += NT) {
        const int row = i / CPR, ch = i - row * CPR;
        uint4 *p = reinterpret_cast<uint4 *>(stage + C::TILE + row * LD + ch * 16);
        uint4 v4 = *p;
        uint32_t *v = reinterpret_cast<uint32_t *>(&v4);
        uint32_t any = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t m = 0;
          if constexpr (E4M3) {
            const uint32_t x = v[k] & 0x7f7f7f7fu;
            m = ((x + 0x01010101u) & 0x80808080u) >> 7;  // 1 where the byte is 0x7f
            m *= 0xffu;
          } else {
            const uint32_t x = v[k] & 0x7fff7fffu;
            m = ((x + 0x00800080u) & 0x80008000u) >> 15;  // 1 where the exponent is full
            m *= 0xffffu;
          }
          v[k] &= ~m;
          any |= m;
        }
        if (any) {
          *p = v4;
          atomicOr(&band[row >> 5], 1u << (row & 31));
        }
      }
      __syncthreads();
      hot[0] = band[0], hot[1] = band[1];
    }

    // --- scores
    float s[NG][4];
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[j][k] = 0.0f;
    const uint32_t krow = ks + (wt * TPW + (lane & 7) + (lane & 8)) * LD + (lane >> 4) * 16;
#pragma unroll
    for (int jp = 0; jp < NG / 2; ++jp) {
      // four matrices: groups 2jp, 2jp + 1 of 8 tokens x two 16-byte chunks
#pragma unroll
      for (int c = 0; c < CPR; c += 2) {
        uint32_t r[4];
        const uint32_t a = krow + jp * 16 * LD + c * 16;
        if (c + 1 < CPR) ldm4(a, r);
        else ldm2(a, r);
        if constexpr (E4M3) {
          mma<true>(s[2 * jp], qf[c], cvt_lo(r[0]), cvt_hi(r[0]));
          mma<true>(s[2 * jp + 1], qf[c], cvt_lo(r[1]), cvt_hi(r[1]));
          if (c + 1 < CPR) {
            mma<true>(s[2 * jp], qf[c + 1 < KS ? c + 1 : 0], cvt_lo(r[2]), cvt_hi(r[2]));
            mma<true>(s[2 * jp + 1], qf[c + 1 < KS ? c + 1 : 0], cvt_lo(r[3]), cvt_hi(r[3]));
          }
        } else {
          mma<false>(s[2 * jp], qf[c / 2], r[0], r[2]);
          mma<false>(s[2 * jp + 1], qf[c / 2], r[1], r[3]);
        }
      }
    }

    // --- running softmax
    float inv[NG][2];  // 2^-ev
    float m0 = M0, m1 = M1;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const int col = wt * TPW + 8 * j + 2 * q4;
      float f0 = cq, f1 = cq, e0 = 0.0f, e1 = 0.0f;
      inv[j][0] = inv[j][1] = 1.0f;
      if constexpr (E4M3) {
        const char2 a = *reinterpret_cast<const char2 *>(ke + col);
        const char2 v = *reinterpret_cast<const char2 *>(ve + col);
        f0 = cq * pow2i(a.x), f1 = cq * pow2i(a.y);
        e0 = v.x, e1 = v.y;
        inv[j][0] = pow2i(-v.x), inv[j][1] = pow2i(-v.y);
      }
      s[j][0] = fmaf(s[j][0], f0, e0);
      s[j][1] = fmaf(s[j][1], f1, e1);
      s[j][2] = fmaf(s[j][2], f0, e0);
      s[j][3] = fmaf(s[j][3], f1, e1);
      if (edge) {
        const int t = t0 + col;
        if (t >= lim0) s[j][0] = -INFINITY;
        if (t + 1 >= lim0) s[j][1] = -INFINITY;
        if (t >= lim1) s[j][2] = -INFINITY;
        if (t + 1 >= lim1) s[j][3] = -INFINITY;
        if (t >= held) inv[j][0] = 0.0f;  // no token: its exponent is not one
        if (t + 1 >= held) inv[j][1] = 0.0f;
      }
      m0 = fmaxf(m0, fmaxf(s[j][0], s[j][1]));
      m1 = fmaxf(m1, fmaxf(s[j][2], s[j][3]));
    }
    m0 = fmaxf(m0, __shfl_xor_sync(~0u, m0, 1));
    m1 = fmaxf(m1, __shfl_xor_sync(~0u, m1, 1));
    m0 = fmaxf(m0, __shfl_xor_sync(~0u, m0, 2));
    m1 = fmaxf(m1, __shfl_xor_sync(~0u, m1, 2));
    const float u0 = m0 == -INFINITY ? 0.0f : m0 - BIAS, u1 = m1 == -INFINITY ? 0.0f : m1 - BIAS;
    if (__any_sync(~0u, m0 != M0 || m1 != M1)) {
      const float c0 = m0 == -INFINITY ? 1.0f : ex2(M0 - m0);
      const float c1 = m1 == -INFINITY ? 1.0f : ex2(M1 - m1);
      l0 *= c0, l1 *= c1;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] *= c0, o[i][1] *= c0, o[i][2] *= c1, o[i][3] *= c1;
      M0 = m0, M1 = m1;
    }
    uint32_t p[NG / 2][4];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const float a = ex2(s[j][0] - u0), b = ex2(s[j][1] - u0);
      const float c = ex2(s[j][2] - u1), d = ex2(s[j][3] - u1);
      l0 = fmaf(a, inv[j][0], fmaf(b, inv[j][1], l0));
      l1 = fmaf(c, inv[j][0], fmaf(d, inv[j][1], l1));
      p[j / 2][(j & 1) * 2] = pack<E4M3>(a, b);
      p[j / 2][(j & 1) * 2 + 1] = pack<E4M3>(c, d);
    }

    // --- weighted values
    const uint32_t vrow = vs + (wt * TPW + (lane & 7) + (lane & 8)) * LD + (lane >> 4) * 16;
#pragma unroll
    for (int kk = 0; kk < NG / 2; ++kk) {
#pragma unroll
      for (int c = 0; c < CPR; c += 2) {
        uint32_t r[4];
        const uint32_t a = vrow + kk * 16 * LD + c * 16;
        if (c + 1 < CPR) ldm4t(a, r);
        else ldm2t(a, r);
        if constexpr (E4M3) {
          const uint32_t x0 = __byte_perm(r[0], 0, 0x3120), x1 = __byte_perm(r[1], 0, 0x3120);
          mma<true>(o[2 * c], p[kk], cvt_lo(x0), cvt_lo(x1));
          mma<true>(o[2 * c + 1], p[kk], cvt_hi(x0), cvt_hi(x1));
          if (c + 1 < CPR) {
            constexpr int last = D / 8 - 1;
            const uint32_t y0 = __byte_perm(r[2], 0, 0x3120), y1 = __byte_perm(r[3], 0, 0x3120);
            mma<true>(o[2 * c + 2 <= last ? 2 * c + 2 : 0], p[kk], cvt_lo(y0), cvt_lo(y1));
            mma<true>(o[2 * c + 3 <= last ? 2 * c + 3 : 0], p[kk], cvt_hi(y0), cvt_hi(y1));
          }
        } else {
          mma<false>(o[c], p[kk], r[0], r[1]);
          mma<false>(o[c + 1], p[kk], r[2], r[3]);
        }
      }
    }
    if (hot[0] | hot[1]) {  // rare: the elements taken out above
      const int lg = w.ps_log2, pm = (1 << lg) - 1;
      for (int k = 0; k < TPW; ++k) {
        const int row = wt * TPW + k, t = t0 + row;
        if (!((row < 32 ? hot[0] : hot[1]) >> (row & 31) & 1)) continue;
        const int id = w.table[cur.b * w.tstride + (t >> lg)];
        const uint8_t *v = w.v + id * w.vps + ((static_cast<int64_t>(head) << lg) + (t & pm)) * C::DB;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x;
            if constexpr (E4M3) {
              const int d = 16 * (i / 2) + 4 * q4 + 2 * e + (i & 1);
              x = (v[d] & 0x7f) == 0x7f ? NAN : 0.0f;
            } else {
              const uint16_t u = reinterpret_cast<const uint16_t *>(v)[8 * i + 2 * q4 + e];
              x = (u & 0x7f80) == 0x7f80 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : 0.0f;
            }
            if (t < lim0) o[i][e] += x;
            if (t < lim1) o[i][2 + e] += x;
          }
      }
      __syncthreads();
      if (tid < 2) band[tid] = 0;
    }

    // --- next tile; at the end of the item or of the span, leave the partial result
    const bool last = cur.t + 1 == cur.nt || cur.x + 1 == hi;
    const uint32_t slot = (pre ? cur.j : cum1[cur.b] + cur.j) + blockIdx.x;
    if (cur.x + 1 < hi) step(cur);
    else ++cur.x;
    if (!last) continue;
    fresh = true;
    l0 += __shfl_xor_sync(~0u, l0, 1);
    l1 += __shfl_xor_sync(~0u, l1, 1);
    l0 += __shfl_xor_sync(~0u, l0, 2);
    l1 += __shfl_xor_sync(~0u, l1, 2);
    if constexpr (WT > 1) {
      float *jm = join + RT * C::OLD, *jl = jm + WT * RT;
      const int r = wr * 16 + g;
      __syncthreads();  // the join area of the item before is free
      if (q4 == 0) {
        jm[wt * RT + r] = M0, jm[wt * RT + r + 8] = M1;
        jl[wt * RT + r] = l0, jl[wt * RT + r + 8] = l1;
      }
      __syncthreads();
      float t0m = -INFINITY, t1m = -INFINITY;
#pragma unroll
      for (int v = 0; v < WT; ++v) {
        t0m = fmaxf(t0m, jm[v * RT + r]);
        t1m = fmaxf(t1m, jm[v * RT + r + 8]);
      }
      const float z0 = t0m == -INFINITY ? 0.0f : t0m, z1 = t1m == -INFINITY ? 0.0f : t1m;
      l0 = l1 = 0.0f;
#pragma unroll
      for (int v = 0; v < WT; ++v) {
        l0 += jl[v * RT + r] * ex2(jm[v * RT + r] - z0);
        l1 += jl[v * RT + r + 8] * ex2(jm[v * RT + r + 8] - z1);
      }
      const float c0 = ex2(M0 - z0), c1 = ex2(M1 - z1);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] *= c0, o[i][1] *= c0, o[i][2] *= c1, o[i][3] *= c1;
      M0 = t0m, M1 = t1m;
      float *a = join + r * C::OLD + q4 * 2, *c = a + 8 * C::OLD;
#pragma unroll
      for (int v = 0; v < WT; ++v) {  // the warps in turn: a fixed order of the sum
        if (wt == v) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            float2 *pa = reinterpret_cast<float2 *>(a + 8 * i), *pc = reinterpret_cast<float2 *>(c + 8 * i);
            if (v > 0) {
              const float2 x = *pa, y = *pc;
              o[i][0] += x.x, o[i][1] += x.y, o[i][2] += y.x, o[i][3] += y.y;
            }
            if (v + 1 < WT) {
              *pa = make_float2(o[i][0], o[i][1]);
              *pc = make_float2(o[i][2], o[i][3]);
            }
          }
        }
        if (v + 1 < WT) __syncthreads();
      }
      if (wt != WT - 1) continue;
    }
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int r = wr * 16 + g + 8 * a;
      if (row0 + r >= rows) continue;
      const float l = a ? l1 : l0, M = a ? M1 : M0;
      const float f = l == 0.0f ? 0.0f : 1.0f / l;
      const int64_t at = static_cast<int64_t>(slot) * RT + r;
      float *dst = P.po + at * D;
      if constexpr (E4M3) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          *reinterpret_cast<float4 *>(dst + 16 * c + 4 * q4) =
              make_float4(o[2 * c][2 * a] * f, o[2 * c + 1][2 * a] * f, o[2 * c][2 * a + 1] * f,
                          o[2 * c + 1][2 * a + 1] * f);
      } else {
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<float2 *>(dst + 8 * c + 2 * q4) =
              make_float2(o[c][2 * a] * f, o[c][2 * a + 1] * f);
      }
      if (q4 == 0) P.pl[at] = l == 0.0f ? -INFINITY : M - BIAS + log2f(l);
    }
  }
  cp_wait<0>();
}

template <int D, bool E4M3, int WR, int WT>
cudaError_t span_go(const SpanParams &p, int64_t tiles, int *grid, cudaStream_t s) {
  using C = SpanCfg<D, E4M3, WR, WT>;
  const int smem = C::FIXED + 8 * (p.w.B + 1);
  auto *f = span_kernel<D, E4M3, WR, WT>;
  static Slots slots;  // of this kernel, per device
  int sms = 0, occ = 0;
  const cudaError_t e = slots.get(reinterpret_cast<const void *>(f), C::NT, C::FIXED, C::FIXED + 8 * (kMaxB + 1),
                                  &sms, &occ);
  if (e != cudaSuccess) return e;
  // CTAs per SM: what registers allow, and what this call's shared memory does
  const int by_smem = kSmSmem / (smem + 1024);
  int64_t n = static_cast<int64_t>(sms) * (occ < by_smem ? occ : by_smem > 0 ? by_smem : 1);
  if (n > kMaxGrid) n = kMaxGrid;
  if (n > tiles) n = tiles;
  if (n < 1) n = 1;
  *grid = static_cast<int>(n);
  f<<<*grid, C::NT, smem, s>>>(p);
  return cudaGetLastError();
}

template <int D, bool E4M3>
cudaError_t span_any(const SpanParams &p, int wr, int64_t tiles, int *grid, cudaStream_t s) {
  switch (wr) {
    case 1: return span_go<D, E4M3, 1, 4>(p, tiles, grid, s);
    case 2: return span_go<D, E4M3, 2, 2>(p, tiles, grid, s);
    case 3: return span_go<D, E4M3, 3, 1>(p, tiles, grid, s);
    default: return span_go<D, E4M3, 4, 1>(p, tiles, grid, s);
  }
}

}  // namespace kv
