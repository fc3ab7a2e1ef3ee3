// kv_dense.cuh -- the dense kernel of spec_attend: partial attention of the
// query rows of all sequences over the prefix that they share.
//
// Mathematics: as in the span kernel (kv_span.cuh), but the stored exponents
// go into the operands: within a tile of 128 tokens the keys enter as
// y 2^(ek - E), the values as u 2^(ev - F), E and F seven below the tile's
// largest exponents.  That is exact in float16 for tokens down to 2^22 below
// the tile's largest, so that a score needs one multiplication, by a factor
// that all of a row's scores of the tile share, and the weights (of 16 bits, as
// there) are P_j = 2^(z_j + F - M), l = sum_tiles 2^-F sum_j P_j.  l is kept 2^-25
// times as large: a tile of zeros (F = -107) adds 2^(15 + 107 - 25) a token, which
// 2^30 tokens keep finite, one of the largest exponent (F = 112) 2^(11 - 112 - 25),
// still normal.  The running maximum M follows only where a row's maximum passes
// it by more than 4 (float16 P with a bias of 2^11; 8 in bfloat16): otherwise
// nothing that is summed is scaled (a published technique).
//
// Bound: the tensor cores, and next to them the exponentials (16384 for each
// 128 x 128 tile beside 2 x 512 cycles of products).  A CTA takes 256 query
// rows of one key/value head, as two tiles of 128 rows that share each key and
// value tile.  A key tile is taken in two halves of 64 tokens with a score buffer
// each, so that a row tile's next scores are formed beside its softmax, and the
// other row tile's products beside both.  Scores (2 x 2 x 64 columns) and outputs
// are in TMEM; a softmax thread has a row of its own, so nothing is reduced across
// lanes; the weights go back to TMEM over the scores, as the left operand of P V.
//
// Roles: warps 0-3 and 4-7 queries, softmax and output of a row tile each; warps
// 8-11 bring keys, 12-15 values into shared memory (e4m3 through registers as
// float16, a tile ahead, bfloat16 by asynchronous copies); warps 16 and 17
// issue the products of a row tile each, as soon as its operands are there.
// Two stages of keys and of values.
//
// Measured: 256 x 9 queries of 32 heads (9216 rows a key/value head of 128) over
// 8192 e4m3 tokens 437 us, 707 TFLOP/s, 37 % of the products' rate; tensor pipe 31 %
// active, one instruction issued every other cycle, and of 10 warps per issue 2.2
// wait for instructions: the roles' code is larger than the nearest instruction cache.
// Heads of 128, 96 and 64 in e4m3 spill 80, 32 and 20 bytes a thread.
#pragma once

#include <cuda_fp16.h>

#include "kv_span.h"
#include "kv_tc.cuh"

namespace kv {

constexpr int DN_NT = 640;     // threads
constexpr int DN_FETCH = 128;  // of them loading keys; as many load values
constexpr int DN_TILE = 128;   // key tokens per tile
constexpr int DN_RING = 8;     // tiles whose exponents are kept
// Registers per thread: at launch (5 warpgroups), softmax (2), loading (2), the rest.
constexpr int DN_REGS = 96, DN_SOFT = 120, DN_LOAD = 96, DN_REST = 48;
static_assert(2 * DN_SOFT + 2 * DN_LOAD + DN_REST <= 5 * DN_REGS, "registers");

template <int D>
struct DenseCfg {
  static constexpr int SUBS = (D + 63) / 64;        // chunks of 64 elements (128 bytes)
  static constexpr int OP = SUBS * DN_TILE * 128;   // bytes of an operand of 128 rows
  static constexpr int Q = 0, K = 2 * OP, V = 4 * OP, OPER = 6 * OP;
};

struct DenseShared {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t sfull[2][2], pfull[2][2];         // per row tile and score buffer
  uint64_t odone[2], ofull[2], drain[2];     // per row tile
  uint64_t consts[DN_RING], qfull[2];
  int exps[2][DN_RING];      // E, F
  uint32_t tmem, dead;
  uint32_t sum[DN_NT / 32];
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(DN_NT, 1) dense_kernel(const __grid_constant__ SpanParams P) {
  using C = DenseCfg<D>;
  constexpr float BIAS = E4M3 ? 11.0f : 0.0f, SLACK = E4M3 ? 4.0f : 8.0f;
  constexpr float SUM = E4M3 ? 0x1p-25f : 1.0f, SUM_LOG = E4M3 ? 25.0f : 0.0f;  // factor of the sum of weights
  constexpr float kNone = -1e30f;  // maximum of no scores
  extern __shared__ uint8_t raw[];
  uint8_t *sm = raw + (-s32(raw) & 1023);  // operands: 1024-byte aligned
  DenseShared &S = *reinterpret_cast<DenseShared *>(sm + C::OPER);
  uint32_t *cum = reinterpret_cast<uint32_t *>(sm + C::OPER + sizeof(DenseShared));  // B + 1
  const uint32_t base = s32(sm);

  const View &w = P.w;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = P.G, B = w.B;

  // --- rows before each sequence
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(s32(&S.kfull[i]), E4M3 ? DN_FETCH / 32 : DN_FETCH), bar_init(s32(&S.kempty[i]), 2);
      bar_init(s32(&S.vfull[i]), E4M3 ? DN_FETCH / 32 : DN_FETCH), bar_init(s32(&S.vempty[i]), 2);
      for (int k = 0; k < 2; ++k) bar_init(s32(&S.sfull[i][k]), 1), bar_init(s32(&S.pfull[i][k]), 4);
      bar_init(s32(&S.odone[i]), 1), bar_init(s32(&S.ofull[i]), 1), bar_init(s32(&S.drain[i]), 1);
    }
    for (int i = 0; i < DN_RING; ++i) bar_init(s32(&S.consts[i]), 2);
    bar_init(s32(&S.qfull[0]), 4), bar_init(s32(&S.qfull[1]), 4);
    S.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) tmem_alloc(&S.tmem, 512);
  const int per = (B + DN_NT - 1) / DN_NT, b0 = min(tid * per, B), b1 = min(b0 + per, B);
  uint32_t a = 0;
  for (int b = b0; b < b1; ++b) {
    int own, n;
    row_shape(w, b, own, n);
    cum[b] = a;
    a += n * G;
  }
  uint32_t e = a;
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(~0u, e, o);
    if (lane >= o) e += t;
  }
  if (lane == 31) S.sum[warp] = e;
  tc_before();
  __syncthreads();
  tc_after();
  e -= a;
  uint32_t rows = 0;
  for (int v = 0; v < DN_NT / 32; ++v) {
    if (v < warp) e += S.sum[v];
    rows += S.sum[v];
  }
  for (int b = b0; b < b1; ++b) {
    cum[b] += e;
    if (blockIdx.x == 0) P.plan.rows[b] = cum[b];
  }
  if (tid == 0) {
    cum[B] = rows;
    if (blockIdx.x == 0) P.plan.rows[B] = rows;
  }
  __syncthreads();
  const uint32_t tmem = S.tmem;
  volatile uint32_t *dead = &S.dead;
  const int nt = (w.prefix + DN_TILE - 1) / DN_TILE;      // key tiles of an item
  const int nj = (rows + DN_ROWS - 1) / DN_ROWS;          // items of a key/value head
  const uint32_t W = static_cast<uint32_t>(nt) * nj * w.Hkv, ctas = min(gridDim.x, W);
  const bool idle = blockIdx.x >= ctas;
  const uint32_t lo = idle ? 0 : static_cast<uint32_t>(static_cast<uint64_t>(W) * blockIdx.x / ctas);
  const uint32_t hi = idle ? 0 : static_cast<uint32_t>(static_cast<uint64_t>(W) * (blockIdx.x + 1) / ctas);
  const int tiles = static_cast<int>(hi - lo);
  const int item0 = idle ? 0 : lo / nt, first0 = idle ? 0 : lo - item0 * nt;

  // All products that this thread issued are done, also where a wait gave up:
  // TMEM goes back behind this.
  auto drained = [&](int i) {
    mma_commit(s32(&S.drain[i]));
    uint32_t late = 0;
    bar_wait(s32(&S.drain[i]), 0, &late);
    if (late) *dead = 1;
  };

  if (warp < 8) {
    regs_to<DN_SOFT, DN_REGS>();
    // ================================================= softmax and output
    const int half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 TMEM lanes a warp
    const uint32_t oc = tmem + lanes + 256 + half * 128;
    const uint32_t wb = base + C::Q + half * C::OP + (warp & 3) * 32 * 128;  // the warp's query rows
    const int r = tid;  // row of the item
    int item = item0, tt = first0;
    float M = kNone, l = 0.0f, qc = 0.0f;
    float kt = 0.0f, F = 0.0f, invF = 1.0f;  // of the tile
    bool fresh = true;
    int g = 0;  // items
    for (int u = 0; u < 2 * tiles; ++u) {
      const int t = u >> 1;  // half u & 1 of tile t
      if (fresh) {  // the row's query; the products with the item before are done
        const uint32_t row = item % nj * DN_ROWS + r;
        int64_t off = -1;
        if (row < rows) {
          int b = 0, h = B;
          while (h - b > 1) {
            const int m = (b + h) >> 1;
            if (cum[m] <= row) b = m;
            else h = m;
          }
          const int y = row - cum[b], i = y / G;
          off = b * P.qs0 + i * P.qs1 + (item / nj * G + y - i * G) * P.qs2;
        }
        // into shared memory by the warp's 32 rows together, neighbouring lanes
        // neighbouring chunks; then a row by its own thread
        constexpr int CH = D / 8;
        uint4 v[CH];
        auto at = [&](int y, int c) {
          return wb + (c >> 3) * (DN_TILE * 128) + y * 128 + (((c ^ y) & 7) << 4);
        };
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int x = lane + 32 * k, y = x / CH;
          const int64_t o = __shfl_sync(~0u, off, y);
          v[k] = make_uint4(0, 0, 0, 0);
          if (o >= 0) {
            const __nv_bfloat16 *src = P.q + o + 8 * (x - y * CH);
            if (P.qvec) {
              v[k] = __ldg(reinterpret_cast<const uint4 *>(src));
            } else {
              const uint16_t *u = reinterpret_cast<const uint16_t *>(src);
              v[k] = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int x = lane + 32 * k, y = x / CH;
          sts128(at(y, x - y * CH), v[k]);
        }
        qc = P.c;
        if constexpr (E4M3) {
          // bring the row's largest finite magnitude to [2^10, 2^11): exact in
          // float16 for all elements above 2^-28 of it
          __syncwarp();
          uint32_t m = 0;
          auto most = [&](uint32_t u) {
            const uint32_t a = u & 0x7fffu, b = u >> 16 & 0x7fffu;
            m = max(m, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
          };
#pragma unroll
          for (int k = 0; k < CH; ++k) {
            v[k] = lds128(at(lane, k));
            most(v[k].x), most(v[k].y), most(v[k].z), most(v[k].w);
          }
          const int eq = max(static_cast<int>(m >> 7) - 127 - 10, -100);
          qc = P.c * pow2i(eq);
          const float f = pow2i(-eq);
          auto two = [&](uint32_t u) {
            return pack<true>(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xffff0000u) * f);
          };
#pragma unroll
          for (int k = 0; k < CH; ++k)
            sts128(at(lane, k), make_uint4(two(v[k].x), two(v[k].y), two(v[k].z), two(v[k].w)));
        }
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(s32(&S.qfull[half]));
        M = kNone, l = 0.0f;
      }
      if (!(u & 1)) {
        kt = qc;
        if constexpr (E4M3) {
          bar_wait(s32(&S.consts[t % DN_RING]), t / DN_RING & 1, dead);
          const int fe = S.exps[1][t % DN_RING];
          kt = qc * pow2i(S.exps[0][t % DN_RING]);
          F = static_cast<float>(fe);
          invF = pow2i(-fe - 13) * (SUM * 0x1p13f);  // 2^-F SUM, subnormal for the largest F
        }
      }
      const uint32_t sc = tmem + lanes + half * 128 + (u & 1) * 64;
      bar_wait(s32(&S.sfull[half][u & 1]), t & 1, dead);
      tc_after();
      float s[64];
#pragma unroll
      for (int c = 0; c < 64; c += 16) tmem_ld16(sc + c, s + c);
      tmem_wait_ld(s, 64);
      const int n = w.prefix - tt * DN_TILE - (u & 1) * 64;  // tokens from here on
      float ks = kt;  // still to be multiplied by
      if (n < 64) {   // masked behind the multiplication: a factor of 0 would make NaN of -inf
        ks = 1.0f;
#pragma unroll
        for (int c = 0; c < 64; ++c) s[c] = c >= n ? -INFINITY : s[c] * kt;
      }
      float m2[2] = {s[0], s[1]};
#pragma unroll
      for (int c = 2; c < 62; c += 4) m2[0] = max3(m2[0], s[c], s[c + 1]), m2[1] = max3(m2[1], s[c + 2], s[c + 3]);
      const float m = fmaf(max3(fmaxf(m2[0], m2[1]), s[62], s[63]), ks, F);
      if (__any_sync(~0u, fresh || m > M + SLACK)) {
        const float nm = fmaxf(M, m), f = ex2(M - nm);
        M = nm;
        l *= f;
        if (!fresh) {
          bar_wait(s32(&S.odone[half]), u - 1 & 1, dead);  // products up to the half tile before
          tc_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tmem_ld16(oc + c, o);
            tmem_wait_ld(o, 16);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= f;
            tmem_st16(oc + c, reinterpret_cast<const uint32_t *>(o));
          }
          tmem_wait_st();
        }
      }
      const float2 k2 = {ks, ks}, b2 = {F - M + BIAS, F - M + BIAS};
      float2 acc[2] = {{0, 0}, {0, 0}};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 z = fma2(make_float2(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), k2, b2);
          z.x = ex2(z.x), z.y = ex2(z.y);
          acc[i & 1] = add2(acc[i & 1], z);
          p[i] = pack<E4M3>(z.x, z.y);
        }
        tmem_st16(sc + 16 * c, p);  // over scores that are read
      }
      acc[0] = add2(acc[0], acc[1]);
      l = fmaf(acc[0].x + acc[0].y, invF, l);
      tmem_wait_st();
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive(s32(&S.pfull[half][u & 1]));

      const bool last = (u & 1) && (tt + 1 == nt || t + 1 == tiles);
      if (last) {
        const int64_t at = static_cast<int64_t>(item + blockIdx.x) * DN_ROWS + r;
        const bool there = static_cast<uint32_t>(item % nj * DN_ROWS + r) < rows;
        const float f = l == 0.0f ? 0.0f : 1.0f / l;
        if (there) P.pl[at] = l == 0.0f ? -INFINITY : M - (BIAS - SUM_LOG) + log2f(l);
        bar_wait(s32(&S.ofull[half]), g++ & 1, dead);
        tc_after();
        // rows leave through the shared memory of the item's queries, 16 columns
        // at a time in two buffers, so that a store covers whole sectors
        float *dst = P.po + (at - lane) * D + (lane & 3) * 4;
        const uint32_t there32 = __ballot_sync(~0u, there);
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          const uint32_t buf = wb + (c & 16) * 128;
          float o[16];
          tmem_ld16(oc + c, o);
          tmem_wait_ld(o, 16);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sts128(buf + lane * 64 + ((i ^ lane >> 1) & 3) * 16,
                   make_uint4(__float_as_uint(o[4 * i] * SUM * f), __float_as_uint(o[4 * i + 1] * SUM * f),
                              __float_as_uint(o[4 * i + 2] * SUM * f), __float_as_uint(o[4 * i + 3] * SUM * f)));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int y = 8 * i + (lane >> 2);
            const uint4 x = lds128(buf + y * 64 + ((lane ^ y >> 1) & 3) * 16);
            if (there32 >> y & 1) *reinterpret_cast<uint4 *>(dst + y * D + c) = x;
          }
        }
        __syncwarp();
        tc_before();
      }
      fresh = last;
      if ((u & 1) && ++tt == nt) tt = 0, ++item;
    }
  } else if (warp < 16) {
    regs_to<DN_LOAD, DN_REGS>();
    // ===================================== keys (four warps), values (four)
    const bool vs = warp >= 12;
    const int p = tid & DN_FETCH - 1;
    const uint8_t *src = vs ? w.v : w.k;
    const int64_t stride = vs ? w.vps : w.kps;
    const uint32_t dst0 = base + (vs ? C::V : C::K);
    uint64_t *full = vs ? S.vfull : S.kfull, *empty = vs ? S.vempty : S.kempty;
    const int lg = w.ps_log2, pm = (1 << lg) - 1;
    int item = item0, tt = first0;
    if constexpr (E4M3) {
      constexpr int CPR = D / 16;                     // 16-byte chunks of a row
      constexpr int PASS = DN_TILE * CPR / DN_FETCH;  // of a tile, per thread
      static_assert(DN_TILE * CPR % DN_FETCH == 0, "chunks");
      int id[PASS], ide = -1;  // page ids of the tile to be fetched next
      auto pages = [&](int tile) {
        const int t0 = tile * DN_TILE;
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
          const int tok = t0 + (p + i * DN_FETCH) / CPR;
          id[i] = tok < w.prefix ? ldg_now(w.ptable + (tok >> lg)) : -1;
        }
        ide = t0 + 4 * lane < w.prefix ? ldg_now(w.ptable + (t0 + 4 * lane >> lg)) : -1;
      };
      uint4 q[PASS] = {};
      uint32_t ex = 0;  // exponents of the lane's four tokens, the first `live` of them there
      int live = 0;
      // A chunk without a page is read from page 0 and put to zero in store(): the
      // loads stand in a row without branches.
      auto fetch = [&](int it, int tile) {
        if (w.n_pages == 0) return;
        const uint32_t row0 = static_cast<uint32_t>(it / nj) << lg;
        const int t0 = tile * DN_TILE;
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
          const int x = p + i * DN_FETCH, row = x / CPR;
          const uint32_t pg = static_cast<uint32_t>(id[i]) < static_cast<uint32_t>(w.n_pages) ? id[i] : 0;
          q[i] = ldg_now16(src + pg * stride + (row0 + (t0 + row & pm)) * D + (x - row * CPR) * 16);
        }
        // (masked when it is used: nothing here waits for a load)
        live = static_cast<uint32_t>(ide) < static_cast<uint32_t>(w.n_pages) ? min(max(w.prefix - t0 - 4 * lane, 0), 4) : 0;
        ex = ldg_now32((vs ? w.ve : w.ke) + ((static_cast<int64_t>(live ? ide : 0) * w.Hkv + it / nj) << lg) +
                       (t0 + 4 * lane & pm));
      };
      auto store = [&](uint32_t dst, int E) {
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
          const int x = p + i * DN_FETCH, row = x / CPR, f = 2 * (x - row * CPR);
          const int e = static_cast<int8_t>(__shfl_sync(~0u, ex, row >> 2) >> 8 * (row & 3));
          const float one = pow2i(max(e - E, -126));  // e - E <= 7
          const uint32_t two = pack<true>(one, one), is = e == -128 ? 0u : ~0u;
          const __half2 sc = *reinterpret_cast<const __half2 *>(&two);
          auto scaled = [&](uint32_t h) {
            const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&h), sc);
            return *reinterpret_cast<const uint32_t *>(&y);
          };
          const uint4 b = make_uint4(q[i].x & is, q[i].y & is, q[i].z & is, q[i].w & is);
          const uint4 lo4 = make_uint4(scaled(cvt_lo(b.x)), scaled(cvt_hi(b.x)), scaled(cvt_lo(b.y)), scaled(cvt_hi(b.y)));
          const uint4 hi4 = make_uint4(scaled(cvt_lo(b.z)), scaled(cvt_hi(b.z)), scaled(cvt_lo(b.w)), scaled(cvt_hi(b.w)));
          const uint32_t to = dst + (f >> 3) * (DN_TILE * 128) + row * 128;
          const uint32_t c0 = ((f ^ row) & 7) << 4, c1 = ((f + 1 ^ row) & 7) << 4;
          const bool swap = f & 8;  // lanes of one row: all eight chunk positions at once
          sts128(to + (swap ? c1 : c0), swap ? hi4 : lo4);
          sts128(to + (swap ? c0 : c1), swap ? lo4 : hi4);
        }
      };
      // the loads of a tile are issued when the tile before is stored
      if (tiles > 0) pages(tt), fetch(item, tt);
      for (int t = 0; t < tiles; ++t) {
        if (live < 4) {  // -128 where there is no token
          const uint32_t in = (1u << 8 * live) - 1;
          ex = (ex & in) | (0x80808080u & ~in);
        }
        int E = -128;  // seven below the tile's largest exponent
#pragma unroll
        for (int i = 0; i < 4; ++i) E = max(E, static_cast<int>(static_cast<int8_t>(ex >> 8 * i)));
        E = max(__reduce_max_sync(~0u, E), kExpMin) - 7;
        if (p == 0) {
          S.exps[vs][t % DN_RING] = E;
          bar_arrive(s32(&S.consts[t % DN_RING]));
        }
        if (++tt == nt) tt = 0, ++item;
        if (t + 1 < tiles) pages(tt);
        if (t >= 2) bar_wait(s32(empty + (t & 1)), (t >> 1) - 1 & 1, dead);
        store(dst0 + (t & 1) * C::OP, E);
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(s32(full + (t & 1)));
        if (t + 1 < tiles) fetch(item, tt);
      }
    } else {
      constexpr int CPR = D / 8;
      for (int t = 0; t < tiles; ++t) {
        if (t >= 2) bar_wait(s32(empty + (t & 1)), (t >> 1) - 1 & 1, dead);
        const uint32_t row0 = static_cast<uint32_t>(item / nj) << lg, dst = dst0 + (t & 1) * C::OP;
#pragma unroll
        for (int i = 0; i < CPR; ++i) {
          const int x = p + i * DN_FETCH, row = x / CPR, f = x - row * CPR, tok = tt * DN_TILE + row;
          const int id = tok < w.prefix ? __ldg(w.ptable + (tok >> lg)) : -1;
          const bool ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(w.n_pages);
          const uint32_t at = ((row0 + (tok & pm)) * D + f * 8) * 2;
          cp16(dst + (f >> 3) * (DN_TILE * 128) + row * 128 + (((f ^ row) & 7) << 4),
               ok ? src + id * stride + at : src, ok);
        }
        // arrives when this thread's copies are in
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(s32(full + (t & 1))) : "memory");
        if (++tt == nt) tt = 0, ++item;
      }
      cp_wait<0>();
    }
  } else {
    regs_to<DN_REST, DN_REGS>();
    // =========================================================== products
    if (warp < 18) {
    // one lane issues, chosen by elect.sync, and all that its products are
    // described by is the warp's: kept in uniform registers, where they are wanted
    const int half = __shfl_sync(~0u, warp, 0) - 16;
    const uint32_t base = __shfl_sync(~0u, s32(sm), 0), tmem = __shfl_sync(~0u, S.tmem, 0);
    const int tiles = __shfl_sync(~0u, static_cast<int>(hi - lo), 0);
    const int nt = __shfl_sync(~0u, (w.prefix + DN_TILE - 1) / DN_TILE, 0);
    constexpr uint32_t sdesc = mma_desc(E4M3, 128, 64, false, false);
    constexpr uint32_t odesc = mma_desc(E4M3, 128, D, false, true);
    const uint64_t qd = smem_desc(base + C::Q + half * C::OP, 16, 1024), kd = smem_desc(base + C::K, 16, 1024);
    const uint64_t vd = smem_desc(base + C::V, DN_TILE * 128, 1024);
    const uint32_t sc = tmem + half * 128, oc = tmem + 256 + half * 128;
    int g = 0;
    // Half tile u, tile tt of its item: scores into buffer u & 1 ...
    auto scores = [&](int u, int tt) {
      const int t = u >> 1, st = t & 1;
      if (!(u & 1) && (t == 0 || tt == 0)) bar_wait(s32(&S.qfull[half]), g++ & 1, dead);
      // the weights of half tile u - 2 are read; behind an item, all of it is done
      const bool behind = u > 0 && !(u & 1) && tt == 0;
      if (u >= 2) bar_wait(s32(&S.odone[half]), behind ? u - 1 & 1 : u & 1, dead);
      if (!(u & 1)) bar_wait(s32(&S.kfull[st]), t >> 1 & 1, dead);
      if (!E4M3) fence_async();  // the copies' writes, before the products' reads
      tc_after();
      if (elected() && !*dead) {
        const uint64_t kk = kd + st * (C::OP >> 4) + (u & 1) * (64 * 128 >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int off = (k >> 2) * (DN_TILE * 128) + (k & 3) * 32 >> 4;
          mma_ss(sc + (u & 1) * 64, qd + off, kk + off, sdesc, k > 0);
        }
        mma_commit(s32(&S.sfull[half][u & 1]));
        if (u & 1) mma_commit(s32(&S.kempty[st]));
      }
      __syncwarp();
    };
    // ... and its weighted values.
    auto values = [&](int u, int tt) {
      const int t = u >> 1, st = t & 1;
      const bool last = (u & 1) && (tt + 1 == nt || t + 1 == tiles);
      // (parities tell one phase from the next only: no phase is skipped)
      if (last) bar_wait(s32(&S.odone[half]), u - 1 & 1, dead);
      if (!(u & 1)) bar_wait(s32(&S.vfull[st]), t >> 1 & 1, dead);
      if (!E4M3) fence_async();
      bar_wait(s32(&S.pfull[half][u & 1]), t & 1, dead);
      tc_after();
      if (elected() && !*dead) {
        const uint64_t vv = vd + st * (C::OP >> 4) + (u & 1) * (64 * 128 >> 4);
        const bool fresh = !(u & 1) && (t == 0 || tt == 0);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ts(oc, sc + (u & 1) * 64 + 8 * k, vv + (k * 2048 >> 4), odesc, !fresh || k > 0);
        mma_commit(s32(&S.odone[half]));
        if (u & 1) mma_commit(s32(&S.vempty[st]));
        if (last) mma_commit(s32(&S.ofull[half]));
      }
      __syncwarp();
    };
    int tt = __shfl_sync(~0u, first0, 0);
    for (int t = 0; t < tiles; ++t) {
      // the next half tile's scores before these weights, except behind an item's
      // last, whose output has to be out before the next item's queries are in
      const bool last = tt + 1 == nt || t + 1 == tiles;
      if (t == 0 || tt == 0) scores(2 * t, tt);
      scores(2 * t + 1, tt);
      values(2 * t, tt);
      if (!last) scores(2 * t + 2, tt + 1);
      values(2 * t + 1, tt);
      if (++tt == nt) tt = 0;
    }
    if (elected()) drained(half);
    __syncwarp();
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 16) tmem_free(tmem, 512);
  if (tid == 0) P.plan.lost[blockIdx.x] = S.dead;
}

template <int D, bool E4M3>
cudaError_t dense_go(const SpanParams &p, int64_t tiles, int *grid, cudaStream_t s) {
  constexpr int fixed = 1024 + DenseCfg<D>::OPER + sizeof(DenseShared);
  static_assert(fixed + 4 * (kMaxB + 1) <= 232448, "shared memory");
  auto *f = dense_kernel<D, E4M3>;
  static Slots slots;
  int sms = 0, occ = 0;
  constexpr int smem = fixed + 4 * (kMaxB + 1);
  const cudaError_t e = slots.get(reinterpret_cast<const void *>(f), DN_NT, smem, smem, &sms, &occ);
  if (e != cudaSuccess) return e;
  int64_t n = sms < kMaxDense ? sms : kMaxDense;
  if (n > tiles) n = tiles;
  if (n < 1) n = 1;
  *grid = static_cast<int>(n);
  f<<<*grid, DN_NT, fixed + 4 * (kMaxB + 1), s>>>(p);
  return cudaGetLastError();
}

}  // namespace kv
