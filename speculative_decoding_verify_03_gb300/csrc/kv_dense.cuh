// kv_dense.cuh -- the dense kernel of spec_attend: partial attention of the
// query rows of all sequences over the prefix that they share.
//
// Mathematics: as in the span kernel (kv_span.cuh), but the stored exponents
// go into the operands: within a tile of 128 tokens the keys enter as
// y 2^(ek - E), the values as u 2^(ev - F), E and F seven below the tile's
// largest exponents.  That is exact in float16 for tokens down to 2^22 below
// the tile's largest, so that a score needs one multiplication, by a factor
// that all of a row's scores of the tile share, and the weights are
// P_j = 2^(z_j + F - M), l = sum_tiles 2^-F sum_j P_j.  The running maximum M
// follows only where a row's maximum passes it by more than 4 (float16 P with
// a bias of 2^11; 8 in bfloat16): otherwise nothing that is summed is scaled.
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
// 8-15 bring keys and values into shared memory (e4m3 through registers as
// float16, a tile ahead, bfloat16 by asynchronous copies); warps 16 and 17
// issue the products of a row tile each, as soon as its operands are there.
// Two stages of keys and of values.
#pragma once

#include <cuda_fp16.h>

#include "kv_span.h"
#include "kv_tc.cuh"

namespace kv {

constexpr int DN_NT = 640;     // threads
constexpr int DN_FETCH = 256;  // of them loading
constexpr int DN_TILE = 128;   // key tokens per tile
constexpr int DN_RING = 8;     // tiles whose exponents are kept
// Registers per thread: at launch (5 warpgroups), softmax (2), loading (2), the rest.
constexpr int DN_REGS = 96, DN_SOFT = 136, DN_LOAD = 80, DN_REST = 48;
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
  int2 exps[DN_RING];        // E, F
  uint32_t qmax[DN_ROWS];    // largest finite magnitude of a row, as bfloat16 bits
  uint32_t tmem, dead;
  uint32_t sum[DN_NT / 32];
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(DN_NT, 1) dense_kernel(const __grid_constant__ SpanParams P) {
  using C = DenseCfg<D>;
  constexpr float BIAS = E4M3 ? 11.0f : 0.0f, SLACK = E4M3 ? 4.0f : 8.0f;
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
    for (int i = 0; i < DN_RING; ++i) bar_init(s32(&S.consts[i]), 1);
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
    const int r = tid;  // row of the item
    int item = item0, tt = first0;
    float M = kNone, l = 0.0f, qc = 0.0f;
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
        // the warp's 32 rows together: neighbouring lanes, neighbouring chunks
        constexpr int CH = D / 8;
        uint4 v[CH];
        if constexpr (E4M3) S.qmax[r] = 0;
        __syncwarp();
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
        qc = P.c;
        if constexpr (E4M3) {
          // bring each row's largest finite magnitude to [2^10, 2^11): exact in
          // float16 for all elements above 2^-28 of it
#pragma unroll
          for (int k = 0; k < CH; ++k) {
            uint32_t m = 0;
            auto most = [&](uint32_t u) {
              const uint32_t a = u & 0x7fffu, b = u >> 16 & 0x7fffu;
              m = max(m, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
            };
            most(v[k].x), most(v[k].y), most(v[k].z), most(v[k].w);
            atomicMax(&S.qmax[warp * 32 + (lane + 32 * k) / CH], m);
          }
          __syncwarp();
          const int eq = max(static_cast<int>(S.qmax[r] >> 7) - 127 - 10, -100);
          qc = P.c * pow2i(eq);
#pragma unroll
          for (int k = 0; k < CH; ++k) {
            const float f = pow2i(-__shfl_sync(~0u, eq, (lane + 32 * k) / CH));
            auto two = [&](uint32_t u) {
              return pack<true>(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xffff0000u) * f);
            };
            v[k] = make_uint4(two(v[k].x), two(v[k].y), two(v[k].z), two(v[k].w));
          }
        }
        const uint32_t qb = base + C::Q + half * C::OP + (warp & 3) * 32 * 128;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const int x = lane + 32 * k, y = x / CH, c = x - y * CH;
          sts128(qb + (c >> 3) * (DN_TILE * 128) + y * 128 + (((c ^ y) & 7) << 4), v[k]);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(s32(&S.qfull[half]));
        M = kNone, l = 0.0f;
      }
      float kt = qc, F = 0.0f, invF = 1.0f;
      if constexpr (E4M3) {
        bar_wait(s32(&S.consts[t % DN_RING]), t / DN_RING & 1, dead);
        const int2 x = S.exps[t % DN_RING];
        kt = qc * pow2i(x.x);
        F = static_cast<float>(x.y);
        invF = pow2i(-x.y);
      }
      const uint32_t sc = tmem + lanes + half * 128 + (u & 1) * 64;
      bar_wait(s32(&S.sfull[half][u & 1]), t & 1, dead);
      tc_after();
      float s[64];
#pragma unroll
      for (int c = 0; c < 64; c += 16) tmem_ld16(sc + c, s + c);
      tmem_wait_ld(s, 64);
      const int n = w.prefix - tt * DN_TILE - (u & 1) * 64;  // tokens from here on
      if (n < 64) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c >= n) s[c] = -INFINITY;
      }
      float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < 64; c += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) m4[i] = fmaxf(m4[i], s[c + i]);
      const float m = fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), kt, F);
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
      const float2 k2 = {kt, kt}, b2 = {F - M + BIAS, F - M + BIAS};
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
        if (there) P.pl[at] = l == 0.0f ? -INFINITY : M - BIAS + log2f(l);
        bar_wait(s32(&S.ofull[half]), g++ & 1, dead);
        tc_after();
        float *dst = P.po + at * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          tmem_ld16(oc + c, o);
          tmem_wait_ld(o, 16);
          if (there) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4 *>(dst + c + i) = make_float4(o[i] * f, o[i + 1] * f, o[i + 2] * f, o[i + 3] * f);
          }
        }
        tc_before();
      }
      fresh = last;
      if ((u & 1) && ++tt == nt) tt = 0, ++item;
    }
  } else if (warp < 16) {
    regs_to<DN_LOAD, DN_REGS>();
    // ============================================ queries, keys and values
    const int p = tid - 256;
    const int lg = w.ps_log2, pm = (1 << lg) - 1;
    int item = item0, tt = first0;
    if constexpr (E4M3) {
      constexpr int CPR = D / 16, ALL = DN_TILE * CPR;      // 16-byte chunks of a row, of a tile
      constexpr int PASS = (ALL + DN_FETCH - 1) / DN_FETCH;  // chunks per thread
      int id[PASS], ide = -1;  // page ids of the tile to be fetched next
      auto pages = [&](int tile) {
        const int t0 = tile * DN_TILE;
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
          const int x = p + i * DN_FETCH, tok = t0 + x / CPR;
          id[i] = (ALL % DN_FETCH == 0 || x < ALL) && tok < w.prefix ? ldg_now(w.ptable + (tok >> lg)) : -1;
        }
        ide = t0 + 4 * lane < w.prefix ? ldg_now(w.ptable + (t0 + 4 * lane >> lg)) : -1;
      };
      auto fetch = [&](uint4 (&q)[PASS], const uint8_t *src, int64_t stride, int it, int tile) {
        const uint32_t row0 = static_cast<uint32_t>(it / nj) << lg;
        const int t0 = tile * DN_TILE;
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
          const int x = p + i * DN_FETCH, row = x / CPR;
          q[i] = make_uint4(0, 0, 0, 0);
          if (static_cast<uint32_t>(id[i]) < static_cast<uint32_t>(w.n_pages))
            q[i] = ldg_now16(src + id[i] * stride + (row0 + (t0 + row & pm)) * D + (x - row * CPR) * 16);
        }
      };
      // exponents of the lane's four tokens; -128 where there is none
      auto exps = [&](const int8_t *src, int it, int tile) {
        const int tok = tile * DN_TILE + 4 * lane, n = w.prefix - tok;
        uint32_t v = 0x80808080u;
        if (static_cast<uint32_t>(ide) < static_cast<uint32_t>(w.n_pages)) {
          v = ldg_now32(src + ((static_cast<int64_t>(ide) * w.Hkv + it / nj) << lg) + (tok & pm));
          if (n < 4) {
            const uint32_t in = (1u << 8 * n) - 1;
            v = (v & in) | (0x80808080u & ~in);
          }
        }
        return v;
      };
      auto top = [&](uint32_t v) {  // seven below the tile's largest
        int m = -128;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, static_cast<int>(static_cast<int8_t>(v >> 8 * i)));
        return max(__reduce_max_sync(~0u, m), kExpMin) - 7;
      };
      auto store = [&](uint32_t dst, const uint4 (&q)[PASS], uint32_t v, int E) {
#pragma unroll
        for (int i = 0; i < PASS; ++i) {
          const int x = p + i * DN_FETCH, row = x / CPR, f = 2 * (x - row * CPR);
          const uint32_t word = __shfl_sync(~0u, v, row >> 2);
          if (ALL % DN_FETCH && x >= ALL) break;
          const int d = static_cast<int8_t>(word >> 8 * (row & 3)) - E;  // <= 7
          const float one = pow2i(max(d, -126));
          const uint32_t two = pack<true>(one, one);
          const __half2 sc = *reinterpret_cast<const __half2 *>(&two);
          auto scaled = [&](uint32_t h) {
            const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&h), sc);
            return *reinterpret_cast<const uint32_t *>(&y);
          };
          const uint4 lo4 = make_uint4(scaled(cvt_lo(q[i].x)), scaled(cvt_hi(q[i].x)), scaled(cvt_lo(q[i].y)),
                                       scaled(cvt_hi(q[i].y)));
          const uint4 hi4 = make_uint4(scaled(cvt_lo(q[i].z)), scaled(cvt_hi(q[i].z)), scaled(cvt_lo(q[i].w)),
                                       scaled(cvt_hi(q[i].w)));
          const uint32_t to = dst + (f >> 3) * (DN_TILE * 128) + row * 128;
          const uint32_t c0 = ((f ^ row) & 7) << 4, c1 = ((f + 1 ^ row) & 7) << 4;
          const bool swap = f & 8;  // lanes of one row: all eight chunk positions at once
          sts128(to + (swap ? c1 : c0), swap ? hi4 : lo4);
          sts128(to + (swap ? c0 : c1), swap ? lo4 : hi4);
        }
      };
      auto next = [&](int &it, int &tile) {
        if (++tile == nt) tile = 0, ++it;
      };
      // the loads of a tile's keys are issued when the keys before are stored, and
      // so the values': a tile ahead
      uint4 k[PASS], v[PASS];
      uint32_t ek = 0, ev = 0;
      if (tiles > 0) {
        pages(tt);
        fetch(k, w.k, w.kps, item, tt);
        ek = exps(w.ke, item, tt);
        fetch(v, w.v, w.vps, item, tt);
        ev = exps(w.ve, item, tt);
      }
      for (int t = 0; t < tiles; ++t) {
        const int st = t & 1, E = top(ek), F = top(ev);
        next(item, tt);
        if (t + 1 < tiles) pages(tt);
        if (t >= 2) bar_wait(s32(&S.kempty[st]), (t >> 1) - 1 & 1, dead);
        store(base + C::K + st * C::OP, k, ek, E);
        if (p == 0) S.exps[t % DN_RING] = make_int2(E, F);
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(s32(&S.kfull[st]));
        if (p == 0) bar_arrive(s32(&S.consts[t % DN_RING]));
        if (t + 1 < tiles) {
          fetch(k, w.k, w.kps, item, tt);
          ek = exps(w.ke, item, tt);
        }
        if (t >= 2) bar_wait(s32(&S.vempty[st]), (t >> 1) - 1 & 1, dead);
        store(base + C::V + st * C::OP, v, ev, F);
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(s32(&S.vfull[st]));
        if (t + 1 < tiles) {
          fetch(v, w.v, w.vps, item, tt);
          ev = exps(w.ve, item, tt);
        }
      }
    } else {
      constexpr int CPR = D / 8;
      auto copy = [&](uint32_t dst, const uint8_t *src, int64_t stride, int it, int tile, uint64_t *bar) {
        const uint32_t row0 = static_cast<uint32_t>(it / nj) << lg;
#pragma unroll
        for (int i = 0; i < CPR / 2; ++i) {
          const int x = p + i * DN_FETCH, row = x / CPR, f = x - row * CPR, tok = tile * DN_TILE + row;
          const int id = tok < w.prefix ? __ldg(w.ptable + (tok >> lg)) : -1;
          const bool ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(w.n_pages);
          const uint32_t at = ((row0 + (tok & pm)) * D + f * 8) * 2;
          cp16(dst + (f >> 3) * (DN_TILE * 128) + row * 128 + (((f ^ row) & 7) << 4),
               ok ? src + id * stride + at : src, ok);
        }
        // arrives when this thread's copies are in
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(s32(bar)) : "memory");
      };
      for (int t = 0; t < tiles; ++t) {
        const int st = t & 1;
        if (t >= 2) bar_wait(s32(&S.kempty[st]), (t >> 1) - 1 & 1, dead);
        copy(base + C::K + st * C::OP, w.k, w.kps, item, tt, &S.kfull[st]);
        if (t >= 2) bar_wait(s32(&S.vempty[st]), (t >> 1) - 1 & 1, dead);
        copy(base + C::V + st * C::OP, w.v, w.vps, item, tt, &S.vfull[st]);
        if (++tt == nt) tt = 0, ++item;
      }
      cp_wait<0>();
    }
  } else {
    regs_to<DN_REST, DN_REGS>();
    // =========================================================== products
    if (warp < 18) {
    const int half = warp - 16;
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
      if (lane == 0 && !*dead) {
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
      if (lane == 0 && !*dead) {
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
    int tt = first0;
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
    if (lane == 0) drained(half);
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
  int64_t n = sms < kMaxGrid ? sms : kMaxGrid;
  if (n > tiles) n = tiles;
  if (n < 1) n = 1;
  *grid = static_cast<int>(n);
  f<<<*grid, DN_NT, fixed + 4 * (kMaxB + 1), s>>>(p);
  return cudaGetLastError();
}

}  // namespace kv
