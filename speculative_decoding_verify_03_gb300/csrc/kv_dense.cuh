// kv_dense.cuh -- the dense kernel of spec_attend and spec_attend_tree: partial
// attention of the query rows of all sequences over the prefix that they share, or
// of a tree's many query rows over their sequence's own tokens.
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
// Two stages of keys and of values.  Where no item has more than 128 rows the second
// row tile's warps stand aside.
//
// Own items (OWN): the nodes of a drafted tree over their sequence's own tokens.  The
// row tiles are those of a sequence and key/value head, the tiles of all items are
// numbered through as in the span kernel, a row's mask says what it sees of the
// step's tokens (64 bits at a time, only where a tile holds some), and of values that
// not all rows see the ones that are not finite are taken out of the tile and added,
// at the item's end, to the rows that see them.
//
// The roles' loops together have to stay in the instruction cache: with polls, query
// loads and products unrolled the code was 161 KB, the cache that a GPC shares was 80 %
// busy with it, and the first line below took 437 us.  So what runs once an item is a
// loop of a few instructions, and a role's loop stands once in the code (54 KB, 67 KB
// with own items).
//
// Measured: 256 x 9 queries of 32 heads (9216 rows a key/value head of 128) over
// 8192 e4m3 tokens 285 us, 1085 TFLOP/s, 57 % of the products' rate: tensor pipe 46 %
// active, 58 % of the issue slots used (over bfloat16 tokens a call takes 7 % less: the
// conversions).  16 trees of 64 nodes of 32 heads over
// 2000..8192 tokens 100 us, 840 TFLOP/s: 34 tiles and two items a CTA, whose ends show (an
// item costs about three tiles beside its own, DN_ITEM).
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

// Where a role is among the CTA's tiles: tile tt of nt of an item.  Prefix items
// are numbered through; own items are of sequence b, key/value head `head`, row
// tile rt of `per`, with `own` tokens before the step's n.
struct DenseAt {
  int tt, nt, item;
  int b, head, rt, per, own, n;
};

struct DenseShared {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t sfull[2][2], pfull[2][2];         // per row tile and score buffer
  uint64_t odone[2], ofull[2], drain[2];     // per row tile
  uint64_t consts[DN_RING], qfull[2];
  int exps[2][DN_RING];      // E, F
  uint32_t last[DN_RING];    // the tile is the CTA's last one of its item
  uint32_t hot[DN_RING];     // own items: a byte for each loading warp that took out values
  uint32_t tmem, dead;
  uint32_t sum[DN_NT / 32], sum1[DN_NT / 32];
};

// The NaN and infinities among elements c .. c + 15 of the values of tokens t0 ..
// end - 1, which were taken out of the products, added to a row that sees them.
template <int D, bool E4M3>
__device__ __noinline__ void add_odd(const View &w, int b, int head, int own, int t0, int end, const int32_t *mask, int c, float *o) {
  const int lg = w.ps_log2, pm = (1 << lg) - 1;
  for (int t = max(t0, own); t < end; ++t) {
    const int j = t - own;
    if (!(mask[j >> 5] >> (j & 31) & 1)) continue;
    const int id = w.table[b * w.tstride + (t >> lg)];
    if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(w.n_pages)) continue;
    const uint8_t *v = w.v + id * w.vps + ((static_cast<int64_t>(head) << lg) + (t & pm)) * D * (E4M3 ? 1 : 2);
    for (int i = 0; i < 16; ++i) {
      if constexpr (E4M3) {
        if ((v[c + i] & 0x7f) == 0x7f) o[i] += NAN;
      } else {
        const uint16_t u = reinterpret_cast<const uint16_t *>(v)[c + i];
        if ((u & 0x7f80) == 0x7f80) o[i] += __uint_as_float(static_cast<uint32_t>(u) << 16);
      }
    }
  }
}

template <int D, bool E4M3, bool OWN>
__global__ void __launch_bounds__(DN_NT, 1) dense_kernel(const __grid_constant__ SpanParams P) {
  using C = DenseCfg<D>;
  constexpr float BIAS = E4M3 ? 11.0f : 0.0f, SLACK = E4M3 ? 4.0f : 8.0f;
  constexpr float SUM = E4M3 ? 0x1p-25f : 1.0f, SUM_LOG = E4M3 ? 25.0f : 0.0f;  // factor of the sum of weights
  constexpr float kNone = -1e30f;  // maximum of no scores
  extern __shared__ uint8_t raw[];
  uint8_t *sm = raw + (-s32(raw) & 1023);  // operands: 1024-byte aligned
  DenseShared &S = *reinterpret_cast<DenseShared *>(sm + C::OPER);
  // B + 1 words: query rows before each sequence; own items: tiles before it, then items
  uint32_t *cum = reinterpret_cast<uint32_t *>(sm + C::OPER + sizeof(DenseShared));
  uint32_t *cum1 = cum + P.w.B + 1;
  const uint32_t base = s32(sm);

  cudaTriggerProgrammaticLaunchCompletion();  // for the call's next kernel (launch())
  const View &w = P.w;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = P.G, B = w.B;

  // --- rows before each sequence
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(s32(&S.kfull[i]), E4M3 ? DN_FETCH / 32 : DN_FETCH), bar_init(s32(&S.kempty[i]), P.halves);
      bar_init(s32(&S.vfull[i]), E4M3 ? DN_FETCH / 32 : DN_FETCH), bar_init(s32(&S.vempty[i]), P.halves);
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
  uint32_t a = 0, a1 = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    int own, n;
    row_shape(w, b, own, n);
    cum[b] = a;
    if constexpr (OWN) {
      const uint32_t j = (n * G + DN_ROWS - 1) / DN_ROWS * w.Hkv;
      cum1[b] = a1;
      a1 += j;
      a += j * ((own + n + DN_TILE - 1) / DN_TILE);
    } else {
      a += n * G;
    }
  }
  uint32_t e = a, e1 = a1;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(~0u, e, o), t1 = OWN ? __shfl_up_sync(~0u, e1, o) : 0;
    if (lane >= o) e += t, e1 += t1;
  }
  if (lane == 31) {
    S.sum[warp] = e;
    if (OWN) S.sum1[warp] = e1;
  }
  tc_before();
  __syncthreads();
  tc_after();
  e -= a, e1 -= a1;
  // sums of the warps before: a lane each
  static_assert(DN_NT / 32 <= 32, "warps");
  const uint32_t of = lane < DN_NT / 32 ? S.sum[lane] : 0, of1 = OWN && lane < DN_NT / 32 ? S.sum1[lane] : 0;
  uint32_t up = of, up1 = of1;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(~0u, up, o), t1 = OWN ? __shfl_up_sync(~0u, up1, o) : 0;
    if (lane >= o) up += t, up1 += t1;
  }
  // all query rows; own items: all tiles, all items
  const uint32_t rows = __shfl_sync(~0u, up, 31), items = __shfl_sync(~0u, up1, 31);
  e += __shfl_sync(~0u, up - of, warp), e1 += __shfl_sync(~0u, up1 - of1, warp);
  uint32_t *out0 = OWN ? P.plan.tiles : P.plan.rows;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    cum[b] += e;
    if (OWN) cum1[b] += e1;
    if (blockIdx.x == 0) {
      out0[b] = cum[b];
      if (OWN) P.plan.items[b] = cum1[b];
    }
  }
  if (tid == 0) {
    cum[B] = rows;
    if (OWN) cum1[B] = items;
    if (blockIdx.x == 0) {
      out0[B] = rows;
      if (OWN) P.plan.items[B] = items;
    }
  }
  __syncthreads();
  const uint32_t tmem = S.tmem;
  volatile uint32_t *dead = &S.dead;
  const int nj = (rows + DN_ROWS - 1) / DN_ROWS;          // prefix: items of a key/value head
  const uint32_t cost = OWN ? cost_of_item(rows, gridDim.x, B, DN_ITEM) : 0;
  const uint32_t W = OWN ? rows + cost * items : static_cast<uint32_t>((w.prefix + DN_TILE - 1) / DN_TILE) * nj * w.Hkv;
  const uint32_t ctas = min(gridDim.x, W);
  bool idle = blockIdx.x >= ctas;
  uint32_t lo = idle ? 0 : static_cast<uint32_t>(static_cast<uint64_t>(W) * blockIdx.x / ctas);
  uint32_t hi = idle ? 0 : static_cast<uint32_t>(static_cast<uint64_t>(W) * (blockIdx.x + 1) / ctas);
  if (OWN && cost) {
    lo = tile_at(w, cum, cum1, cost, DN_TILE, lo), hi = tile_at(w, cum, cum1, cost, DN_TILE, hi);
    idle |= lo >= hi;
  }
  const int tiles = static_cast<int>(hi - lo);
  // --- the first tile, and the next one
  auto shape = [&](DenseAt &x) {
    row_shape(w, x.b, x.own, x.n);
    x.per = (x.n * G + DN_ROWS - 1) / DN_ROWS;
    x.nt = (x.own + x.n + DN_TILE - 1) / DN_TILE;
  };
  auto begin = [&]() {
    DenseAt x = {};
    x.nt = 1;
    if (idle) return x;
    if constexpr (OWN) {
      int r = B;
      while (r - x.b > 1) {
        const int m = (x.b + r) >> 1;
        if (cum[m] <= lo) x.b = m;
        else r = m;
      }
      shape(x);
      const uint32_t y = lo - cum[x.b], j = y / x.nt;
      x.head = j / x.per;
      x.rt = j - x.head * x.per;
      x.tt = y - j * x.nt;
    } else {
      x.nt = (w.prefix + DN_TILE - 1) / DN_TILE;
      x.item = lo / x.nt;
      x.tt = lo - x.item * x.nt;
    }
    return x;
  };
  auto step = [&](DenseAt &x) {  // there is a next tile
    if (++x.tt < x.nt) return;
    x.tt = 0;
    if constexpr (OWN) {
      if (++x.rt < x.per) return;
      x.rt = 0;
      if (++x.head < w.Hkv) return;
      x.head = 0;
      do ++x.b;
      while (x.b + 1 < B && cum[x.b + 1] == cum[x.b]);
      shape(x);
    } else {
      ++x.item;
    }
  };

  // All products that this thread issued are done, also where a wait gave up:
  // TMEM goes back behind this.
  auto drained = [&](int i) {
    mma_commit(s32(&S.drain[i]));
    uint32_t late = 0;
    bar_wait(s32(&S.drain[i]), 0, &late);
    if (late) *dead = 1;
  };

  if (warp < 8) {
    if (warp < 4 * P.halves) {
      regs_to<DN_SOFT, DN_REGS>();
      // ================================================= softmax and output
      const int half = warp >> 2;
      const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 TMEM lanes a warp
      const uint32_t oc = tmem + lanes + 256 + half * 128;
      const uint32_t wb = base + C::Q + half * C::OP + (warp & 3) * 32 * 128;  // the warp's query rows
      const int r = tid;  // row of the item
      DenseAt x = begin();
      float M = kNone, l = 0.0f, qc = 0.0f;
      float kt = 0.0f, F = 0.0f, invF = 1.0f;  // of the tile
      bool fresh = true;
      int node = -1;  // own items: the row's place in the step
      int begun = 0;  // own items: the CTA's first tile of the item
      int g = 0;  // items
#pragma unroll 1
      for (int u = 0; u < 2 * tiles; ++u) {
        const int t = u >> 1;  // half u & 1 of tile t
        if (fresh) {  // the row's query; the products with the item before are done
          const uint32_t row = (OWN ? x.rt : x.item % nj) * DN_ROWS + r;
          int64_t off = -1;
          if (OWN) {
            node = -1;
            if (row < static_cast<uint32_t>(x.n * G)) {
              node = row / G;
              off = x.b * P.qs0 + node * P.qs1 + (x.head * G + static_cast<int>(row) - node * G) * P.qs2;
            }
          } else if (row < rows) {
            int b = 0, h = B;
            while (h - b > 1) {
              const int m = (b + h) >> 1;
              if (cum[m] <= row) b = m;
              else h = m;
            }
            const int y = row - cum[b], i = y / G;
            off = b * P.qs0 + i * P.qs1 + (x.item / nj * G + y - i * G) * P.qs2;
          }
          // into shared memory by the warp's 32 rows together, neighbouring lanes
          // neighbouring chunks; then a row by its own thread
          // (loops, not one long piece of code: an item's first tile would wait for its
          // instructions)
          constexpr int CH = D / 8;
          auto at = [&](int y, int c) {
            return wb + (c >> 3) * (DN_TILE * 128) + y * 128 + (((c ^ y) & 7) << 4);
          };
          if (P.qvec) {
#pragma unroll 4
            for (int k = 0; k < CH; ++k) {
              const int z = lane + 32 * k, y = z / CH, c = z - y * CH;
              const int64_t o = __shfl_sync(~0u, off, y);
              cp16(at(y, c), P.q + (o < 0 ? 0 : o + 8 * c), o >= 0);
            }
            cp_commit();
            cp_wait<0>();
          } else {
#pragma unroll 1
            for (int k = 0; k < CH; ++k) {
              const int z = lane + 32 * k, y = z / CH, c = z - y * CH;
              const int64_t o = __shfl_sync(~0u, off, y);
              uint4 v = make_uint4(0, 0, 0, 0);
              if (o >= 0) {
                const uint16_t *u = reinterpret_cast<const uint16_t *>(P.q + o + 8 * c);
                v = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
              }
              sts128(at(y, c), v);
            }
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
#pragma unroll 2
            for (int k = 0; k < CH; ++k) {
              const uint4 v = lds128(at(lane, k));
              most(v.x), most(v.y), most(v.z), most(v.w);
            }
            const int eq = max(static_cast<int>(m >> 7) - 127 - 10, -100);
            qc = P.c * pow2i(eq);
            const float f = pow2i(-eq);
            auto two = [&](uint32_t u) {
              return pack<true>(__uint_as_float(u << 16) * f, __uint_as_float(u & 0xffff0000u) * f);
            };
#pragma unroll 2
            for (int k = 0; k < CH; ++k) {
              const uint4 v = lds128(at(lane, k));
              sts128(at(lane, k), make_uint4(two(v.x), two(v.y), two(v.z), two(v.w)));
            }
          }
          fence_async();
          __syncwarp();
          if (lane == 0) bar_arrive(s32(&S.qfull[half]));
          M = kNone, l = 0.0f;
          begun = t;
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
        // tokens from here on that all rows see
        const int n = (OWN ? x.own : w.prefix) - x.tt * DN_TILE - (u & 1) * 64;
        float ks = kt;  // still to be multiplied by
        if (n < 64) {   // masked behind the multiplication: a factor of 0 would make NaN of -inf
          ks = 1.0f;
          if constexpr (OWN) {
            uint64_t see = 0;
            if (node >= 0)
              see = seen_nodes(P.mask + (static_cast<int64_t>(x.b) * w.N + node) * P.mask_words, P.mask_words, x.n, -n);
            const uint32_t see0 = static_cast<uint32_t>(see), see1 = static_cast<uint32_t>(see >> 32);
#pragma unroll
            for (int c = 0; c < 64; ++c) s[c] = (c < 32 ? see0 : see1) >> (c & 31) & 1 ? s[c] * kt : -INFINITY;
          } else {
#pragma unroll
            for (int c = 0; c < 64; ++c) s[c] = c >= n ? -INFINITY : s[c] * kt;
          }
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

        const bool last = (u & 1) && (x.tt + 1 == x.nt || t + 1 == tiles);
        if (last) {
          const uint32_t slot = (OWN ? cum1[x.b] + x.head * x.per + x.rt : x.item) + blockIdx.x;
          const int64_t at = static_cast<int64_t>(slot) * DN_ROWS + r;
          const bool there = OWN ? node >= 0 : static_cast<uint32_t>(x.item % nj * DN_ROWS + r) < rows;
          const float f = l == 0.0f ? 0.0f : 1.0f / l;
          if (there) P.pl[at] = l == 0.0f ? -INFINITY : M - (BIAS - SUM_LOG) + log2f(l);
          bar_wait(s32(&S.ofull[half]), g++ & 1, dead);
          tc_after();
          int hot0 = t + 1;  // own items: the first tile that values were taken out of
          if constexpr (OWN) {
            const volatile uint32_t *hot = S.hot;
            for (int k = t; k >= begun && (x.tt - (t - k) + 1) * DN_TILE > x.own; --k)
              if (hot[k % DN_RING]) hot0 = k;
          }
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
            if (OWN && hot0 <= t && node >= 0) {  // rare: to the rows that see them
              const int t0 = (x.tt - (t - hot0)) * DN_TILE;
              float more[16] = {};
              add_odd<D, E4M3>(w, x.b, x.head, x.own, t0, min(x.own + x.n, (x.tt + 1) * DN_TILE),
                               P.mask + (static_cast<int64_t>(x.b) * w.N + node) * P.mask_words, c, more);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] += more[i];
            }
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
        if ((u & 1) && t + 1 < tiles) step(x);
      }
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
    DenseAt x = begin();
    // own items: the tile holds tokens that not all rows see; then no NaN or infinity
    // of their values goes into a product, where a weight of zero would spread it
    auto banded = [&]() { return OWN && vs && (x.tt + 1) * DN_TILE > x.own; };
    // tokens of the item's list and the pages that hold them
    auto held = [&]() { return OWN ? x.own + x.n : w.prefix; };
    auto list = [&]() { return OWN ? w.table + x.b * w.tstride : w.ptable; };
    auto head_of = [&]() { return static_cast<uint32_t>(OWN ? x.head : x.item / nj); };
    if constexpr (E4M3) {
      constexpr int CPR = D / 16;                     // 16-byte chunks of a row
      constexpr int PASS = DN_TILE * CPR / DN_FETCH;  // of a tile, per thread
      static_assert(DN_TILE * CPR % DN_FETCH == 0, "chunks");
      // A thread's chunk and, in each pass, its row.  Rows of 4 or 8 chunks: eight
      // neighbouring lanes have four chunks of two rows, an even and an odd one, whose
      // float16 chunks 2c (or 2c + 1) are in eight different groups of banks; the
      // passes are RPP rows apart, and the warp's 32 rows are a lane's each for the scales.
      constexpr bool EVEN = CPR == 8 || CPR == 4;
      constexpr int RPP = EVEN ? DN_FETCH / CPR : 1, RPW = RPP / 4;  // rows of a pass, of a warp
      const int wl = warp & 3, sub = CPR == 8 ? lane >> 2 & 3 : lane >> 2, chunk = CPR == 8 ? (lane & 3) | lane >> 4 << 2 : lane & 3;
      auto row_of = [&](int i) { return EVEN ? wl * RPW + sub + RPP * i : (p + i * DN_FETCH) / CPR; };
      auto chunk_of = [&](int i) { return EVEN ? chunk : p + i * DN_FETCH - row_of(i) * CPR; };
      int ids = -1, idn = -1;  // pages of tokens 16 j .. of the tile to be fetched next, j = lane & 7; of the one behind it
      auto pages = [&](int tt) {
        const int tok = tt * DN_TILE + 16 * (lane & 7);
        return tok < held() ? ldg_now(list() + (tok >> lg)) : -1;
      };
      uint4 q[PASS] = {};
      uint32_t ex = 0;  // exponents of the lane's four tokens, the first `live` of them there
      int live = 0;
      const bool any = w.n_pages > 0;
      // A chunk without a page is read from page 0 and put to zero below: the loads
      // stand in a row without branches.  Where tokens 16 j .. of the tile begin is worked
      // out once, by lane j; a pass's rows are a few of 16 such.
      auto page = [&](int id) { return static_cast<uint32_t>(id) < static_cast<uint32_t>(w.n_pages); };
      const uint8_t *begins = src;
      auto places = [&]() {
        const int id = page(ids) ? ids : 0;
        const uint32_t in = (head_of() << lg) + (x.tt * DN_TILE + 16 * (lane & 7) & pm);
        begins = src + id * stride + static_cast<uint64_t>(in) * D;
      };
      auto load = [&](int i) {
        const int row = row_of(i);
        const uint8_t *from = reinterpret_cast<const uint8_t *>(
            __shfl_sync(~0u, reinterpret_cast<unsigned long long>(begins), CPR == 8 ? i : row >> 4));
        if (any) q[i] = ldg_now16(from + ((row & 15) * D + chunk_of(i) * 16));
      };
      // (masked when they are used: nothing here waits for a load)
      auto load_exps = [&]() {
        const int t0 = x.tt * DN_TILE, id = __shfl_sync(~0u, ids, lane >> 2);
        live = page(id) ? min(max(held() - t0 - 4 * lane, 0), 4) : 0;
        if (any)
          ex = ldg_now32((vs ? w.ve : w.ke) + ((static_cast<int64_t>(live ? id : 0) * w.Hkv + head_of()) << lg) +
                         (t0 + 4 * lane & pm));
      };
      bool ahead = false;
      // tile t goes to shared memory, then tile t + 1 is asked for (t = -1: the first one)
#pragma unroll 1
      for (int t = -1; t < tiles; ++t) {
        const bool more = t + 1 < tiles;
        bool partial = false;
        int E = -128;        // seven below the tile's largest exponent
        int band = DN_TILE;  // own items: the first row of values that not all rows see
        if (t >= 0) {
          partial = __any_sync(~0u, live < 4);
          if (live < 4) {  // -128 where there is no token
            const uint32_t in = (1u << 8 * live) - 1;
            ex = (ex & in) | (0x80808080u & ~in);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) E = max(E, static_cast<int>(static_cast<int8_t>(ex >> 8 * i)));
          E = max(__reduce_max_sync(~0u, E), kExpMin) - 7;
          if (p == 0) {
            S.exps[vs][t % DN_RING] = E;
            if (!vs) S.last[t % DN_RING] = x.tt + 1 == x.nt || t + 1 == tiles;
            bar_arrive(s32(&S.consts[t % DN_RING]));
          }
          if (OWN && vs) band = x.own - x.tt * DN_TILE;
        }
        const uint32_t was = ex;
        if (more) {
          if (t >= 0) step(x);
          ids = ahead ? idn : pages(x.tt);
        }
        ahead = t + 2 < tiles && x.tt + 1 < x.nt;
        if (ahead) idn = pages(x.tt + 1);
        if (t >= 0) {
          // the factors 2^(e - E) of the warp's rows, twice in a word: a lane each (e - E <= 7)
          auto factor = [&](int e) {
            const float one = pow2i(max(e - E, -126));
            return pack<true>(one, one);
          };
          const int mine = wl * RPW + lane % (EVEN ? RPW : 1) + RPP * (lane / (EVEN ? RPW : 1));
          const int exr = EVEN ? static_cast<int8_t>(__shfl_sync(~0u, was, mine >> 2 & 31) >> 8 * (mine & 3)) : 0;
          const uint32_t factors = EVEN ? factor(exr) : 0;
          uint32_t two[PASS];
          if constexpr (EVEN) {
#pragma unroll
            for (int i = 0; i < PASS; ++i) two[i] = __shfl_sync(~0u, factors, i * RPW + sub);
            if (partial) {
#pragma unroll
              for (int i = 0; i < PASS; ++i) {
                const uint32_t is = __shfl_sync(~0u, exr, i * RPW + sub) == -128 ? 0u : ~0u;
                q[i].x &= is, q[i].y &= is, q[i].z &= is, q[i].w &= is;
              }
            }
          }
          if (t >= 2) bar_wait(s32(empty + (t & 1)), (t >> 1) - 1 & 1, dead);
          const uint32_t dst = dst0 + (t & 1) * C::OP;
          auto to = [&](int i, int c) {  // chunk c of the row's float16 elements
            return dst + (c >> 3) * (DN_TILE * 128) + row_of(i) * 128 + (((c ^ row_of(i)) & 7) << 4);
          };
#pragma unroll
          for (int i = 0; i < PASS; ++i) {
            const int row = row_of(i), f = 2 * chunk_of(i);
            if constexpr (!EVEN) {
              const int e = static_cast<int8_t>(__shfl_sync(~0u, was, row >> 2) >> 8 * (row & 3));
              two[i] = factor(e);
              const uint32_t is = e == -128 ? 0u : ~0u;
              q[i].x &= is, q[i].y &= is, q[i].z &= is, q[i].w &= is;
            }
            const __half2 sc = *reinterpret_cast<const __half2 *>(&two[i]);
            auto scaled = [&](uint32_t h) {
              const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&h), sc);
              return *reinterpret_cast<const uint32_t *>(&y);
            };
            const uint4 b = q[i];
            const uint4 lo4 = make_uint4(scaled(cvt_lo(b.x)), scaled(cvt_hi(b.x)), scaled(cvt_lo(b.y)), scaled(cvt_hi(b.y)));
            const uint4 hi4 = make_uint4(scaled(cvt_lo(b.z)), scaled(cvt_hi(b.z)), scaled(cvt_lo(b.w)), scaled(cvt_hi(b.w)));
            const bool swap = !EVEN && f & 8;  // lanes of one row: all eight chunk positions at once
            sts128(to(i, swap ? f + 1 : f), swap ? hi4 : lo4);
            sts128(to(i, swap ? f : f + 1), swap ? lo4 : hi4);
          }
          if constexpr (OWN) {
            if (vs) {
              bool odd = false;
              if (band < DN_TILE) {  // what is NaN among these values comes out again
#pragma unroll 1
                for (int i = 0; i < 2 * PASS; ++i) {
                  if (row_of(i >> 1) < band) continue;
                  const uint32_t at = to(i >> 1, 2 * chunk_of(i >> 1) + (i & 1));
                  uint4 v = lds128(at);
                  uint32_t any = 0;
                  auto clean = [&](uint32_t u) {  // 1 where the exponent is full
                    const uint32_t m = (((u & 0x7fff7fffu) + 0x04000400u) & 0x80008000u) >> 15;
                    any |= m;
                    return u & ~(m * 0xffffu);
                  };
                  v = make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
                  if (any) sts128(at, v);
                  odd |= any != 0;
                }
              }
              odd = __any_sync(~0u, odd);
              if (lane == 0) reinterpret_cast<volatile uint8_t *>(&S.hot[t % DN_RING])[wl] = odd;
            }
          }
          fence_async();
          __syncwarp();
          if (lane == 0) bar_arrive(s32(full + (t & 1)));
        }
        if (more) {
          places();
#pragma unroll
          for (int i = 0; i < PASS; ++i) load(i);
          load_exps();
          if (OWN && ahead) {  // the tile behind that one comes to L2: a row a thread
            const int id = __shfl_sync(~0u, idn, p >> 4), tok = (x.tt + 1) * DN_TILE + p;
            if (page(id) && tok < held())
              prefetch_l2(src + id * stride + static_cast<uint64_t>((head_of() << lg) + (tok & pm)) * D);
          }
        }
      }
    } else {
      constexpr int CPR = D / 8;
#pragma unroll 1
      for (int t = 0; t < tiles; ++t) {
        if (t >= 2) bar_wait(s32(empty + (t & 1)), (t >> 1) - 1 & 1, dead);
        if (p == 0) {
          if (!vs) S.last[t % DN_RING] = x.tt + 1 == x.nt || t + 1 == tiles;
          bar_arrive(s32(&S.consts[t % DN_RING]));
        }
        const uint32_t row0 = head_of() << lg, dst = dst0 + (t & 1) * C::OP;
        const int32_t *ids = list();
        const int end = held();
        if (OWN && banded()) {  // through registers
          const int first = x.own - x.tt * DN_TILE;
          bool odd = false;
#pragma unroll 4
          for (int i = 0; i < CPR; ++i) {
            const int z = p + i * DN_FETCH, row = z / CPR, f = z - row * CPR, tok = x.tt * DN_TILE + row;
            const int id = tok < end ? __ldg(ids + (tok >> lg)) : -1;
            uint4 q = make_uint4(0, 0, 0, 0);
            if (static_cast<uint32_t>(id) < static_cast<uint32_t>(w.n_pages))
              q = __ldg(reinterpret_cast<const uint4 *>(src + id * stride + ((row0 + (tok & pm)) * D + f * 8) * 2));
            uint32_t *u = reinterpret_cast<uint32_t *>(&q);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t m = (((u[k] & 0x7fff7fffu) + 0x00800080u) & 0x80008000u) >> 15;  // 1 where the exponent is full
              if (row < first) m = 0;
              odd |= m != 0;
              u[k] &= ~(m * 0xffffu);
            }
            sts128(dst + (f >> 3) * (DN_TILE * 128) + row * 128 + (((f ^ row) & 7) << 4), q);
          }
          odd = __any_sync(~0u, odd);
          if (lane == 0) reinterpret_cast<volatile uint8_t *>(&S.hot[t % DN_RING])[warp & 3] = odd;
          fence_async();
          bar_arrive(s32(full + (t & 1)));
        } else {
#pragma unroll
          for (int i = 0; i < CPR; ++i) {
            const int z = p + i * DN_FETCH, row = z / CPR, f = z - row * CPR, tok = x.tt * DN_TILE + row;
            const int id = tok < end ? __ldg(ids + (tok >> lg)) : -1;
            const bool ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(w.n_pages);
            const uint32_t at = ((row0 + (tok & pm)) * D + f * 8) * 2;
            cp16(dst + (f >> 3) * (DN_TILE * 128) + row * 128 + (((f ^ row) & 7) << 4),
                 ok ? src + id * stride + at : src, ok);
          }
          if (OWN && vs && lane == 0) reinterpret_cast<volatile uint8_t *>(&S.hot[t % DN_RING])[warp & 3] = 0;
          // arrives when this thread's copies are in
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(s32(full + (t & 1))) : "memory");
        }
        if (t + 1 < tiles) step(x);
      }
      cp_wait<0>();
    }
  } else {
    regs_to<DN_REST, DN_REGS>();
    // =========================================================== products
    if (warp < 16 + P.halves) {
    // one lane issues, chosen by elect.sync, and all that its products are
    // described by is the warp's: kept in uniform registers, where they are wanted
    const int half = __shfl_sync(~0u, warp, 0) - 16;
    const uint32_t base = __shfl_sync(~0u, s32(sm), 0), tmem = __shfl_sync(~0u, S.tmem, 0);
    const int tiles = __shfl_sync(~0u, static_cast<int>(hi - lo), 0);
    constexpr uint32_t sdesc = mma_desc(E4M3, 128, 64, false, false);
    constexpr uint32_t odesc = mma_desc(E4M3, 128, D, false, true);
    const uint64_t qd = smem_desc(base + C::Q + half * C::OP, 16, 1024), kd = smem_desc(base + C::K, 16, 1024);
    const uint64_t vd = smem_desc(base + C::V, DN_TILE * 128, 1024);
    const uint32_t sc = tmem + half * 128, oc = tmem + 256 + half * 128;
    int g = 0;
    // Half tile u (begin: the CTA's first one of its item): scores into buffer u & 1 ...
    auto scores = [&](int u, bool begin) {
      const int t = u >> 1, st = t & 1;
      if (begin) bar_wait(s32(&S.qfull[half]), g++ & 1, dead);
      // the weights of half tile u - 2 are read; behind an item, all of it is done
      const bool behind = u > 0 && begin;
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
    auto values = [&](int u, bool begin, bool end) {
      const int t = u >> 1, st = t & 1;
      const bool last = (u & 1) && end;
      // (parities tell one phase from the next only: no phase is skipped)
      if (last) bar_wait(s32(&S.odone[half]), u - 1 & 1, dead);
      if (!(u & 1)) bar_wait(s32(&S.vfull[st]), t >> 1 & 1, dead);
      if (!E4M3) fence_async();
      bar_wait(s32(&S.pfull[half][u & 1]), t & 1, dead);
      tc_after();
      if (elected() && !*dead) {
        const uint64_t vv = vd + st * (C::OP >> 4) + (u & 1) * (64 * 128 >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ts(oc, sc + (u & 1) * 64 + 8 * k, vv + (k * 2048 >> 4), odesc, !begin || k > 0);
        mma_commit(s32(&S.odone[half]));
        if (u & 1) mma_commit(s32(&S.vempty[st]));
        if (last) mma_commit(s32(&S.ofull[half]));
      }
      __syncwarp();
    };
    // The next half tile's scores come before these weights, except behind an item's
    // last, whose output has to be out before the next item's queries are in.  (One
    // copy each of the two in the code: the roles' loops together are to stay in the
    // instruction cache.)
    int next = 0;
    bool end = false;  // of the item, behind this tile
#pragma unroll 1
    for (int u = 0; u < 2 * tiles; ++u) {
      const bool begin = next == u;  // of the item: its scores were not formed ahead
      if (!(u & 1)) {
        bar_wait(s32(&S.consts[(u >> 1) % DN_RING]), (u >> 1) / DN_RING & 1, dead);
        end = __shfl_sync(~0u, S.last[(u >> 1) % DN_RING], 0);
      }
      const int upto = (u & 1) && end ? u : u + 1;
#pragma unroll 1
      for (; next <= upto; ++next) scores(next, begin && next == u);
      values(u, begin, end);
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
  wait_for_first(P);
}

template <int D, bool E4M3, bool OWN = false>
cudaError_t dense_go(const SpanParams &p, int64_t tiles, int *grid, cudaStream_t s) {
  constexpr int fixed = 1024 + DenseCfg<D>::OPER + sizeof(DenseShared);
  constexpr int smem = fixed + (OWN ? 8 : 4) * (kMaxB + 1);
  static_assert(smem <= 232448, "shared memory");
  auto *f = dense_kernel<D, E4M3, OWN>;
  static Slots slots;
  int sms = 0, occ = 0;
  const cudaError_t e = slots.get(reinterpret_cast<const void *>(f), DN_NT, smem, smem, &sms, &occ);
  if (e != cudaSuccess) return e;
  int64_t n = sms < kMaxDense ? sms : kMaxDense;
  if (n > tiles) n = tiles;
  if (n < 1) n = 1;
  *grid = static_cast<int>(n);
  return launch(f, *grid, DN_NT, smem, s, p);
}

}  // namespace kv
