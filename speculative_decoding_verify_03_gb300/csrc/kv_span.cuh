// kv_span.cuh -- the span kernel of spec_attend: partial attention of a few
// query rows over a span of key tiles (see kv_span.h for the work's cut).
//
// Mathematics, in powers of two: z_j = scale log2(e) q.k_j and, with the
// stored exponents, k_j = 2^ek y_j, v_j = 2^ev u_j: the tensor cores form
// q.y_j, the column factor 2^ek is applied to the score, and the weight that
// multiplies u_j is P_j = 2^(z_j + ev_j - M), M the running maximum of
// z_j + ev_j.  So no exponent of v enters a 16-bit operand, and the sum of
// weights is l = sum_j P_j 2^-ev_j.  o = (sum_j P_j u_j) / l,
// lse2 = M + log2 l.  y and u are exact in float16 and each row of q is scaled
// by a power of two into its range; P is biased by 2^8, so that weights down to
// 2^-33 of the largest survive.  The sum is kept 2^-12 times as large: a token
// of zeros (e = -100) adds 2^(8 + 100 - 12), which 2^30 of them keep finite, one of
// the largest exponent (119) 2^-123, still normal.  (Products of e4m3, with q as a sum of two, would
// need no conversion of the keys, but are summed with about 14 bits: lse came
// out 2e-4 off.)  bfloat16 caches: the same with ek = ev = 0 in bfloat16: a product
// has both operands in one 16-bit type, and float16 does not hold all values of
// the cache, so the weights are rounded to 8 bits there (the error of 16 heads of
// 64 over 1001 + 0..300 tokens against 64 bits 0.0022, the output's own rounding
// 0.0017); a second product with what the rounding left would cost as much again.
//
// Layout: a CTA has WR x WT warps; a warp works on 16 rows and 64 / WT tokens
// of each tile with m16n8k16 products, and keeps its own running maximum, sum
// and output in registers; the WT warps of a row tile are joined at the end of
// an item.  K and V tiles come through a ring of asynchronous copies, rows
// padded to an odd multiple of 16 bytes (ldmatrix without bank conflicts).
// e4m3 bytes go through ldmatrix as pairs: a key row's four bytes per lane are
// the two halves of one k16 step (the order of d within a step is free as long
// as q has the same), and the transposed value pairs give two n8 tiles, even
// and odd d, after one byte permute.  Page ids are looked up two tiles ahead of
// their use, exponents turned into factors once per tile, and with 16 rows the
// next items' queries come with their first tile (short contexts are many items
// of a few tiles).
//
// Bound and measured: 8 x 5 queries of 64 heads (40 rows a key/value head of 128)
// over 40000..65536 e4m3 tokens 340 us, 2.5 TB/s or 37 % of a copy's rate: about
// 1900 cycles per 64-token tile and SM, where the bytes alone would take 707.
// No pipe is full (tensor 40 %, ALU 39 %, issue 44 %): three warps a
// scheduler wait for one another's products, loads and barriers, and each of the
// three row warps converts the whole tile for itself, about two thirds of the
// ALU's work.  Over bfloat16 tokens, without conversions, 340 us are 5.0 TB/s (74 %).
// 512 x 2..9 queries of 16 heads of 64 over 0..300 bfloat16 tokens 134 us (2.5
// TB/s): what an item costs once.  A prompt of 2048 tokens at position 0, 32 heads:
// 344 us (100 TFLOP/s of what its queries see; each row tile walks all keys).
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
  // Rows of 4, 8 or 16 chunks lie one after the other, chunks swapped by the row
  // number; others are padded to an odd number of chunks.  Either way the eight
  // rows of an ldmatrix matrix are in eight different groups of banks.
  static constexpr bool SWAP = (CPR & (CPR - 1)) == 0;
  static constexpr int LD = SWAP ? DB : (CPR | 1) * 16;  // row pitch in shared memory
  __device__ static constexpr int swap(int row) { return !SWAP ? 0 : CPR == 4 ? row >> 1 & 3 : row & 7; }
  __device__ static constexpr int at(int row, int ch) { return row * LD + (ch ^ swap(row)) * 16; }
  static constexpr int TILE = kTile * LD;            // bytes of a K or V tile
  static constexpr int STAGE = 2 * TILE;
  static constexpr int ST = STAGE > 30000 || (WR == 1 && D == 64) ? 2 : 3;  // stages
  static constexpr int OLD = D + 4;                  // pitch of the joined output
  static constexpr int JOIN = WT > 1 ? (RT * OLD + 2 * WT * RT) * 4 : 0;
  static constexpr int CONSTS = E4M3 ? ST * kTile * 16 : 0;  // a token's factors, per stage
  static constexpr int QLD = 2 * D + 16;                     // pitch of the queries, 16 rows only
  static constexpr int QBUF = WR == 1 ? 3 * RT * QLD : 0;
  static constexpr int FIXED = ST * STAGE + JOIN + CONSTS + QBUF + 384;
  static constexpr int MIN_CTAS = WR == 1 ? (D == 64 ? 5 : 3) : WR == 3 ? 4 : 3;
};

// An item: sequence, key/value head, row tile; row tiles of a head, own tokens
// before the step, tokens in the step.
struct Cursor {
  int b, head, rt, per, own, n;
};
// What a tile is, in shared memory (four of them: the current one and the next).
struct TileInfo {
  int t0, held, head, b;      // first token; tokens of the item's list; head, sequence
  int row0, rows, own, slot;  // first row of the item, rows of the sequence; partial result
  int first, last, pad[2];    // first or last tile of the item in this span
  int page[4];                // page of each 16 tokens, -1: none
};

template <int D, bool E4M3, int WR, int WT>
__global__ void __launch_bounds__(32 * WR *WT, SpanCfg<D, E4M3, WR, WT>::MIN_CTAS)
    span_kernel(const __grid_constant__ SpanParams P) {
  using C = SpanCfg<D, E4M3, WR, WT>;
  constexpr int NT = C::NT, RT = C::RT, LD = C::LD, ST = C::ST, CPR = C::CPR;
  constexpr int TPW = kTile / WT;   // tokens of a tile per warp
  constexpr int TPP = TPW < 32 ? TPW : 32;  // tokens of a pass: what registers hold
  constexpr int NG = TPP / 8;       // groups of 8 tokens
  constexpr float BIAS = E4M3 ? 8.0f : 0.0f;
  constexpr float SUM = E4M3 ? 0x1p-12f : 1.0f, SUM_LOG = E4M3 ? 12.0f : 0.0f;  // factor of the sum of weights
  extern __shared__ __align__(128) uint8_t sm[];
  uint8_t *stages = sm;
  float *join = reinterpret_cast<float *>(sm + ST * C::STAGE);
  float4 *consts = reinterpret_cast<float4 *>(sm + ST * C::STAGE + C::JOIN);  // 2^ek, ev, 2^-ev SUM
  uint8_t *qbuf = sm + ST * C::STAGE + C::JOIN + C::CONSTS;
  TileInfo *info = reinterpret_cast<TileInfo *>(qbuf + C::QBUF);  // 4
  Cursor *cursor = reinterpret_cast<Cursor *>(info + 4);           // of the newest description
  uint32_t *band = reinterpret_cast<uint32_t *>(cursor + 1) + 1;   // 2 words
  uint32_t *wsum = band + 2;                                       // 2 words per warp
  uint32_t *cum0 = reinterpret_cast<uint32_t *>(sm + C::FIXED);  // B + 1: tiles or rows before b
  uint32_t *cum1 = cum0 + P.w.B + 1;                             // B + 1: items before b (own)

  // the merge kernel may be set up meanwhile; it waits for this grid's end
  cudaTriggerProgrammaticLaunchCompletion();
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
    uint32_t e0 = a0, e1 = a1;  // inclusive over the warp, then exclusive over the CTA
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t0 = __shfl_up_sync(~0u, e0, o), t1 = __shfl_up_sync(~0u, e1, o);
      if (lane >= o) e0 += t0, e1 += t1;
    }
    if (lane == 31) wsum[2 * warp] = e0, wsum[2 * warp + 1] = e1;
    if (tid < 2) band[tid] = 0;
    __syncthreads();
    e0 -= a0, e1 -= a1;
    uint32_t all0 = 0, all1 = 0;
#pragma unroll
    for (int v = 0; v < NT / 32; ++v) {
      if (v < warp) e0 += wsum[2 * v], e1 += wsum[2 * v + 1];
      all0 += wsum[2 * v], all1 += wsum[2 * v + 1];
    }
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) {
      const uint32_t t0 = cum0[b], t1 = cum1[b];
      cum0[b] = e0, cum1[b] = e1;
      e0 += t0, e1 += t1;
    }
    if (tid == 0) cum0[B] = all0, cum1[B] = all1;
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
  // --- descriptions of the tiles to come: the first tile of an item by one thread
  auto describe = [&](const Cursor &c, uint32_t x, int t) {
    TileInfo &T = info[x & 3];
    T.t0 = t * kTile, T.held = c.own + c.n, T.head = c.head, T.b = c.b;
    T.row0 = c.rt * RT, T.rows = pre ? rows_all : c.n * G, T.own = c.own;
    T.slot = (pre ? 0 : cum1[c.b]) + c.head * c.per + c.rt + blockIdx.x;
    T.first = 1, T.last = x + 1 == hi || T.t0 + kTile >= T.held;
  };
  auto enter = [&](Cursor &c) {  // shape of sequence c.b
    row_shape(w, c.b, c.own, c.n);
    c.per = (c.n * G + RT - 1) / RT;
  };
  auto begin = [&](Cursor &c) {
    uint32_t y = lo;
    if (pre) {
      c.b = 0, c.per = pnj, c.own = w.prefix, c.n = 0;
    } else {
      c.b = before(lo);
      y -= cum0[c.b];
      enter(c);
    }
    const int nt = (c.own + c.n + kTile - 1) / kTile, j = y / nt;
    c.head = j / c.per;
    c.rt = j - c.head * c.per;
    describe(c, lo, y - j * nt);
  };
  auto next_item = [&](Cursor &c) {
    if (++c.rt < c.per) return;
    c.rt = 0;
    if (++c.head < w.Hkv) return;
    c.head = 0;
    do ++c.b;
    while (cum0[c.b + 1] == cum0[c.b]);
    enter(c);
  };
  // tile x < hi from tile x - 1, by a warp: its words side by side
  auto advance = [&](uint32_t x) {
    const TileInfo &A = info[(x - 1) & 3];
    if (A.last) {
      if (lane == 0) {
        Cursor c = *cursor;
        next_item(c);
        describe(c, x, 0);
        *cursor = c;
      }
    } else if (lane < 12) {
      int v = reinterpret_cast<const int *>(&A)[lane];
      if (lane == 0) v += kTile;                                          // t0
      if (lane == 8) v = 0;                                               // first
      if (lane == 9) v = x + 1 == hi || A.t0 + 2 * kTile >= A.held;       // last
      reinterpret_cast<int *>(&info[x & 3])[lane] = v;
    }
    __syncwarp();
  };
  const int lg = w.ps_log2, pm = (1 << lg) - 1;
  // --- page of 16 tokens (group i of four) of a tile, -1 where there is none
  auto page = [&](const TileInfo &T, int i) {
    const int tok = T.t0 + 16 * i;
    if (tok >= T.held) return -1;
    const int id = __ldg((pre ? w.ptable : w.table + T.b * w.tstride) + (tok >> lg));
    return static_cast<uint32_t>(id) < static_cast<uint32_t>(w.n_pages) ? id : -1;
  };
  // --- copies of tile x into its stage
  auto fetch = [&](uint32_t x, const TileInfo &T) {
    const uint32_t ks = s32(stages + x % ST * C::STAGE), vs = ks + C::TILE;
    const int left = T.held - T.t0;  // tokens of the tile that there are
    const uint32_t row0 = (static_cast<uint32_t>(T.head) << lg) + (T.t0 & pm);
    if (NT % CPR == 0 && lg >= 6) {  // one page: a pointer each, then constant steps
      const int id = T.page[0], r = tid / CPR, ch = tid % CPR;
      const uint32_t at = (row0 + r) * C::DB + ch * 16;
      const uint8_t *kp = w.k + (id < 0 ? 0 : id) * w.kps + at, *vp = w.v + (id < 0 ? 0 : id) * w.vps + at;
#pragma unroll
      for (int i = 0; i < (kTile * CPR + NT - 1) / NT; ++i) {
        const int row = r + i * (NT / CPR);
        if (kTile * CPR % NT == 0 || row < kTile) {
          const bool ok = id >= 0 && row < left;
          cp16(ks + C::at(row, ch), kp + i * (NT / CPR) * C::DB, ok);
          cp16(vs + C::at(row, ch), vp + i * (NT / CPR) * C::DB, ok);
        }
      }
    } else {
      const uint32_t first = static_cast<uint32_t>(T.head) << lg;
#pragma unroll
      for (int i = 0; i < (kTile * CPR + NT - 1) / NT; ++i) {
        const int y = tid + i * NT, row = y / CPR, ch = y - row * CPR;
        if (kTile * CPR % NT && y >= kTile * CPR) break;
        const int id = T.page[row >> 4];
        const uint32_t at = (first + ((T.t0 + row) & pm)) * C::DB + ch * 16;
        const bool ok = id >= 0 && row < left;
        cp16(ks + C::at(row, ch), w.k + (ok ? id * w.kps + at : 0), ok);
        cp16(vs + C::at(row, ch), w.v + (ok ? id * w.vps + at : 0), ok);
      }
    }
  };
  // --- a token's exponents and the factors made of them
  auto exps = [&](const TileInfo &T, int i) {
    const int id = T.page[i >> 4];
    int e = 0;
    if (id >= 0 && T.t0 + i < T.held) {
      const int64_t at = ((static_cast<int64_t>(id) * w.Hkv + T.head) << lg) + ((T.t0 + i) & pm);
      e = (static_cast<int>(__ldg(w.ke + at)) & 0xffff) | static_cast<int>(__ldg(w.ve + at)) << 16;
    }
    return e;
  };
  auto factors = [&](uint32_t x, int i, int e) {
    const int ek = static_cast<int16_t>(e & 0xffff), ev = e >> 16;
    consts[x % ST * kTile + i] = make_float4(pow2i(ek), static_cast<float>(ev), pow2i(-ev) * SUM, 0.0f);
  };
  // --- row r (of all rows of the item's sequence, or of the prefix): its query
  // and the tokens that it sees; null past the last row
  auto query = [&](const TileInfo &T, int r, int &lim) -> const __nv_bfloat16 * {
    lim = 0;
    if (r >= T.rows) return nullptr;
    const int b = pre ? before(r) : T.b, rr = pre ? r - static_cast<int>(cum0[b]) : r;
    const int i = rr / G, gg = rr - i * G;
    lim = pre ? w.prefix : T.own + i + 1;
    return P.q + b * P.qs0 + i * P.qs1 + (T.head * G + gg) * P.qs2;
  };
  // --- 16 rows: the queries of the item that begins with a tile, slot k of 3
  auto queries = [&](const TileInfo &T, int k) {
    constexpr int CH = D / 8;
    for (int x = tid; x < RT * CH; x += NT) {
      const int r = x / CH, ch = x - r * CH;
      int lim;
      const __nv_bfloat16 *src = query(T, T.row0 + r, lim);
      uint8_t *dst = qbuf + (k * RT + r) * C::QLD + ch * 16;
      if (P.qvec) {
        cp16(s32(dst), src ? src + 8 * ch : P.q, src != nullptr);
      } else {
        for (int i = 0; i < 8; ++i)
          reinterpret_cast<uint16_t *>(dst)[i] =
              src ? __ldg(reinterpret_cast<const uint16_t *>(src) + 8 * ch + i) : 0;
      }
    }
  };

  if (warp == 0) {
    if (lane == 0) {
      Cursor c;
      begin(c);
      *cursor = c;
    }
    __syncwarp();
    for (int i = 1; i < ST && lo + i < hi; ++i) advance(lo + i);
  }
  __syncthreads();
  if (tid < 4 * ST && lo + (tid >> 2) < hi) {  // the first tiles' page ids
    TileInfo &T = info[(lo + (tid >> 2)) & 3];
    T.page[tid & 3] = page(T, tid & 3);
  }
  int slot_in = 0, slot_out = 0;  // query slots (16 rows)
  __syncthreads();
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) {
    if (lo + i < hi) {
      const TileInfo &T = info[(lo + i) & 3];
      if (WR == 1 && T.first) {
        queries(T, slot_in);
        slot_in = slot_in == 2 ? 0 : slot_in + 1;
      }
      fetch(lo + i, T);
      if (E4M3 && tid < kTile) factors(lo + i, tid, exps(T, tid));
    }
    cp_commit();
  }

  constexpr int KQ = D / 16;  // k steps of q.k
  uint32_t qf[KQ][4];
  float o[D / 8][4];
  float M0, M1, l0, l1;
  float cq0 = P.c, cq1 = P.c;  // score factors of rows g and g + 8: scale log2 e 2^eq
  int lim0 = 0, lim1 = 0;      // tokens that they see
  int rows = 0;                // rows of the item
  int free_to = 0;             // tokens that every row sees

  for (uint32_t x = lo; x < hi; ++x) {
    cp_wait<ST - 2>();
    __syncthreads();
    const TileInfo &T = info[x & 3];
    // the copies of a tile to come, then the description of the one behind it
    int idn = -1, exn = 0;
    const bool take = x + ST - 1 < hi, more = x + ST < hi;
    if (take) {
      const TileInfo &A = info[(x + ST - 1) & 3];
      if (WR == 1 && A.first) {
        queries(A, slot_in);
        slot_in = slot_in == 2 ? 0 : slot_in + 1;
      }
      fetch(x + ST - 1, A);
      if (E4M3 && tid < kTile) exn = exps(A, tid);
    }
    cp_commit();
    if (more && warp == 0) {
      advance(x + ST);
      if (lane < 4) idn = page(info[(x + ST) & 3], lane);
    }

    if (T.first) {  // a new item: its rows' queries, in registers
      rows = T.rows - T.row0;
      free_to = pre ? w.prefix : T.own + T.row0 / G + 1;
      const __nv_bfloat16 *src[2];
      src[0] = query(T, T.row0 + wr * 16 + g, lim0);
      src[1] = query(T, T.row0 + wr * 16 + g + 8, lim1);
      const uint8_t *qs = qbuf + (slot_out * RT + g) * C::QLD;
      if (WR == 1) slot_out = slot_out == 2 ? 0 : slot_out + 1;
      auto word = [&](int a, int d) -> uint32_t {  // elements d, d + 1 of row g + 8 a
        if (WR == 1) return *reinterpret_cast<const uint32_t *>(qs + 8 * a * C::QLD + 2 * d);
        if (!src[a]) return 0;
        if (P.qvec) return __ldg(reinterpret_cast<const uint32_t *>(src[a] + d));
        const uint32_t x = __ldg(reinterpret_cast<const uint16_t *>(src[a] + d));
        const uint32_t y = __ldg(reinterpret_cast<const uint16_t *>(src[a] + d + 1));
        return x | y << 16;
      };
      if constexpr (E4M3) {
        // bring each row's largest finite magnitude to [2^10, 2^11): exact in
        // float16 for all elements above 2^-28 of it
        uint32_t m0 = 0, m1 = 0;
#pragma unroll
        for (int k = 0; k < KQ; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            qf[k][i] = word(i & 1, 16 * k + 4 * q4 + (i & 2));  // d as the key's bytes
            const uint32_t x = qf[k][i] & 0x7fffu, y = qf[k][i] >> 16 & 0x7fffu;
            const uint32_t m = max(x < 0x7f80u ? x : 0u, y < 0x7f80u ? y : 0u);
            if (i & 1) m1 = max(m1, m);
            else m0 = max(m0, m);
          }
        m0 = max(m0, __shfl_xor_sync(~0u, m0, 1)), m1 = max(m1, __shfl_xor_sync(~0u, m1, 1));
        m0 = max(m0, __shfl_xor_sync(~0u, m0, 2)), m1 = max(m1, __shfl_xor_sync(~0u, m1, 2));
        const int eq0 = max(static_cast<int>(m0 >> 7) - 127 - 10, -100);
        const int eq1 = max(static_cast<int>(m1 >> 7) - 127 - 10, -100);
        cq0 = P.c * pow2i(eq0), cq1 = P.c * pow2i(eq1);
        const float f0 = pow2i(-eq0), f1 = pow2i(-eq1);
#pragma unroll
        for (int k = 0; k < KQ; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f = i & 1 ? f1 : f0;
            qf[k][i] = pack<true>(__uint_as_float(qf[k][i] << 16) * f, __uint_as_float(qf[k][i] & 0xffff0000u) * f);
          }
      } else {
#pragma unroll
        for (int k = 0; k < KQ; ++k) {
          const int d = 16 * k + 2 * q4;
          qf[k][0] = word(0, d), qf[k][1] = word(1, d);
          qf[k][2] = word(0, d + 8), qf[k][3] = word(1, d + 8);
        }
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = 0.0f;
      M0 = M1 = -INFINITY;
      l0 = l1 = 0.0f;
    }
    uint8_t *stage = stages + x % ST * C::STAGE;
    const uint32_t ks = s32(stage), vs = ks + C::TILE;
    const float4 *fac = consts + x % ST * kTile;
    const int t0 = T.t0, held = T.held;
    const bool edge = t0 + kTile > free_to;
    // Tokens that some row of the tile does not see but that are present: a
    // NaN or infinity among their values would reach every row through a zero
    // weight.  Take such elements out; add them below to the rows that see them.
    const bool banded = edge && !pre && held > free_to;
    uint32_t hot[2] = {0, 0};
    if (banded) {
      const int first = max(free_to - t0, 0), last = min(held - t0, kTile);
      for (int i = first * CPR + tid; i < last * CPR; i += NT) {
        const int row = i / CPR, ch = i - row * CPR;
        uint4 *p = reinterpret_cast<uint4 *>(stage + C::TILE + C::at(row, ch));
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

#pragma unroll 1
    for (int tp = wt * TPW; tp < (wt + 1) * TPW; tp += TPP) {
    // --- scores
    float s[NG][4];
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[j][k] = 0.0f;
    // ldmatrix: this lane's row, and its chunk c + (lane >> 4), c even
    const uint32_t lrow = (tp + (lane & 15)) * LD, lch = ((lane >> 4) ^ C::swap(lane & 15)) << 4;
    const uint32_t krow = ks + lrow;
#pragma unroll
    for (int jp = 0; jp < NG / 2; ++jp) {
      // four matrices: groups 2jp, 2jp + 1 of 8 tokens x two 16-byte chunks
#pragma unroll
      for (int c = 0; c < CPR; c += 2) {
        uint32_t r[4];
        const uint32_t a = krow + jp * 16 * LD + (C::SWAP ? c * 16 ^ lch : c * 16 + lch);
        if (c + 1 < CPR) ldm4(a, r);
        else ldm2(a, r);
        if constexpr (E4M3) {
          mma<true>(s[2 * jp], qf[c], cvt_lo(r[0]), cvt_hi(r[0]));
          mma<true>(s[2 * jp + 1], qf[c], cvt_lo(r[1]), cvt_hi(r[1]));
          if (c + 1 < CPR) {
            constexpr int top = KQ - 1;
            mma<true>(s[2 * jp], qf[c + 1 <= top ? c + 1 : 0], cvt_lo(r[2]), cvt_hi(r[2]));
            mma<true>(s[2 * jp + 1], qf[c + 1 <= top ? c + 1 : 0], cvt_lo(r[3]), cvt_hi(r[3]));
          }
        } else {
          mma<false>(s[2 * jp], qf[c / 2], r[0], r[2]);
          mma<false>(s[2 * jp + 1], qf[c / 2], r[1], r[3]);
        }
      }
    }

    // --- running softmax
    float m0 = M0, m1 = M1;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const int col = tp + 8 * j + 2 * q4;
      if constexpr (E4M3) {
        const float4 a = fac[col], b = fac[col + 1];
        s[j][0] = fmaf(s[j][0], cq0 * a.x, a.y);
        s[j][1] = fmaf(s[j][1], cq0 * b.x, b.y);
        s[j][2] = fmaf(s[j][2], cq1 * a.x, a.y);
        s[j][3] = fmaf(s[j][3], cq1 * b.x, b.y);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) s[j][k] *= P.c;
      }
      if (edge) {
        const int t = t0 + col;
        if (t >= lim0) s[j][0] = -INFINITY;
        if (t + 1 >= lim0) s[j][1] = -INFINITY;
        if (t >= lim1) s[j][2] = -INFINITY;
        if (t + 1 >= lim1) s[j][3] = -INFINITY;
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
      float i0 = 1.0f, i1 = 1.0f;  // 2^-ev SUM
      if constexpr (E4M3) {
        const int col = tp + 8 * j + 2 * q4;
        i0 = fac[col].z, i1 = fac[col + 1].z;
      }
      l0 = fmaf(a, i0, fmaf(b, i1, l0));
      l1 = fmaf(c, i0, fmaf(d, i1, l1));
      p[j / 2][(j & 1) * 2] = pack<E4M3>(a, b);
      p[j / 2][(j & 1) * 2 + 1] = pack<E4M3>(c, d);
    }

    // --- weighted values
    const uint32_t vrow = vs + lrow;
#pragma unroll
    for (int kk = 0; kk < NG / 2; ++kk) {
#pragma unroll
      for (int c = 0; c < CPR; c += 2) {
        uint32_t r[4];
        const uint32_t a = vrow + kk * 16 * LD + (C::SWAP ? c * 16 ^ lch : c * 16 + lch);
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
    }
    if (hot[0] | hot[1]) {  // rare: the elements taken out above
      for (int k = 0; k < TPW; ++k) {
        const int row = wt * TPW + k, t = t0 + row;
        if (!((row < 32 ? hot[0] : hot[1]) >> (row & 31) & 1)) continue;
        const int id = w.table[T.b * w.tstride + (t >> lg)];
        const uint8_t *v = w.v + id * w.vps + ((static_cast<int64_t>(T.head) << lg) + (t & pm)) * C::DB;
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

    if (more && tid < 4) info[(x + ST) & 3].page[tid] = idn;
    if (E4M3 && take && tid < kTile) factors(x + ST - 1, tid, exn);

    // --- at the end of the item or of the span, leave the partial result
    if (!T.last) continue;
    const uint32_t slot = T.slot;
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
      if (r >= rows) continue;
      const float l = a ? l1 : l0, M = a ? M1 : M0;
      const float f = l == 0.0f ? 0.0f : 1.0f / l;
      const int64_t at = static_cast<int64_t>(slot) * RT + r;
      float *dst = P.po + at * D;
      if constexpr (E4M3) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          *reinterpret_cast<float4 *>(dst + 16 * c + 4 * q4) =
              make_float4(o[2 * c][2 * a] * SUM * f, o[2 * c + 1][2 * a] * SUM * f, o[2 * c][2 * a + 1] * SUM * f,
                          o[2 * c + 1][2 * a + 1] * SUM * f);
      } else {
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<float2 *>(dst + 8 * c + 2 * q4) =
              make_float2(o[c][2 * a] * f, o[c][2 * a + 1] * f);
      }
      if (q4 == 0) P.pl[at] = l == 0.0f ? -INFINITY : M - (BIAS - SUM_LOG) + log2f(l);
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
