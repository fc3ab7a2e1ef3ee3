// kv_pages.cu -- entries and pages of the cache on the move: an accepted path's
// entries to consecutive positions, page tables over a pool with reference
// counts (grow, shrink, free, fork), and copies of pages.
//
// Compact: a place is never behind the entry that goes to it (path[j] >= j), and
// never that of a later one, so entries may be moved in increasing order.  A CTA
// takes a sequence and a head, a thread 16 bytes of an entry; a pass's loads all
// come before its stores.
//
// Tables: one cluster of CTAs does a whole call, so that counts, sums and
// assignments can wait for one another.  What each row needs is summed over the
// rows by every CTA for itself; where that is little the first CTA goes on alone,
// without the cluster's barriers.  Then the counts are read, 32 a thread, and the
// free pages numbered by sums over the warp, the CTA and the cluster, in the
// order of the page ids: page of number k goes to the row in whose sum k falls.
// The counts go to the CTAs in turns of 1024 (in eight long pieces the lowest free
// pages were a few CTAs' work alone: 64 x 1024 of them 12 us in place of 7).
// Nothing depends on the order of atomics: they add to counts, or or bits.
//
// Bound: the chain of loads and cluster barriers; copies by memory.  Measured (replayed
// calls): four entries each of 256 accepted paths, 8 heads of 128 in bfloat16, 5.7 us.
// 512 rows' room for nine tokens (287 pages of 98304) and back 10.7 us for both calls, 2.8
// where there is nothing to do; 64 x 1024 pages of 262144 and back 19 us.  31 forks each
// of 8 rows of 23 .. 31 pages of 128 tokens and back 18 us, the copies of their last pages
// (62 MB in and out) 8.0 us, 7.8 TB/s: what was read just before is in L2.
// Free pages are looked for from the lowest number on, so these hold where some of the
// first pages are free.  Where they are taken, the counts up to the first free page are
// read, and read again by the pass that gives pages; with few entries by one CTA, 32768
// counts a round: 512 rows' nine tokens and back with the first 90 % of the pool taken 16.6
// us of 98304 pages, 29.8 of 262144 (10.4 and 10.1 with as many taken anywhere).
#include <cooperative_groups.h>

#include <type_traits>
#include <utility>

#include "kv_common.cuh"
#include "spec_tree.h"

namespace {

namespace cg = cooperative_groups;
using kv::View;

// ------------------------------------------------------------------ compact
constexpr int MV_NT = 256;

struct MP {
  View w;
  uint8_t *k, *v;
  int8_t *ke, *ve;
  const int32_t *path, *acc;
  int32_t *status;
};

template <bool E4M3>
__global__ void __launch_bounds__(MV_NT) compact_kernel(const __grid_constant__ MP P, int D) {
  const View &w = P.w;
  const int b = blockIdx.y, head = blockIdx.x, tid = threadIdx.x;
  const int a = P.acc[b], len = w.len[b];
  const int32_t *path = P.path + static_cast<int64_t>(b) * w.N;
  const int own = len - w.prefix;
  int st = a < 0 || a >= w.N ? SPEC_ROW_BAD_TREE : 0, bad = 0;
  if (!st)
    for (int j = 1 + tid; j <= a; j += MV_NT) {
      const int at = path[j], before = path[j - 1];
      bad |= at <= before || at >= w.N || (j == 1 && before != 0);
    }
  if (__syncthreads_or(bad)) st = SPEC_ROW_BAD_TREE;
  if (len < w.prefix) st |= SPEC_ROW_BAD_LENGTH;
  else if (!st && a > 0 && own + static_cast<int64_t>(path[a]) >= static_cast<int64_t>(w.max_pages) << w.ps_log2)
    st |= SPEC_ROW_BAD_LENGTH;
  const bool go = !st && a > 0;  // of the whole CTA
  const int DB = E4M3 ? D : 2 * D, CPR = DB / 16;
  const int cols = 2 * CPR + (E4M3 ? 1 : 0);  // 16 bytes of a key or a value; both exponents
  const int per = MV_NT / cols;               // entries of a pass
  const int col = tid % cols, sub = tid / cols;
  const int pm = (1 << w.ps_log2) - 1;
  const uint32_t np = static_cast<uint32_t>(w.n_pages);
  const int32_t *ids = w.table + b * w.tstride;
  int lost = 0;
  if (go)
    for (int j0 = 1; j0 <= a; j0 += per) {
      const int j = j0 + sub;
      const bool mine = sub < per && j <= a;
      int64_t to = 0;
      bool put = false;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (mine) {
        const int s = own + path[j], d = own + j;
        if (s != d) {
          const int sp = ids[s >> w.ps_log2], dp = ids[d >> w.ps_log2];
          put = static_cast<uint32_t>(sp) < np && static_cast<uint32_t>(dp) < np;
          lost |= !put;
          const int64_t sr = (static_cast<int64_t>(head) << w.ps_log2) + (s & pm);
          const int64_t dr = (static_cast<int64_t>(head) << w.ps_log2) + (d & pm);
          if (put) {
            if (col < CPR) {
              to = dp * w.kps + dr * DB + col * 16;
              x = *reinterpret_cast<const uint4 *>(P.k + sp * w.kps + sr * DB + col * 16);
            } else if (col < 2 * CPR) {
              to = dp * w.vps + dr * DB + (col - CPR) * 16;
              x = *reinterpret_cast<const uint4 *>(P.v + sp * w.vps + sr * DB + (col - CPR) * 16);
            } else if constexpr (E4M3) {
              const int64_t page = static_cast<int64_t>(w.Hkv) << w.ps_log2;
              to = dp * page + dr;
              x.x = static_cast<uint8_t>(P.ke[sp * page + sr]);
              x.y = static_cast<uint8_t>(P.ve[sp * page + sr]);
            }
          }
        }
      }
      __syncthreads();
      if (put) {
        if (col < CPR) *reinterpret_cast<uint4 *>(P.k + to) = x;
        else if (col < 2 * CPR) *reinterpret_cast<uint4 *>(P.v + to) = x;
        else if constexpr (E4M3) P.ke[to] = static_cast<int8_t>(x.x), P.ve[to] = static_cast<int8_t>(x.y);
      }
      __syncthreads();
    }
  if (__syncthreads_or(lost)) st |= SPEC_ROW_BAD_PAGE;
  if (P.status && head == 0 && tid == 0) P.status[b] = st;
}

// --------------------------------------------------------------------- copy
constexpr int CY_NT = 128;

struct YP {
  uint8_t *k, *v;
  int8_t *ke, *ve;
  const int32_t *copies;
  int64_t kps, vps;
  int32_t n_pages, Hkv, page, row;  // row: bytes of an entry and head
};

// Grid: heads by triples.  The entries of a head are side by side in a page.
__global__ void __launch_bounds__(CY_NT) copy_kernel(const __grid_constant__ YP P) {
  const int32_t *c = P.copies + static_cast<int64_t>(blockIdx.x / P.Hkv) * 3;
  const int head = blockIdx.x % P.Hkv;
  const int src = c[0], dst = c[1], n = min(c[2], P.page);
  if (static_cast<uint32_t>(src) >= static_cast<uint32_t>(P.n_pages) ||
      static_cast<uint32_t>(dst) >= static_cast<uint32_t>(P.n_pages) || n <= 0 || src == dst)
    return;
  const int64_t in = static_cast<int64_t>(head) * P.page * P.row;
  const uint4 *ks = reinterpret_cast<const uint4 *>(P.k + src * P.kps + in), *vs = reinterpret_cast<const uint4 *>(P.v + src * P.vps + in);
  uint4 *kd = reinterpret_cast<uint4 *>(P.k + dst * P.kps + in), *vd = reinterpret_cast<uint4 *>(P.v + dst * P.vps + in);
  const int chunks = n * P.row / 16;  // rows are multiples of 16 bytes
  int i = threadIdx.x;
  for (; i + 3 * CY_NT < chunks; i += 4 * CY_NT) {
    uint4 x[4], y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = __ldcs(ks + i + u * CY_NT), y[u] = __ldcs(vs + i + u * CY_NT);
#pragma unroll
    for (int u = 0; u < 4; ++u) __stcs(kd + i + u * CY_NT, x[u]), __stcs(vd + i + u * CY_NT, y[u]);
  }
  for (; i < chunks; i += CY_NT) {
    const uint4 x = __ldcs(ks + i), y = __ldcs(vs + i);
    __stcs(kd + i, x), __stcs(vd + i, y);
  }
  if (P.ke) {
    const int64_t page = static_cast<int64_t>(P.Hkv) * P.page, at = static_cast<int64_t>(head) * P.page;
    for (int t = threadIdx.x; t < n; t += CY_NT) {
      P.ke[dst * page + at + t] = P.ke[src * page + at + t];
      P.ve[dst * page + at + t] = P.ve[src * page + at + t];
    }
  }
}

// ------------------------------------------------------------------- tables
constexpr int TB_NT = 1024;   // threads of a CTA
constexpr int TB_CTAS = 8;    // of the cluster
constexpr int TB_EACH = 32;   // counts of a thread and round: 8 loads of 4
constexpr uint32_t TB_ALONE = 4096;  // entries that one CTA sees to alone

struct Pool {
  int32_t *refs, *table, *held;
  int64_t tstride;
  int32_t B, max_pages, n_pages, prefix, ps_log2;
  bool vec;  // refs is 16-byte aligned
};

struct TableShared {
  uint16_t list[TB_NT * TB_EACH];  // free pages of the CTA's parts of a round: warp, place in its 1024 counts
  unsigned long long warp2[TB_NT / 32];
  uint32_t count[2][TB_NT / 32];  // free pages of the warps' parts of a round, by the round's parity
  uint32_t first[TB_NT / 32];     // their numbers in the round
  uint32_t number[TB_NT / 32];    // what a warp's places on the list are behind their pages' numbers
  uint32_t all;                   // free pages of the round
};

// Who works on the tables: the whole cluster, or its first CTA.
struct Team {
  unsigned rank, ctas;
  __device__ void sync() const {
    if (ctas > 1) cg::this_cluster().sync();
    else __syncthreads();
  }
  __device__ int64_t round() const { return static_cast<int64_t>(ctas) * TB_NT * TB_EACH; }
};

// Exclusive sum over the CTA's threads; *all: the whole sum.  Barriers on both sides.
template <class T>
__device__ T cta_sum(T x, T *warps, T *all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T e = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(~0u, e, o);
    if (lane >= o) e += t;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = e;
  __syncthreads();
  const T mine = warps[lane];
  T s = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(~0u, s, o);
    if (lane >= o) s += t;
  }
  *all = __shfl_sync(~0u, s, 31);
  return e - x + __shfl_sync(~0u, s - mine, warp);
}

// a[0 .. n], b[0 .. n]: sums of a[0 .. n), b[0 .. n) before each entry, by the whole
// CTA (both in one word of 64 bits: no sum reaches 2^32).
__device__ void sum_up(uint32_t *a, uint32_t *b, int n, unsigned long long *warps) {
  const int per = (n + TB_NT - 1) / TB_NT, i0 = min(static_cast<int>(threadIdx.x) * per, n), i1 = min(i0 + per, n);
  unsigned long long mine = 0, all;
  for (int i = i0; i < i1; ++i) mine += a[i] | static_cast<unsigned long long>(b[i]) << 32;
  unsigned long long at = cta_sum(mine, warps, &all);
  for (int i = i0; i < i1; ++i) {
    const uint32_t x = a[i], y = b[i];
    a[i] = static_cast<uint32_t>(at);
    b[i] = static_cast<uint32_t>(at >> 32);
    at += x | static_cast<unsigned long long>(y) << 32;
  }
  if (threadIdx.x == 0) a[n] = static_cast<uint32_t>(all), b[n] = static_cast<uint32_t>(all >> 32);
  __syncthreads();
}

// The largest i < n with cum[i] <= x (x < cum[n]).
__device__ __forceinline__ int before(const uint32_t *cum, int n, uint32_t x) {
  int l = 0, r = n;
  while (r - l > 1) {
    const int m = (l + r) >> 1;
    if (cum[m] <= x) l = m;
    else r = m;
  }
  return l;
}
// The same for several x, whose loads do not wait for one another.
template <int K>
__device__ __forceinline__ void before(const uint32_t *cum, int n, const uint32_t (&x)[K], int (&i)[K]) {
#pragma unroll
  for (int u = 0; u < K; ++u) i[u] = 0;
  for (int s = n > 1 ? 1 << (31 - __clz(n - 1)) : 0; s; s >>= 1)
#pragma unroll
    for (int u = 0; u < K; ++u)
      if (i[u] + s < n && cum[i[u] + s] <= x[u]) i[u] += s;
}

// f(K, i) for i = from, from + K stride, .. below n: for i, i + stride, .. as far as they
// are below n; K is one where no thread has more, since a group costs what all of it does.
template <int K, class F>
__device__ __forceinline__ void in_groups(uint32_t from, uint32_t stride, uint32_t n, F f) {
  if (n <= stride) {
    if (from < n) f(std::integral_constant<int, 1>{}, from);
  } else {
    for (uint32_t i = from; i < n; i += K * stride) f(std::integral_constant<int, K>{}, i);
  }
}

// Of the thread's 32 counts from count i0 on (the warp's part: 1024 counts), those
// that are of free pages: bit 4 u + k is count i0 + 128 u + 4 lane + k.
__device__ uint32_t free_bits(const Pool &P, int64_t i0) {
  i0 += 4 * (threadIdx.x & 31);
  uint32_t bits = 0;
  if (P.vec && i0 + 7 * 128 + 4 <= P.n_pages) {
    int4 x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = __ldcg(reinterpret_cast<const int4 *>(P.refs + i0 + 128 * u));
#pragma unroll
    for (int u = 0; u < 8; ++u)
      bits |= (static_cast<uint32_t>(x[u].x <= 0) | static_cast<uint32_t>(x[u].y <= 0) << 1 |
               static_cast<uint32_t>(x[u].z <= 0) << 2 | static_cast<uint32_t>(x[u].w <= 0) << 3) << (4 * u);
  } else {
#pragma unroll 1
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = i0 + 128 * u + k;
        if (i < P.n_pages && __ldcg(P.refs + i) <= 0) bits |= 1u << (4 * u + k);
      }
  }
  return bits;
}

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ uint32_t sum_to(uint32_t x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(~0u, x, o);
    if ((threadIdx.x & 31) >= o) x += t;
  }
  return x;
}

// Takes the lowest free pages for the rows of cum (n + 1 sums of what they need):
// give(row, k, page) for the k-th page of each row that is served, that is whose
// sum is within what the pool has.  Returns the number of free pages, or any
// number from the rows' sum on.  All CTAs of the team call it, after a team's
// barrier behind the last change of a count.  A round's parts of 1024 counts go to
// the CTAs in turn, so that each has its share of the pages that are given: the
// lowest ones are in the first parts.
template <class F>
__device__ uint32_t take_pages(const Pool &P, const uint32_t *cum, int n, const Team &team, TableShared &S, F give) {
  const unsigned rank = team.rank, ctas = team.ctas;
  const int64_t round = team.round();
  const uint32_t total = cum[n];
  if (total == 0) return 0;
  const int rounds = static_cast<int>((P.n_pages + round - 1) / round);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t bits = 0;           // the thread's free pages of the round,
  uint32_t size = 0, first = 0;  // those of the CTA's warp `lane`, the number of the first of them in the round
  int turn = 0;
  auto count = [&](int r) -> uint32_t {  // free pages of round r
    bits = free_bits(P, r * round + (static_cast<int64_t>(warp) * ctas + rank) * 1024);
    uint32_t *mine = S.count[turn++ & 1];
    const uint32_t c = __reduce_add_sync(~0u, __popc(bits));
    if (lane == 0) mine[warp] = c;
    if (ctas == 1) {
      __syncthreads();
      size = mine[lane];
      const uint32_t to = sum_to(size);
      first = to - size;
      return __shfl_sync(~0u, to, 31);
    }
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    if (warp == 0) {  // the parts' order: warps, then CTAs
      uint32_t x[TB_CTAS], all = 0, ahead = 0;
#pragma unroll
      for (unsigned c = 0; c < TB_CTAS; ++c) x[c] = *cl.map_shared_rank(mine + lane, c);
#pragma unroll
      for (unsigned c = 0; c < TB_CTAS; ++c) {
        if (c < rank) ahead += x[c];
        all += x[c];
      }
      const uint32_t to = sum_to(all);
      S.first[lane] = to - all + ahead;
      if (lane == 31) S.all = to;
    }
    __syncthreads();
    size = mine[lane];
    first = S.first[lane];
    return S.all;
  };
  uint32_t found = 0;
  int counted = 0;
  for (; counted < rounds && found < total; ++counted) found += count(counted);
  // rows up to the last one whose sum the pool has
  const uint32_t limit = found >= total ? total : cum[before(cum, n, found)];
  uint32_t sum = 0;
  for (int r = 0; r < rounds && sum < limit; ++r) {
    const uint32_t here = counted == 1 ? found : count(r);  // one round: as counted
    // The warps' places on the CTA's list, for those that are given.
    const uint32_t number = sum + first, given = number < limit ? min(limit - number, size) : 0;
    const uint32_t to = sum_to(given);
    if (warp == 0) S.number[lane] = number - (to - given);
    const uint32_t mine = __shfl_sync(~0u, to, 31);  // of the CTA
    const uint32_t base = __shfl_sync(~0u, to - given, warp), end = base + __shfl_sync(~0u, given, warp);
    if (base < end) {
      // a warp's pages in the order of u, lane, k: sums over the lanes for each u,
      // four of them in a word (32 x 4 counts fit eight bits)
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        lo |= __popc(bits >> (4 * u) & 15) << (8 * u);
        hi |= __popc(bits >> (16 + 4 * u) & 15) << (8 * u);
      }
      uint32_t el = sum_to(lo), eh = sum_to(hi);
      const uint32_t al = __shfl_sync(~0u, el, 31), ah = __shfl_sync(~0u, eh, 31);
      el -= lo, eh -= hi;
      uint32_t at = base;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        uint32_t k = at + ((u < 4 ? el : eh) >> (8 * (u & 3)) & 255);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const bool is = bits >> (4 * u + v) & 1;
          if (is && k < end) S.list[k] = static_cast<uint16_t>(warp * 1024 + 128 * u + 4 * lane + v);
          k += is;
        }
        at += (u < 4 ? al : ah) >> (8 * (u & 3)) & 255;
      }
    }
    __syncthreads();
    in_groups<4>(threadIdx.x, TB_NT, mine, [&](auto K_, uint32_t k0) {
      constexpr int K = decltype(K_)::value;
      uint32_t x[K];
      int id[K], row[K];
#pragma unroll
      for (int u = 0; u < K; ++u) {
        const uint32_t k = min(k0 + u * TB_NT, mine - 1), e = S.list[k];
        x[u] = k + S.number[e >> 10];
        id[u] = static_cast<int>(r * round + (static_cast<int64_t>(e >> 10) * ctas + rank) * 1024 + (e & 1023));
      }
      before(cum, n, x, row);
#pragma unroll
      for (int u = 0; u < K; ++u)
        if (k0 + u * TB_NT < mine) give(row[u], x[u] - cum[row[u]], id[u]);
    });
    __syncthreads();
    sum += here;
  }
  return found;
}

struct RP {
  Pool p;
  const int32_t *len;
  int32_t *status;
  int32_t n;
};

// Pages that a row of `held` is to hold for `len` + n tokens; -1: bad.
__device__ __forceinline__ int wanted(const Pool &P, int len, int n, int held, int *st) {
  const int64_t t = static_cast<int64_t>(len) + n - P.prefix;
  const int64_t want = len == -1 ? 0 : (t + (1 << P.ps_log2) - 1) >> P.ps_log2;
  *st = len < -1 || (len >= 0 && t < 0) || want > P.max_pages || held < 0 || held > P.max_pages ? SPEC_ROW_BAD_LENGTH : 0;
  return *st ? -1 : static_cast<int>(want);
}

__global__ void __cluster_dims__(TB_CTAS, 1, 1) __launch_bounds__(TB_NT) resize_kernel(const __grid_constant__ RP R) {
  extern __shared__ __align__(16) uint8_t tm[];
  TableShared &S = *reinterpret_cast<TableShared *>(tm);
  uint32_t *cum = reinterpret_cast<uint32_t *>(tm + sizeof(TableShared));  // B + 1 pages to take, B + 1 pages to give back, B held
  const Pool &P = R.p;
  Team team = {cg::this_cluster().block_rank(), TB_CTAS};
  const int B = P.B, tid = threadIdx.x;
  uint32_t *gone = cum + B + 1;
  int32_t *has = reinterpret_cast<int32_t *>(gone + B + 1);
  for (int b = tid; b < B; b += TB_NT) {
    const int held = P.held[b];
    int st;
    const int want = wanted(P, R.len[b], R.n, held, &st);
    has[b] = held;
    cum[b] = want > held ? want - held : 0;
    gone[b] = want >= 0 && want < held ? held - want : 0;
    if (team.rank == 0 && R.status) R.status[b] = st;
  }
  // the status words are written; what is held and the lengths have been read by all,
  // so that all come to the same sums whatever one of them does behind the wait
  auto read = cg::this_cluster().barrier_arrive();
  __syncthreads();
  sum_up(cum, gone, B, S.warp2);
  cg::this_cluster().barrier_wait(std::move(read));
  if (!(cum[B] | gone[B])) return;
  if (cum[B] + gone[B] <= TB_ALONE) {
    if (team.rank) return;
    team.ctas = 1;
  }
  if (gone[B]) {
    const uint32_t np = static_cast<uint32_t>(P.n_pages), many = gone[B], stride = team.ctas * TB_NT;
    in_groups<8>(team.rank * TB_NT + tid, stride, many, [&](auto K_, uint32_t x0) {
      constexpr int K = decltype(K_)::value;
      uint32_t x[K];
      int id[K], of[K];
#pragma unroll
      for (int u = 0; u < K; ++u) x[u] = min(x0 + u * stride, many - 1);
      before(gone, B, x, of);
#pragma unroll
      for (int u = 0; u < K; ++u)  // the last gone[row + 1] - gone[row] entries of the row
        if (x0 + u * stride < many)
          id[u] = P.table[of[u] * P.tstride + has[of[u]] - static_cast<int>(gone[of[u] + 1] - x[u])];
#pragma unroll
      for (int u = 0; u < K; ++u) {
        if (x0 + u * stride >= many) continue;
        if (static_cast<uint32_t>(id[u]) < np) atomicSub(P.refs + id[u], 1);
        else if (R.status) atomicOr(R.status + of[u], SPEC_ROW_BAD_PAGE);
      }
    });
    team.sync();  // the counts
  }
  const uint32_t found = take_pages(P, cum, B, team, S, [&](int row, uint32_t k, int32_t id) {
    P.table[row * P.tstride + has[row] + k] = id;
    P.refs[id] = 1;
  });
  for (int b = team.rank * TB_NT + tid; b < B; b += team.ctas * TB_NT) {
    const uint32_t take = cum[b + 1] - cum[b], give = gone[b + 1] - gone[b];
    if (take && cum[b + 1] > found) {
      if (R.status) atomicOr(R.status + b, SPEC_ROW_NO_PAGES);
    } else if (take | give) {
      P.held[b] = has[b] + static_cast<int>(take) - static_cast<int>(give);
    }
  }
  // no CTA ends while another one may read its part of the sums
  if (team.ctas > 1 && cum[B]) team.sync();
}

struct FP {
  Pool p;
  int32_t *len;
  const int32_t *src, *dst;
  int32_t *copies, *status;
  int32_t n;
};

__global__ void __cluster_dims__(TB_CTAS, 1, 1) __launch_bounds__(TB_NT) fork_kernel(const __grid_constant__ FP F) {
  extern __shared__ __align__(16) uint8_t tm[];
  TableShared &S = *reinterpret_cast<TableShared *>(tm);
  // n + 1 pages to take, n + 1 pages to share, B first forks to each row, n lengths of the sources, n flags
  uint32_t *cum = reinterpret_cast<uint32_t *>(tm + sizeof(TableShared));
  const Pool &P = F.p;
  Team team = {cg::this_cluster().block_rank(), TB_CTAS};
  const int n = F.n, tid = threadIdx.x, lg = P.ps_log2;
  const uint32_t B = static_cast<uint32_t>(P.B), np = static_cast<uint32_t>(P.n_pages);
  uint32_t *shared = cum + n + 1, *first = shared + n + 1;
  int32_t *lens = reinterpret_cast<int32_t *>(first + P.B);
  uint8_t *fine = reinterpret_cast<uint8_t *>(lens + n);
  for (int b = tid; b < P.B; b += TB_NT) first[b] = ~0u;
  __syncthreads();
  for (int j = tid; j < n; j += TB_NT) {
    const uint32_t d = F.dst[j];
    if (d < B) atomicMin(first + d, static_cast<uint32_t>(j));
  }
  __syncthreads();
  for (int j = tid; j < n; j += TB_NT) {
    const uint32_t s = F.src[j], d = F.dst[j];
    int st = 0, need = 0, full = 0, len = 0;
    if (s >= B || d >= B || s == d || first[d] != static_cast<uint32_t>(j)) {
      st = SPEC_ROW_BAD_FORK;
    } else {
      len = F.len[s];
      const int held = P.held[s], taken = P.held[d];
      const int64_t t = len == -1 ? 0 : static_cast<int64_t>(len) - P.prefix;
      if (taken != 0) {
        st = SPEC_ROW_BAD_FORK;
      } else if (len < -1 || t < 0 || held < 0 || held > P.max_pages || (t + (1 << lg) - 1) >> lg > held) {
        st = SPEC_ROW_BAD_LENGTH;
      } else {
        full = static_cast<int>(t >> lg);
        need = (t & ((1 << lg) - 1)) != 0;
      }
    }
    cum[j] = need;
    shared[j] = full;
    lens[j] = len;
    fine[j] = !st;
    if (team.rank == 0) {
      if (F.status) F.status[j] = st;
      F.copies[3 * j] = F.copies[3 * j + 1] = -1, F.copies[3 * j + 2] = 0;
    }
  }
  // status words and copies are written, lengths and what is held have been read by all
  auto read = cg::this_cluster().barrier_arrive();
  __syncthreads();
  sum_up(cum, shared, n, S.warp2);
  cg::this_cluster().barrier_wait(std::move(read));
  if (cum[n] + shared[n] <= TB_ALONE) {
    if (team.rank) return;
    team.ctas = 1;
  }
  const uint32_t found = take_pages(P, cum, n, team, S, [&](int j, uint32_t, int32_t id) {
    const int full = static_cast<int>(shared[j + 1] - shared[j]);
    const int old = P.table[F.src[j] * P.tstride + full];
    P.table[F.dst[j] * P.tstride + full] = id;
    P.refs[id] = 1;
    if (static_cast<uint32_t>(old) < np) {
      F.copies[3 * j] = old;
      F.copies[3 * j + 1] = id;
      F.copies[3 * j + 2] = lens[j] - P.prefix - (full << lg);
    } else if (F.status) {
      atomicOr(F.status + j, SPEC_ROW_BAD_PAGE);
    }
  });
  const uint32_t stride = team.ctas * TB_NT, many = shared[n];
  in_groups<4>(team.rank * TB_NT + tid, stride, many, [&](auto K_, uint32_t x0) {
    constexpr int K = decltype(K_)::value;
    uint32_t x[K];
    int id[K], of[K];
    bool on[K];
#pragma unroll
    for (int u = 0; u < K; ++u) x[u] = min(x0 + u * stride, many - 1);
    before(shared, n, x, of);
#pragma unroll
    for (int u = 0; u < K; ++u) {
      const uint32_t to = cum[of[u] + 1];
      on[u] = x0 + u * stride < many && !(to > cum[of[u]] && to > found);
      x[u] -= shared[of[u]];
      if (on[u]) id[u] = P.table[F.src[of[u]] * P.tstride + static_cast<int>(x[u])];
    }
#pragma unroll
    for (int u = 0; u < K; ++u) {
      if (!on[u]) continue;
      P.table[F.dst[of[u]] * P.tstride + static_cast<int>(x[u])] = id[u];
      if (static_cast<uint32_t>(id[u]) < np) atomicAdd(P.refs + id[u], 1);
      else if (F.status) atomicOr(F.status + of[u], SPEC_ROW_BAD_PAGE);
    }
  });
  for (int k = team.rank * TB_NT + tid; k < n; k += team.ctas * TB_NT) {
    if (!fine[k]) continue;
    const uint32_t take = cum[k + 1] - cum[k];
    if (take && cum[k + 1] > found) {
      if (F.status) atomicOr(F.status + k, SPEC_ROW_NO_PAGES);
      continue;
    }
    P.held[F.dst[k]] = static_cast<int>(shared[k + 1] - shared[k] + take);
    F.len[F.dst[k]] = lens[k];
  }
  // no CTA ends while another one may read its part of the sums
  if (team.ctas > 1 && cum[n]) team.sync();
}

spec_status check_pool(const spec_kv_pool *p, Pool &P) {
  if (!p || p->B < 0 || p->max_pages < 0 || p->n_pages < 0 || p->page_size < 1 || p->prefix_len < 0 ||
      p->table_row_stride < p->max_pages)
    return SPEC_ERR_INVALID_ARG;
  const int lg = kv::log2_page(p->page_size);
  if (lg < 0 || p->B > kv::kMaxB || static_cast<int64_t>(p->max_pages) * p->page_size > (1 << 30) ||
      static_cast<int64_t>(p->max_pages) * p->B > INT32_MAX || p->prefix_len > (1 << 30))
    return SPEC_ERR_UNSUPPORTED;
  const uintptr_t all = reinterpret_cast<uintptr_t>(p->refs) | reinterpret_cast<uintptr_t>(p->table) |
                        reinterpret_cast<uintptr_t>(p->held);
  if (all % 4) return SPEC_ERR_INVALID_ARG;
  if (p->B > 0 && ((p->n_pages > 0 && !p->refs) || (p->max_pages > 0 && !p->table) || !p->held))
    return SPEC_ERR_INVALID_ARG;
  P = {p->refs, p->table, p->held, p->table_row_stride, p->B, p->max_pages, p->n_pages, p->prefix_len, lg,
       reinterpret_cast<uintptr_t>(p->refs) % 16 == 0};
  return SPEC_OK;
}

}  // namespace

extern "C" spec_status spec_kv_compact(const spec_kv_cache *cache, const spec_kv_batch *batch,
                                       const int32_t *path, const int32_t *accepted_len,
                                       int32_t *row_status, void *stream) {
  MP P = {};
  const spec_status st = kv::make_view(cache, batch, true, P.w);
  if (st != SPEC_OK) return st;
  if (P.w.N > SPEC_TREE_MAX) return SPEC_ERR_UNSUPPORTED;
  if (P.w.B == 0) return SPEC_OK;
  if (!path || !accepted_len || reinterpret_cast<uintptr_t>(path) % 4 ||
      reinterpret_cast<uintptr_t>(accepted_len) % 4 || reinterpret_cast<uintptr_t>(row_status) % 4)
    return SPEC_ERR_INVALID_ARG;
  P.k = static_cast<uint8_t *>(cache->k_pages);
  P.v = static_cast<uint8_t *>(cache->v_pages);
  P.ke = cache->k_exp;
  P.ve = cache->v_exp;
  P.path = path;
  P.acc = accepted_len;
  P.status = row_status;
  const dim3 grid(P.w.Hkv, P.w.B);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->format == SPEC_KV_E4M3) compact_kernel<true><<<grid, MV_NT, 0, s>>>(P, cache->head_dim);
  else compact_kernel<false><<<grid, MV_NT, 0, s>>>(P, cache->head_dim);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

extern "C" spec_status spec_kv_copy(const spec_kv_cache *cache, const int32_t *copies, int32_t n,
                                    void *stream) {
  spec_kv_batch none = {};  // the cache's own checks
  View w;
  spec_status st = kv::make_view(cache, &none, false, w);
  if (st != SPEC_OK) return st;
  if (n < 0) return SPEC_ERR_INVALID_ARG;
  if (n > 1 << 20) return SPEC_ERR_UNSUPPORTED;
  if (n == 0 || cache->n_pages == 0) return SPEC_OK;
  const bool e4m3 = cache->format == SPEC_KV_E4M3;
  if (!copies || reinterpret_cast<uintptr_t>(copies) % 4 || !cache->k_pages || !cache->v_pages ||
      (e4m3 && (!cache->k_exp || !cache->v_exp)))
    return SPEC_ERR_INVALID_ARG;
  uintptr_t all = reinterpret_cast<uintptr_t>(cache->k_pages) | reinterpret_cast<uintptr_t>(cache->v_pages);
  if (e4m3) all |= reinterpret_cast<uintptr_t>(cache->k_exp) | reinterpret_cast<uintptr_t>(cache->v_exp);
  if (all % 16) return SPEC_ERR_INVALID_ARG;
  YP P = {static_cast<uint8_t *>(cache->k_pages), static_cast<uint8_t *>(cache->v_pages),
          e4m3 ? cache->k_exp : nullptr, e4m3 ? cache->v_exp : nullptr, copies, w.kps, w.vps,
          cache->n_pages, cache->n_kv_heads, cache->page_size, cache->head_dim * (e4m3 ? 1 : 2)};
  copy_kernel<<<static_cast<unsigned>(n) * cache->n_kv_heads, CY_NT, 0, static_cast<cudaStream_t>(stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

extern "C" spec_status spec_kv_resize(const spec_kv_pool *pool, const int32_t *kv_len, int32_t n_step,
                                      int32_t *row_status, void *stream) {
  RP R = {};
  const spec_status st = check_pool(pool, R.p);
  if (st != SPEC_OK) return st;
  if (n_step < 0) return SPEC_ERR_INVALID_ARG;
  if (n_step > 1 << 30) return SPEC_ERR_UNSUPPORTED;
  if (pool->B == 0) return SPEC_OK;
  if (!kv_len || (reinterpret_cast<uintptr_t>(kv_len) | reinterpret_cast<uintptr_t>(row_status)) % 4)
    return SPEC_ERR_INVALID_ARG;
  R.len = kv_len;
  R.n = n_step;
  R.status = row_status;
  const int smem = sizeof(TableShared) + (3 * pool->B + 2) * 4;
  static std::atomic<bool> ready[kv::kDevices] = {};
  if (!kv::allow_shared(reinterpret_cast<const void *>(resize_kernel), sizeof(TableShared) + (3 * kv::kMaxB + 2) * 4, ready)) return SPEC_ERR_CUDA;
  resize_kernel<<<TB_CTAS, TB_NT, smem, static_cast<cudaStream_t>(stream)>>>(R);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

extern "C" spec_status spec_kv_fork(const spec_kv_pool *pool, int32_t *kv_len, const int32_t *src,
                                    const int32_t *dst, int32_t n, int32_t *copies, int32_t *fork_status,
                                    void *stream) {
  FP F = {};
  const spec_status st = check_pool(pool, F.p);
  if (st != SPEC_OK) return st;
  if (n < 0) return SPEC_ERR_INVALID_ARG;
  if (n > kv::kMaxB) return SPEC_ERR_UNSUPPORTED;
  if (n == 0) return SPEC_OK;
  const uintptr_t all = reinterpret_cast<uintptr_t>(kv_len) | reinterpret_cast<uintptr_t>(src) |
                        reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(copies) |
                        reinterpret_cast<uintptr_t>(fork_status);
  if (!src || !dst || !copies || all % 4 || (pool->B > 0 && !kv_len)) return SPEC_ERR_INVALID_ARG;
  F.len = kv_len;
  F.src = src;
  F.dst = dst;
  F.n = n;
  F.copies = copies;
  F.status = fork_status;
  const int smem = sizeof(TableShared) + (2 * (n + 1) + pool->B + n) * 4 + n;
  static std::atomic<bool> ready[kv::kDevices] = {};
  if (!kv::allow_shared(reinterpret_cast<const void *>(fork_kernel), sizeof(TableShared) + (4 * kv::kMaxB + 2) * 4 + kv::kMaxB, ready)) return SPEC_ERR_CUDA;
  fork_kernel<<<TB_CTAS, TB_NT, smem, static_cast<cudaStream_t>(stream)>>>(F);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
