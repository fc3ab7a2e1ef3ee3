// spec_tree.cu -- trees of drafted tokens: what each node sees, and the walk
// along the tokens that the target drew.
//
// Mask: row i of a tree's mask is the bit of i or-ed to the row of its parent.
// One CTA per sequence, a thread per node, by doubling: after k rounds a row
// holds the node's 2^k nearest ancestors, so a tree of depth d takes
// ceil(log2(d + 1)) rounds, whose number a chain of 512 makes 9.  The mask stays
// in shared memory and leaves it in whole words.
//
// Accept: a warp per sequence.  Its nodes are in shared memory, 32 are compared
// at a time, and the lowest match is the next node: about 60 clocks a step, and
// nothing but the first loads waits for memory.
//
// Bound: both by their launch and a chain of two loads: 2.7 us each for one tree of 26
// nodes (replayed calls), 2.9 and 3.3 us for 256 trees of 64.
#include <cuda_runtime.h>

#include <cstdint>

#include "spec_kv.h"
#include "spec_tree.h"

namespace {

constexpr int TW = SPEC_TREE_MAX / 32;  // words of a mask row at most
constexpr int AC_ROWS = 4;              // sequences per CTA of the walk

struct TP {
  const int32_t *parents, *gam;
  int32_t *mask, *depth, *status;
  int32_t gm, W;
};

// gamma_b, or -1 where it is not in [0, gm].
__device__ __forceinline__ int gamma_of(const int32_t *gam, int b, int gm) {
  const int g = gam ? gam[b] : gm;
  return g < 0 || g > gm ? -1 : g;
}

// Grid: sequences.  Shared memory: rows of the mask (an odd number of words
// apart), then jumps.
__global__ void __launch_bounds__(SPEC_TREE_MAX) mask_kernel(const __grid_constant__ TP P) {
  extern __shared__ uint32_t sm[];
  const int N = P.gm + 1, W = P.W, pitch = W | 1;
  const int b = blockIdx.x, i = threadIdx.x;
  uint32_t *row = sm + i * pitch;
  int32_t *jump = reinterpret_cast<int32_t *>(sm + N * pitch);
  const int g = gamma_of(P.gam, b, P.gm);
  int at = 0;
  bool bad = false;
  if (i > 0 && i <= g) {
    at = P.parents[static_cast<int64_t>(b) * P.gm + i - 1];
    bad = at < 0 || at >= i;
  }
  int st = g < 0 ? SPEC_ROW_BAD_GAMMA : 0;
  if (__syncthreads_or(bad)) st |= SPEC_ROW_BAD_TREE;
  const bool live = !st && i <= g;
  if (i < N) {
    for (int w = 0; w < W; ++w) row[w] = 0;
    if (live) row[i >> 5] = 1u << (i & 31);
    jump[i] = live ? at : 0;
  }
  // the root is node 0 of every mask: rounds end when all jumps have come to it
  while (__syncthreads_or(live && at != 0)) {
    uint32_t more[TW];
    int next = 0;
    if (live) {
      next = jump[at];
#pragma unroll
      for (int w = 0; w < TW; ++w)
        if (w < W) more[w] = sm[at * pitch + w];
    }
    __syncthreads();
    if (live) {
#pragma unroll
      for (int w = 0; w < TW; ++w)
        if (w < W) row[w] |= more[w];
      jump[i] = at = next;
    }
  }
  if (live) {
    row[0] |= 1u;
    if (P.depth) {
      int d = -1;
      for (int w = 0; w < W; ++w) d += __popc(row[w]);
      P.depth[static_cast<int64_t>(b) * N + i] = d;
    }
  } else if (i < N && P.depth) {
    P.depth[static_cast<int64_t>(b) * N + i] = 0;
  }
  __syncthreads();
  int32_t *out = P.mask + static_cast<int64_t>(b) * N * W;
  for (int x = i; x < N * W; x += blockDim.x) out[x] = static_cast<int32_t>(sm[x / W * pitch + x % W]);
  if (P.status && i == 0) P.status[b] = st;
}

struct CP {
  const int32_t *target, *draft, *parents, *gam;
  int32_t *acc, *next, *path, *tokens, *status;
  int32_t B, gm;
};

// Shared memory per warp: parents and drafts of nodes 0 .. gm, target tokens.
__global__ void __launch_bounds__(32 * AC_ROWS) accept_kernel(const __grid_constant__ CP P) {
  extern __shared__ int32_t am[];
  const int N = P.gm + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x * AC_ROWS + warp;
  if (b >= P.B) return;
  int32_t *up = am + warp * 3 * N, *tok = up + N, *tgt = tok + N;
  const int64_t r = static_cast<int64_t>(b);
  const int g = gamma_of(P.gam, b, P.gm);
  bool bad = false;
  for (int j = lane; j <= g; j += 32) {
    const int p = j ? P.parents[r * P.gm + j - 1] : -1;
    bad |= j && (p < 0 || p >= j);
    up[j] = p;
    tok[j] = j ? P.draft[r * P.gm + j - 1] : -1;
    tgt[j] = P.target[r * N + j];
  }
  int st = g < 0 ? SPEC_ROW_BAD_GAMMA : 0;
  if (__any_sync(~0u, bad)) st |= SPEC_ROW_BAD_TREE;
  __syncwarp();
  int at = 0, n = 0, t = -1;
  int32_t *path = P.path ? P.path + r * N : nullptr;
  int32_t *tokens = P.tokens ? P.tokens + r * P.gm : nullptr;
  while (!st) {
    t = tgt[at];
    if (t < 0) {
      st = SPEC_ROW_BAD_TOKEN;
      break;
    }
    if (path && lane == 0) path[n] = at;
    int child = 0;  // a child's number is above its parent's
    for (int j0 = (at + 1) & ~31; j0 <= g; j0 += 32) {
      const int j = j0 + lane;
      const unsigned hit = __ballot_sync(~0u, j > 0 && j <= g && up[j] == at && tok[j] == t);
      if (hit) {
        child = j0 + __ffs(hit) - 1;
        break;
      }
    }
    if (!child) break;
    if (tokens && lane == 0) tokens[n] = t;
    ++n;
    at = child;
  }
  if (st) n = -1, t = -1;  // no nodes visited
  __syncwarp();            // the walk's stores come before these
  if (path)
    for (int j = n + 1 + lane; j < N; j += 32) path[j] = -1;
  if (tokens)
    for (int j = max(n, 0) + lane; j < P.gm; j += 32) tokens[j] = -1;
  if (lane == 0) {
    P.acc[b] = max(n, 0);
    P.next[b] = t;
    if (P.status) P.status[b] = st;
  }
}

bool aligned(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

spec_status check(int32_t B, int32_t gamma_max) {
  if (B < 0 || gamma_max < 0) return SPEC_ERR_INVALID_ARG;
  return gamma_max >= SPEC_TREE_MAX ? SPEC_ERR_UNSUPPORTED : SPEC_OK;
}

}  // namespace

extern "C" spec_status spec_tree_mask(int32_t B, int32_t gamma_max, const int32_t *parents,
                                      const int32_t *gamma_per_row, int32_t *mask, int32_t *depth,
                                      int32_t *row_status, void *stream) {
  const spec_status c = check(B, gamma_max);
  if (c != SPEC_OK || B == 0) return c;
  if (!mask || (gamma_max > 0 && !parents) || !aligned(parents) || !aligned(gamma_per_row) ||
      !aligned(mask) || !aligned(depth) || !aligned(row_status))
    return SPEC_ERR_INVALID_ARG;
  TP P = {parents, gamma_per_row, mask, depth, row_status, gamma_max, (gamma_max + 32) / 32};
  const int N = gamma_max + 1, threads = (N + 31) / 32 * 32;
  const int smem = (N * (P.W | 1) + N) * 4;  // 36 KB at most
  mask_kernel<<<B, threads, smem, static_cast<cudaStream_t>(stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

extern "C" spec_status spec_tree_accept(int32_t B, int32_t gamma_max, const int32_t *target_tokens,
                                        const int32_t *draft_tokens, const int32_t *parents,
                                        const int32_t *gamma_per_row, int32_t *accepted_len,
                                        int32_t *next_token, int32_t *path, int32_t *path_tokens,
                                        int32_t *row_status, void *stream) {
  const spec_status c = check(B, gamma_max);
  if (c != SPEC_OK || B == 0) return c;
  if (!target_tokens || !accepted_len || !next_token || (gamma_max > 0 && (!draft_tokens || !parents)))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(target_tokens) || !aligned(draft_tokens) || !aligned(parents) || !aligned(gamma_per_row) ||
      !aligned(accepted_len) || !aligned(next_token) || !aligned(path) || !aligned(path_tokens) ||
      !aligned(row_status))
    return SPEC_ERR_INVALID_ARG;
  CP P = {target_tokens, draft_tokens, parents, gamma_per_row, accepted_len, next_token,
          path, path_tokens, row_status, B, gamma_max};
  const int smem = AC_ROWS * 3 * (gamma_max + 1) * 4;  // 24 KB at most
  accept_kernel<<<(B + AC_ROWS - 1) / AC_ROWS, 32 * AC_ROWS, smem, static_cast<cudaStream_t>(stream)>>>(P);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
