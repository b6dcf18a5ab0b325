// Append of new keys and values to a paged cache (lin_step.h).
//
// cache[page_table[r][t / P]][t % P][h] <- new[r][j][h] for t = pos[r] + rank(j),
// where rank(j) is j for a step, a prompt or an accepted prefix, and j's depth
// on the accepted path for a draft tree.
//
// A pure copy, bound by HBM (read + write of the rows written) for a prompt and
// by one launch's chain of dependent loads (count, position, page id, rows) for
// a step. One warp moves one token: it owns whole rows, so tokens may land in
// any order of pages, and it looks the page up once for all heads of K and V.
// The rows' loads are issued before the page lookup, whose latency they hide.
// 8 prompts of 2k-4k tokens, 8 heads of 128 in bf16: 33.5 us, 0.89 of the measured
// copy bandwidth; one token of each of 256 requests: 3.0 us, the launch.

#include "common.cuh"
#include "step_internal.h"

namespace lin {
namespace {

constexpr int kAppendWarps = 4;
// 16-byte loads in flight per lane: 8 x 32 lanes x 16 B = 4 KB, K and V of
// one token of 8 heads x 128 in bf16
constexpr int kAppendUnroll = 8;

__global__ void __launch_bounds__(kAppendWarps * 32)
kv_append_kernel(const lin_kv_cache_t c, const lin_kv_append_args_t a, int row_shift, int chunks) {
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  if (item >= int64_t(a.batch) * a.n) return;
  const int r = static_cast<int>(item / a.n), j = static_cast<int>(item % a.n);
  int rank = j;
  if (a.n_tok) {
    const int count = a.n_tok[r];
    if (count < 0 || count > a.n) {
      if (lane == 0 && a.pos[r] >= 0) report(a.status, LIN_ST_BAD_ACCEPT);
      return;
    }
    if (j >= count) return;
  }
  if (a.parent) {
    // lane d holds draft d's parent; the path is walked up from accept_node
    const int par = lane < a.n ? a.parent[int64_t(r) * a.n + lane] : -1;
    const int node = a.accept_node[r];
    const bool bad = __any_sync(~0u, lane < a.n && (par < -1 || par >= lane)) || node < -1 || node >= a.n;
    if (bad) {
      if (lane == 0 && a.pos[r] >= 0) report(a.status, LIN_ST_BAD_TREE);
      return;
    }
    uint32_t path = 0;
    for (int at = node; at >= 0; at = __shfl_sync(~0u, par, at)) path |= 1u << at;
    if (!((path >> j) & 1u)) return;
    rank = __popc(path & ((1u << j) - 1u));
  }
  const char* ks = static_cast<const char*>(a.k) + r * a.req_stride + j * a.token_stride;
  const char* vs = static_cast<const char*>(a.v) + r * a.req_stride + j * a.token_stride;
  char* kd = nullptr;
  char* vd = nullptr;
  // K's chunks, then V's
  for (int c0 = 0; c0 < 2 * chunks; c0 += 32 * kAppendUnroll) {
    uint4 v[kAppendUnroll];
#pragma unroll
    for (int i = 0; i < kAppendUnroll; ++i) {
      const int x = c0 + i * 32 + lane;
      if (x < 2 * chunks)
        v[i] = __ldcs(reinterpret_cast<const uint4*>(x < chunks ? ks : vs) + (x < chunks ? x : x - chunks));
    }
    if (!kd) {
      const int pos = a.pos[r];
      if (pos < 0) return;
      const int64_t t = int64_t(pos) + rank;
      const int64_t pg = t / c.page_size;
      if (pg >= a.max_pages) {
        if (lane == 0) report(a.status, LIN_ST_BAD_SEQLEN);
        return;
      }
      const int id = a.page_table[r * a.page_table_stride + pg];
      if (id < 0 || id >= c.num_pages) {
        if (lane == 0) report(a.status, LIN_ST_BAD_PAGE);
        return;
      }
      const int64_t at = a.layer * c.layer_stride + id * c.page_stride + (t - pg * c.page_size) * c.token_stride;
      kd = static_cast<char*>(c.k) + at;
      vd = static_cast<char*>(c.v) + at;
    }
#pragma unroll
    for (int i = 0; i < kAppendUnroll; ++i) {
      const int x = c0 + i * 32 + lane;
      if (x < 2 * chunks) {
        const int y = x < chunks ? x : x - chunks;
        const int64_t off = (y >> row_shift) * c.head_stride + (int64_t(y & ((1 << row_shift) - 1)) << 4);
        *reinterpret_cast<uint4*>((x < chunks ? kd : vd) + off) = v[i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const lin_kv_cache_t& c, const lin_kv_append_args_t& a, cudaStream_t s) {
  const int row = c.head_dim * dtype_size(c.dtype) / 16;  // 8 .. 64, a power of two
  int shift = 0;
  while ((1 << shift) < row) ++shift;
  const int64_t items = int64_t(a.batch) * a.n;
  const int64_t blocks = (items + kAppendWarps - 1) / kAppendWarps;
  if (blocks > INT32_MAX || int64_t(c.num_kv_heads) * row > INT32_MAX / 4) return cudaErrorInvalidValue;
  kv_append_kernel<<<static_cast<unsigned>(blocks), kAppendWarps * 32, 0, s>>>(c, a, shift, c.num_kv_heads * row);
  return cudaGetLastError();
}

}  // namespace lin
