// What the kernels of chunk attention share: the plan of a call, and the split of a
// batch's work over the CTAs.
//
// An item is up to `rows` rows of one request: m consecutive new tokens times the query
// heads of one kv head (or a block of them, where they are more than the rows). Its last
// token sees keys(j) tokens of the cache, and it counts as keys(j) + item_cost, the cost
// of its start and end. The items of the whole batch, laid end to end, are cut into one
// equal range per CTA (lengths are read on the device), so causal prompts, ragged
// batches and a few rows over a long cache load the SMs alike. A border inside an item
// moves up to the end of a tile of tk keys, one within its cost to its start. An item
// inside one range is finished there; one that crosses a border leaves (value sums, m,
// sum) of each piece in the workspace, and a second kernel joins them in range order, so
// results do not depend on timing. A request's items have a closed sum (keys grow by m
// from one to the next), so no kernel has to lay the items out.
//
// Batches of many items per CTA (the tensor-memory kernel) are not cut, where the lengths,
// which a call's room says nothing of, allow that: a CTA takes the next item from a counter
// whenever it begins one. So the items under way at a time are neighbours, which share their
// keys and values in L2. A request's items come longest first. An item whose turn comes
// after u units begins when u / CTAs of them are done at the latest, so the last end can be
// told before: the counter is used where it lies within 1 / kManyItems of an equal share.
// Whole items, so again the result does not depend on who took them.
#pragma once

#include <cuda.h>
#include <math.h>

#include "attn_common.cuh"
#include "prompt_internal.h"

namespace lin {
namespace chunk {

constexpr int64_t kLongest = attn::kLongest;

// By the counter and by ranges, us (and the last end by the counter in equal shares): 64 x
// 1-512 tokens after 200-8,000, 16 / 2 heads of 256 (1.1) 1,350 and 1,515, 32 / 8 of 128 904
// and 967, 8,192 after 120,000 (1.1) 11,454 and 13,421; 8 prompts of 4,096, 16 / 2 of 128,
// 446 and 445, with one token after 24,000 before them (1.1) 451 and 458, after 12,000 behind
// them (1.4) 536 and 454, after 128,000 1,805 and 473; 256 single tokens after 1,000, the
// last after 4,000 (1.2) 225 and 202, after 16,000 (1.9) 346 and 213; 64 tokens after 129,000
// in a call with room for 32,768 1,569 and 83.
constexpr int kManyItems = 4;

struct Split {       // the item that begins in range c and goes on past it
  int parts;         // 0: there is none
  int row0, tokens;  // its packed rows
  int head0, heads;  // its query heads
};

struct Plan {
  lin_kv_cache_t c;
  lin_attn_chunk_args_t a;
  int group;        // query heads per kv head
  int bheads;       // of an item
  int blocks;       // items that share a kv head's group
  int m;            // tokens of an item
  int rows;         // most rows of an item: m * bheads and less
  int heads;        // kv heads * blocks
  int tk;           // keys of a tile
  int grid, item_cost;
  int box;          // tokens of a TMA box of the cache; 0: none
  int q_box;        // and of one of the queries, a row tile's
  float scale_log2;  // |scale| log2(e), never 0; q is negated where scale < 0
  uint32_t negate;
  uint32_t page_mul, page_shift;    // t / page_size = (mulhi(t, mul) + t) >> shift
  uint32_t bhead_mul, bhead_shift;  // row / bheads
  float* part;       // [2 grid][D / 4][rows][4] value sums of unfinished pieces: a warp's rows side by side
  float2* part_ml;   // [2 grid][rows] their (maximum, sum)
  Split* split;      // [grid]
  int* ticket;       // [0] items handed out so far, [1] whether they are: share_kernel's; NULL: they are not
  int64_t items;     // of the batch at most
};

__device__ __forceinline__ int page_of(const Plan& p, int t) { return (__umulhi(t, p.page_mul) + t) >> p.page_shift; }
__device__ __forceinline__ int token_of(const Plan& p, int row) { return (__umulhi(row, p.bhead_mul) + row) >> p.bhead_shift; }

// A piece of an item as the roles of a CTA see it.
struct Piece {
  int r;             // request; -1: no more pieces
  int hk;            // kv head
  int head0, heads;  // query heads
  int row0, tokens;  // packed rows
  int pos;           // position of the first one (negative where kv_len < n)
  int keys;          // tokens that the last one sees
  int t0, t1;        // tiles here
  int whole;         // all of the item's: outputs; else the part's index is in `part`
  int part;
};

// Request r as a row of items.
struct Req {
  int cu, n, base;   // first packed row, rows, position of the first
  int items, few;    // per head; the first `few` see one key at most and count as one
};

// Whether the batch's items are taken one by one.
__device__ __forceinline__ bool one_by_one(const Plan& p) { return p.ticket && p.ticket[1]; }

__device__ __forceinline__ int64_t longest(const Plan& p) { return min(int64_t(p.a.max_pages) * p.c.page_size, kLongest); }

__device__ __forceinline__ Req request(const Plan& p, int r, bool tell) {
  Req q;
  const int len = p.a.kv_len[r], begin = p.a.cu_seqlens[r], end = p.a.cu_seqlens[r + 1];
  q.items = q.n = 0;
  if (len < 0) return q;
  if (len > longest(p) || begin < 0 || end < begin || end > p.a.tokens) {
    if (tell) report(p.a.status, LIN_ST_BAD_SEQLEN);
    return q;
  }
  q.cu = begin, q.n = end - begin, q.base = len - q.n;
  q.items = (q.n + p.m - 1) / p.m;
  q.few = 0;
  if (q.base <= 1) q.few = min(q.items - 1, static_cast<int>((1 - int64_t(q.base)) / p.m));
  if (len <= 1) q.few = q.items;
  return q;
}

// Keys that item j counts: what its last token sees, one at least.
__device__ __forceinline__ int64_t keys_of(const Plan& p, const Req& q, int j) {
  const int64_t k = int64_t(q.base) + min(int64_t(j + 1) * p.m, int64_t(q.n));
  return k > 1 ? k : 1;
}

// Units of a head's items before item j.
__device__ __forceinline__ int64_t units_before(const Plan& p, const Req& q, int j) {
  const int64_t few = q.few, x = j;
  int64_t u = int64_t(p.item_cost) * x + (x < few ? x : few);
  if (x > few) {
    u += (x - few) * q.base + int64_t(p.m) * ((x * (x + 1) - few * (few + 1)) / 2);
    if (j == q.items) u -= int64_t(q.items) * p.m - q.n;
  }
  return u;
}

__device__ __forceinline__ int range_of(int64_t unit, int64_t ranges, int64_t total) {
  return static_cast<int>(((unit + 1) * ranges - 1) / total);
}

// Where a CTA is in its range: one thread's, which hands the pieces out.
struct Walk {
  int64_t pos, end, total, ranges;  // where the item begins and the range ends among all units
  Req q;
  int r, h, j, t0;
};

struct WalkShared {
  int64_t scan[16], at;
  int r;
};

// The CTA's range, from a scan over the requests by all NT threads. False where
// there is no work for it.
template <int NT>
__device__ __forceinline__ bool walk_begin(const Plan& p, Walk& w, WalkShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int batch = p.a.batch, span = (batch + NT - 1) / NT;
  const int r0 = min(batch, tid * span), r1 = min(batch, r0 + span);
  int64_t mine = 0;
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    const Req q = request(p, r, blockIdx.x == 0);
    if (q.items) mine += units_before(p, q, q.items) * p.heads;
  }
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) sh.scan[warp] = upto;
  __syncthreads();
  w.total = 0;
#pragma unroll
  for (int x = 0; x < NT / 32; ++x) {
    if (x < warp) upto += sh.scan[x];
    w.total += sh.scan[x];
  }
  // a range holds a tile at least, so every range of an item has one of its tiles
  // (but the last, where the border before it moved past them all)
  const int64_t most = w.total / p.tk;
  w.ranges = most < 1 ? 1 : most < gridDim.x ? most : gridDim.x;
  if (blockIdx.x >= w.ranges || w.total == 0) {
    if (tid == 0) p.split[blockIdx.x].parts = 0;
    return false;
  }
  const int64_t cur = w.total * blockIdx.x / w.ranges;
  w.end = w.total * (blockIdx.x + 1) / w.ranges;
  if (cur >= upto - mine && cur < upto) {
    int64_t at = upto - mine;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
      const Req q = request(p, r, false);
      const int64_t n = q.items ? units_before(p, q, q.items) * p.heads : 0;
      if (cur < at + n) {
        sh.r = r, sh.at = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  w.r = sh.r;
  w.q = request(p, w.r, false);
  const int64_t per_head = units_before(p, w.q, w.q.items);
  int64_t off = cur - sh.at;
  w.h = static_cast<int>(off / per_head);
  off -= w.h * per_head;
  int lo = 0, hi = w.q.items - 1;  // the last item that begins at or before the border
#pragma unroll 1
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (units_before(p, w.q, mid) <= off)
      lo = mid;
    else
      hi = mid - 1;
  }
  w.j = lo;
  off -= units_before(p, w.q, lo);
  w.pos = cur - off;
  off -= p.item_cost;
  w.t0 = off > 0 ? static_cast<int>((off + p.tk - 1) / p.tk) : 0;
  return true;
}

// The next piece, r = -1 at the range's end. Leaves the range's split there.
__device__ __forceinline__ Piece walk_next(const Plan& p, Walk& w) {
  Piece x;
#pragma unroll 1
  while (w.pos < w.end) {
    const int64_t keys = keys_of(p, w.q, w.j);
    const int tiles = static_cast<int>((keys + p.tk - 1) / p.tk);
    const int64_t upto = w.end - w.pos - p.item_cost;
    const int t1 = upto >= keys ? tiles : upto > 0 ? static_cast<int>((upto + p.tk - 1) / p.tk) : 0;
    const int t0 = w.t0;
    const bool found = t1 > t0;
    if (found) {
      const int kv = w.h / p.blocks, hb = w.h - kv * p.blocks;
      x.r = w.r, x.hk = kv;
      x.head0 = kv * p.group + hb * p.bheads, x.heads = min(p.bheads, p.group - hb * p.bheads);
      x.row0 = w.q.cu + w.j * p.m, x.tokens = min(p.m, w.q.n - w.j * p.m);
      x.pos = w.q.base + w.j * p.m;
      x.keys = max(0, x.pos + x.tokens);
      x.t0 = t0, x.t1 = t1;
      x.whole = t0 == 0 && t1 == tiles;
      x.part = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
    }
    if (t1 < tiles) {  // the range ends inside the item
      Split s;
      s.parts = 0;
      if (t0 == 0 && t1 > 0) {
        s.parts = range_of(w.pos + p.item_cost + int64_t(tiles - 1) * p.tk, w.ranges, w.total) - blockIdx.x + 1;
        s.row0 = x.row0, s.tokens = x.tokens, s.head0 = x.head0, s.heads = x.heads;
      }
      p.split[blockIdx.x] = s;
      w.end = -1;
    } else {
      w.pos += keys + p.item_cost;
      w.t0 = 0;
      if (w.pos >= w.end) {
        p.split[blockIdx.x].parts = 0;
      } else if (++w.j == w.q.items) {
        w.j = 0;
        if (++w.h == p.heads) {
          w.h = 0;
#pragma unroll 1
          do {
            w.q = request(p, ++w.r, false);
          } while (w.q.items == 0);
        }
      }
    }
    if (found) return x;
  }
  x.r = -1;
  return x;
}

// Tensor maps of the layer's keys and values and of the queries.
struct Maps {
  CUtensorMap k, v, q;
};

// Hands out whole items by the counter, by a whole warp.
struct Tickets {
  int r0;           // lane l looks at request r0 + l
  int64_t base;     // items before these
  int64_t upto;     // and up to the lane's request, of these
  Req q;
  __device__ __forceinline__ void look(const Plan& p, int r) {
    const int lane = threadIdx.x & 31;
    r0 = r;
    q.items = q.n = 0;
    if (r0 + lane < p.a.batch) q = request(p, r0 + lane, false);
    upto = int64_t(q.items) * p.heads;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += x;
    }
  }
  __device__ __forceinline__ void begin(const Plan& p) {
    base = 0;
    look(p, 0);
  }
  __device__ __forceinline__ Piece next(const Plan& p) {
    const int lane = threadIdx.x & 31;
    Piece x;
    x.r = -1;
    int64_t at = lane == 0 ? atomicAdd(p.ticket, 1) : 0;
    at = __shfl_sync(~0u, at, 0);
    // (cu_seqlens that overlap could have more, and wrap the counter)
    if (at >= p.items) return x;
    uint32_t past;
#pragma unroll 1
    while ((past = __ballot_sync(~0u, at < base + upto)) == 0) {
      base += __shfl_sync(~0u, upto, 31);
      if (r0 + 32 >= p.a.batch) return x;
      look(p, r0 + 32);
    }
    const int l = __ffs(past) - 1;
    const int items = __shfl_sync(~0u, q.items, l), n = __shfl_sync(~0u, q.n, l);
    const int64_t off = at - base - (__shfl_sync(~0u, upto, l) - int64_t(items) * p.heads);
    const int h = static_cast<int>(off / items), j = items - 1 - static_cast<int>(off - int64_t(h) * items);
    const int kv = h / p.blocks, hb = h - kv * p.blocks;
    x.r = r0 + l, x.hk = kv;
    x.head0 = kv * p.group + hb * p.bheads, x.heads = min(p.bheads, p.group - hb * p.bheads);
    x.row0 = __shfl_sync(~0u, q.cu, l) + j * p.m, x.tokens = min(p.m, n - j * p.m);
    x.pos = __shfl_sync(~0u, q.base, l) + j * p.m;
    x.keys = max(0, x.pos + x.tokens);
    x.t0 = 0, x.t1 = (max(x.keys, 1) + p.tk - 1) / p.tk;
    x.whole = 1, x.part = 2 * blockIdx.x + 1;
    return x;
  }
};

// One translation unit per head_dim and kind of kernel.
cudaError_t launch_mma_d64(const Plan& p, cudaStream_t s);
cudaError_t launch_umma_d64(const Plan& p, const Maps& m, cudaStream_t s);
cudaError_t launch_mma_d128(const Plan& p, cudaStream_t s);
cudaError_t launch_umma_d128(const Plan& p, const Maps& m, cudaStream_t s);
cudaError_t launch_mma_d256(const Plan& p, cudaStream_t s);
cudaError_t launch_umma_d256(const Plan& p, const Maps& m, cudaStream_t s);

}  // namespace chunk
}  // namespace lin
