// What the kernels of decode attention share: the plan of a call, the split of
// a batch's work over the CTAs, and the end of a piece of work.
//
// A unit is kUnit tokens of one item = (request, kv head, block of rows), and an
// item counts as item_cost units more, for what its start and end take. The
// units of the whole batch, laid end to end, are cut into one equal range per
// CTA (lengths are read on the device), so a batch of ragged lengths and a
// single long request load the SMs alike. A border among an item's first
// item_cost units moves to the item's start. An item inside one range is finished
// there; one that crosses a border leaves (value sums, m, sum) of each piece in
// the workspace, and a second kernel joins them in range order, so results do
// not depend on timing.
#pragma once

#include <math.h>

#include "common.cuh"
#include "step_internal.h"
#include "umma.cuh"

namespace lin {
namespace attn {

constexpr float kSlack = 8.0f;
constexpr int kUnit = 64;  // tokens of a work unit
// A part's sum where its item is not to be written: a bad tree, or a wait that ran out
constexpr float kLeftOut = -1.0f;

struct Plan {
  lin_kv_cache_t c;
  lin_attn_args_t a;
  int group;          // query heads per key-value head
  int rows;           // n_q * group
  int grid;           // CTAs of the main kernel
  int block_rows;     // rows of an item
  int row_blocks;     // items of one (request, kv head)
  int item_cost;      // of an item besides its tokens, in units
  int whole;          // items are short and stay whole: every border moves to an item's start
  float scale_log2;   // |scale| log2(e); q is negated where scale < 0
  uint32_t negate;
  float slack;        // kSlack in units of q.k
  uint32_t page_mul, page_shift;    // t / page_size = (mulhi(t, mul) + t) >> shift, t < 2^31
  uint32_t group_mul, group_shift;  // the same for row / group
  uint32_t block_mul, block_shift;  // and for item / row_blocks
  float* part;        // [2 grid][block_rows][D] value sums of unfinished pieces
  float2* part_ml;    // [2 grid][block_rows] their (maximum, sum or kLeftOut)
  longlong2* split;   // [grid] the item that begins in range c and goes on past
                      // it (or -1), and its number of parts
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// the next bf16 part of a pair of weights; the pair keeps what is left
__device__ __forceinline__ uint32_t take_bf16(float& a, float& b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  a -= __low2float(h);
  b -= __high2float(h);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// t / page_size, the query token of a row, the kv head of an item
__device__ __forceinline__ int page_of(const Plan& p, int t) { return (__umulhi(t, p.page_mul) + t) >> p.page_shift; }
__device__ __forceinline__ int query_of(const Plan& p, int q) { return (__umulhi(q, p.group_mul) + q) >> p.group_shift; }
__device__ __forceinline__ int head_of(const Plan& p, int it) { return (__umulhi(it, p.block_mul) + it) >> p.block_shift; }

// Units of a request: at least one where it has an output to write.
__device__ __forceinline__ int units_of(int len, int64_t most) {
  return len < 0 || len > most ? 0 : len == 0 ? 1 : (len - 1) / kUnit + 1;
}

// The longest request allowed: token indices, and those that loads run ahead by,
// stay clear of the 32-bit end.
constexpr int64_t kLongest = (int64_t(1) << 31) - 65536;
__device__ __forceinline__ int64_t longest(const Plan& p) {
  return min(int64_t(p.a.max_pages) * p.c.page_size, kLongest);
}

// Where a CTA is in its range.
struct Walk {
  int64_t base, end, total, ranges;  // where the item and the range lie among all units
  int64_t most;   // longest request allowed
  int per_req;    // items of a request
  int r, len, u;  // the request, its length and units
  int next_len;   // the next request's length, loaded a piece early
  int it, t0;     // its item, and the item's first unit here
  longlong2 split;
};

// The piece's end: the first of the item's units past it.
__device__ __forceinline__ int walk_until(const Plan& p, const Walk& w) {
  const int64_t upto = w.end - w.base - p.item_cost;
  return static_cast<int>(upto >= w.u ? w.u : upto > 0 && !p.whole ? upto : 0);
}

// The CTA's range, from a scan over the requests' lengths by all NT threads.
// False where there is no work for it.
template <int NT>
__device__ __forceinline__ bool walk_begin(const Plan& p, Walk& w, int64_t (&s_scan)[NT / 32], int64_t (&s_first)[2]) {
  const lin_attn_args_t& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  w.most = longest(p);
  w.per_req = p.c.num_kv_heads * p.row_blocks;
  w.split = make_longlong2(-1, 0);
  const int span = (a.batch + NT - 1) / NT;
  const int r0 = min(a.batch, tid * span), r1 = min(a.batch, r0 + span);
  int64_t mine = 0;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    const int len = a.kv_len[r];
    if (len > w.most && blockIdx.x == 0) report(a.status, LIN_ST_BAD_SEQLEN);
    const int u = units_of(len, w.most);
    if (u > 0) mine += int64_t(u + p.item_cost) * w.per_req;
  }
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) s_scan[warp] = upto;
  __syncthreads();
  w.total = 0;
#pragma unroll
  for (int x = 0; x < NT / 32; ++x) {
    if (x < warp) upto += s_scan[x];
    w.total += s_scan[x];
  }
  w.ranges = w.total < gridDim.x ? w.total : gridDim.x;
  if (blockIdx.x >= w.ranges) {
    if (tid == 0) p.split[blockIdx.x].x = -1;
    return false;
  }
  const int64_t cur = w.total * blockIdx.x / w.ranges;
  w.end = w.total * (blockIdx.x + 1) / w.ranges;
  if (cur >= upto - mine && cur < upto) {
    int64_t at = upto - mine;
    int r = r0;
    for (;; ++r) {
      const int u = units_of(a.kv_len[r], w.most);
      const int64_t n = u > 0 ? int64_t(u + p.item_cost) * w.per_req : 0;
      if (cur < at + n) break;
      at += n;
    }
    s_first[0] = r;
    s_first[1] = at;
  }
  __syncthreads();
  w.r = static_cast<int>(s_first[0]);
  w.len = a.kv_len[w.r];
  w.next_len = w.r + 1 < a.batch ? a.kv_len[w.r + 1] : -1;
  w.u = units_of(w.len, w.most);
  w.it = static_cast<int>((cur - s_first[1]) / (w.u + p.item_cost));
  w.base = s_first[1] + int64_t(w.it) * (w.u + p.item_cost);
  w.t0 = p.whole ? 0 : max(0, static_cast<int>(cur - w.base) - p.item_cost);
  if (walk_until(p, w) > w.t0) return true;
  if (tid == 0) p.split[blockIdx.x].x = -1;
  return false;
}

// On to the next piece; false at the range's end.
__device__ __forceinline__ bool walk_next(const Plan& p, Walk& w, int t1) {
  if (t1 < w.u) {
    if (w.t0 == 0) {
      // the item goes on: its last unit lies in the range whose end is the first past it
      const int64_t last = w.base + w.u + p.item_cost - 1;
      w.split.x = int64_t(w.r) * w.per_req + w.it;
      w.split.y = ((last + 1) * w.ranges - 1) / w.total - blockIdx.x + 1;
    }
    return false;
  }
  w.base += w.u + p.item_cost;
  if (w.base >= w.end) return false;
  w.t0 = 0;
  if (++w.it == w.per_req) {
    w.it = 0;
    do {
      ++w.r;
      w.len = w.next_len;
      w.next_len = w.r + 1 < p.a.batch ? p.a.kv_len[w.r + 1] : -1;
      w.u = units_of(w.len, w.most);
    } while (w.u == 0);
  }
  return walk_until(p, w) > 0;
}

// What each draft sees of the drafts, by one warp: lane j's set goes to see[j].
__device__ __forceinline__ void draft_sets(const Plan& p, int r, uint32_t (&see)[32], int& bad_out) {
  const lin_attn_args_t& a = p.a;
  const int lane = threadIdx.x & 31;
  uint32_t set = (2u << lane) - 1u;
  bool bad = false;
  if (a.parent) {
    const int par = lane < a.n_q ? a.parent[int64_t(r) * a.n_q + lane] : -1;
    bad = __any_sync(~0u, lane < a.n_q && (par < -1 || par >= lane));
    set = 1u << lane;
    if (!bad)
      // parents come first: in n_q rounds every node has its parent's set
      for (int j = 0; j < a.n_q; ++j) {
        const uint32_t s = __shfl_sync(~0u, set, j);
        if (par == j) set |= s;
      }
  }
  see[lane] = set;
  if (lane == 0) {
    bad_out = bad;
    if (bad) report(a.status, LIN_ST_BAD_TREE);
  }
}

// Joins the KG value sums [KG][ROWS][PITCH >= D] and (m, sum) [KG][ROWS] of a piece in
// shared memory and writes the outputs of a whole item, or the piece's part (or,
// with t1 within the piece, what is summed so far, which carry_in takes up).
// All NT threads.
template <int D, int KG, int ROWS, int NT, int PITCH = D>
__device__ __forceinline__ void finish_piece(const Plan& p, const Walk& w, int t1, const float* merge,
                                             const float2* merge_ml, bool bad) {
  const lin_attn_args_t& a = p.a;
  const int hk = head_of(p, w.it), row0 = (w.it - hk * p.row_blocks) * ROWS;
  const bool whole = w.t0 == 0 && t1 == w.u;
  const int64_t part = 2 * int64_t(blockIdx.x) + (w.t0 == 0 ? 1 : 0);
  constexpr int LANES = D / 4 < 32 ? D / 4 : 32;  // threads of a row, so many steps of 4 channels
  constexpr int STEPS = D / 4 / LANES, AT = NT / LANES;
  const int lane = threadIdx.x % LANES;
#pragma unroll 1  // once per piece: what counts is how much code it brings in
  for (int i = 0; i < (ROWS + AT - 1) / AT; ++i) {
    const int row = threadIdx.x / LANES + i * AT, q = row0 + row;
    if (row >= ROWS || q >= p.rows) continue;
    float2 ml[KG];
    float4 y[KG][STEPS];
#pragma unroll
    for (int k = 0; k < KG; ++k) {
      ml[k] = merge_ml[k * ROWS + row];
#pragma unroll
      for (int x = 0; x < STEPS; ++x)
        y[k][x] = *reinterpret_cast<const float4*>(merge + (k * ROWS + row) * PITCH + (x * LANES + lane) * 4);
    }
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int k = 0; k < KG; ++k) top = fmaxf(top, ml[k].x);
    float4 v[STEPS];
#pragma unroll
    for (int x = 0; x < STEPS; ++x) v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < KG; ++k) {
      // 0 where a copy saw nothing (a NaN sum goes on)
      const float f = ml[k].y == 0.0f ? 0.0f : ml[k].x == top ? 1.0f : exp2_fast(ml[k].x - top);
      sum = fmaf(f, ml[k].y, sum);
#pragma unroll
      for (int x = 0; x < STEPS; ++x) {
        v[x].x = fmaf(f, y[k][x].x, v[x].x), v[x].y = fmaf(f, y[k][x].y, v[x].y);
        v[x].z = fmaf(f, y[k][x].z, v[x].z), v[x].w = fmaf(f, y[k][x].w, v[x].w);
      }
    }
    const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int j = query_of(p, q);
    const int64_t out = ((int64_t(w.r) * a.n_q + j) * a.num_q_heads + hk * p.group + q - j * p.group) * D;
#pragma unroll
    for (int x = 0; x < STEPS; ++x) {
      const int d = (x * LANES + lane) * 4;
      if (!whole) {
        *reinterpret_cast<float4*>(p.part + (part * ROWS + row) * D + d) = v[x];
      } else if (bad) {
      } else if (a.out_dtype == LIN_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + out + d) =
            make_float4(v[x].x * scale, v[x].y * scale, v[x].z * scale, v[x].w * scale);
      } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v[x].x * scale, v[x].y * scale);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(v[x].z * scale, v[x].w * scale);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out + d) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
    if (!whole && lane == 0) p.part_ml[part * ROWS + row] = make_float2(top, bad ? kLeftOut : sum);
  }
}

// Joins the piece's part, the sums so far, into the first of the value sums that
// finish_piece is to join. All NT threads, each with the channels that it wrote.
template <int D, int ROWS, int NT, int PITCH>
__device__ __forceinline__ void carry_in(const Plan& p, const Walk& w, float* merge, float2* merge_ml) {
  const int64_t part = 2 * int64_t(blockIdx.x) + (w.t0 == 0 ? 1 : 0);
  constexpr int LANES = D / 4 < 32 ? D / 4 : 32, STEPS = D / 4 / LANES;
  const int lane = threadIdx.x % LANES, row0 = (w.it - head_of(p, w.it) * p.row_blocks) * ROWS;
#pragma unroll 1
  for (int row = threadIdx.x / LANES; row < ROWS && row0 + row < p.rows; row += NT / LANES) {
    const float2 now = merge_ml[row], was = p.part_ml[part * ROWS + row];
    const float top = fmaxf(now.x, was.x);
    const float f = now.y == 0.0f ? 0.0f : now.x == top ? 1.0f : exp2_fast(now.x - top);
    const float g = was.y == 0.0f ? 0.0f : was.x == top ? 1.0f : exp2_fast(was.x - top);
#pragma unroll
    for (int x = 0; x < STEPS; ++x) {
      float4& v = *reinterpret_cast<float4*>(merge + row * PITCH + (x * LANES + lane) * 4);
      const float4 y = *reinterpret_cast<const float4*>(p.part + (part * ROWS + row) * D + (x * LANES + lane) * 4);
      v.x = fmaf(g, y.x, f * v.x), v.y = fmaf(g, y.y, f * v.y);
      v.z = fmaf(g, y.z, f * v.z), v.w = fmaf(g, y.w, f * v.w);
    }
    // every lane of the row has read its (m, sum)
    __syncwarp(LANES == 32 ? ~0u : ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1)));
    if (lane == 0) merge_ml[row] = make_float2(top, fmaf(g, was.y, f * now.y));
  }
}

// One translation unit per head_dim and kind of kernel.
cudaError_t launch_d64(const Plan& p, int row_tiles, int grid, cudaStream_t s);
cudaError_t launch_d128(const Plan& p, int row_tiles, int grid, cudaStream_t s);
cudaError_t launch_d256(const Plan& p, int row_tiles, int grid, cudaStream_t s);
cudaError_t launch_umma_d64(const Plan& p, int grid, cudaStream_t s);
cudaError_t launch_umma_d128(const Plan& p, int grid, cudaStream_t s);
cudaError_t launch_umma_d256(const Plan& p, int grid, cudaStream_t s);

}  // namespace attn
}  // namespace lin
