// Block tables, positions and slot maps of a batch's new tokens (lin_prompt.h).
//
//   need[r] = ceil((len + n) / P) - ceil(len / P),  before = its exclusive sum,
//   table[r][ceil(len / P) + i] = free[before[r] + i],  cu = the running sum of n,
//   position = len + j (or + depth),  slot = table[r][(len + j) / P] P + (len + j) % P
//
// Bound by latency: a launch, the lengths, a block scan, the first page ids (256 requests
// of one token 5.7 us, 64 chunks of up to 2,048 tokens 5.6 us). One
// launch: every CTA scans the whole batch by itself (a kernel in front would cost more
// than the repeated loads, which come from L2) and then serves kPlanTokens packed
// rows. The scan leaves a mark at the row where a request begins, and a row's request
// is the last mark at or before it; that has no cost per request, so a batch of
// thousands of requests of one token and one request of 100,000 go the same way. The
// row that is the first of its page writes the table's entry.

#include "common.cuh"
#include "prompt_internal.h"

namespace lin {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanTokens = 2048;  // rows of a CTA
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int64_t kPlanLongest = (int64_t(1) << 31) - 65536;  // of a request, as attention takes it

struct Request {
  int len, n;    // cached tokens (-1: padding or left out), rows among the packed tokens
  int need;      // new pages
  int bad;       // status bits
};

__device__ __forceinline__ int pages_of(int tokens, int page) { return tokens > 0 ? (tokens - 1) / page + 1 : 0; }

// What the request itself says; rows past the end and short pages come from the sums.
__device__ __forceinline__ Request look_at(const lin_kv_plan_args_t& a, int r) {
  Request q;
  q.len = a.length[r];
  q.n = a.n_new ? a.n_new[r] : a.n;
  q.need = q.bad = 0;
  if (q.len < 0) {
    q.len = -1, q.n = 0;
    return q;
  }
  const int64_t most = min(int64_t(a.max_pages) * a.page_size, kPlanLongest);
  if (q.n < 0) q.n = 0, q.bad = LIN_ST_BAD_SEQLEN;
  if (int64_t(q.len) + q.n > most) q.bad = LIN_ST_BAD_SEQLEN;
  if (a.parent) {
    const int32_t* par = a.parent + int64_t(r) * a.n;
    bool ok = true;
    for (int j = 0; j < a.n; ++j) {
      const int up = par[j];
      ok &= up >= -1 && up < j;
    }
    if (!ok) q.bad |= LIN_ST_BAD_TREE;
  }
  if (q.bad)
    q.len = -1;
  else if (a.free_pages)
    q.need = pages_of(q.len + q.n, a.page_size) - pages_of(q.len, a.page_size);
  return q;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const lin_kv_plan_args_t a) {
  __shared__ int s_req[kPlanTokens];     // request that begins at this row, or -1
  __shared__ int s_before[kPlanTokens];  // its first free page's index, or -1: left out
  __shared__ int64_t s_tok[kPlanWarps], s_page[kPlanWarps];
  __shared__ int s_last[kPlanWarps], s_taken[kPlanWarps];
  __shared__ int64_t s_start;  // first row of the request that covers row 0 of the CTA
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = int64_t(blockIdx.x) * kPlanTokens;
  for (int i = tid; i < kPlanTokens; i += kPlanThreads) s_req[i] = -1;

  // ---- the batch's running sums ---------------------------------------------------
  const int span = (a.batch + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(a.batch, tid * span), r1 = min(a.batch, r0 + span);
  int64_t tok = 0, page = 0;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    const Request q = look_at(a, r);
    tok += q.n, page += q.need;
  }
  const int64_t my_tok = tok, my_page = page;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, tok, o), y = __shfl_up_sync(~0u, page, o);
    if (lane >= o) tok += x, page += y;
  }
  if (lane == 31) s_tok[warp] = tok, s_page[warp] = page;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w)
    if (w < warp) tok += s_tok[w], page += s_page[w];
  tok -= my_tok, page -= my_page;  // before this thread's requests

  // ---- marks of the requests with rows here; the first CTA writes what goes by request ----
  int taken = 0;
  for (int r = r0; r < r1; ++r) {
    const Request q = look_at(a, r);
    const int64_t end = tok + q.n;
    int bad = q.bad;
    bool in = q.len >= 0;
    if (in && end > a.tokens) in = false, bad |= LIN_ST_BAD_SEQLEN;
    if (in && q.need > 0 && page + q.need > a.num_free) in = false, bad |= LIN_ST_NO_PAGES;
    if (in && q.need > 0) taken = static_cast<int>(page + q.need);
    if (q.n > 0 && end > row0 && tok < row0 + kPlanTokens) {
      const int o = tok > row0 ? static_cast<int>(tok - row0) : 0;
      s_req[o] = r;
      s_before[o] = in ? static_cast<int>(q.need > 0 ? page : 0) : -1;
      if (o == 0) s_start = tok;
    }
    if (blockIdx.x == 0) {
      if (bad) report(a.status, bad);
      if (a.kv_len) a.kv_len[r] = in ? q.len + q.n : -1;
      if (a.cu_seqlens) a.cu_seqlens[r + 1] = static_cast<int>(min(end, int64_t(INT32_MAX)));
    }
    tok = end, page += q.need;
  }
  if (blockIdx.x == 0) {
#pragma unroll
    for (int o = 16; o; o >>= 1) taken = max(taken, __shfl_xor_sync(~0u, taken, o));
    if (lane == 0) s_taken[warp] = taken;
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    if (a.cu_seqlens) a.cu_seqlens[0] = 0;
    if (a.taken) {
      for (int w = 1; w < kPlanWarps; ++w) taken = max(taken, s_taken[w]);
      *a.taken = taken;
    }
  }
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) total += s_tok[w];

  // ---- rows: warp w has kPlanTokens / kPlanWarps of them --------------------------------
  constexpr int ROWS = kPlanTokens / kPlanWarps;
  int last[ROWS / 32];
  int most = -1;
#pragma unroll
  for (int i = 0; i < ROWS / 32; ++i) {
    const int o = warp * ROWS + i * 32 + lane;
    const uint32_t marks = __ballot_sync(~0u, s_req[o] >= 0);
    const uint32_t upto = marks & (~0u >> (31 - lane));
    last[i] = upto ? warp * ROWS + i * 32 + 31 - __clz(upto) : most;
    if (marks) most = warp * ROWS + i * 32 + 31 - __clz(marks);
  }
  if (lane == 0) s_last[warp] = most;
  __syncthreads();
  int carry = -1;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w)
    if (w < warp) carry = max(carry, s_last[w]);
#pragma unroll
  for (int i = 0; i < ROWS / 32; ++i) {
    const int o = warp * ROWS + i * 32 + lane;
    const int64_t row = row0 + o;
    if (row >= a.tokens) continue;
    const int mark = max(last[i], carry);
    int position = -1;
    int64_t slot = -1;
    const int before = row < total && mark >= 0 ? s_before[mark] : -1;
    if (before >= 0) {
      const int r = s_req[mark], len = a.length[r];
      const int j = static_cast<int>(row - (mark == 0 ? s_start : row0 + mark));
      const int at = len + j, pg = at / a.page_size, in_page = at - pg * a.page_size;
      position = at;
      if (a.parent) {
        const int32_t* par = a.parent + int64_t(r) * a.n;
        position = len;
        for (int up = par[j]; up >= 0; up = par[up]) ++position;
      }
      const int have = pages_of(len, a.page_size);
      int32_t* entry = a.page_table + r * a.page_table_stride + pg;
      int id;
      if (a.free_pages && pg >= have) {
        id = a.free_pages[before + pg - have];
        if (in_page == 0) *entry = id;
      } else {
        id = *entry;
      }
      if (id >= 0 && id < a.num_pages)
        slot = int64_t(id) * a.page_size + in_page;
      else
        report(a.status, LIN_ST_BAD_PAGE);
    }
    if (a.position) a.position[row] = position;
    if (a.slot) a.slot[row] = slot;
  }
}

}  // namespace

cudaError_t launch_kv_plan(const lin_kv_plan_args_t& a, cudaStream_t s) {
  const int blocks = a.tokens > 0 ? (a.tokens - 1) / kPlanTokens + 1 : 1;
  kv_plan_kernel<<<blocks, kPlanThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace lin
