// Decode attention over a paged key-value cache (lin_step.h).
//
//   out[r][j][h] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t - m)
//
// in one pass over the visible tokens with the running maximum m and sum. One
// CTA takes one (request, query token, query head); its warps take every
// fourth token, a lane holds head_dim / 32 channels, and the warps' (m, sum,
// values) are joined in shared memory at the end.

#include <math.h>

#include "common.cuh"
#include "step_internal.h"

namespace lin {
namespace {

constexpr int kWarps = 4;

template <int D, int DT>
__global__ void __launch_bounds__(kWarps * 32)
attn_simple_kernel(const lin_kv_cache_t c, const lin_attn_args_t a) {
  constexpr int E = D / 32;
  __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x % a.num_q_heads, j = blockIdx.x / a.num_q_heads % a.n_q;
  const int r = blockIdx.x / a.num_q_heads / a.n_q;
  const int hk = h / (a.num_q_heads / c.num_kv_heads);
  const int len = a.kv_len[r];
  if (len < 0) return;
  if (len > int64_t(a.max_pages) * c.page_size) {
    if (threadIdx.x == 0) report(a.status, LIN_ST_BAD_SEQLEN);
    return;
  }
  const int base = len - a.n_q;
  uint32_t see = (2u << j) - 1u;
  if (a.parent) {
    const int par = lane < a.n_q ? a.parent[int64_t(r) * a.n_q + lane] : -1;
    if (__any_sync(~0u, lane < a.n_q && (par < -1 || par >= lane))) {
      if (threadIdx.x == 0) report(a.status, LIN_ST_BAD_TREE);
      return;
    }
    see = 0;
    for (int at = j; at >= 0; at = __shfl_sync(~0u, par, at)) see |= 1u << at;
  }
  const char* qp = static_cast<const char*>(a.q) + r * a.req_stride + j * a.token_stride;
  float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = load_elem(qp, h * D + lane + 32 * i, DT) * a.scale;
    o[i] = 0.0f;
  }
  for (int t = warp; t < len; t += kWarps) {
    if (t >= base && !((see >> (t - base)) & 1u)) continue;
    const int pg = t / c.page_size;
    const int id = a.page_table[r * a.page_table_stride + pg];
    if (id < 0 || id >= c.num_pages) {
      if (lane == 0) report(a.status, LIN_ST_BAD_PAGE);
      continue;
    }
    const int64_t at = a.layer * c.layer_stride + id * c.page_stride +
                       int64_t(t - pg * c.page_size) * c.token_stride + hk * c.head_stride;
    const char* kp = static_cast<const char*>(c.k) + at;
    const char* vp = static_cast<const char*>(c.v) + at;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(q[i], load_elem(kp, lane + 32 * i, DT), s);
#pragma unroll
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(~0u, s, w);
    const float m2 = fmaxf(m, s);
    const float f = m == m2 ? 1.0f : expf(m - m2), p = expf(s - m2);
    l = fmaf(l, f, p);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = fmaf(o[i], f, p * load_elem(vp, lane + 32 * i, DT));
    m = m2;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) sm_o[warp][lane + 32 * i] = o[i];
  if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
  __syncthreads();
  float top = -INFINITY, sum = 0.0f, f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_m[w]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = sm_l[w] != 0.0f ? expf(sm_m[w] - top) : 0.0f;  // a NaN stays one
    sum += f[w] * sm_l[w];
  }
  const int64_t out = ((int64_t(r) * a.n_q + j) * a.num_q_heads + h) * D;
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += f[w] * sm_o[w][d];
    store_elem(a.out, out + d, a.out_dtype, sum != 0.0f ? v / sum : 0.0f);
  }
}

}  // namespace

size_t attn_workspace(const lin_kv_cache_t&, const lin_attn_args_t&) { return 0; }

cudaError_t launch_attn_decode(const lin_kv_cache_t& c, const lin_attn_args_t& a, void*, cudaStream_t s) {
  const int64_t blocks = int64_t(a.batch) * a.n_q * a.num_q_heads;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  const bool b = c.dtype == LIN_BF16;
  if (c.head_dim == 64)
    (b ? attn_simple_kernel<64, LIN_BF16> : attn_simple_kernel<64, LIN_F32>)<<<grid, kWarps * 32, 0, s>>>(c, a);
  else if (c.head_dim == 128)
    (b ? attn_simple_kernel<128, LIN_BF16> : attn_simple_kernel<128, LIN_F32>)<<<grid, kWarps * 32, 0, s>>>(c, a);
  else
    (b ? attn_simple_kernel<256, LIN_BF16> : attn_simple_kernel<256, LIN_F32>)<<<grid, kWarps * 32, 0, s>>>(c, a);
  return cudaGetLastError();
}

}  // namespace lin
