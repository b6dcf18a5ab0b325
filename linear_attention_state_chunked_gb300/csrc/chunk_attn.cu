// Chunk attention over a paged key-value cache (lin_prompt.h): the join of split items
// and the host side. The main kernels are in chunk_umma.cuh and chunk_mma.cuh.

#include "chunk_common.cuh"

namespace lin {
namespace chunk {
namespace {

constexpr int kJoinWarps = 8;

// The item that begins in range c and goes on past it has the parts, in token order,
// 2c + 1 and then 2c' of the ranges c' = c + 1, ... A warp per row; blockIdx.y takes
// every gridDim.y-th set of rows.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Plan p) {
  constexpr int V = D / 32;
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  // the stream's next launch is ordered behind this grid alone: every block waits
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Split s = p.split[c];
  if (s.parts == 0) return;
  auto index = [&](int i, int row) { return (2 * int64_t(c) + (i == 0 ? 1 : 2 * i)) * p.rows + row; };
  for (int row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); row < s.tokens * p.bheads; row += gridDim.y * kJoinWarps) {
    const int t = token_of(p, row), h = row - t * p.bheads;
    if (h >= s.heads) continue;
    float top = -INFINITY;
    bool out = false;
    for (int i = lane; i < s.parts; i += 32) {
      const float2 ml = p.part_ml[index(i, row)];
      top = fmaxf(top, ml.x);
      out |= ml.y == attn::kLeftOut;
    }
    if (__any_sync(~0u, out)) continue;  // left out after a wait that ran out
#pragma unroll
    for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
    float sum = 0.0f, v[V];
#pragma unroll
    for (int x = 0; x < V; ++x) v[x] = 0.0f;
#pragma unroll 4
    for (int i = 0; i < s.parts; ++i) {
      const int64_t at = index(i, row);
      const float2 ml = p.part_ml[at];
      // 0 where a part saw nothing (a NaN sum goes on)
      const float f = ml.y == 0.0f ? 0.0f : ml.x == top ? 1.0f : attn::exp2_fast(ml.x - top);
      sum = fmaf(f, ml.y, sum);
#pragma unroll
      for (int x = 0; x < V; x += 2) {
        const float2 y = *reinterpret_cast<const float2*>(p.part + at * D + lane * V + x);
        v[x] = fmaf(f, y.x, v[x]), v[x + 1] = fmaf(f, y.y, v[x + 1]);
      }
    }
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t at = (int64_t(s.row0 + t) * p.a.num_q_heads + s.head0 + h) * D + lane * V;
#pragma unroll
    for (int x = 0; x < V; x += 2) {
      if (p.a.out_dtype == LIN_F32)
        *reinterpret_cast<float2*>(static_cast<float*>(p.a.out) + at + x) = make_float2(v[x] * f, v[x + 1] * f);
      else
        *reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(p.a.out) + at + x) =
            __floats2bfloat162_rn(v[x] * f, v[x + 1] * f);
    }
  }
}

// Which kernel a call takes.
struct Shape {
  bool umma;
  int rows, tk, ctas, item_cost;
};

Shape shape_of(const lin_kv_cache_t& c, const lin_attn_chunk_args_t& a, int out_dtype) {
  if (c.dtype == LIN_BF16 && out_dtype == LIN_BF16) {
    const int64_t rows = int64_t(a.tokens) * (a.num_q_heads / c.num_kv_heads);  // of a kv head
    const bool two = c.head_dim <= 128 && rows > 128 * int64_t(a.batch);
    return {true, two ? 256 : 128, 128, 1, 192};
  }
  const int row_bytes = c.head_dim * dtype_size(c.dtype);
  return {false, 64, row_bytes >= 512 ? 16 : 32, row_bytes <= 256 ? 3 : row_bytes == 512 ? 2 : 1, 64};
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) sms = device_sm_count(dev);
  return sms > 0 ? sms : 152;  // no device: the size of a GB300
}

size_t bytes_of(const lin_kv_cache_t& c, const Shape& f) {
  const size_t grid = size_t(sm_count()) * f.ctas;
  return 2 * grid * f.rows * (c.head_dim * sizeof(float) + sizeof(float2)) + grid * sizeof(Split);
}

// Granlund and Montgomery's division by an invariant: s = ceil(log2 d),
// mul = floor(2^32 (2^s - d) / d) + 1
void divide_by(int64_t d, uint32_t& mul, uint32_t& shift) {
  shift = 0;
  while ((int64_t(1) << shift) < d) ++shift;
  mul = static_cast<uint32_t>((((uint64_t(1) << shift) - d) << 32) / d + 1);
}

}  // namespace
}  // namespace chunk

size_t chunk_need(const lin_kv_cache_t& c, const lin_attn_chunk_args_t& a) {
  return chunk::bytes_of(c, chunk::shape_of(c, a, a.out_dtype));
}

size_t chunk_workspace(const lin_kv_cache_t& c, const lin_attn_chunk_args_t& a) {
  // of every kernel that a call over this cache may take
  size_t most = 0;
  lin_attn_chunk_args_t x = a;
  x.batch = 1;
  for (const int out : {LIN_BF16, LIN_F32})
    for (const int tokens : {1, 129}) {
      x.tokens = tokens;
      const size_t n = chunk::bytes_of(c, chunk::shape_of(c, x, out));
      if (n > most) most = n;
    }
  return most;
}

cudaError_t launch_attn_chunk(const lin_kv_cache_t& c, const lin_attn_chunk_args_t& a, void* ws, cudaStream_t s) {
  const chunk::Shape f = chunk::shape_of(c, a, a.out_dtype);
  chunk::Plan p;
  p.c = c;
  p.a = a;
  p.group = a.num_q_heads / c.num_kv_heads;
  p.rows = f.rows;
  p.blocks = (p.group + f.rows - 1) / f.rows;
  p.bheads = (p.group + p.blocks - 1) / p.blocks;
  p.blocks = (p.group + p.bheads - 1) / p.bheads;
  p.m = f.rows / p.bheads;
  p.heads = c.num_kv_heads * p.blocks;
  p.tk = f.tk;
  p.grid = chunk::sm_count() * f.ctas;
  p.item_cost = f.item_cost;
  p.scale_log2 = fabsf(a.scale) * 1.4426950408889634f;  // log2(e)
  if (p.scale_log2 < 0x1p-126f) p.scale_log2 = 0x1p-126f;  // not 0: hidden scores are -inf
  p.slack = attn::kSlack / p.scale_log2;
  p.negate = !(a.scale < 0.0f) ? 0u : c.dtype == LIN_BF16 ? 0x80008000u : 0x80000000u;
  chunk::divide_by(c.page_size, p.page_mul, p.page_shift);
  chunk::divide_by(p.bheads, p.bhead_mul, p.bhead_shift);
  char* w = static_cast<char*>(ws);
  p.part = reinterpret_cast<float*>(w);
  w += size_t(2) * p.grid * p.rows * c.head_dim * sizeof(float);
  p.part_ml = reinterpret_cast<float2*>(w);
  w += size_t(2) * p.grid * p.rows * sizeof(float2);
  p.split = reinterpret_cast<chunk::Split*>(w);
  cudaError_t e;
  if (f.umma)
    e = c.head_dim == 64    ? chunk::launch_umma_d64(p, s)
        : c.head_dim == 128 ? chunk::launch_umma_d128(p, s)
                            : chunk::launch_umma_d256(p, s);
  else
    e = c.head_dim == 64    ? chunk::launch_mma_d64(p, s)
        : c.head_dim == 128 ? chunk::launch_mma_d128(p, s)
                            : chunk::launch_mma_d256(p, s);
  if (e != cudaSuccess) return e;
  // the join's launch overlaps the main kernel, and it waits there for its end
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(p.grid, 4);
  cfg.blockDim = dim3(chunk::kJoinWarps * 32);
  return c.head_dim == 64    ? cudaLaunchKernelEx(&cfg, chunk::join_kernel<64>, p)
         : c.head_dim == 128 ? cudaLaunchKernelEx(&cfg, chunk::join_kernel<128>, p)
                             : cudaLaunchKernelEx(&cfg, chunk::join_kernel<256>, p);
}

}  // namespace lin
