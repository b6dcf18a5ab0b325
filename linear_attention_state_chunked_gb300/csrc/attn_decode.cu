// Decode attention over a paged key-value cache (lin_step.h): the join of split
// items and the host side. The main kernel is in attn_kernel.cuh.

#include "attn_kernel.cuh"

namespace lin {
namespace attn {
namespace {

constexpr int kJoinWarps = 8, kRowWarps = 16;
constexpr int kJoinRows = 16;    // most rows of an item side by side in the grid
constexpr int kMaxRanges = 1024;
constexpr int kShortUnits = 4;   // of a request: see shape_of

// The item that begins in range c and goes on past it has the parts, in token
// order, 2c + 1 and then 2c' of the ranges c' = c + 1, ... They are joined in that
// order (where a row has kRowWarps warps, each takes every kRowWarps-th), so the result
// does not depend on timing.
//
// Bound by the latency of dependent loads (split, sums, values). Many items, few
// parts each: a block for every range, a warp per row, and most find no split. Few
// items, many parts: a block for every item's row, which works out from the lengths
// (while the main kernel runs) which ranges hold it, loads all sums at once and
// the values by 16 warps (one request of 60,000 tokens, one kv head, 304 parts:
// 24 us in all with a block for every range's row, 18 so).
struct Split {
  int parts, hk, rb;
  int64_t r;
};
__device__ __forceinline__ bool split_of(const Plan& p, int c, Split& s) {
  const longlong2 split = p.split[c];
  if (split.x < 0) return false;
  const int64_t head = split.x / p.row_blocks;
  s.rb = static_cast<int>(split.x - head * p.row_blocks);
  s.r = head / p.c.num_kv_heads;
  s.hk = static_cast<int>(head - s.r * p.c.num_kv_heads);
  s.parts = static_cast<int>(split.y);
  return true;
}
// Index of part i's row, and of a row's first output.
__device__ __forceinline__ int64_t part_row(const Plan& p, int c, int i, int row) {
  return (2 * int64_t(c) + (i == 0 ? 1 : 2 * i)) * p.block_rows + row;
}
template <int D>
__device__ __forceinline__ int64_t out_row(const Plan& p, const Split& s, int q) {
  const int j = query_of(p, q);
  return ((s.r * p.a.n_q + j) * p.a.num_q_heads + s.hk * p.group + q - j * p.group) * D;
}
// a part's share of the joined sums (0 where it saw nothing; a NaN sum goes on)
__device__ __forceinline__ float share_of(float2 ml, float top) {
  return ml.y == 0.0f ? 0.0f : ml.x == top ? 1.0f : exp2_fast(ml.x - top);
}
template <int V>
__device__ __forceinline__ void load_values(const float* src, float (&x)[V]) {
  if constexpr (V == 2) {
    const float2 y = *reinterpret_cast<const float2*>(src);
    x[0] = y.x, x[1] = y.y;
  } else {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const float4 y = *reinterpret_cast<const float4*>(src + k);
      x[k] = y.x, x[k + 1] = y.y, x[k + 2] = y.z, x[k + 3] = y.w;
    }
  }
}

// The range that holds this unit.
__device__ __forceinline__ int range_of(int64_t unit, int64_t ranges, int64_t total) {
  return static_cast<int>(((unit + 1) * ranges - 1) / total);
}

// A warp per row.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Plan p) {
  constexpr int V = D / 32;
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Split s;
  if (!split_of(p, c, s)) return;
  const int q = s.rb * p.block_rows + row;
  if (row >= p.block_rows || q >= p.rows) return;
  float top = -INFINITY;
  bool out = false;
  for (int i = lane; i < s.parts; i += 32) {
    const float2 ml = p.part_ml[part_row(p, c, i, row)];
    top = fmaxf(top, ml.x);
    out |= ml.y == kLeftOut;
  }
  if (__any_sync(~0u, out)) return;  // a request left out
#pragma unroll
  for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
  float sum = 0.0f, v[V];
#pragma unroll
  for (int x = 0; x < V; ++x) v[x] = 0.0f;
#pragma unroll 4
  for (int i = 0; i < s.parts; ++i) {
    const int64_t at = part_row(p, c, i, row);
    const float2 ml = p.part_ml[at];
    float x[V];
    load_values<V>(p.part + at * D + lane * V, x);
    const float f = share_of(ml, top);
    sum = fmaf(f, ml.y, sum);
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = fmaf(f, x[k], v[k]);
  }
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t at = out_row<D>(p, s, q) + lane * V;
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    if (p.a.out_dtype == LIN_F32)
      *reinterpret_cast<float2*>(static_cast<float*>(p.a.out) + at + k) = make_float2(v[k] * f, v[k + 1] * f);
    else
      *reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(p.a.out) + at + k) =
          __floats2bfloat162_rn(v[k] * f, v[k + 1] * f);
  }
}

// A block per row of an item: block (item, y).
template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) join_row_kernel(const Plan p) {
  constexpr int V = D / 32, NT = kRowWarps * 32;
  __shared__ float s_f[kMaxRanges], s_v[kRowWarps][D], s_top[kRowWarps], s_sum[kRowWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_req = p.c.num_kv_heads * p.row_blocks, it = blockIdx.x % per_req;
  Split s;
  s.r = blockIdx.x / per_req;
  s.hk = head_of(p, it);
  s.rb = it - s.hk * p.row_blocks;
  // where the item lies among all units, as in walk_begin (every warp by itself)
  const int64_t most = longest(p);
  int64_t before = 0, total = 0;
  for (int r = lane; r < p.a.batch; r += 32) {
    const int u = units_of(p.a.kv_len[r], most);
    const int64_t n = u > 0 ? int64_t(u + p.item_cost) * per_req : 0;
    total += n;
    if (r < s.r) before += n;
  }
#pragma unroll
  for (int w = 16; w; w >>= 1) {
    before += __shfl_xor_sync(~0u, before, w);
    total += __shfl_xor_sync(~0u, total, w);
  }
  const int u = units_of(p.a.kv_len[s.r], most);
  int c = 0;
  s.parts = 1;
  if (u > 0) {
    const int64_t ranges = total < p.grid ? total : p.grid, base = before + int64_t(it) * (u + p.item_cost);
    // borders among the first item_cost units have moved to the item's start
    c = range_of(base + p.item_cost, ranges, total);
    s.parts = range_of(base + u + p.item_cost - 1, ranges, total) - c + 1;
  }
  // Every block waits, those of a request without units too: the stream's next
  // launch is ordered behind this grid alone, which therefore must not end
  // before the main kernel, the last reader of the lengths and writer of `split`.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (s.parts == 1) return;
  for (int row = blockIdx.y; row < p.block_rows; row += gridDim.y) {
    const int q = s.rb * p.block_rows + row;
    if (q >= p.rows) return;
    constexpr int MOST = kMaxRanges / NT;
    float2 ml[MOST];
    float top = -INFINITY;
    bool out = false;
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      const int i = tid + k * NT;
      ml[k] = i < s.parts ? p.part_ml[part_row(p, c, i, row)] : make_float2(-INFINITY, 0.0f);
    }
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      top = fmaxf(top, ml[k].x);
      out |= ml[k].y == kLeftOut;
    }
#pragma unroll
    for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
    if (lane == 0) s_top[warp] = top;
    if (__syncthreads_or(out)) return;  // a request left out
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, s_top[w]);
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      const int i = tid + k * NT;
      const float f = share_of(ml[k], top);
      if (i < s.parts) s_f[i] = f;
      sum = fmaf(f, ml[k].y, sum);
    }
#pragma unroll
    for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    float v[V];
#pragma unroll
    for (int x = 0; x < V; ++x) v[x] = 0.0f;
#pragma unroll(D <= 128 ? 10 : 8)
    for (int i = warp; i < s.parts; i += kRowWarps) {
      float x[V];
      load_values<V>(p.part + part_row(p, c, i, row) * D + lane * V, x);
      const float f = s_f[i];
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = fmaf(f, x[k], v[k]);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) s_v[warp][lane * V + k] = v[k];
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) sum += s_sum[w];
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t at = out_row<D>(p, s, q);
    for (int d = tid; d < D; d += NT) {
      float x = 0.0f;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) x += s_v[w][d];
      store_elem(p.a.out, at + d, p.a.out_dtype, x * f);
    }
    __syncthreads();
  }
}

template <int D>
cudaError_t launch_join(cudaLaunchConfig_t& cfg, const Plan& p, int grid, int64_t items) {
  const int rows = p.rows < p.block_rows ? p.rows : p.block_rows;
  if (items * 8 > grid) {  // fewer than 8 parts to an item
    cfg.gridDim = dim3(grid, (rows + kJoinWarps - 1) / kJoinWarps);
    cfg.blockDim = dim3(kJoinWarps * 32);
    return cudaLaunchKernelEx(&cfg, join_kernel<D>, p);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(items), rows < kJoinRows ? rows : kJoinRows);
  cfg.blockDim = dim3(kRowWarps * 32);
  return cudaLaunchKernelEx(&cfg, join_row_kernel<D>, p);
}

// Which kernel a call takes, the rows of its items and its CTAs per SM.
// item_cost, in units of 64 tokens: an item's start and end take about 6 us of an
// SM on tcgen05 against 0.9 us per unit, and 4 us of a CTA against 1.5 us per
// unit (two CTAs to an SM) on warp-level MMA.
struct Shape {
  bool umma;
  int block_rows, ctas, item_cost;
  // Items of up to so many units stay whole, as the join takes longer than their
  // tokens one after another (one token, 1 and 256 requests of 128-256 tokens: bf16
  // heads of 64 6.4 and 10.2 us against 7.9 and 14.5, of 256 9.7 and 38.3 against 10.5
  // and 38.9; one request of 512 tokens 10.4 against 8.9; fp32, 64-128 tokens: heads of
  // 64 6.9 and 16.0 against 7.6 and 17.9, of 256 12.1 and 48.0 against 12.6 and 50.0,
  // 256 tokens 19.5 against 15.8). What the page table allows decides, as the lengths
  // are the device's: short requests with a wide table are split.
  int whole_units;
};

template <int D>
int ctas_of(bool bf16, int rt) {
  if (bf16) return rt == 1 ? Cfg<D, LIN_BF16, 1>::CTAS : rt == 2 ? Cfg<D, LIN_BF16, 2>::CTAS : Cfg<D, LIN_BF16, 4>::CTAS;
  return rt == 1 ? Cfg<D, LIN_F32, 1>::CTAS : rt == 2 ? Cfg<D, LIN_F32, 2>::CTAS : Cfg<D, LIN_F32, 4>::CTAS;
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) sms = device_sm_count(dev);
  return sms > 0 ? sms : 152;  // no device: the size of a GB300
}

// bf16 caches: up to 16 rows per (request, kv head) on warp-level MMA, more on
// tcgen05 in blocks of 32, 64 or 128 (64 requests of 500-8,000 tokens, 2 kv heads, 64
// and 128 rows: heads of 64 72 and 129 us against 74 and 131 on warp-level MMA, of
// 128 85 and 140 against 118 and 218, of 256 125 and 178 against 245 and 469; 32 rows:
// 48, 70 and 106 against 45, 69 and 133).
// But 17 to 32 rows of requests of up to 256 tokens go as two blocks of 16, for an
// item's start and end take longer there than reading it twice: 4 drafts of a group
// of 8, 2 kv heads, 1 and 256 requests of 128-256 tokens: heads of 64 6.8 and 17.8 us
// against 8.4 and 27.6, of 128 8.7 and 38.6 against 10.8 and 42.4. Heads of 256 leave
// room for one CTA to an SM, so there only while each block has an SM to itself (32
// requests 11.8 us against 14.9; 64 21.0 against 16.8; 256 71.0 against 62.6).
// fp32 caches: warp-level MMA in blocks of 16, 32 or 64. So do fp32 outputs of bf16
// caches, whose long sums tcgen05 does not round (64 requests of 500-8,000 tokens, 2
// kv heads of 128, 32, 64 and 128 rows: 81, 140 and 260 us, where it took 76, 102
// and 170; 4 of 64, 32 rows: 86 against 135).
int batch_in_two(const lin_kv_cache_t& c) { return sm_count() / 2 / c.num_kv_heads; }  // heads of 256
Shape shape_of(const lin_kv_cache_t& c, int batch, int rows, int64_t units, int out_dtype) {
  const bool b = c.dtype == LIN_BF16;
  const bool bb = b && out_dtype == LIN_BF16;
  const bool in_two = units <= kShortUnits && (c.head_dim < 256 || batch <= batch_in_two(c));
  if (bb && rows > 16 && (rows > 32 || !in_two)) return {true, rows <= 32 ? 32 : rows <= 64 ? 64 : 128, 1, 7, 4};
  const int rt = rows <= 16 || bb ? 1 : rows <= 32 ? 2 : 4;
  return {false, 16 * rt, c.head_dim == 64 ? ctas_of<64>(b, rt) : c.head_dim == 128 ? ctas_of<128>(b, rt) : ctas_of<256>(b, rt), b ? 3 : 2, b ? 4 : 2};
}

// CTAs of the main kernel: what is resident at once, or one per unit where the
// longest request allowed would give fewer.
int grid_of(const lin_kv_cache_t& c, int batch, int rows, int64_t units, const Shape& f) {
  const int64_t blocks = (rows + f.block_rows - 1) / f.block_rows;
  const int64_t items = int64_t(batch) * c.num_kv_heads * blocks;
  const int64_t most = units > 1 && items < INT32_MAX ? items * units : items;
  const int64_t sms = sm_count(), full = sms * f.ctas < kMaxRanges ? sms * f.ctas : kMaxRanges;
  return static_cast<int>(most < full && most > 0 ? most : full);
}

int rows_of(const lin_kv_cache_t& c, const lin_attn_args_t& a) { return a.n_q * (a.num_q_heads / c.num_kv_heads); }
int64_t units_most(const lin_kv_cache_t& c, const lin_attn_args_t& a) {
  return (int64_t(a.max_pages) * c.page_size + kUnit - 1) / kUnit;
}
size_t bytes_of(const lin_kv_cache_t& c, const Shape& f, size_t grid) {
  return 2 * grid * f.block_rows * (c.head_dim * sizeof(float) + sizeof(float2)) + grid * sizeof(longlong2);
}

// Granlund and Montgomery's division by an invariant: s = ceil(log2 d),
// mul = floor(2^32 (2^s - d) / d) + 1
void divide_by(int64_t d, uint32_t& mul, uint32_t& shift) {
  shift = 0;
  while ((int64_t(1) << shift) < d) ++shift;
  mul = static_cast<uint32_t>((((uint64_t(1) << shift) - d) << 32) / d + 1);
}

}  // namespace
}  // namespace attn

// What this call uses.
size_t attn_need(const lin_kv_cache_t& c, const lin_attn_args_t& a) {
  const int rows = attn::rows_of(c, a);
  const int64_t units = attn::units_most(c, a);
  const attn::Shape f = attn::shape_of(c, a.batch, rows, units, a.out_dtype);
  return attn::bytes_of(c, f, attn::grid_of(c, a.batch, rows, units, f));
}

// The most that a call uses of up to this batch, so many rows and pages, and either
// output type. Within one kind of kernel that grows with each of them, so the
// kinds' largest calls do (shape_of's borders).
size_t attn_workspace(const lin_kv_cache_t& c, const lin_attn_args_t& a) {
  const int rows = attn::rows_of(c, a);
  const int64_t units = attn::units_most(c, a);
  size_t most = 0;
  for (const int out : {LIN_BF16, LIN_F32})
    for (const int b : {attn::batch_in_two(c), a.batch})
      for (const int r : {16, 32, 64, rows})
        for (const int64_t u : {int64_t(attn::kShortUnits), units}) {
          const int x = b < a.batch ? b : a.batch, y = r < rows ? r : rows;
          const int64_t z = u < units ? u : units;
          const attn::Shape f = attn::shape_of(c, x, y, z, out);
          const size_t n = attn::bytes_of(c, f, attn::grid_of(c, x, y, z, f));
          if (n > most) most = n;
        }
  return most;
}

cudaError_t launch_attn_decode(const lin_kv_cache_t& c, const lin_attn_args_t& a, void* ws, cudaStream_t s) {
  attn::Plan p;
  p.c = c;
  p.a = a;
  p.group = a.num_q_heads / c.num_kv_heads;
  p.rows = attn::rows_of(c, a);
  const int64_t units = attn::units_most(c, a);
  const attn::Shape f = attn::shape_of(c, a.batch, p.rows, units, a.out_dtype);
  const int grid = attn::grid_of(c, a.batch, p.rows, units, f);
  p.grid = grid;
  p.block_rows = f.block_rows;
  p.item_cost = f.item_cost;
  p.whole = int64_t(a.max_pages) * c.page_size <= int64_t(f.whole_units) * attn::kUnit;
  p.row_blocks = (p.rows + f.block_rows - 1) / f.block_rows;
  p.scale_log2 = fabsf(a.scale) * 1.4426950408889634f;  // log2(e)
  p.slack = attn::kSlack / p.scale_log2;  // infinite where scale is 0: one reference does
  p.negate = !(a.scale < 0.0f) ? 0u : c.dtype == LIN_BF16 ? 0x80008000u : 0x80000000u;
  attn::divide_by(c.page_size, p.page_mul, p.page_shift);
  attn::divide_by(p.group, p.group_mul, p.group_shift);
  attn::divide_by(p.row_blocks, p.block_mul, p.block_shift);
  char* w = static_cast<char*>(ws);
  p.part = reinterpret_cast<float*>(w);
  w += size_t(2) * grid * f.block_rows * c.head_dim * sizeof(float);
  p.part_ml = reinterpret_cast<float2*>(w);
  w += size_t(2) * grid * f.block_rows * sizeof(float2);
  p.split = reinterpret_cast<longlong2*>(w);
  const int rt = f.block_rows / 16;
  cudaError_t e;
  if (f.umma)
    e = c.head_dim == 64    ? attn::launch_umma_d64(p, grid, s)
        : c.head_dim == 128 ? attn::launch_umma_d128(p, grid, s)
                            : attn::launch_umma_d256(p, grid, s);
  else
    e = c.head_dim == 64    ? attn::launch_d64(p, rt, grid, s)
        : c.head_dim == 128 ? attn::launch_d128(p, rt, grid, s)
                            : attn::launch_d256(p, rt, grid, s);
  if (e != cudaSuccess || p.whole) return e;
  // the join's launch overlaps the main kernel, and it waits there for its end
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int64_t items = int64_t(a.batch) * c.num_kv_heads * p.row_blocks;
  return c.head_dim == 64    ? attn::launch_join<64>(cfg, p, grid, items)
         : c.head_dim == 128 ? attn::launch_join<128>(cfg, p, grid, items)
                             : attn::launch_join<256>(cfg, p, grid, items);
}

}  // namespace lin
