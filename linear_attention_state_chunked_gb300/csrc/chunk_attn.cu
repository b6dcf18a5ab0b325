// Chunk attention over a paged key-value cache (lin_prompt.h): the join of split items
// and the host side. The main kernels are in chunk_umma.cuh and chunk_mma.cuh.

#include <cudaTypedefs.h>

#include "chunk_common.cuh"

namespace lin {
namespace chunk {
namespace {

constexpr int kJoinWarps = 8;
constexpr int kJoinRows = 32;      // rows of a block: a lane each
constexpr int kManyParts = 8;      // of an item: see launch_attn_chunk
constexpr int kShareThreads = 512;

// Whether the batch's items are taken one by one: where the last one ends in time
// (chunk_common.cuh). Of a request's last head that is the item from which on the items get
// shorter by more (m) than passes until their turn (their units / CTAs). One block.
__global__ void __launch_bounds__(kShareThreads) share_kernel(const Plan p) {
  __shared__ int64_t s_sum[kShareThreads / 32], s_late[kShareThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, batch = p.a.batch;
  const int span = (batch + kShareThreads - 1) / kShareThreads;
  const int r0 = min(batch, tid * span), r1 = min(batch, r0 + span);
  // units of this thread's requests, and the last end with none before them, in units x CTAs
  int64_t mine = 0, late = 0;
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    const Req q = request(p, r, false);
    if (q.items == 0) continue;
    const int64_t turn = int64_t(p.grid) - 1 - q.base / p.m;
    const int j = static_cast<int>(max(int64_t(0), min(int64_t(q.items) - 1, turn)));
    mine += units_before(p, q, q.items) * p.heads;
    late = max(late, mine - units_before(p, q, j + 1) + (keys_of(p, q, j) + p.item_cost) * p.grid);
  }
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += x;
  }
  late += upto - mine;
#pragma unroll
  for (int o = 16; o; o >>= 1) late = max(late, __shfl_xor_sync(~0u, late, o));
  if (lane == 31) s_sum[warp] = upto, s_late[warp] = late;
  __syncthreads();
  if (tid == 0) {
    int64_t total = 0, last = 0;
#pragma unroll
    for (int x = 0; x < kShareThreads / 32; ++x) last = max(last, total + s_late[x]), total += s_sum[x];
    p.ticket[0] = 0;
    p.ticket[1] = last <= total + total / kManyItems;
  }
}

// The x-th of the ranges whose last item goes on past them, by a whole warp; false
// where there are fewer.
__device__ __forceinline__ bool find_split(const Plan& p, int x, int& range, Split& s) {
  const int lane = threadIdx.x & 31;
  for (int c = 0; c < p.grid; c += 32) {
    const uint32_t some = __ballot_sync(~0u, c + lane < p.grid && p.split[c + lane].parts > 0);
    const int n = __popc(some);
    if (x < n) {
      range = c + static_cast<int>(__fns(some, 0, x + 1));
      s = p.split[range];
      return true;
    }
    x -= n;
  }
  return false;
}

// The item that begins in range c and goes on past it has the parts, in token order,
// 2c + 1 and then 2c' of the ranges c' = c + 1, ... A lane joins a row, so that a part's
// loads are whole lines. WP warps share the parts (each takes every WP-th, and they are
// added in a fixed order), the others the channels. Bound by the latency of dependent
// loads: split, sums, values.
template <int D, int WP>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Plan p) {
  constexpr int WC = kJoinWarps / WP;                   // warps side by side
  constexpr int CG = WP == 1 ? D / 4 / WC : 4;          // a warp's groups of 4 channels
  constexpr int CH = WC * CG * 4;                       // a block's channels
  __shared__ float s_out[kJoinRows][CH + 4];
  __shared__ float s_sum[kJoinRows];
  __shared__ float4 s_part[WP > 1 ? WP : 1][CG][kJoinRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wp = warp % WP, wc = warp / WP;
  if (one_by_one(p)) return;
  Split s;
  int c;
  if (!find_split(p, blockIdx.x, c, s)) return;
  const int row0 = blockIdx.y * kJoinRows, row = row0 + lane;
  if (row0 >= s.tokens * p.bheads) return;
  const int ch0 = blockIdx.z * CH;
  auto part = [&](int i) { return int64_t(2) * c + (i == 0 ? 1 : 2 * i); };
  float top = -INFINITY;
  bool out = false;
#pragma unroll 8
  for (int i = 0; i < s.parts; ++i) {
    const float2 ml = p.part_ml[part(i) * p.rows + row];
    top = fmaxf(top, ml.x);
    out |= ml.y == attn::kLeftOut;
  }
  float sum = 0.0f;
  float4 v[CG];
#pragma unroll
  for (int k = 0; k < CG; ++k) v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int i = wp; i < s.parts; i += WP) {
    const float2 ml = p.part_ml[part(i) * p.rows + row];
    const float4* src = reinterpret_cast<const float4*>(p.part) + (part(i) * (D / 4) + ch0 / 4 + wc * CG) * p.rows + row;
    float4 y[CG];
#pragma unroll
    for (int k = 0; k < CG; ++k) y[k] = src[int64_t(k) * p.rows];
    // 0 where a part saw nothing (a NaN sum goes on)
    const float f = ml.y == 0.0f ? 0.0f : ml.x == top ? 1.0f : attn::exp2_fast(ml.x - top);
    sum = fmaf(f, ml.y, sum);
#pragma unroll
    for (int k = 0; k < CG; ++k) {
      v[k].x = fmaf(f, y[k].x, v[k].x), v[k].y = fmaf(f, y[k].y, v[k].y);
      v[k].z = fmaf(f, y[k].z, v[k].z), v[k].w = fmaf(f, y[k].w, v[k].w);
    }
  }
  if constexpr (WP > 1) {
    s_out[lane][warp] = sum;  // (joined below)
#pragma unroll
    for (int k = 0; k < CG; ++k) s_part[wp][k][lane] = v[k];
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int x = 0; x < WP; ++x) sum += s_out[lane][x];
#pragma unroll
    for (int k = 0; k < CG; ++k) {
      v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int x = 0; x < WP; ++x) {
        const float4 y = s_part[x][k][lane];
        v[k].x += y.x, v[k].y += y.y, v[k].z += y.z, v[k].w += y.w;
      }
    }
    __syncthreads();
  }
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (wp == 0) {
#pragma unroll
    for (int k = 0; k < CG; ++k)
      *reinterpret_cast<float4*>(&s_out[lane][(wc * CG + k) * 4]) = make_float4(v[k].x * f, v[k].y * f, v[k].z * f, v[k].w * f);
  }
  if (warp == 0) s_sum[lane] = out ? attn::kLeftOut : 0.0f;
  __syncthreads();
  // rows as they lie in the outputs
  constexpr int PER = CH / 4;  // threads of a row
  for (int x = threadIdx.x; x < kJoinRows * PER; x += kJoinWarps * 32) {
    const int r = x / PER, q = row0 + r, t = token_of(p, q), h = q - t * p.bheads;
    if (t >= s.tokens || h >= s.heads || s_sum[r] == attn::kLeftOut) continue;  // left out after a wait that ran out
    const float4 y = *reinterpret_cast<const float4*>(&s_out[r][x % PER * 4]);
    const int64_t at = (int64_t(s.row0 + t) * p.a.num_q_heads + s.head0 + h) * D + ch0 + x % PER * 4;
    if (p.a.out_dtype == LIN_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.a.out) + at) = y;
    } else {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.a.out) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
  }
}

// Which kernel a call takes.
struct Shape {
  bool umma;
  int rows, tk, ctas, item_cost;
};

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) sms = device_sm_count(dev);
  return sms > 0 ? sms : 152;  // no device: the size of a GB300
}

// Whether an item has two row tiles of 128 (heads of 64 and 128): where a request has more
// rows than one tile, and the call more work than `kTwoFrom` tiles of 128 x 128 for each SM,
// by what the host knows of it. Two read a tile of K and V for twice the rows and share the
// unit better, one makes more and shorter items. Heads of 128, one against two: 64 tokens
// after 1,000 18.3 and 21.7 us, 256 after 8,000 33.9 and 40.9, 512 after 8,000 46.8 and
// 45.1, 32 x 64 after 4,000 89 and 76, 32 after 400,000 105 and 96.
constexpr int kTwoFrom = 20;

bool two_tiles(const lin_kv_cache_t& c, const lin_attn_chunk_args_t& a) {
  const int64_t rows = int64_t(a.tokens) * (a.num_q_heads / c.num_kv_heads);  // of a kv head
  const double keys = double(a.max_pages) * c.page_size;
  return rows > 128 * int64_t(a.batch) && double(rows) * c.num_kv_heads * keys > double(kTwoFrom) * 128 * 128 * sm_count();
}

// item_cost: what an item's start and end take, in keys (tensor-memory kernel, 2 prompts of
// 4,096 tokens: as 96 keys 183 us, as 192 156, as 320 140, as 384 137).
Shape shape_of(const lin_kv_cache_t& c, int out_dtype, bool two) {
  if (c.dtype == LIN_BF16 && out_dtype == LIN_BF16) {
    two = two && c.head_dim <= 128;
    return {true, two ? 256 : 128, !two ? 128 : c.head_dim == 64 ? 96 : 80, 1, 384};
  }
  const int row_bytes = c.head_dim * dtype_size(c.dtype);
  return {false, 64, row_bytes >= 512 ? 16 : 32, c.head_dim == 256 ? 1 : c.head_dim == 128 ? 2 : 3, c.head_dim == 256 ? 128 : 64};
}

size_t bytes_of(const lin_kv_cache_t& c, const Shape& f) {
  const size_t grid = size_t(sm_count()) * f.ctas;
  return 2 * grid * f.rows * (c.head_dim * sizeof(float) + sizeof(float2)) + grid * sizeof(Split) + 16;
}

// Granlund and Montgomery's division by an invariant: s = ceil(log2 d),
// mul = floor(2^32 (2^s - d) / d) + 1
void divide_by(int64_t d, uint32_t& mul, uint32_t& shift) {
  shift = 0;
  while ((int64_t(1) << shift) < d) ++shift;
  mul = static_cast<uint32_t>((((uint64_t(1) << shift) - d) << 32) / d + 1);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }
  return fn;
}

// A layer's K or V as [page][head][token][channel], in boxes of 64 channels x `box` tokens.
// False where the strides are none that a tensor map takes.
bool encode(CUtensorMap* map, const lin_kv_cache_t& c, void* base, int layer, int box) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(c.head_dim) * 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.num_kv_heads), static_cast<cuuint64_t>(c.num_pages)};
  // (the stride of an axis of one is not looked at)
  const cuuint64_t strides[3] = {c.page_size > 1 ? static_cast<cuuint64_t>(c.token_stride) : row,
                                 c.num_kv_heads > 1 ? static_cast<cuuint64_t>(c.head_stride) : row,
                                 c.num_pages > 1 ? static_cast<cuuint64_t>(c.page_stride) : row};
  const cuuint32_t boxes[4] = {64, static_cast<cuuint32_t>(box), 1, 1}, ones[4] = {1, 1, 1, 1};
  char* at = static_cast<char*>(base) + (c.num_layers > 1 ? layer * c.layer_stride : 0);
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, at, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The packed queries as [token][head][channel], in boxes of 64 channels of an item's heads.
bool encode_q(CUtensorMap* map, const lin_kv_cache_t& c, const lin_attn_chunk_args_t& a, int heads, int tokens) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(c.head_dim) * 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(a.num_q_heads), static_cast<cuuint64_t>(a.tokens)};
  const cuuint64_t strides[2] = {row, a.tokens > 1 ? static_cast<cuuint64_t>(a.token_stride) : row * a.num_q_heads};
  const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)}, ones[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_join(const Plan& p, int64_t items, int rows, cudaStream_t s) {
  const unsigned x = static_cast<unsigned>(items < p.grid ? items : p.grid), y = (rows + kJoinRows - 1) / kJoinRows;
  if (items * kManyParts > p.grid)
    join_kernel<D, 1><<<dim3(x, y, 1), kJoinWarps * 32, 0, s>>>(p);
  else
    join_kernel<D, kJoinWarps><<<dim3(x, y, D / 16), kJoinWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace chunk

size_t chunk_need(const lin_kv_cache_t& c, const lin_attn_chunk_args_t& a) {
  return chunk::bytes_of(c, chunk::shape_of(c, a.out_dtype, chunk::two_tiles(c, a)));
}

size_t chunk_workspace(const lin_kv_cache_t& c, const lin_attn_chunk_args_t&) {
  // of every kernel that a call over this cache may take
  size_t most = 0;
  for (const int out : {LIN_BF16, LIN_F32})
    for (const bool two : {false, true}) {
      const size_t n = chunk::bytes_of(c, chunk::shape_of(c, out, two));
      if (n > most) most = n;
    }
  return most;
}

cudaError_t launch_attn_chunk(const lin_kv_cache_t& c, const lin_attn_chunk_args_t& a, void* ws, cudaStream_t s) {
  const chunk::Shape f = chunk::shape_of(c, a.out_dtype, chunk::two_tiles(c, a));
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
  p.negate = !(a.scale < 0.0f) ? 0u : c.dtype == LIN_BF16 ? 0x80008000u : 0x80000000u;
  chunk::divide_by(c.page_size, p.page_mul, p.page_shift);
  chunk::divide_by(p.bheads, p.bhead_mul, p.bhead_shift);
  char* w = static_cast<char*>(ws);
  p.part = reinterpret_cast<float*>(w);
  w += size_t(2) * p.grid * p.rows * c.head_dim * sizeof(float);
  p.part_ml = reinterpret_cast<float2*>(w);
  w += size_t(2) * p.grid * p.rows * sizeof(float2);
  p.split = reinterpret_cast<chunk::Split*>(w);
  w += size_t(p.grid) * sizeof(chunk::Split);
  // Items of the batch at most. Where it could have many for a CTA, a first launch tells by
  // the lengths whether they are taken one by one.
  const int64_t items = p.items = int64_t(p.heads) * (a.tokens / p.m + a.batch);
  p.ticket = f.umma && items >= int64_t(chunk::kManyItems) * p.grid && items < (1 << 30) ? reinterpret_cast<int*>(w) : nullptr;
  if (p.ticket) {
    chunk::share_kernel<<<1, chunk::kShareThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  p.box = p.q_box = 0;
  cudaError_t e;
  if (f.umma) {
    chunk::Maps m = {};
    int box = 32;  // of whole pages and tiles
    while (box >= 8 && (c.page_size % box || p.tk % box)) box /= 2;
    if (box >= 8 && chunk::encode(&m.k, c, c.k, a.layer, box) && chunk::encode(&m.v, c, c.v, a.layer, box)) p.box = box;
    // a row tile of whole tokens is one box of the queries
    if (128 % p.bheads == 0 && chunk::encode_q(&m.q, c, a, p.bheads, 128 / p.bheads)) p.q_box = 128 / p.bheads;
    e = c.head_dim == 64    ? chunk::launch_umma_d64(p, m, s)
        : c.head_dim == 128 ? chunk::launch_umma_d128(p, m, s)
                            : chunk::launch_umma_d256(p, m, s);
  } else {
    e = c.head_dim == 64    ? chunk::launch_mma_d64(p, s)
        : c.head_dim == 128 ? chunk::launch_mma_d128(p, s)
                            : chunk::launch_mma_d256(p, s);
  }
  if (e != cudaSuccess) return e;
  // Few items have many parts each (one request's last tokens over a long cache), which
  // the warps of a block then share (8 tokens after 100,000: 39 us, rows alone 65; 32 x 32
  // after 4,000, the other way: 52, and 84 with shared parts).
  const int64_t most = int64_t(a.tokens) * p.bheads;
  const int rows = most < p.rows ? static_cast<int>(most) : p.rows;
  return c.head_dim == 64    ? chunk::launch_join<64>(p, items, rows, s)
         : c.head_dim == 128 ? chunk::launch_join<128>(p, items, rows, s)
                             : chunk::launch_join<256>(p, items, rows, s);
}

}  // namespace lin
