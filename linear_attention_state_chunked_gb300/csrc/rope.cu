// Rotary positions of new queries and keys, with the append to a paged cache
// (lin_prompt.h):
//   (x, y) -> m (x cos a - y sin a, y cos a + x sin a),  a = position inv_freq,
// over the pairs of the first rot_dim channels of every head; the turned keys, and the
// values as they are, go straight to their rows of the cache.
//
// Bound by HBM for a prompt (every row read and written once: 32,768 tokens of 16 + 2 heads
// of 128 in bf16 62.5 us, 0.79 of a copy's bandwidth) and by one launch's chain of dependent
// loads for a step (256 tokens 3.3 us). A CTA takes a few tokens: it makes their cosines and
// sines once, in shared memory, for all heads, and looks their rows up once; then a
// thread moves an item, two 16-byte chunks that hold each other's partners. Where rot_dim
// ends inside an item a thread moves one chunk, whose partners are its own (pairs: 100 of
// 128 channels 91 us) or come from the row's copy in shared memory (halves: 124 us).
//
// The angle. In fp32 position * inv_freq is off by up to 2^-24 of itself, 0.06 at a
// million. Here it is a fraction of a turn in 64-bit fixed point: inv_freq / 2 pi has an
// error of about 2^-64 turns, the product with the position wraps by itself, and what is
// left of it is rounded once to fp32, a relative 2^-24 of at most half a turn.

#include "common.cuh"
#include "prompt_internal.h"

namespace lin {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 8;   // most tokens of a CTA
constexpr int kRopeMaxDim = 256;

enum RopeMode { kHalf = 0, kPairs = 1, kAny = 2 };  // kAny: rot_dim that does not end with an item

// inv_freq / 2 pi in units of 2^-64 turns, modulo a turn.
__device__ __forceinline__ uint64_t turns_of(float inv_freq) {
  constexpr uint64_t kTwoPi = 0x28be60db9391054aull;  // 2^64 / 2 pi
  const uint32_t bits = __float_as_uint(inv_freq);
  const int exp = static_cast<int>((bits >> 23) & 255);
  const uint64_t m = exp ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int up = (exp ? exp : 1) - 150;  // inv_freq = m 2^up
  const uint64_t lo = m * kTwoPi, hi = __umul64hi(m, kTwoPi);
  uint64_t t;
  if (up >= 64)
    t = 0;
  else if (up >= 0)
    t = lo << up;
  else if (up > -64)
    t = (lo >> -up) | (hi << (64 + up));
  else
    t = up > -128 ? hi >> (-up - 64) : 0;
  return bits >> 31 ? 0 - t : t;
}

template <int DT>
struct Chunk {  // 16 bytes
  static constexpr int V = DT == LIN_BF16 ? 8 : 4;
  static __device__ __forceinline__ void get(const uint4& u, float (&v)[V]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == LIN_BF16) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        v[i] = __uint_as_float(w[i]);
      }
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&v)[V]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == LIN_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[i] = __float_as_uint(v[i]);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// blockDim = (items of a head, heads side by side). A token's rows: its nq queries, nk
// keys and nv values.
template <int DT, int MODE>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const lin_kv_cache_t c, const lin_rope_args_t a, int per_cta, int nq, int nk, int nv) {
  constexpr int V = Chunk<DT>::V;
  __shared__ float2 s_cs[kRopeTokens * kRopeMaxDim / 2];
  __shared__ int64_t s_off[kRopeTokens];  // of the token's row in the cache, or -1
  __shared__ int s_live[kRopeTokens];
  __shared__ uint4 s_row[MODE == kAny ? 2 * kRopeThreads : 1];  // rows of this step and the last
  const int tx = threadIdx.x, ty = threadIdx.y, tid = ty * blockDim.x + tx, nt = blockDim.x * blockDim.y;
  const int t0 = blockIdx.x * per_cta, count = min(per_cta, a.tokens - t0);
  const int half = a.rot_dim >> 1;

  if (tid < count) {
    const int pos = a.position[t0 + tid];
    s_live[tid] = pos >= 0;
    int64_t off = -1;
    if (nv > 0 && pos >= 0) {
      const int64_t slot = a.slot[t0 + tid];
      const int64_t page = slot / c.page_size;
      if (slot >= 0 && page < c.num_pages)
        off = a.layer * c.layer_stride + page * c.page_stride + (slot - page * c.page_size) * c.token_stride;
      else if (slot >= 0)
        report(a.status, LIN_ST_BAD_PAGE);
    }
    s_off[tid] = off;
  }
  for (int i = tid; i < count * half; i += nt) {
    const int t = i / half, pair = i - t * half;
    const int64_t turn = static_cast<int64_t>(turns_of(a.inv_freq[pair]) * static_cast<uint64_t>(int64_t(a.position[t0 + t])));
    float s, co;
    sincospif(static_cast<float>(turn) * 0x1p-63f, &s, &co);
    s_cs[i] = make_float2(co * a.scale, s * a.scale);
  }
  __syncthreads();

  const int rows = nq + nk + nv, many = count * rows;
  const int row_bytes = a.head_dim * (DT == LIN_BF16 ? 2 : 4);
  // chunks of this thread's item and the pair of the first one's first channel
  int c0, c1, pair;
  bool turned, second = true;
  if constexpr (MODE == kHalf) {
    turned = tx * V < half;
    c0 = turned ? tx : 2 * tx;
    c1 = turned ? tx + half / V : 2 * tx + 1;
    pair = tx * V;
  } else if constexpr (MODE == kPairs) {
    c0 = 2 * tx, c1 = c0 + 1;
    turned = c0 * V < a.rot_dim;
    pair = tx * V;
  } else {
    c0 = c1 = tx, pair = 0;
    turned = tx * V < a.rot_dim;
    second = false;
  }
  // every thread takes as many steps: kAny has barriers
  int t = 0, row = ty, buf = 0;
  for (int x = 0; x < many; x += blockDim.y) {
    while (row >= rows) row -= rows, ++t;
    const bool live = x + ty < many && s_live[t];
    const int what = row < nq ? 0 : row < nq + nk ? 1 : 2;
    const int head = what == 0 ? row : what == 1 ? row - nq : row - nq - nk;
    const char* src = static_cast<const char*>(what == 0 ? a.q : what == 1 ? a.k : a.v) +
                      int64_t(t0 + t) * (what == 0 ? a.q_stride : what == 1 ? a.k_stride : a.v_stride) + int64_t(head) * row_bytes;
    uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
    if (live) {
      u0 = __ldcs(reinterpret_cast<const uint4*>(src) + c0);
      if (second) u1 = __ldcs(reinterpret_cast<const uint4*>(src) + c1);
    }
    const uint4* mine = s_row;  // the row's chunks
    if constexpr (MODE == kAny) {
      if (!a.interleaved) {  // (or partners lie in the thread's own chunk)
        uint4* at = s_row + (buf * blockDim.y + ty) * blockDim.x;
        at[tx] = u0;
        mine = at;
        buf ^= 1;
        __syncthreads();
      }
    }
    if (live && turned && what < 2) {
      float v0[V], v1[V], w0[V], w1[V];
      Chunk<DT>::get(u0, v0);
      Chunk<DT>::get(u1, v1);
      const float2* cs = s_cs + t * half + pair;
      if constexpr (MODE == kHalf) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 y = cs[i];
          w0[i] = v0[i] * y.x - v1[i] * y.y;
          w1[i] = v1[i] * y.x + v0[i] * y.y;
        }
      } else if constexpr (MODE == kPairs) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const float2 y = cs[i], z = cs[V / 2 + i];
          w0[2 * i] = v0[2 * i] * y.x - v0[2 * i + 1] * y.y;
          w0[2 * i + 1] = v0[2 * i + 1] * y.x + v0[2 * i] * y.y;
          w1[2 * i] = v1[2 * i] * z.x - v1[2 * i + 1] * z.y;
          w1[2 * i + 1] = v1[2 * i + 1] * z.x + v1[2 * i] * z.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int ch = tx * V + i;
          w0[i] = v0[i];
          if (ch < a.rot_dim) {
            const bool lower = a.interleaved ? !(i & 1) : ch < half;
            const float2 y = cs[a.interleaved ? ch >> 1 : lower ? ch : ch - half];
            const float z = a.interleaved ? v0[i ^ 1] : load_elem(mine, lower ? ch + half : ch - half, DT);
            w0[i] = lower ? v0[i] * y.x - z * y.y : v0[i] * y.x + z * y.y;
          }
        }
      }
      u0 = Chunk<DT>::put(w0);
      if (second) u1 = Chunk<DT>::put(w1);
    }
    if (live) {
      char* out = what == 0 ? static_cast<char*>(a.q_out) : what == 1 ? static_cast<char*>(a.k_out) : nullptr;
      if (out) {
        out += int64_t(t0 + t) * (what == 0 ? a.q_out_stride : a.k_out_stride) + int64_t(head) * row_bytes;
        reinterpret_cast<uint4*>(out)[c0] = u0;
        if (second) reinterpret_cast<uint4*>(out)[c1] = u1;
      }
      if (what > 0 && s_off[t] >= 0) {
        char* to = static_cast<char*>(what == 1 ? c.k : c.v) + s_off[t] + head * c.head_stride;
        reinterpret_cast<uint4*>(to)[c0] = u0;
        if (second) reinterpret_cast<uint4*>(to)[c1] = u1;
      }
    }
    row += blockDim.y;
  }
}

template <int DT>
cudaError_t run_rope(const lin_kv_cache_t* cache, const lin_rope_args_t& a, cudaStream_t s) {
  constexpr int V = Chunk<DT>::V;
  const int nq = a.q_out ? a.num_q_heads : 0, nk = a.k_out || cache ? a.num_k_heads : 0, nv = cache ? a.num_k_heads : 0;
  const bool items = a.head_dim % (2 * V) == 0 && a.rot_dim % (2 * V) == 0;
  const int tx = items ? a.head_dim / (2 * V) : a.head_dim / V;
  const int ty = kRopeThreads / tx;
  // tokens of a CTA: as many as leave several CTAs for every SM
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) sms = device_sm_count(dev);
  if (sms <= 0) sms = 152;  // no device: the size of a GB300
  int per_cta = a.tokens / (8 * sms);
  per_cta = per_cta < 1 ? 1 : per_cta > kRopeTokens ? kRopeTokens : per_cta;
  lin_kv_cache_t c = {};
  if (cache) c = *cache;
  const int blocks = (a.tokens - 1) / per_cta + 1;
  auto kern = !items ? rope_kernel<DT, kAny> : a.interleaved ? rope_kernel<DT, kPairs> : rope_kernel<DT, kHalf>;
  kern<<<blocks, dim3(tx, ty), 0, s>>>(c, a, per_cta, nq, nk, nv);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const lin_kv_cache_t* cache, const lin_rope_args_t& a, cudaStream_t s) {
  return a.dtype == LIN_BF16 ? run_rope<LIN_BF16>(cache, a, s) : run_rope<LIN_F32>(cache, a, s);
}

}  // namespace lin
