// Norms around a block with its gate, scale and residual (lin_step.h), in one
// pass over the row:
//   t = x rs(x; group) w_post act(gate),  h = residual + scale scale_w t,
//   y = h rs(h; row) w_pre,               rs(z; S) = (mean_S z^2 + eps)^(-1/2)
//
// Bound by HBM: every array is read or written once; a row lives in registers
// between its two norms. A row belongs to a set of whole warps (several rows
// share a CTA where rows are short), a thread to vectors of 8 consecutive
// channels, so group sums of 8 .. 256 channels are butterflies inside a warp
// and row sums add one barrier. Where 8-element vectors do not fit (an odd
// width or row start) a thread owns single channels instead.

#include "common.cuh"
#include "step_internal.h"

namespace lin {
namespace {

constexpr int kNormThreads = 512;   // most threads of one row
constexpr int kNormBlock = 256;     // rows shorter than this share a CTA

template <int DT, int VEC>
struct Raw;  // VEC elements as loaded
template <> struct Raw<LIN_F32, 8> {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    a = q[0], b = q[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
};
template <> struct Raw<LIN_BF16, 8> {
  uint4 a;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Raw<LIN_F32, 1> {
  float a;
  __device__ __forceinline__ void load(const void* p, int64_t i) { a = static_cast<const float*>(p)[i]; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = a; }
};
template <> struct Raw<LIN_BF16, 1> {
  uint16_t a;
  __device__ __forceinline__ void load(const void* p, int64_t i) { a = static_cast<const uint16_t*>(p)[i]; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = bf16_bits_to_f32(a); }
};

template <int DT>
__device__ __forceinline__ void put(void* p, int64_t i, const float (&v)[8]) {
  Vec8<DT>::store(static_cast<char*>(p) + i * (DT == LIN_BF16 ? 2 : 4), v);
}
template <int DT>
__device__ __forceinline__ void put(void* p, int64_t i, const float (&v)[1]) {
  store_elem(p, i, DT, v[0]);
}

__device__ __forceinline__ float warp_sum(float v, int width) {
  for (int o = width >> 1; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Sum over the `tpr` threads (whole warps) of one row; every thread of the
// block calls it. part: a row's 32 floats.
__device__ __forceinline__ float row_sum(float v, float* part, int tpr, int tx) {
  v = warp_sum(v, 32);
  if (tpr == 32) return v;
  if ((tx & 31) == 0) part[tx >> 5] = v;
  __syncthreads();
  const int warps = tpr >> 5;
  v = (tx & 31) < warps ? part[tx & 31] : 0.0f;
  v = warp_sum(v, 32);
  __syncthreads();
  return v;
}

// How the first norm's sums are taken: over the row, over aligned sets of
// lanes, or through shared memory.
enum GroupMode { kGroupNone = 0, kGroupRow = 1, kGroupLanes = 2, kGroupShared = 3 };

template <int XT, int IOT, int HT, int VEC, int NV>
__global__ void __launch_bounds__(VEC == 8 ? kNormThreads : 1024) block_norm_kernel(const lin_norm_args_t a, int mode, int shared_floats) {
  extern __shared__ float sm[];
  const int tpr = blockDim.x, tx = threadIdx.x;
  float* part = sm + threadIdx.y * 32;
  float* gsum = sm + blockDim.y * 32 + threadIdx.y * shared_floats;
  const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  const int C = a.channels;
  const bool live = row < a.rows;
  Raw<XT, VEC> rx[NV];
  Raw<IOT, VEC> rg[NV];
  Raw<HT, VEC> rr[NV];
  // every load of the row is in flight before the first sum
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * tpr + tx) * VEC;
    if (live && c < C) {
      rx[v].load(a.x, row * a.x_stride + c);
      if (a.gate) rg[v].load(a.gate, row * a.gate_stride + c);
      if (a.residual) rr[v].load(a.residual, row * a.residual_stride + c);
    }
  }
  float t[NV][VEC];
  float ss[NV], all = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const bool in = live && (v * tpr + tx) * VEC < C;
    if (in) rx[v].get(t[v]);
    ss[v] = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if (!in) t[v][i] = 0.0f;
      ss[v] = fmaf(t[v][i], t[v][i], ss[v]);
    }
    all += ss[v];
  }
  if (mode != kGroupNone) {
    const float inv = 1.0f / static_cast<float>(a.group);
    if (mode == kGroupRow) {
      const float s = rsqrtf(row_sum(all, part, tpr, tx) * inv + a.eps);
#pragma unroll
      for (int v = 0; v < NV; ++v) ss[v] = s;
    } else if (mode == kGroupLanes) {
#pragma unroll
      for (int v = 0; v < NV; ++v) ss[v] = rsqrtf(warp_sum(ss[v], a.group / VEC) * inv + a.eps);
    } else {
      // sums of single vectors, then a warp to each group in a fixed order
      const int per = a.group / VEC, groups = C / a.group, warps = tpr >> 5;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if ((v * tpr + tx) * VEC < C) gsum[v * tpr + tx] = ss[v];
      __syncthreads();
      for (int g = tx >> 5; g < groups; g += warps) {
        float s = 0.0f;
        for (int i = tx & 31; i < per; i += 32) s += gsum[g * per + i];
        s = warp_sum(s, 32);
        __syncwarp();
        if ((tx & 31) == 0) gsum[g * per] = rsqrtf(s * inv + a.eps);
      }
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int x = v * tpr + tx;
        if (x * VEC < C) ss[v] = gsum[x - x % per];
      }
    }
  }
  all = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * tpr + tx) * VEC;
    if (!live || c >= C) continue;
    float w[VEC];
    if (mode != kGroupNone) {
      Raw<IOT, VEC> rw;
      rw.load(a.w_post, c % a.group);
      rw.get(w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) t[v][i] *= ss[v] * w[i];
    }
    if (a.gate) {
      rg[v].get(w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float sig = __fdividef(1.0f, 1.0f + expf(-w[i]));  // 0 where expf overflows
        t[v][i] *= a.gate_act == LIN_ACT_SILU ? w[i] * sig : sig;
      }
    }
    if (a.scale_w) {
      Raw<IOT, VEC> rw;
      rw.load(a.scale_w, c);
      rw.get(w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) t[v][i] *= w[i];
    }
    if (a.residual) {
      rr[v].get(w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) t[v][i] = fmaf(a.scale, t[v][i], w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) t[v][i] *= a.scale;
    }
    if (a.h_out) put<HT>(a.h_out, row * a.h_stride + c, t[v]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) all = fmaf(t[v][i], t[v][i], all);
  }
  if (!a.w_pre) return;
  const float s = rsqrtf(row_sum(all, part, tpr, tx) / static_cast<float>(C) + a.eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * tpr + tx) * VEC;
    if (!live || c >= C) continue;
    Raw<IOT, VEC> rw;
    float w[VEC];
    rw.load(a.w_pre, c);
    rw.get(w);
#pragma unroll
    for (int i = 0; i < VEC; ++i) t[v][i] *= s * w[i];
    put<IOT>(a.y, row * a.y_stride + c, t[v]);
  }
}

bool vec_ok(const void* p, int64_t stride) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0);
}

template <int XT, int IOT, int HT, int VEC, int NV>
cudaError_t run(const lin_norm_args_t& a, int tpr, int rows, int mode, cudaStream_t s) {
  const int shared = mode == kGroupShared ? (a.channels + VEC - 1) / VEC : 0;
  const size_t smem = sizeof(float) * rows * (32 + shared);
  auto kern = block_norm_kernel<XT, IOT, HT, VEC, NV>;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const int64_t blocks = (a.rows + rows - 1) / rows;
  kern<<<static_cast<unsigned>(blocks), dim3(tpr, rows), smem, s>>>(a, mode, shared);
  return cudaGetLastError();
}

template <int XT, int IOT, int HT>
cudaError_t pick(const lin_norm_args_t& a, cudaStream_t s) {
  const bool vec = a.channels % 8 == 0 && (!a.w_post || a.group % 8 == 0) && vec_ok(a.x, a.x_stride) &&
                   vec_ok(a.gate, a.gate_stride) && vec_ok(a.residual, a.residual_stride) &&
                   vec_ok(a.h_out, a.h_stride) && vec_ok(a.y, a.y_stride) && vec_ok(a.w_post, 0) &&
                   vec_ok(a.scale_w, 0) && vec_ok(a.w_pre, 0);
  const int per = vec ? 8 : 1;
  const int vecs = (a.channels + per - 1) / per;
  const int most = vec ? kNormThreads : 1024;
  // the fewest vectors per thread, of 1, 2, 4, 8 (and 32 single channels)
  int nv = 1;
  while (vecs > most * nv) nv *= 2;
  const int tpr = ((vecs + nv - 1) / nv + 31) / 32 * 32;
  const int rows = tpr >= kNormBlock ? 1 : kNormBlock / tpr;
  int mode = kGroupNone;
  if (a.w_post) {
    const int lanes = a.group / per;
    mode = a.group == a.channels ? kGroupRow
           : lanes <= 32 && (lanes & (lanes - 1)) == 0 ? kGroupLanes : kGroupShared;
  }
  if (vec) {
    if (nv == 1) return run<XT, IOT, HT, 8, 1>(a, tpr, rows, mode, s);
    if (nv == 2) return run<XT, IOT, HT, 8, 2>(a, tpr, rows, mode, s);
    if (nv == 4) return run<XT, IOT, HT, 8, 4>(a, tpr, rows, mode, s);
    return run<XT, IOT, HT, 8, 8>(a, tpr, rows, mode, s);
  }
  if (nv <= 4) {
    const int t4 = ((vecs + 3) / 4 + 31) / 32 * 32;
    return run<XT, IOT, HT, 1, 4>(a, t4, t4 >= kNormBlock ? 1 : kNormBlock / t4, mode, s);
  }
  return run<XT, IOT, HT, 1, 32>(a, 1024, 1, mode, s);
}

}  // namespace

cudaError_t launch_block_norm(const lin_norm_args_t& a, cudaStream_t s) {
  const bool x32 = a.x_dtype == LIN_F32, i32 = a.io_dtype == LIN_F32, h32 = a.h_dtype == LIN_F32;
  if (x32)
    return i32 ? (h32 ? pick<LIN_F32, LIN_F32, LIN_F32>(a, s) : pick<LIN_F32, LIN_F32, LIN_BF16>(a, s))
               : (h32 ? pick<LIN_F32, LIN_BF16, LIN_F32>(a, s) : pick<LIN_F32, LIN_BF16, LIN_BF16>(a, s));
  return i32 ? (h32 ? pick<LIN_BF16, LIN_F32, LIN_F32>(a, s) : pick<LIN_BF16, LIN_F32, LIN_BF16>(a, s))
             : (h32 ? pick<LIN_BF16, LIN_BF16, LIN_F32>(a, s) : pick<LIN_BF16, LIN_BF16, LIN_BF16>(a, s));
}

}  // namespace lin
