// Norms around a block with its gate, scale and residual (lin_step.h), in one
// pass over the row:
//   t = x rs(x; group) w_post act(gate),  h = residual + scale scale_w t,
//   y = h rs(h; row) w_pre,               rs(z; S) = (mean_S z^2 + eps)^(-1/2)
//
// Bound by HBM: every array is read or written once; a row lives in registers
// between its two norms. A row belongs to a set of whole warps (several rows
// share a CTA where rows are short), a thread to vectors of 8 consecutive
// channels, so group sums of 8 .. 256 channels are butterflies inside a warp
// and row sums add one barrier. Rows of an odd width start anywhere in a vector
// of 8, but all arrays of one call alike: there the vectors are shifted (channel
// c0 - shift on), and only a row's first and last are taken by elements. Where
// the arrays differ in that, or groups do not end with vectors, a thread owns
// single channels instead.
// 32,768 rows of 32 x 128 channels, fp32 in, gate and output bf16: 171 us, 0.93 of
// the measured copy bandwidth; 4,097 rows of 1,533 (shifted): 15.5 us, by single
// channels 27.9; one row of 4096: 2.8 us, the launch.
// Far from that bound: single channels of rows of more than 4096, 32 to a thread, which
// spill (4,096 rows of 6,000 in groups of 1,500, bf16: 920 us for a floor of 29), and
// rows of more than 16,384 channels, 8 vectors to a thread (1,024 rows of 20,480:
// 74 us for 25).

#include "common.cuh"
#include "step_internal.h"

namespace lin {
namespace {

constexpr int kNormThreads = 512;   // most threads of one row
constexpr int kNormBlock = 256;     // rows shorter than this share a CTA
constexpr int kManyRows = 2048;     // rows that fill the GPU several times over

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

// The elements c0 .. c0 + 7 of a row at `p` + `row` that lie in [0, C), 0 elsewhere.
template <int DT>
__device__ __forceinline__ void load_part(Raw<DT, 8>& r, const void* p, int64_t row, int c0, int C) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = c0 + i >= 0 && c0 + i < C ? load_elem(p, row + c0 + i, DT) : 0.0f;
  Vec8<DT>::store(&r, v);  // exact: the values are of that type
}
template <int DT>
__device__ __forceinline__ void put_part(void* p, int64_t row, int c0, int C, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c0 + i >= 0 && c0 + i < C) store_elem(p, row + c0 + i, DT, v[i]);
}

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

// 1 / (1 + 2^(-x log2 e)) in four instructions (the gate alone would else bound a
// long prompt's call by its instructions): off by about (|x| + 4) 2^-24 of itself,
// from the exponent's product; 0 below x = -87.3, where it would be less than the
// smallest normal number (and SiLU, 1e-36 and less, 0 with it).
__device__ __forceinline__ float sigmoid(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// How the first norm's sums are taken: over the row, over aligned sets of
// lanes, or through shared memory.
enum GroupMode { kGroupNone = 0, kGroupRow = 1, kGroupLanes = 2, kGroupShared = 3 };

// VEC 8 with SH: shifted vectors (the group is the row, if any).
template <int XT, int IOT, int HT, int VEC, int NV, bool SH>
__global__ void __launch_bounds__(VEC == 8 ? kNormThreads : 1024)
block_norm_kernel(const lin_norm_args_t a, int mode, int shared_floats) {
  extern __shared__ float sm[];
  const int tpr = blockDim.x, tx = threadIdx.x;
  float* part = sm + threadIdx.y * 32;
  float* gsum = sm + blockDim.y * 32 + threadIdx.y * shared_floats;
  const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  const int C = a.channels;
  const bool live = row < a.rows;
  const int shift = SH ? static_cast<int>((row * a.x_stride) & 7) : 0;
  auto chan = [&](int v) { return (v * tpr + tx) * VEC - shift; };
  auto in = [&](int c) { return live && c < C && (!SH || c > -VEC); };
  auto whole = [&](int c) { return !SH || (c >= 0 && c + VEC <= C); };
  Raw<XT, VEC> rx[NV];
  Raw<IOT, VEC> rg[NV];
  Raw<HT, VEC> rr[NV];
  // every load of the row is in flight before the first sum
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = chan(v);
    if (!in(c)) continue;
    if (whole(c)) {
      rx[v].load(a.x, row * a.x_stride + c);
      if (a.gate) rg[v].load(a.gate, row * a.gate_stride + c);
      if (a.residual) rr[v].load(a.residual, row * a.residual_stride + c);
    } else if constexpr (SH) {
      load_part(rx[v], a.x, row * a.x_stride, c, C);
      if (a.gate) load_part(rg[v], a.gate, row * a.gate_stride, c, C);
      if (a.residual) load_part(rr[v], a.residual, row * a.residual_stride, c, C);
    }
  }
  float t[NV][VEC];
  float ss[NV], all = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const bool mine = in(chan(v));
    if (mine) rx[v].get(t[v]);
    ss[v] = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if (!mine) t[v][i] = 0.0f;
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
  // VEC weights from channel c on
  auto weights = [&](const void* w, int c, float (&out)[VEC]) {
    if constexpr (SH) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) out[i] = c + i >= 0 && c + i < C ? load_elem(w, c + i, IOT) : 0.0f;
    } else {
      Raw<IOT, VEC> rw;
      rw.load(w, c);
      rw.get(out);
    }
  };
  all = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = chan(v);
    if (!in(c)) continue;
    float w[VEC];
    if (mode != kGroupNone) {
      // groups of whole lanes are powers of two wide
      weights(a.w_post, mode == kGroupRow ? c : mode == kGroupLanes ? c & (a.group - 1) : c % a.group, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) t[v][i] *= ss[v] * w[i];
    }
    if (a.gate) {
      rg[v].get(w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float sig = sigmoid(w[i]);
        t[v][i] *= a.gate_act == LIN_ACT_SILU ? w[i] * sig : sig;
      }
    }
    if (a.scale_w) {
      weights(a.scale_w, c, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) t[v][i] *= w[i];
    }
    if (a.residual) {
      rr[v].get(w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) t[v][i] = fmaf(a.scale, t[v][i], w[i]);
    } else if (a.scale != 1.0f) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) t[v][i] *= a.scale;
    }
    if (a.h_out) {
      if (whole(c))
        put<HT>(a.h_out, row * a.h_stride + c, t[v]);
      else if constexpr (SH)
        put_part<HT>(a.h_out, row * a.h_stride, c, C, t[v]);
    }
    if (a.w_pre) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) all = fmaf(t[v][i], t[v][i], all);
    }
  }
  if (!a.w_pre) return;
  const float s = rsqrtf(row_sum(all, part, tpr, tx) / static_cast<float>(C) + a.eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = chan(v);
    if (!in(c)) continue;
    float w[VEC];
    weights(a.w_pre, c, w);
#pragma unroll
    for (int i = 0; i < VEC; ++i) t[v][i] *= s * w[i];
    if (whole(c))
      put<IOT>(a.y, row * a.y_stride + c, t[v]);
    else if constexpr (SH)
      put_part<IOT>(a.y, row * a.y_stride, c, C, t[v]);
  }
}

bool vec_ok(const void* p, int64_t stride) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0);
}
// the row starts at the same place of a vector of 8 as x's
bool shift_ok(const void* p, int64_t stride, int dt, int64_t x_stride) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (8 * dtype_size(dt)) == 0 && (stride - x_stride) % 8 == 0);
}

template <int XT, int IOT, int HT, int VEC, int NV, bool SH = false>
cudaError_t run(const lin_norm_args_t& a, int tpr, int mode, cudaStream_t s) {
  const int rows = tpr >= kNormBlock ? 1 : kNormBlock / tpr;
  const int shared = mode == kGroupShared ? (a.channels + VEC - 1) / VEC : 0;
  const size_t smem = sizeof(float) * rows * (32 + shared);
  auto kern = block_norm_kernel<XT, IOT, HT, VEC, NV, SH>;
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
  const bool shift = !vec && (!a.w_post || a.group == a.channels) && shift_ok(a.x, a.x_stride, XT, a.x_stride) &&
                     shift_ok(a.gate, a.gate_stride, IOT, a.x_stride) &&
                     shift_ok(a.residual, a.residual_stride, HT, a.x_stride) &&
                     shift_ok(a.h_out, a.h_stride, HT, a.x_stride) && shift_ok(a.y, a.y_stride, IOT, a.x_stride);
  int mode = kGroupNone;
  if (a.w_post) {
    const int lanes = vec ? a.group / 8 : a.group;
    mode = a.group == a.channels ? kGroupRow
           : lanes <= 32 && (lanes & (lanes - 1)) == 0 ? kGroupLanes : kGroupShared;
  }
  if (vec || shift) {
    const int vecs = vec ? a.channels / 8 : (a.channels + 14) / 8;
    // Vectors per thread: one, or two where many long rows let bytes in flight
    // count for more than threads (8192 rows of 4096 channels 60.9 to 53.4 us; rows
    // of 512, 41.4 against 42.4; shifted rows of 1533, 15.4 against 17.8), and more
    // where kNormThreads demand it.
    int nv = vec && a.rows >= kManyRows && vecs >= 256 ? 2 : 1;
    while (vecs > kNormThreads * nv) nv *= 2;
    const int tpr = ((vecs + nv - 1) / nv + 31) / 32 * 32;
    if (vec) {
      if (nv == 1) return run<XT, IOT, HT, 8, 1>(a, tpr, mode, s);
      if (nv == 2) return run<XT, IOT, HT, 8, 2>(a, tpr, mode, s);
      if (nv == 4) return run<XT, IOT, HT, 8, 4>(a, tpr, mode, s);
      return run<XT, IOT, HT, 8, 8>(a, tpr, mode, s);
    }
    if (nv == 1) return run<XT, IOT, HT, 8, 1, true>(a, tpr, mode, s);
    if (nv == 2) return run<XT, IOT, HT, 8, 2, true>(a, tpr, mode, s);
    if (nv == 4) return run<XT, IOT, HT, 8, 4, true>(a, tpr, mode, s);
    if (a.channels <= 4096 * 8 - 8) return run<XT, IOT, HT, 8, 8, true>(a, tpr, mode, s);
  }
  if (a.channels <= 4096) return run<XT, IOT, HT, 1, 4>(a, ((a.channels + 3) / 4 + 31) / 32 * 32, mode, s);
  return run<XT, IOT, HT, 1, 32>(a, 1024, mode, s);
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
