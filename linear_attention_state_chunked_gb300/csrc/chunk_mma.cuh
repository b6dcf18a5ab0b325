// Chunk attention on warp-level MMA: fp32 caches, and bf16 caches with fp32 outputs.
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = 2^(s_t - m),  s_t = scale log2(e) q.k_t
//
// over the tokens up to the query's own; one pass over tiles of TK keys with a running
// maximum m and sum per row. A warp owns 16 rows (tokens x query heads of one kv head)
// and keeps their softmax state and value sums in registers. Four warps have an item's 64
// rows; for heads of 256, whose rows leave room for one block on an SM, there are two such
// groups, which take every other tile and are joined at a piece's end (fp32, 1,000 tokens
// after 1,000, 16 / 4 heads: of 256 811 us with one group, 615 with two, and 600 now; of 128,
// where two blocks fit, 310 and 335, and 289 now). K and V
// tiles come by 16-byte asynchronous copies (pages may end anywhere), two tiles ahead,
// swizzled so that no fragment load conflicts. fp32 operands go as two tf32 parts, three products
// (attn_kernel.cuh); the tensor unit cuts off below the last place of what it adds to,
// so the products of 32 channels of a score, and of 16 tokens, are added with rounding.
// 8 x 1-300 tokens after 0-2,000, 12 / 4 heads of 64, fp32: 101 us, 39 TFLOP/s; 4 x 1,000
// after 1,000, 16 / 4 heads of 64, 128 and 256: fp32 492, 1,092 and 2,331 us (either output
// type), bf16 caches with fp32 outputs 192, 325 and 798 (with bf16 outputs, chunk_umma.cuh's,
// 54, 68 and 128). Registers
// leave two or three warps to a scheduler, and no unit is full (heads of 128: tensor pipe
// 45%, ALU 44%, issue 53%): what bounds it is how little of a warp's splits, products and
// softmax goes on beside another's. Splitting a tile once for the block in shared memory,
// instead of in each warp, took as long (101 us, heads of 128 289 to 302).
#pragma once

#include "attn_kernel.cuh"
#include "chunk_common.cuh"

namespace lin {
namespace chunk {

template <int D_, int DT_>
struct MCfg {
  static constexpr int D = D_, DT = DT_;
  static constexpr bool BF = DT == LIN_BF16;
  static constexpr int ES = BF ? 2 : 4, ROWB = D * ES;
  static constexpr int GROUPS = D == 256 ? 2 : 1, GT = 128, NT = GROUPS * GT, ROWS = 64;
  static constexpr int TK = ROWB >= 512 ? 16 : 32;
  static constexpr int STAGES = GROUPS == 1 ? 3 : 4, STAGE = 2 * TK * ROWB;
  static constexpr int QB = ROWS * ROWB;
  static constexpr int SMEM = STAGES * STAGE + QB;
  static constexpr int CTAS = D == 256 ? 1 : D == 128 ? 2 : 3;
  static_assert(SMEM * CTAS <= 220 * 1024 && SMEM >= GT * (D / 2 + 4) * 4, "");
};

// Barriers of a group's four warps.
__device__ __forceinline__ bool group_any(int group, bool x) {
  int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(static_cast<int>(x)), "r"(group + 1)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void group_wait(int group) { asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory"); }

template <class C, int PT>
__global__ void __launch_bounds__(C::NT, C::CTAS) chunk_mma_kernel(const Plan p) {
  using namespace attn;
  constexpr int D = C::D, TK = C::TK, NT = C::NT, GT = C::GT, ROWB = C::ROWB, CPR = ROWB / 16;
  constexpr bool BF = C::BF;
  constexpr int NB = TK / 8;  // key blocks of a tile
  constexpr uint32_t ALL = TK == 32 ? ~0u : (1u << (TK & 31)) - 1u;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ WalkShared s_walk;
  __shared__ Piece s_piece;
  __shared__ uint32_t s_valid[4];
  const int tid = threadIdx.x, lane = tid & 31, group = tid / C::GT, gtid = tid % C::GT, warp = gtid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const lin_kv_cache_t& c = p.c;
  const lin_attn_chunk_args_t& a = p.a;
  Walk w;
  if (!walk_begin<NT>(p, w, s_walk)) return;
  const uint32_t ring = umma::smem_u32(smem), qs = ring + C::STAGES * C::STAGE;

  while (true) {
    __syncthreads();  // the last piece is done with shared memory
    if (tid == 0) s_piece = walk_next(p, w);
    __syncthreads();
    const Piece x = s_piece;
    if (x.r < 0) break;
    const char* kb = static_cast<const char*>(c.k) + a.layer * c.layer_stride + x.hk * c.head_stride;
    const char* vb = static_cast<const char*>(c.v) + a.layer * c.layer_stride + x.hk * c.head_stride;
    const int32_t* table = a.page_table + x.r * a.page_table_stride;

    // lane l of every warp looks up key l % TK of a tile
    int key = x.t0 * TK + (lane & (TK - 1));
    int id = key < x.keys ? table[page_of(p, key)] : -1;
    auto fill = [&](int, int stage) {
      const bool live = static_cast<uint32_t>(id) < static_cast<uint32_t>(c.num_pages);
      if (key < x.keys && !live && tid < TK) report(a.status, LIN_ST_BAD_PAGE);
      const int64_t off = live ? id * c.page_stride + (key - page_of(p, key) * c.page_size) * c.token_stride : 0;
      const uint32_t valid = __ballot_sync(~0u, live) & ALL;
      if (tid == 0) s_valid[stage] = valid;
      const uint32_t dst = ring + stage * C::STAGE;
#pragma unroll
      for (int i = 0; i < TK * CPR / NT; ++i) {
        const int y = i * NT + tid, row = y / CPR, ch = y % CPR;
        const int64_t o = __shfl_sync(~0u, off, row) + ch * 16;
        const bool ok = (valid >> row) & 1u;
        cp16(dst + chunk_at<ROWB>(row, ch), kb + o, ok);
        cp16(dst + TK * ROWB + chunk_at<ROWB>(row, ch), vb + o, ok);
      }
      key += TK;
      id = key < x.keys ? table[page_of(p, key)] : -1;
    };

    // ---- queries: row = token * bheads + head --------------------------------------
    for (int y = tid; y < C::ROWS * CPR; y += NT) {
      const int row = y / CPR, ch = y % CPR;
      const int i = token_of(p, row), h = row - i * p.bheads;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (i < x.tokens && h < x.heads) {
        v = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.q) + int64_t(x.row0 + i) * a.token_stride +
                                            int64_t(x.head0 + h) * ROWB + ch * 16);
        v.x ^= p.negate, v.y ^= p.negate, v.z ^= p.negate, v.w ^= p.negate;
      }
      *reinterpret_cast<uint4*>(smem + C::STAGES * C::STAGE + chunk_at<ROWB>(row, ch)) = v;
    }
    // tokens that this thread's two rows see
    int sees[2];
    bool mine[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int row = warp * 16 + g + 8 * k, i = token_of(p, row);
      mine[k] = i < x.tokens && row - i * p.bheads < x.heads;
      sees[k] = mine[k] ? max(0, x.pos + i + 1) : 0;
    }
    const int all_see = max(0, x.pos + 1);  // what every row of the item sees

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    // Tile i of the piece lies in stage i % STAGES and is group i % GROUPS's; GROUPS tiles
    // at a time, and as many (2 with one group) under way.
    constexpr int STEP = C::GROUPS, AHEAD = C::STAGES - STEP;
    const int tiles = x.t1 - x.t0;
    auto fill_next = [&](int i) {
#pragma unroll
      for (int k = 0; k < STEP; ++k)
        if (i + k < tiles) fill(i + k, (i + k) % C::STAGES);
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < AHEAD; i += STEP) fill_next(i);
#pragma unroll 1
    for (int i0 = 0; i0 < tiles; i0 += STEP) {
      cp_wait<AHEAD / STEP - 1>();
      __syncthreads();  // these tiles are there, and the last ones have been used
      fill_next(i0 + AHEAD);
      const int i = i0 + group;
      if (i >= tiles) continue;
      const int key0 = (x.t0 + i) * TK, stage = i % C::STAGES;
      const uint32_t ks = ring + stage * C::STAGE, vs = ks + TK * ROWB;

      // ---- scores ---------------------------------------------------------------
      float s[NB][4];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[n][k] = 0.0f;
      if constexpr (BF) {
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          uint32_t qa[4];
          ldsm4(qa, qs + chunk_at<ROWB>(warp * 16 + (lane & 15), 2 * d + (lane >> 4)));
#pragma unroll
          for (int n = 0; n < NB; n += 2) {
            uint32_t b[4];  // keys n and n + 1, channels 16 d on
            ldsm4(b, ks + chunk_at<ROWB>(n * 8 + (lane & 7) + (lane >> 4) * 8, 2 * d + ((lane >> 3) & 1)));
            mma_bf16(s[n], qa, b[0], b[1]);
            mma_bf16(s[n + 1], qa, b[2], b[3]);
          }
        }
      } else {
#pragma unroll 1
        for (int d0 = 0; d0 < D / 8; d0 += 4) {
          float part[NB][4];
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) part[n][k] = 0.0f;
#pragma unroll
          for (int dd = 0; dd < 4; ++dd) {
            const int d = d0 + dd;
            uint32_t q[4], hi[4], lo[4];
            ldsm4(q, qs + chunk_at<ROWB>(warp * 16 + (lane & 15), 2 * d + (lane >> 4)));
#pragma unroll
            for (int k = 0; k < 4; ++k) split_tf32(__uint_as_float(q[k]), hi[k], lo[k]);
            // a sum's three products wait for one another: those of all keys in turn
            uint32_t bh[NB][2], bl[NB][2];
#pragma unroll
            for (int n = 0; n < NB; n += 2) {
              uint32_t b[4];
              ldsm4(b, ks + chunk_at<ROWB>(n * 8 + (lane & 7) + (lane >> 4) * 8, 2 * d + ((lane >> 3) & 1)));
#pragma unroll
              for (int k = 0; k < 4; ++k) split_tf32(__uint_as_float(b[k]), bh[n + k / 2][k & 1], bl[n + k / 2][k & 1]);
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) mma_tf32(part[n], lo, bh[n][0], bh[n][1]);
#pragma unroll
            for (int n = 0; n < NB; ++n) mma_tf32(part[n], hi, bl[n][0], bl[n][1]);
#pragma unroll
            for (int n = 0; n < NB; ++n) mma_tf32(part[n], hi, bh[n][0], bh[n][1]);
          }
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[n][k] += part[n][k];
        }
      }

      // ---- softmax ----------------------------------------------------------------
      const uint32_t valid = s_valid[stage];
      const bool masked = key0 + TK > all_see || valid != ALL;
      uint32_t vis[2] = {~0u, ~0u};
      if (masked) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int n = sees[k] - key0;
          vis[k] = n <= 0 ? 0u : n >= 32 ? valid : valid & ((1u << n) - 1u);
        }
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (!((vis[k >> 1] >> (n * 8 + 2 * t4 + (k & 1))) & 1u)) s[n][k] = -INFINITY;
      }
      float z[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < NB; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * k], s[n][2 * k + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2)) * p.scale_log2;
        if (mx > m[k]) {
          const float f = exp2_fast(m[k] - mx);  // 0 at first
          m[k] = mx, l[k] *= f;
#pragma unroll
          for (int y = 0; y < D / 8; ++y) o[y][2 * k] *= f, o[y][2 * k + 1] *= f;
        }
        z[k] = m[k] == -INFINITY ? 0.0f : -m[k];
      }
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s[n][k] = exp2_fast(fmaf(s[n][k], p.scale_log2, z[k >> 1]));
          l[k >> 1] += s[n][k];
        }

      // Values that are infinite or NaN: 0 in the product, added by themselves to the
      // rows that see them (0 NaN is NaN, and hidden ones must have no part).
      if (masked) {
        bool wild = false;
        for (int y = gtid; y < TK * CPR; y += GT) {
          const uint4 v = *reinterpret_cast<const uint4*>(smem + (vs - ring) + y * 16);
          const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            wild |= (q[k] & 0x7f800000u) == 0x7f800000u || (BF && (q[k] & 0x7f80u) == 0x7f80u);
        }
        if (group_any(group, wild)) {
#pragma unroll 1
          for (int t = 0; t < TK; ++t) {
#pragma unroll
            for (int y = 0; y < D / 8; ++y)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int ch = y * 8 + 2 * t4 + k;
                const unsigned char* at = smem + (vs - ring) + chunk_at<ROWB>(t, ch * C::ES / 16) + ch * C::ES % 16;
                const float v = load_elem(at, 0, C::DT);
                if (!isfinite(v)) {
                  if ((vis[0] >> t) & 1u) o[y][k] += v;
                  if ((vis[1] >> t) & 1u) o[y][2 + k] += v;
                }
              }
          }
          group_wait(group);
          for (int y = gtid; y < TK * ROWB / 4; y += GT) {
            uint32_t& v = reinterpret_cast<uint32_t*>(smem + (vs - ring))[y];
            if (BF)
              v = finite_bf16(v);
            else if ((v & 0x7f800000u) == 0x7f800000u)
              v = 0;
          }
          group_wait(group);
        }
      }

      // ---- value sums: the products of 16 tokens at a time are added with rounding ----
      if constexpr (BF) {
#pragma unroll
        for (int n = 0; n < NB; n += 2) {
          uint32_t pa[PT][4];
          float y[8] = {s[n][0], s[n][1], s[n][2], s[n][3], s[n + 1][0], s[n + 1][1], s[n + 1][2], s[n + 1][3]};
#pragma unroll
          for (int part = 0; part < PT; ++part)
#pragma unroll
            for (int k = 0; k < 4; ++k) pa[part][k] = take_bf16(y[2 * k], y[2 * k + 1]);
#pragma unroll
          for (int d = 0; d < D / 8; d += 2) {
            uint32_t b[4];
            ldsm4t(b, vs + chunk_at<ROWB>(n * 8 + (lane & 15), d + (lane >> 4)));
            float u0[4] = {0, 0, 0, 0}, u1[4] = {0, 0, 0, 0};
#pragma unroll
            for (int part = PT - 1; part >= 0; --part) {
              mma_bf16(u0, pa[part], b[0], b[1]);
              mma_bf16(u1, pa[part], b[2], b[3]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) o[d][k] += u0[k], o[d + 1][k] += u1[k];
          }
        }
      } else {
#pragma unroll
        for (int n = 0; n < NB; n += 2) {
          // the k index t4 stands for token 2 t4, t4 + 4 for 2 t4 + 1: what the scores'
          // accumulators hold is the A operand as it is
          uint32_t hi[2][4], lo[2][4];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            split_weight(s[n + y][0], hi[y][0], lo[y][0]);
            split_weight(s[n + y][2], hi[y][1], lo[y][1]);
            split_weight(s[n + y][1], hi[y][2], lo[y][2]);
            split_weight(s[n + y][3], hi[y][3], lo[y][3]);
          }
#pragma unroll
          for (int d = 0; d < D / 8; d += 4) {
            float u[4][4];
#pragma unroll
            for (int z = 0; z < 4; ++z)
#pragma unroll
              for (int k = 0; k < 4; ++k) u[z][k] = 0.0f;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t bh[4][2], bl[4][2];
#pragma unroll
              for (int z = 0; z < 4; ++z)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const uint32_t at = vs + chunk_at<ROWB>((n + y) * 8 + 2 * t4 + k, (d + z) * 2 + (g >> 2)) + (g & 3) * 4;
                  split_tf32(lds32(at), bh[z][k], bl[z][k]);
                }
#pragma unroll
              for (int z = 0; z < 4; ++z) mma_tf32(u[z], lo[y], bh[z][0], bh[z][1]);
#pragma unroll
              for (int z = 0; z < 4; ++z) mma_tf32(u[z], hi[y], bl[z][0], bl[z][1]);
#pragma unroll
              for (int z = 0; z < 4; ++z) mma_tf32(u[z], hi[y], bh[z][0], bh[z][1]);
            }
#pragma unroll
            for (int z = 0; z < 4; ++z)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[d + z][k] += u[z][k];
          }
        }
      }
    }
    cp_wait_all();

    // ---- the piece's end: the second group's sums go to the first --------------------
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      l[k] += __shfl_xor_sync(~0u, l[k], 1);
      l[k] += __shfl_xor_sync(~0u, l[k], 2);
    }
    if constexpr (C::GROUPS == 2) {
      float* const other = reinterpret_cast<float*>(smem) + gtid;  // a thread's values GT apart
      __syncthreads();
      if (group == 1) {
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
#pragma unroll
          for (int k = 0; k < 4; ++k) other[(d * 4 + k) * GT] = o[d][k];
#pragma unroll
        for (int k = 0; k < 2; ++k) other[(D / 2 + k) * GT] = m[k], other[(D / 2 + 2 + k) * GT] = l[k];
      }
      __syncthreads();
      if (group == 1) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float m1 = other[(D / 2 + k) * GT], l1 = other[(D / 2 + 2 + k) * GT], top = fmaxf(m[k], m1);
        // 0 where a group saw nothing (a NaN sum goes on)
        const float f0 = l[k] == 0.0f ? 0.0f : m[k] == top ? 1.0f : exp2_fast(m[k] - top);
        const float f1 = l1 == 0.0f ? 0.0f : m1 == top ? 1.0f : exp2_fast(m1 - top);
        l[k] = fmaf(f0, l[k], f1 * l1), m[k] = top;
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
#pragma unroll
          for (int y = 2 * k; y < 2 * k + 2; ++y) o[d][y] = fmaf(f0, o[d][y], f1 * other[(d * 4 + y) * GT]);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float sum = l[k];
      const int row = warp * 16 + g + 8 * k, i = token_of(p, row);
      const float f = !x.whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
      if (!mine[k]) continue;
      if (x.whole) {
        const int64_t at = (int64_t(x.row0 + i) * a.num_q_heads + x.head0 + row - i * p.bheads) * D + 2 * t4;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          if (a.out_dtype == LIN_F32)
            *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at + d * 8) = make_float2(o[d][2 * k] * f, o[d][2 * k + 1] * f);
          else
            *reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(a.out) + at + d * 8) =
                __floats2bfloat162_rn(o[d][2 * k] * f, o[d][2 * k + 1] * f);
        }
      } else {
        float* to = p.part + ((int64_t(x.part) * (D / 4) + (t4 >> 1)) * p.rows + row) * 4 + (t4 & 1) * 2;
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
          *reinterpret_cast<float2*>(to + int64_t(d) * 8 * p.rows) = make_float2(o[d][2 * k], o[d][2 * k + 1]);
        if (t4 == 0) p.part_ml[int64_t(x.part) * p.rows + row] = make_float2(m[k], sum);
      }
    }
  }
}

template <class C, int PT>
cudaError_t launch_mma(const Plan& p, cudaStream_t s) {
  auto kern = chunk_mma_kernel<C, PT>;
  static bool ready[kMaxDevices];  // set twice at worst, to the same value
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev] = true;
  }
  kern<<<p.grid, C::NT, C::SMEM, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_mma_types(const Plan& p, cudaStream_t s) {
  return p.c.dtype == LIN_F32 ? launch_mma<MCfg<D, LIN_F32>, 1>(p, s) : launch_mma<MCfg<D, LIN_BF16>, 3>(p, s);
}

}  // namespace chunk
}  // namespace lin
