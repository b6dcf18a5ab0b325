// Decode attention over a paged key-value cache (lin_step.h): bf16 caches with up
// to 16 rows per (request, kv head), 32 of short requests, or with fp32 outputs,
// and fp32 caches.
//
//   out[r][j][h] = sum_t p_t v_t / sum_t p_t,  p_t = 2^(s_t - m),
//   s_t = scale log2(e) q.k_t over the tokens that query j sees,
//
// one pass over the cache with a reference m, the sum and the value sum per row.
// The rows of one (request, key-value head) are its n_q x G queries (G query
// heads share the head's keys), so every key is read once for all of them.
//
// Bound by HBM with one row tile in bf16: 2 head_dim elements per token and
// key-value head are read for 4 head_dim flops a row. The tensor work is
// warp-level MMA on 16 rows, which is what a decode step has, and each warp keeps
// its rows' whole softmax state in registers. 256 requests of 1k-16k tokens, 8
// query heads to a kv head of 128: 328-336 us, 0.98 of the measured copy bandwidth.
// fp32 has three tf32 products to an fp32 one, and no unit is full: in trees of 8
// drafts, 24 rows, heads of 64 (32 requests of 8-4,000 tokens: 62 us for a floor of
// 20) the tensor pipe is busy 39% of the time, the schedulers issue 56%, HBM runs at
// 30%. A warp owns one row tile, so with RT tiles every key and value is loaded from
// shared memory and split RT times. 64 requests of 500-8,000 tokens, 2 kv heads, 8, 32
// and 64 rows: heads of 64 63, 114 and 211 us for a floor of 43, of 128 125, 211 and
// 417 for 85, of 256 250, 466 and 765 for 171.
//
// Inside a CTA a group of RT x DS warps (one per 16 rows, and per part of the
// values) shares a ring of S slots of 16 tokens' K and V, filled by 16-byte
// asynchronous copies of its own threads (one bulk copy per row was three times
// slower: a warp issues them one by one). The KG groups take every KG-th slot of
// a piece and are joined in shared memory at its end. Rows of a slot are swizzled
// (16-byte chunk c of row r at c ^ (r % 8)), so every fragment load is free of
// bank conflicts. Tokens past the length, or in a bad page, are filled with zeros
// and masked.
#pragma once

#include "attn_common.cuh"

namespace lin {
namespace attn {

constexpr int kSub = 16;  // tokens of a ring slot

// Warps of one CTA: KG groups x RT row tiles x DS parts of head_dim. DS
// warps share a row tile where rows of 512 bytes and more would otherwise leave
// one warp per scheduler: each makes its channels' part of the scores, which are
// added in shared memory, and its channels' value sums. As many CTAs as leave room for two slots a group and registers
// for the value sums.
template <int D_, int DT_, int RT_>
struct Cfg {
  static constexpr int D = D_, DT = DT_, RT = RT_;
  static constexpr bool BF = DT == LIN_BF16;
  static constexpr int ES = BF ? 2 : 4;
  static constexpr int ROWB = D * ES;                 // bytes of one key or value
  static constexpr int SLOT = 2 * kSub * ROWB;        // K and V of a slot's tokens
  static constexpr int QP = BF ? 1 : 2;               // planes of q: fp32 as two tf32 parts
  static constexpr int QBYTES = QP * 16 * RT * ROWB;
  static constexpr bool MANY = RT >= 2;
  static constexpr int CTAS = ROWB > 256 ? 1 : MANY ? 2 : ROWB == 128 ? 4 : BF ? 2 : 3;
  static constexpr int DS = ROWB <= 256 ? 1 : ROWB == 512 ? 2 : RT == 4 ? 2 : 4;
  static constexpr int NW = ROWB <= 256 ? (MANY ? 8 : 4) : ROWB == 512 ? (MANY ? 16 : 8) : 8;
  // a warp keeps its queries' operands in registers where that costs no occupancy
  static constexpr bool QREG = BF && D <= 128 && !MANY;
  static constexpr int KG = NW / (RT * DS);
  static constexpr int GT = RT * DS * 32;             // threads of a group
  static constexpr int BUDGET = (CTAS == 4 ? 55 : CTAS == 3 ? 73 : CTAS == 2 ? 110 : 216) * 1024;
  static constexpr int SLOTS = (BUDGET - QBYTES) / SLOT / KG;
  static constexpr int S = SLOTS < 12 ? SLOTS : 12;
  static constexpr int RING = KG * S * SLOT;
  static constexpr int SMEM = RING + QBYTES;
  // the groups are joined where the ring and the queries were
  static_assert(S >= 2 && SMEM >= KG * RT * 16 * (D + 2) * 4, "");
};

template <int GT>
__device__ __forceinline__ void group_sync(int kg) {
  if constexpr (GT == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(kg + 1), "n"(GT) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ float lds32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo in two tf32 values of 11 significant bits (the unit reads the upper
// 19 bits of an operand): hi rounded to nearest, by an integer addition as the
// conversion instruction is slower; lo at most 2^12 units of x's last place, so
// that what the unit cuts off is one of them, 2^-23 of x. A NaN x leaves NaN in
// lo whatever becomes of hi, and an infinity does as well.
__device__ __forceinline__ void split_weight(float x, uint32_t& hi, uint32_t& lo) {  // x below kTf32Top
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
// The same for any x: from kTf32Top on hi is cut off, as rounding up would give an
// infinity, and lo's cut is 2^-21 of x.
constexpr float kTf32Top = 0x1.ffep127f;
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (fabsf(x) < kTf32Top ? __float_as_uint(x) + 0x1000u : __float_as_uint(x)) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
// a pair of bf16 values with 0 for infinities and NaN
__device__ __forceinline__ uint32_t finite_bf16(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

// Byte offset of 16-byte chunk `c` of row `r` in rows of ROWB bytes.
template <int ROWB>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return static_cast<uint32_t>(r * ROWB + ((c ^ (r & 7)) << 4));
}

// The same from the offset `at` of chunk 0 of a row r with (r & 7) << 4 added:
// a constant exclusive-or and a constant sum.
__device__ __forceinline__ uint32_t chunk_from(uint32_t at, int c) {
  return (at ^ ((c & 7) << 4)) + (c >> 3) * 128;
}

template <class C, int PT>
__global__ void __launch_bounds__(C::NW * 32, C::CTAS) attn_kernel(const Plan p) {
  constexpr int D = C::D, RT = C::RT, DS = C::DS, KG = C::KG, S = C::S, NT = C::NW * 32, ROWB = C::ROWB;
  constexpr int GT = C::GT, DW = D / DS;  // a warp sums DW channels of the values
  constexpr bool BF = C::BF;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint32_t s_valid[KG][S];  // live tokens of each slot
  __shared__ float4 s_score[DS > 1 ? C::NW : 1][2][DS > 1 ? 32 : 1];  // a warp's share of the scores
  __shared__ uint32_t s_see[32];       // drafts that each query sees
  __shared__ int64_t s_scan[C::NW], s_first[2];
  __shared__ int s_bad;
  asm volatile("griddepcontrol.launch_dependents;");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kg = warp / (RT * DS), gtid = tid - kg * GT, rt = gtid / 32 / DS, ds = gtid / 32 % DS;
  const int g = lane >> 2, t4 = lane & 3;
  const lin_kv_cache_t& c = p.c;
  const lin_attn_args_t& a = p.a;
  Walk w;
  if (!walk_begin<NT>(p, w, s_scan, s_first)) return;

  const uint32_t ring = umma::smem_u32(smem) + kg * (S * C::SLOT);
  const uint32_t qs = umma::smem_u32(smem) + C::RING;
  float* merge = reinterpret_cast<float*>(smem);                       // [KG][16 RT][D]
  float2* merge_ml = reinterpret_cast<float2*>(merge + KG * 16 * RT * D);  // [KG][16 RT]

  while (true) {
    const int t1 = walk_until(p, w), r = w.r;
    const int hk = head_of(p, w.it), row0 = (w.it - hk * p.row_blocks) * 16 * RT;
    const int key_begin = w.t0 * kUnit, key_end = t1 == w.u ? w.len : t1 * kUnit;
    const int base = w.len - a.n_q;  // tokens that every query sees
    const char* kb = static_cast<const char*>(c.k) + a.layer * c.layer_stride + hk * c.head_stride;
    const char* vb = static_cast<const char*>(c.v) + a.layer * c.layer_stride + hk * c.head_stride;
    const int32_t* table = a.page_table + r * a.page_table_stride;

    // ---- slots: lane l of every warp looks up token l % 16 of the slot --------
    const int subs = (key_end - key_begin + kSub - 1) / kSub;
    const int count = subs > kg ? (subs - kg + KG - 1) / KG : 0;  // this group's
    int key = key_begin + kg * kSub + (lane & (kSub - 1));
    int in_page = 0, id = -1;
    auto look = [&]() {  // page id of the next slot's token
      const int page = page_of(p, key);
      in_page = key - page * c.page_size;
      id = key < key_end ? table[page] : -1;
    };
    auto fill = [&](int slot) {
      const bool live = static_cast<uint32_t>(id) < static_cast<uint32_t>(c.num_pages);
      if (key < key_end && !live && gtid == (lane & (kSub - 1))) report(a.status, LIN_ST_BAD_PAGE);
      const int64_t off = live ? id * c.page_stride + in_page * c.token_stride : 0;
      const uint32_t valid = __ballot_sync(~0u, live) & 0xffffu;
      if (gtid == 0) s_valid[kg][slot] = valid;
      constexpr int CPR = ROWB / 16;
      const uint32_t dst = ring + slot * C::SLOT;
#pragma unroll
      for (int i = 0; i < kSub * CPR / GT; ++i) {
        const int x = i * GT + gtid, row = x / CPR, ch = x % CPR;
        const int64_t o = __shfl_sync(~0u, off, row) + ch * 16;
        const bool ok = (valid >> row) & 1u;
        cp16(dst + chunk_at<ROWB>(row, ch), kb + o, ok);
        cp16(dst + kSub * ROWB + chunk_at<ROWB>(row, ch), vb + o, ok);
      }
      key += KG * kSub;
      look();
    };
    look();
#pragma unroll 1
    for (int i = 0; i < S - 1; ++i) {
      if (i < count) fill(i);
      cp_commit();
    }

    // ---- queries and what they see ------------------------------------------
    {
      constexpr int CPR = ROWB / 16;
      const char* qb = static_cast<const char*>(a.q) + r * a.req_stride;
      for (int x = tid; x < 16 * RT * CPR; x += NT) {
        const int row = x / CPR, ch = x % CPR, q = row0 + row;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (q < p.rows) {
          const int j = query_of(p, q), h = hk * p.group + q - j * p.group;
          v = *reinterpret_cast<const uint4*>(qb + j * a.token_stride + h * ROWB + ch * 16);
          v.x ^= p.negate, v.y ^= p.negate, v.z ^= p.negate, v.w ^= p.negate;
        }
        unsigned char* dst = smem + C::RING + chunk_at<ROWB>(row, ch);
        if constexpr (!BF) {
          uint4 lo;
          split_tf32(__uint_as_float(v.x), v.x, lo.x), split_tf32(__uint_as_float(v.y), v.y, lo.y);
          split_tf32(__uint_as_float(v.z), v.z, lo.z), split_tf32(__uint_as_float(v.w), v.w, lo.w);
          *reinterpret_cast<uint4*>(dst + 16 * RT * ROWB) = lo;
        }
        *reinterpret_cast<uint4*>(dst) = v;
      }
      if (warp == 0) draft_sets(p, r, s_see, s_bad);
    }
    __syncthreads();
    const bool bad = s_bad;
    const int qa = row0 + rt * 16 + g, qb2 = qa + 8;
    const uint32_t see0 = qa < p.rows ? s_see[query_of(p, qa)] : 0u;
    const uint32_t see1 = qb2 < p.rows ? s_see[query_of(p, qb2)] : 0u;

    constexpr bool QREG = C::QREG;
    const uint32_t qat = qs + (BF ? chunk_at<ROWB>(rt * 16 + (lane & 15), lane >> 4)
                                  : chunk_at<ROWB>(rt * 16 + g, 0) + t4 * 4);
    uint32_t qf[QREG ? D / 16 : 1][4];
    if constexpr (QREG) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) ldsm4(qf[k], chunk_from(qat, 2 * k));
    }
    float o[DW / 8][4];
#pragma unroll
    for (int n = 0; n < DW / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
    float c0 = -INFINITY, c1 = -INFINITY;  // scores past these move the reference
    float l0 = 0.0f, l1 = 0.0f, z0 = 0.0f, z1 = 0.0f;

    // ---- the pass over this group's slots --------------------------------------
    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      cp_wait<S - 2>();
      group_sync<GT>(kg);  // slot i has landed; slot i - 1 is free
      if (i + S - 1 < count) fill(slot == 0 ? S - 1 : slot - 1);
      cp_commit();
      const uint32_t ks = ring + slot * C::SLOT, vs = ks + kSub * ROWB;
      float s[2][4];  // two column tiles of 8 tokens
      const uint32_t dsb = DS > 1 ? ds * (DW * C::ES) : 0;  // this warp's channels
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[n][x] = 0.0f;
      if constexpr (BF) {
        // even and odd steps sum apart, for chains half as long
        float s2[2][4];
        const uint32_t kat = ks + chunk_at<ROWB>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
#pragma unroll
        for (int x = 0; x < 4; ++x) s2[0][x] = s2[1][x] = 0.0f;
#pragma unroll
        for (int k = 0; k < DW / 16; ++k) {
          uint32_t q[4];
          if constexpr (!QREG) ldsm4(q, chunk_from(qat + dsb, 2 * k));
          uint32_t b[4];
          ldsm4(b, chunk_from(kat + dsb, 2 * k));
          mma_bf16(k & 1 ? s2[0] : s[0], QREG ? qf[QREG ? k : 0] : q, b[0], b[1]);
          mma_bf16(k & 1 ? s2[1] : s[1], QREG ? qf[QREG ? k : 0] : q, b[2], b[3]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) s[0][x] += s2[0][x], s[1][x] += s2[1][x];
      } else {
        const uint32_t kat = ks + chunk_at<ROWB>(g, 0) + t4 * 4;
        // 32 channels to a chain of products, chains joined by rounded additions
#pragma unroll
        for (int k0 = 0; k0 < DW / 8; k0 += 4) {
          float c0[2][4], c1[2][4];
#pragma unroll
          for (int x = 0; x < 4; ++x) c0[0][x] = c0[1][x] = c1[0][x] = c1[1][x] = 0.0f;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t ko = (k0 >> 2) * 128 + dsb;  // 4 steps are one turn of the swizzle
            uint32_t qh[4], ql[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t at = chunk_from(qat + (x & 1) * 8 * ROWB, 2 * y + (x >> 1)) + ko;
              qh[x] = __float_as_uint(lds32(at));
              ql[x] = __float_as_uint(lds32(at + 16 * RT * ROWB));
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              uint32_t h0, w0, h1, w1;
              split_tf32(lds32(chunk_from(kat + n * 8 * ROWB, 2 * y) + ko), h0, w0);
              split_tf32(lds32(chunk_from(kat + n * 8 * ROWB, 2 * y + 1) + ko), h1, w1);
              mma_tf32(c0[n], qh, h0, h1);
              mma_tf32(c1[n], ql, h0, h1);
              mma_tf32(c1[n], qh, w0, w1);
            }
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) s[0][x] += c0[0][x] + c1[0][x], s[1][x] += c0[1][x] + c1[1][x];
        }
      }
      if constexpr (DS > 1) {
        // each of the DS warps has the products of its own channels: add them up,
        // in one order, so that all go on with the same scores
        s_score[warp][0][lane] = make_float4(s[0][0], s[0][1], s[0][2], s[0][3]);
        s_score[warp][1][lane] = make_float4(s[1][0], s[1][1], s[1][2], s[1][3]);
        group_sync<GT>(kg);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float4 sum = s_score[warp - ds][n][lane];
#pragma unroll
          for (int x = 1; x < DS; ++x) {
            const float4 y = s_score[warp - ds + x][n][lane];
            sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
          }
          s[n][0] = sum.x, s[n][1] = sum.y, s[n][2] = sum.z, s[n][3] = sum.w;
        }
      }
      // which of the slot's tokens the two rows see; token n * 8 + 2 t4 + e is
      // bit 8 n + e of the shifted masks
      const uint32_t valid = s_valid[kg][slot];
      const int sh = key_begin + (i * KG + kg) * kSub - base;
      const bool drafts = sh + kSub > 0;
      const bool masked = drafts || valid != 0xffffu;
      uint32_t vis0 = valid, vis1 = valid;
      if (masked) {
        if (drafts) {
          const uint32_t old = sh < 0 ? (1u << -sh) - 1u : 0u;
          vis0 &= sh < 0 ? (see0 << -sh) | old : see0 >> sh;
          vis1 &= sh < 0 ? (see1 << -sh) | old : see1 >> sh;
        }
        vis0 >>= 2 * t4;
        vis1 >>= 2 * t4;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (!((vis0 >> (8 * n + e)) & 1u)) s[n][e] = -INFINITY;
            if (!((vis1 >> (8 * n + e)) & 1u)) s[n][2 + e] = -INFINITY;
          }
      }
      float mx0 = s[0][0], mx1 = s[0][2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        mx0 = fmaxf(mx0, fmaxf(s[n][0], s[n][1]));
        mx1 = fmaxf(mx1, fmaxf(s[n][2], s[n][3]));
      }
      // The weights' reference m follows the maximum only where a score passes it
      // by more than 2^kSlack: weights up to that size lose nothing in fp32, and
      // most slots need neither the rows' maximum nor a rescaling of the sums.
      if (__any_sync(~0u, mx0 > c0 || mx1 > c1)) {
#pragma unroll
        for (int o2 = 1; o2 < 4; o2 <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(~0u, mx0, o2));
          mx1 = fmaxf(mx1, __shfl_xor_sync(~0u, mx1, o2));
        }
        // z = -m scale_log2, 0 while a row has seen nothing
        if (mx0 > c0) {
          const float y = -mx0 * p.scale_log2, f = c0 == -INFINITY ? 0.0f : exp2_fast(y - z0);
          z0 = y, c0 = mx0 + p.slack, l0 *= f;
#pragma unroll
          for (int n = 0; n < DW / 8; ++n) o[n][0] *= f, o[n][1] *= f;
        }
        if (mx1 > c1) {
          const float y = -mx1 * p.scale_log2, f = c1 == -INFINITY ? 0.0f : exp2_fast(y - z1);
          z1 = y, c1 = mx1 + p.slack, l1 *= f;
#pragma unroll
          for (int n = 0; n < DW / 8; ++n) o[n][2] *= f, o[n][3] *= f;
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[n][e] = exp2_fast(fmaf(s[n][e], p.scale_log2, z0));
          s[n][2 + e] = exp2_fast(fmaf(s[n][2 + e], p.scale_log2, z1));
        }
      // A value that some rows do not see may be infinite or NaN, and 0 times
      // that is NaN: slots of drafts are looked over, and where one holds such
      // values they are 0 in the products and are added to the rows that see
      // them by themselves.
      bool wild = false;
      if (masked) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // scale 0 makes NaN of a hidden score
            if (!((vis0 >> (8 * n + e)) & 1u)) s[n][e] = 0.0f;
            if (!((vis1 >> (8 * n + e)) & 1u)) s[n][2 + e] = 0.0f;
          }
        if (drafts && a.n_q > 1) {
          for (int x = lane; x < kSub * ROWB / 16; x += 32) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(vs + x * 16) : "memory");
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              wild |= (w[y] & 0x7f800000u) == 0x7f800000u;
              if (BF) wild |= (w[y] & 0x7f80u) == 0x7f80u;
            }
          }
          wild = __any_sync(~0u, wild);
        }
        if (wild) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll 1
              for (int pair = 0; pair < 4; ++pair) {  // token n * 8 + 2 pair + e
                const int kk = n * 8 + 2 * pair + e, from = (lane & ~3) | pair;
                const float p0 = __shfl_sync(~0u, s[n][e], from), p1 = __shfl_sync(~0u, s[n][2 + e], from);
                const bool v0 = __shfl_sync(~0u, (vis0 >> (8 * n + e)) & 1u, from);
                const bool v1 = __shfl_sync(~0u, (vis1 >> (8 * n + e)) & 1u, from);
#pragma unroll
                for (int x = 0; x < DW / 8; ++x)
#pragma unroll
                  for (int y = 0; y < 2; ++y) {
                    const int d = ds * DW + x * 8 + 2 * t4 + y;
                    float v;
                    if constexpr (BF) {
                      uint16_t h;
                      asm volatile("ld.shared.u16 %0, [%1];"
                                   : "=h"(h) : "r"(vs + chunk_at<ROWB>(kk, d >> 3) + (d & 7) * 2) : "memory");
                      v = bf16_bits_to_f32(h);
                    } else {
                      v = lds32(vs + chunk_at<ROWB>(kk, d >> 2) + (d & 3) * 4);
                    }
                    if (isfinite(v)) continue;
                    if (v0) o[x][y] = fmaf(p0, v, o[x][y]);
                    if (v1) o[x][2 + y] = fmaf(p1, v, o[x][2 + y]);
                  }
              }
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        l0 += s[n][0] + s[n][1];
        l1 += s[n][2] + s[n][3];
      }
      // The unit's own accumulation cuts off below the last place of the sum: over a
      // long cache the loss adds up (4.6e-6 of the outputs at 3,000 tokens, 2.3e-4 at
      // 131,072, always towards 0), so a slot's sums are added by rounded additions
      // (bf16, 256 requests of 1k-16k tokens: less than 0.5% more time).
      if constexpr (BF) {
        const uint32_t vat = vs + chunk_at<ROWB>(lane & 15, lane >> 4);
        uint32_t pf[PT][4];
#pragma unroll
        for (int x = 0; x < PT; ++x) {
          pf[x][0] = take_bf16(s[0][0], s[0][1]);
          pf[x][1] = take_bf16(s[0][2], s[0][3]);
          pf[x][2] = take_bf16(s[1][0], s[1][1]);
          pf[x][3] = take_bf16(s[1][2], s[1][3]);
        }
#pragma unroll
        for (int n = 0; n < DW / 16; ++n) {
          float f0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, f1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          uint32_t b[4];
          ldsm4t(b, chunk_from(vat + ds * (DW * C::ES), 2 * n));
          if (wild) {
#pragma unroll
            for (int x = 0; x < 4; ++x) b[x] = finite_bf16(b[x]);
          }
#pragma unroll
          for (int x = PT - 1; x >= 0; --x) {
            mma_bf16(f0, pf[x], b[0], b[1]);
            mma_bf16(f1, pf[x], b[2], b[3]);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) o[2 * n][x] += f0[x], o[2 * n + 1][x] += f1[x];
        }
      } else {
        // k index t4 | t4 + 4 of a product stands for token 2 t4 | 2 t4 + 1, as
        // the scores lie in registers
        uint32_t ph[2][4], pl[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          split_weight(s[k][0], ph[k][0], pl[k][0]);
          split_weight(s[k][2], ph[k][1], pl[k][1]);
          split_weight(s[k][1], ph[k][2], pl[k][2]);
          split_weight(s[k][3], ph[k][3], pl[k][3]);
        }
        const uint32_t va = vs + ds * (DW * C::ES) + chunk_at<ROWB>(2 * t4, g >> 2) + (g & 3) * 4;
        const uint32_t vb1 = vs + ds * (DW * C::ES) + chunk_at<ROWB>(2 * t4 + 1, g >> 2) + (g & 3) * 4;
#pragma unroll
        for (int n = 0; n < DW / 8; ++n) {
          float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t h0, w0, h1, w1;
            float x0 = lds32(chunk_from(va + k * 8 * ROWB, 2 * n)), x1 = lds32(chunk_from(vb1 + k * 8 * ROWB, 2 * n));
            if (wild) x0 = isfinite(x0) ? x0 : 0.0f, x1 = isfinite(x1) ? x1 : 0.0f;
            split_tf32(x0, h0, w0);
            split_tf32(x1, h1, w1);
            mma_tf32(f, pl[k], h0, h1);
            mma_tf32(f, ph[k], w0, w1);
            mma_tf32(f, ph[k], h0, h1);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) o[n][x] += f[x];
        }
      }
      slot = slot + 1 == S ? 0 : slot + 1;
    }

    // ---- join the groups ---------------------------------------------------------
#pragma unroll
    for (int o2 = 1; o2 < 4; o2 <<= 1) {
      l0 += __shfl_xor_sync(~0u, l0, o2);
      l1 += __shfl_xor_sync(~0u, l1, o2);
    }
    cp_wait<0>();
    __syncthreads();  // every slot is read
    {
      const int row = kg * 16 * RT + rt * 16 + g, d = ds * DW + 2 * t4;
#pragma unroll
      for (int n = 0; n < DW / 8; ++n) {
        *reinterpret_cast<float2*>(merge + row * D + n * 8 + d) = make_float2(o[n][0], o[n][1]);
        *reinterpret_cast<float2*>(merge + (row + 8) * D + n * 8 + d) = make_float2(o[n][2], o[n][3]);
      }
      if (t4 == 0 && ds == 0) {
        merge_ml[row] = make_float2(c0 == -INFINITY ? c0 : -z0, l0);
        merge_ml[row + 8] = make_float2(c1 == -INFINITY ? c1 : -z1, l1);
      }
    }
    __syncthreads();
    finish_piece<D, KG, 16 * RT, NT>(p, w, t1, merge, merge_ml, bad);
    if (!walk_next(p, w, t1)) break;
    __syncthreads();  // the join is read before the ring is filled again
  }
  if (tid == 0) p.split[blockIdx.x] = w.split;
}

template <class C, int PT>
cudaError_t launch_main(const Plan& p, int grid, cudaStream_t s) {
  auto kern = attn_kernel<C, PT>;
  static bool ready[kMaxDevices];  // set twice at worst, to the same value
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev] = true;
  }
  kern<<<grid, C::NW * 32, C::SMEM, s>>>(p);
  return cudaGetLastError();
}

template <int D, int DT>
cudaError_t launch_rows(const Plan& p, int row_tiles, int grid, cudaStream_t s) {
  if constexpr (DT == LIN_BF16) {  // bf16 outputs with larger blocks take the kernels of attn_umma.cuh
    return row_tiles == 4   ? launch_main<Cfg<D, DT, 4>, 3>(p, grid, s)
           : row_tiles == 2 ? launch_main<Cfg<D, DT, 2>, 3>(p, grid, s)
           : p.a.out_dtype == LIN_F32 ? launch_main<Cfg<D, DT, 1>, 3>(p, grid, s)
                                      : launch_main<Cfg<D, DT, 1>, 2>(p, grid, s);
  } else {
    return row_tiles == 1   ? launch_main<Cfg<D, DT, 1>, 1>(p, grid, s)
           : row_tiles == 2 ? launch_main<Cfg<D, DT, 2>, 1>(p, grid, s)
                            : launch_main<Cfg<D, DT, 4>, 1>(p, grid, s);
  }
}

}  // namespace attn
}  // namespace lin
