// Decode attention for more than 16 rows per (request, kv head) over a bf16
// cache, bf16 outputs: a verify of several drafts, or many query heads to a
// key-value head. The products run on the 5th-generation tensor cores.
//
// Warp-level MMA of 16 rows, one m16n8k16 in 8 cycles per scheduler, takes as long
// as the loads at about 24 rows, and tcgen05 some twentieth of that. So its M = 128
// need not be filled with work: the RP (32, 64 or 128) rows are repeated 128 / RP
// times along M, and copy c only ever looks at the c-th share of a tile's tokens:
//   S  = Q K^T      [128 lanes][TK tokens], every lane against every token;
//   P               lane of copy c: weights of its share, 0 elsewhere (the zero
//                   blocks are written once);
//   O += P V        [128 lanes][D]: one online softmax per lane.
// A thread owns a lane: its row's maximum, sum and weights need no exchange
// between threads, and the four softmax warps share the tile's tokens evenly.
// The copies are joined as the pieces of a split are.
//
// What bounds it: in the steady state HBM with 32 rows (0.88 us per 64 tokens and SM
// with heads of 128, floor 0.735; 1.38 of 256, floor 1.47), the softmax warps with
// more (1.00 and 1.74 us for 64 and 128 rows of 128; 0.89 for 64 of 64, floor 0.37),
// where a thread's 32 and 64 weights of a tile take longer than its loads; and in each
// item its start and end, with no loads in flight, about 6 us with 32 rows of 128, 9 of
// 256, 12 with 128 rows, which the split counts (Plan::item_cost). 64 requests of
// 500-8,000 tokens, 2 kv heads, 32, 64 and 128 rows: heads of 64 48, 72 and 129 us for a
// floor of 21, of 128 70, 85 and 140 for 43, of 256 106, 125 and 178 for 85.
//
// Roles: warps 0-3 softmax (thread = TMEM lane), 4-7 load, 8 issues Q K^T, 9
// issues P V (one warp for both would make each wait for the other's operands).
// K and V tiles pass through a ring of U units (16-byte asynchronous copies, as
// pages may end anywhere). S, and P as the A operand, lie in tensor memory, S in
// two buffers and P in NB, so scores, weights and value sums of successive tiles
// overlap. The weights go in PT = 2 bf16 parts (2^-16 together), each a product of
// its own.
//
// The value sums stay in the unit, which cuts off below the last place of what it
// adds to: with 128 rows that takes 1e-4 off the outputs over 16,384 tokens and 8.6e-4
// over 131,072, where a bf16 output is rounded by up to 3.9e-3. So a piece goes in
// runs of up to kRun units, whose sums are joined in fp32 with rounding, and the loss
// stays below 2^-11 (4,096 products of 16 tokens) at any length. (48 requests of
// 60k-131k tokens, 32 rows of 128: 886 us in runs, 876 at a stretch.)
// fp32 outputs take attn_kernel.cuh, which adds every 16 tokens with rounding.
#pragma once

#include "attn_common.cuh"

namespace lin {
namespace attn {

template <int D_, int RP_>
struct UCfg {
  static constexpr int D = D_, RP = RP_, PT = 2;
  static constexpr int TK = D == 64 ? 128 : 64;  // tokens of a tile
  static constexpr int UNIT = TK * D * 2;        // its K, or its V
  static constexpr int COPIES = 128 / RP;
  static constexpr int KW = TK / COPIES;         // a copy's tokens
  // q is the A operand: in tensor memory for heads of up to 128 channels (from
  // shared memory every product reads all 128 lanes of it again, and takes 74
  // cycles for its 16; tensor memory has no room beside O of 256 channels)
  static constexpr bool QT = D <= 128;
  static constexpr int QCOLS = QT ? D / 2 : 0;
  static constexpr int QB = (QT ? RP : 128) * D * 2;
  static constexpr int FREE = 224 * 1024 - QB;
  static constexpr int U = FREE / UNIT < 12 ? FREE / UNIT : 12;
  static constexpr int SMEM = U * UNIT + QB;
  static constexpr int PITCH = D + 4;            // of the joined sums, for the banks
  // tensor memory columns: 2 buffers of S, NB of P (two tokens to a column), O, q
  static constexpr int PCOLS = PT * TK / 2;
  static constexpr int NB = 2 * TK + 2 * PCOLS + D + QCOLS <= 512 ? 2 : 1;
  static constexpr int COLS = 2 * TK + NB * PCOLS + D + QCOLS;
  static constexpr int TMEM = COLS <= 256 ? 256 : 512;
  static constexpr int THREADS = 320;
  static_assert(COLS <= 512 && U >= 4 && SMEM >= 128 * (PITCH + 2) * 4, "");
};

constexpr uint32_t kUmmaWaitTries = 1u << 26;
constexpr int kRun = 512;  // most units of a run

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(umma::smem_u32(bar)) : "memory");
}

// D += A B with A in tensor memory: row i in lane i, two bf16 of a row to a column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      :
      : "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 8 columns of this thread's lane.
__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// True in one lane of the warp, always the same: issues the products and their
// commits. (The compiler keeps what this lane does in uniform registers, which
// the instructions take, where a test of the lane's number leaves moves around
// each of them.)
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) attn_umma_kernel(const Plan p) {
  constexpr int D = C::D, RP = C::RP, PT = C::PT, TK = C::TK, KW = C::KW, U = C::U, NB = C::NB, NT = C::THREADS;
  constexpr int CH = KW < 32 ? KW : 32;  // tokens a thread looks at together
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint64_t b_full[U], b_empty[U], b_s[2], b_sfree[2], b_p[NB], b_pfree[NB], b_q, b_drain;
  __shared__ uint16_t s_valid[16][8];  // live tokens of a tile, 16 to a word; a ring of tiles
  __shared__ uint32_t s_see[32];
  __shared__ int64_t s_scan[NT / 32], s_first[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_bad, s_dead;
  asm volatile("griddepcontrol.launch_dependents;");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const lin_kv_cache_t& c = p.c;
  const lin_attn_args_t& a = p.a;
  if (tid == 0) {
    for (int i = 0; i < U; ++i) umma::mbar_init(&b_full[i], 128 + 4), umma::mbar_init(&b_empty[i], 1);
    for (int i = 0; i < 2; ++i) umma::mbar_init(&b_s[i], 2), umma::mbar_init(&b_sfree[i], 4);
    for (int i = 0; i < NB; ++i) umma::mbar_init(&b_p[i], 4), umma::mbar_init(&b_pfree[i], 1);
    umma::mbar_init(&b_q, 4);
    umma::mbar_init(&b_drain, 2);
    umma::mbar_fence_init();
    s_dead = 0;
  }
  Walk w;
  if (!walk_begin<NT>(p, w, s_scan, s_first)) return;
  if (warp == 8) umma::tmem_alloc(&s_tmem, C::TMEM);
  unsigned char* const qbuf = smem + U * C::UNIT;
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = s_tmem, t_p = tmem + 2 * TK, t_o = t_p + NB * C::PCOLS, t_q = t_o + D;
  float* merge = reinterpret_cast<float*>(smem);
  float2* merge_ml = reinterpret_cast<float2*>(merge + 128 * C::PITCH);

  // the next unit of the ring and its phase, and tiles and runs so far
  int slot = 0;
  uint32_t phase = 0, run = 0, tile0 = 0;
  auto next = [](int& s, uint32_t& ph) {
    if (++s == U) s = 0, ph ^= 1;
  };
  // A thread whose wait runs out waits for nothing more and goes on to the
  // run's end, where all leave: every barrier is still met.
  bool gone = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (gone || umma::mbar_wait(bar, parity, kUmmaWaitTries)) return;
    gone = true;
    s_dead = 1;
    report(a.status, LIN_ST_TIMEOUT);
  };

  int at = w.t0;  // the run's first unit
  while (true) {
    const int t1 = walk_until(p, w), end = min(t1, at + kRun), r = w.r;
    const int hk = head_of(p, w.it), row0 = (w.it - hk * p.row_blocks) * RP;
    const int key_begin = at * kUnit, key_end = end == w.u ? w.len : end * kUnit;
    const int base = w.len - a.n_q;  // tokens that every query sees
    const int tiles = (key_end - key_begin + TK - 1) / TK;

    if (warp < 4) {
      // ---- softmax ---------------------------------------------------------------
      // The queries, row by row, to shared memory: q there (every copy of it), or
      // once, for the lanes to take their rows to tensor memory
      constexpr int CPR = D / 8;
      const uint32_t t_lane = static_cast<uint32_t>(warp * 32) << 16;
      const char* const qsrc = static_cast<const char*>(a.q) + r * a.req_stride + hk * p.group * (D * 2);
#pragma unroll 8
      for (int x = tid; x < RP * CPR; x += 128) {
        const int row = x / CPR, ch = x % CPR, q = row0 + row;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (q < p.rows) {
          const int j = query_of(p, q);
          v = *reinterpret_cast<const uint4*>(qsrc + j * a.token_stride + (q - j * p.group) * (D * 2) + ch * 16);
          v.x ^= p.negate, v.y ^= p.negate, v.z ^= p.negate, v.w ^= p.negate;
        }
#pragma unroll
        for (int k = 0; k < (C::QT ? 1 : C::COPIES); ++k)
          *reinterpret_cast<uint4*>(qbuf + umma::rp_offset(k * RP + row, ch * 8, C::QT ? RP : 128)) = v;
      }
      if (warp == 0) draft_sets(p, r, s_see, s_bad);
      {
        float z[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < D; i += 32) umma::tmem_st32(t_o + t_lane + i, z);
        if (run == 0) {  // other copies' tokens keep weight 0
#pragma unroll 1
          for (int i = 0; i < NB * C::PCOLS; i += 32) umma::tmem_st32(t_p + t_lane + i, z);
        }
      }
      if constexpr (C::QT) {
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int ch = 0; ch < CPR; ch += 2) {
          const uint4 y0 = *reinterpret_cast<const uint4*>(qbuf + umma::rp_offset(tid % RP, ch * 8, RP));
          const uint4 y1 = *reinterpret_cast<const uint4*>(qbuf + umma::rp_offset(tid % RP, ch * 8 + 8, RP));
          const uint32_t v[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
          tmem_st8(t_q + t_lane + ch * 4, v);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      }
      if (!C::QT) umma::fence_smem_to_async();
      umma::fence_before_sync();
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (lane == 0) mbar_arrive(&b_q);
      const int copy = tid / RP, q = row0 + tid % RP;
      const uint32_t see = q < p.rows ? s_see[query_of(p, q)] : 0u;
      float cut = -INFINITY, z = 0.0f, l = 0.0f;  // as in attn_kernel.cuh
      for (int i = 0; i < tiles; ++i) {
        const uint32_t gt = tile0 + i;
        wait(&b_s[gt & 1], (gt >> 1) & 1);
        umma::fence_after_sync();
        const uint32_t t_s = tmem + t_lane + (gt & 1) * TK + copy * KW;
        const int key0 = key_begin + i * TK + copy * KW;  // this copy's first token
        float s[CH];
        // what this row sees of the CH tokens from key0 + x on
        auto sees = [&](int x) {
          const uint16_t* v = &s_valid[gt & 15][(copy * KW + x) / 16];
          uint32_t vis = CH == 16 ? v[0] : v[0] | uint32_t(v[1]) << 16;
          const int sh = key0 + x - base;
          if (sh + CH > 0) vis &= sh >= 0 ? (sh < 32 ? see >> sh : 0u) : (see << -sh) | ((1u << -sh) - 1u);
          return vis;
        };
        auto load = [&](int x) {
          if constexpr (CH == 16)
            umma::tmem_ld16(t_s + x, s);
          else
            umma::tmem_ld32(t_s + x, s);
        };
        constexpr uint32_t ALL = CH == 32 ? ~0u : (1u << (CH & 31)) - 1u;
        float mx = -INFINITY;
#pragma unroll
        for (int x = 0; x < KW; x += CH) {
          load(x);
          const uint32_t vis = sees(x);
          if (vis != ALL) {
#pragma unroll
            for (int k = 0; k < CH; ++k)
              if (!((vis >> k) & 1u)) s[k] = -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < CH; ++k) mx = fmaxf(mx, s[k]);
        }
        float f = 1.0f;
        if (mx > cut) {
          const float y = -mx * p.scale_log2;
          f = cut == -INFINITY ? 0.0f : exp2_fast(y - z);
          z = y, cut = mx + p.slack, l *= f;
        }
        const bool rescale = i > 0 && __any_sync(~0u, f != 1.0f);
        const bool drafts = key_begin + (i + 1) * TK > base && a.n_q > 1;
        // the buffer's last product has read it; where O is touched, all have ended
        if (gt >= NB) wait(&b_pfree[gt % NB], (gt / NB - 1) & 1);
        if (NB > 1 && i > 0 && (rescale || drafts)) wait(&b_pfree[(gt - 1) % NB], ((gt - 1) / NB) & 1);
        umma::fence_after_sync();
        if (rescale) {
#pragma unroll
          for (int x = 0; x < D; x += 32) {
            float o[32];
            umma::tmem_ld32(t_o + t_lane + x, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= f;
            umma::tmem_st32(t_o + t_lane + x, o);
          }
        }
        // values that are infinite or NaN: 0 in the product, added by hand to the
        // rows that see them (only drafts can be hidden from some rows)
        bool wild = false;
        unsigned char* vbuf = nullptr;
        if (drafts) {
          // this tile's V is the unit after its K
          int sl = slot;
          uint32_t ph = phase;
          next(sl, ph);
          vbuf = smem + sl * C::UNIT;
          wait(&b_full[sl], ph);
          const int tile_key = key_begin + i * TK;
          const int from = max(0, base - tile_key), many = min(TK, key_end - tile_key) - from;
          for (int x = tid; x < many * CPR; x += 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(vbuf + umma::rp_offset(from + x / CPR, x % CPR * 8, TK));
            const uint32_t y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              wild |= (y[k] & 0x7f800000u) == 0x7f800000u || (y[k] & 0x7f80u) == 0x7f80u;
          }
          int any;
          asm volatile(
              "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\t"
              "selp.b32 %0, 1, 0, q;\n\t}"
              : "=r"(any)
              : "r"(static_cast<int>(wild))
              : "memory");
          wild = any != 0;
        }
#pragma unroll
        for (int x = 0; x < KW; x += CH) {
          if (KW > CH) load(x);
          const uint32_t vis = sees(x);
#pragma unroll
          for (int k = 0; k < CH; ++k) s[k] = exp2_fast(fmaf(s[k], p.scale_log2, z));
          if (vis != ALL) {
#pragma unroll
            for (int k = 0; k < CH; ++k)
              if (!((vis >> k) & 1u)) s[k] = 0.0f;
          }
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < CH; ++k) sum[k & 3] += s[k];
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          if (wild) {
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
              float o[32];
              umma::tmem_ld32(t_o + t_lane + d, o);
#pragma unroll 1
              for (int k = 0; k < CH; ++k) {
                float pk = 0.0f;
#pragma unroll
                for (int y = 0; y < CH; ++y) pk = y == k ? s[y] : pk;
                const bool seen = (vis >> k) & 1u;
#pragma unroll
                for (int y = 0; y < 32; ++y) {
                  const float v = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(
                      vbuf + umma::rp_offset(copy * KW + x + k, d + y, TK)));
                  if (seen && !isfinite(v)) o[y] = fmaf(pk, v, o[y]);
                }
              }
              umma::tmem_st32(t_o + t_lane + d, o);
            }
          }
#pragma unroll
          for (int part = 0; part < PT; ++part)
#pragma unroll
            for (int k = 0; k < CH; k += 16) {
              uint32_t v[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) v[y] = take_bf16(s[k + 2 * y], s[k + 2 * y + 1]);
              tmem_st8(t_p + t_lane + (gt % NB) * C::PCOLS + part * (TK / 2) + (copy * KW + x + k) / 2, v);
            }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        if (wild) {
          asm volatile("bar.sync 1, 128;" ::: "memory");  // every row has read V
          for (int x = tid; x < C::UNIT / 4; x += 128) {
            uint32_t& v = reinterpret_cast<uint32_t*>(vbuf)[x];
            if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
            if ((v & 0x7f800000u) == 0x7f800000u) v &= 0x0000ffffu;
          }
          umma::fence_smem_to_async();
        }
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_sfree[gt & 1]), mbar_arrive(&b_p[gt % NB]);
        next(slot, phase);
        next(slot, phase);
      }
      if (tiles > 0) wait(&b_pfree[(tile0 + tiles - 1) % NB], ((tile0 + tiles - 1) / NB) & 1);
      umma::fence_after_sync();
      asm volatile("bar.sync 1, 128;" ::: "memory");  // every lane's products are done
#pragma unroll
      for (int x = 0; x < D; x += 32) {
        float o[32];
        umma::tmem_ld32(t_o + t_lane + x, o);
#pragma unroll
        for (int k = 0; k < 32; k += 4)
          *reinterpret_cast<float4*>(merge + tid * C::PITCH + x + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
      }
      merge_ml[tid] = make_float2(cut == -INFINITY ? cut : -z, l);
      umma::fence_before_sync();
    } else if (warp < 8) {
      // ---- loads: warp 4 + x brings the x-th quarter of a tile's tokens ------------
      constexpr int RW = TK / 4, CPR = D / 8;
      const int lw = warp - 4;
      const char* kb = static_cast<const char*>(c.k) + a.layer * c.layer_stride + hk * c.head_stride;
      const char* vb = static_cast<const char*>(c.v) + a.layer * c.layer_stride + hk * c.head_stride;
      const int32_t* table = a.page_table + r * a.page_table_stride;
      int key = key_begin + lw * RW + (lane & (RW - 1));
      int id = key < key_end ? table[page_of(p, key)] : -1;
      // Lane's place in a unit: row lane / CPR + x (32 / CPR) of its warp's rows, so
      // that the swizzle of step x is an exclusive-or with a constant.
      constexpr int STEP = 32 / CPR;
      const uint32_t place = umma::smem_u32(smem) + umma::rp_offset(lw * RW + lane / CPR, (lane % CPR) * 8, TK);
      for (int i = 0; i < tiles; ++i) {
        const bool live = static_cast<uint32_t>(id) < static_cast<uint32_t>(c.num_pages);
        if (key < key_end && !live && lane < RW) report(a.status, LIN_ST_BAD_PAGE);
        const int64_t off = live ? id * c.page_stride + (key - page_of(p, key) * c.page_size) * c.token_stride : 0;
        const uint32_t valid = __ballot_sync(~0u, live);
        key += TK;
        id = key < key_end ? table[page_of(p, key)] : -1;
        if (lane == 0) {
          uint16_t* v = &s_valid[(tile0 + i) & 15][lw * (RW / 16)];
          v[0] = static_cast<uint16_t>(valid);
          if (RW == 32) v[1] = static_cast<uint16_t>(valid >> 16);
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          wait(&b_empty[slot], phase ^ 1);
          const uint32_t dst = place + slot * C::UNIT;
          const char* src = (kv ? vb : kb) + (lane % CPR) * 16;
#pragma unroll
          for (int x = 0; x < RW / STEP; ++x) {
            const int row = x * STEP + lane / CPR;
            const int64_t o = __shfl_sync(~0u, off, row);
            cp16((dst ^ ((x * STEP & 7) << 4)) + x * STEP * 128, src + o, (valid >> row) & 1u);
          }
          // The unit is full when every lane's copies have landed: nobody waits
          // here. (A proxy fence here would wait for all copies in flight; the
          // thread that issues the products has one.)
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(umma::smem_u32(&b_full[slot])) : "memory");
          if (lane == 0) mbar_arrive(&b_full[slot]);  // and passes on s_valid
          next(slot, phase);
        }
      }
    } else {
      // ---- MMA issue: S = Q K^T by warp 8, O += P V by warp 9 -----------------------
      // Descriptors of the buffers' starts; a step within one is a sum to the
      // address field, which holds 18-bit shared-memory addresses / 16.
      const bool scores = warp == 8;
      if (run == 0 && !scores) next(slot, phase);  // K of tile t is unit 2 t, V unit 2 t + 1
      if (scores) {
        constexpr uint32_t id_s = umma::idesc_f16(128, TK, true, false, false);
        const uint64_t q_desc = umma::desc_kmajor(umma::smem_u32(qbuf), 128, 0);
        const uint64_t k_desc = umma::desc_kmajor(umma::smem_u32(smem), TK, 0);
        auto step = [](int rows, int k) { return uint64_t(((k >> 6) * rows * 128 + (k & 63) * 2) >> 4); };
        wait(&b_q, run & 1);
        for (int i = 0; i < tiles; ++i) {
          const uint32_t gt = tile0 + i;
          wait(&b_full[slot], phase);
          wait(&b_sfree[gt & 1], ((gt >> 1) & 1) ^ 1);
          umma::fence_after_sync();
          umma::fence_smem_to_async();
          if (elect_one()) {
            const uint64_t kd = k_desc + slot * (C::UNIT >> 4);
#pragma unroll
            for (int k = 0; k < D; k += 16)
              if constexpr (C::QT)
                mma_ts(tmem + (gt & 1) * TK, t_q + k / 2, kd + step(TK, k), id_s, k > 0);
              else
                umma::mma_f16(tmem + (gt & 1) * TK, q_desc + step(128, k), kd + step(TK, k), id_s, k > 0);
            umma::mma_commit(&b_s[gt & 1]);
            umma::mma_commit(&b_empty[slot]);
            mbar_arrive(&b_s[gt & 1]);  // passes on what the loaders wrote besides the tile
          }
          __syncwarp();
          next(slot, phase);
          next(slot, phase);
        }
      } else {
        constexpr int NV = D < 128 ? D : 128;
        constexpr uint32_t id_o = umma::idesc_f16(128, NV, true, false, true);
        const uint64_t v_desc = umma::desc_mnmajor(umma::smem_u32(smem), TK, 0);
        for (int i = 0; i < tiles; ++i) {
          const uint32_t gt = tile0 + i;
          wait(&b_full[slot], phase);
          umma::fence_smem_to_async();
          wait(&b_p[gt % NB], (gt / NB) & 1);
          umma::fence_after_sync();
          if (elect_one()) {
            const uint64_t vd = v_desc + slot * (C::UNIT >> 4);
            const uint32_t pa = t_p + (gt % NB) * C::PCOLS;
#pragma unroll
            for (int part = PT - 1; part >= 0; --part)
#pragma unroll
              for (int n = 0; n < D; n += NV)
#pragma unroll
                for (int k = 0; k < TK; k += 16)
                  mma_ts(t_o + n, pa + part * (TK / 2) + k / 2, vd + (((n / 64) * (TK * 128) + k * 128) >> 4), id_o, 1);
            umma::mma_commit(&b_pfree[gt % NB]);
            umma::mma_commit(&b_empty[slot]);
          }
          __syncwarp();
          next(slot, phase);
          next(slot, phase);
        }
      }
    }
    __syncthreads();
    if (s_dead) {
      // a wait ran out: let copies and products in flight finish, then leave
      cp_wait_all();
      if (warp >= 8 && elect_one()) {
        umma::mma_commit(&b_drain);
        umma::mbar_wait(&b_drain, 0, kUmmaWaitTries);
      }
      // The parts that this range now leaves unwritten, of the piece at hand and of an
      // item that goes on past the range, count as left out, and their items with them.
      for (int x = tid; x < 2 * RP; x += NT)
        if (x >= RP || w.t0 > 0)
          p.part_ml[2 * int64_t(blockIdx.x) * RP + x] = make_float2(-INFINITY, kLeftOut);
      w.split.x = -1;
      break;
    }
    if (at > w.t0) {
      carry_in<D, RP, NT, C::PITCH>(p, w, merge, merge_ml);
      __syncthreads();
    }
    finish_piece<D, C::COPIES, RP, NT, C::PITCH>(p, w, end, merge, merge_ml, s_bad && end == t1);
    tile0 += tiles;
    ++run;
    at = end;
    if (end == t1) {
      if (!walk_next(p, w, t1)) break;
      at = w.t0;
    }
    umma::fence_smem_to_async();
    __syncthreads();  // the join is read before the ring is filled again
  }
  __syncthreads();
  if (warp == 8) umma::tmem_dealloc(tmem, C::TMEM);
  if (tid == 0) p.split[blockIdx.x] = w.split;
}

template <class C>
cudaError_t launch_umma(const Plan& p, int grid, cudaStream_t s) {
  auto kern = attn_umma_kernel<C>;
  static bool ready[kMaxDevices];  // set twice at worst, to the same value
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev] = true;
  }
  kern<<<grid, C::THREADS, C::SMEM, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_umma_rows(const Plan& p, int grid, cudaStream_t s) {
  switch (p.block_rows) {
    case 32: return launch_umma<UCfg<D, 32>>(p, grid, s);
    case 64: return launch_umma<UCfg<D, 64>>(p, grid, s);
    default: return launch_umma<UCfg<D, 128>>(p, grid, s);
  }
}

}  // namespace attn
}  // namespace lin
