// Chunk attention over bf16 caches with bf16 outputs, on the 5th-generation tensor cores.
//
//   S = Q K^T,  P = 2^(S scale log2(e) - m),  O = sum over tiles of P V,  out = O / sum P
//
// in tiles of 128 rows (new tokens x query heads of one kv head) and TK keys, with a
// running maximum and sum per row. A prompt's floor is the tensor unit's (4 head_dim flops
// per visible row and key), that of a few rows over a long cache HBM's. Measured:
//   8 prompts of 4,096 tokens, 16 / 2 heads of 128             451 us, 1,219 TFLOP/s
//   1,024 tokens after 31,000, 32 / 8 heads of 128             370 us, 1,430 TFLOP/s
//   64 x 1-512 after 200-8,000, 16 / 2 heads of 256          1,350 us,   938 TFLOP/s
//   4 x 1,500-2,500 after 0-3,000, 8 / 8 heads of 64            79 us,   533 TFLOP/s
//   32 x 1-16 after 1,000-16,000, 16 / 2 heads of 128           69 us, 4.5 TB/s
// What bounds prompts now is the chain below and the items' starts and ends: with heads of
// 128 the tensor pipe is busy 49% of the time, with heads of 64, whose products are half as
// long to a weight, 26%, and no unit is full (issue 43%, exponentials 27%). Heads of 256
// (tensor pipe 43%) wait for loads, which begin about a tile ahead, as the rings hold 1.25
// tiles of K and one of V: 5 GB from L2 at 6.8 TB/s, 23% of what L2 gives. Groups of query
// heads that do not divide 128 load their queries by 16-byte copies: 8 prompts of 2,048,
// 28 / 4 heads of 128 814 TFLOP/s, 32 / 4 998.
// The two-tile kernels (128 registers at launch, which setmaxnreg hands out anew) spill some
// 100 bytes.
//
// An item has NQ row tiles. What counts is that the unit always has a product to make: a
// tile's chain (S, its way to the registers, the weights, their way back, P V) is some
// 4,000 cycles long for 128 keys of heads of 128, of which the unit works 1,100. So the
// next S is made while the softmax works on the last, which takes room in tensor memory
// for a second S or for P beside S.
//   NQ = 1 (heads of 256, whose O alone takes half of tensor memory, few rows, and calls with
//   little work): two
//   buffers of S with TK = 128, P in its S's place. A warp issues S, another P V.
//   NQ = 2 (heads of 64 and 128): one S each, which is free once it is in registers, and P
//   beside it: TK = 96 and 80, as S, P and O of both fit. (With TK = 128 and P in S's
//   place, 653 us for 8 prompts of 4,096 tokens, 16 heads of 128.) A warp for each row
//   tile issues its products, as an issue waits until the unit is near it.
//
// Roles: 4 NQ softmax warps (thread = row = tensor-memory lane, so no exchange between
// threads), a warp that loads K and one that loads V, each into a ring of its own, two that
// issue products, one that hands out the pieces (chunk_common.cuh), two that load Q and look
// over values (below). Each goes through the pieces by itself, so one item's end overlaps
// the next one's start. Pages of a multiple of 8 tokens come by TMA, in boxes of 8, 16 or
// 32 tokens; others, whose tokens may begin anywhere in a tile's swizzle, by 16-byte
// asynchronous copies, after which the products need a proxy fence.
//
// P goes back to tensor memory, as the A operand of P V, rounded to
// bf16: one more rounding of 2^-9 rms beside the output's own; the sums are of the
// unrounded weights.
//
// The reference m. A piece's first tile takes its rows' maxima. After that the weights
// are made at once with the reference at hand, and only where a tile's sum of a row passes
// 2^8 are the maxima looked up, the row's sums rescaled and the weights
// made again: a tile in some thousand, which saves the others the pass over the scores.
//
// Hidden values: 0 NaN is NaN, so in tiles that some row of the item does not see whole
// (the last ones) the values are looked over; infinities and NaN are 0 in the product
// and go to the rows that see them by themselves.
//
// The value sums stay in the unit, which cuts off below the last place of what it adds
// to; after kRun tiles they are added to sums in the workspace with rounding, which keeps
// the loss below 2^-11 of the sum p |v| at any length.
#pragma once

#include "chunk_common.cuh"

namespace lin {
namespace chunk {

constexpr int kValidRing = 16, kCheckRing = 8;  // tiles, looked-over tiles under way and some more

template <int D_, int NQ_, bool TMA_>
struct UCfg {
  static constexpr int D = D_, NQ = NQ_;
  static constexpr bool TMA = TMA_;
  static constexpr int TK = NQ == 1 ? 128 : D == 64 ? 96 : 80;
  // a ring unit: 64 or 128 channels of a tile's K, up to 128 of its V
  static constexpr int DK = NQ == 2 && D == 128 ? 128 : 64, KU = D / DK, KB = TK * DK * 2;
  static constexpr int DV = D < 128 ? D : 128, VU = D / DV, VB = TK * DV * 2;
  static constexpr int QT = 128 * D * 2;        // a row tile's queries
  static constexpr int SOFT = 4 * NQ;           // softmax warps
  static constexpr int STAGE = SOFT * 4096;     // where outputs are turned into rows
  // units of the rings: at least a tile of each
  static constexpr int NK = D == 256 ? 5 : DK == 128 ? 3 : 6;
  static constexpr int NV = D == 64 ? 6 : NQ == 2 ? 3 : 2;
  static constexpr int RING = NK * KB + NV * VB;
  static constexpr int SMEM = RING + NQ * QT + STAGE;
  static constexpr int THREADS = SOFT * 32 + 256;
  // tensor memory columns: 2 of S, P in their places or beside, NQ of O
  static constexpr bool APART = NQ == 2;
  static constexpr int T_P = APART ? 2 * TK : 0, P_STEP = APART ? TK / 2 : TK;
  static constexpr int T_O = 512 - NQ * D;
  static constexpr int TMEM = 512;
  static_assert(2 * TK + (APART ? TK : 0) <= T_O && TK % 16 == 0 && NK >= KU && NV >= VU && SMEM <= 224 * 1024, "");
};

constexpr uint32_t kWaitTries = 1u << 24;
constexpr int kRun = 256;     // most tiles whose value sums stay in the unit
constexpr int kPieces = 4;    // pieces handed out ahead
constexpr float kMostSum = 256.0f;  // of a tile's weights, before the reference moves

struct UPiece {
  Piece x;
  int nt[2];    // tiles of the row tiles
  int n;        // the larger
  int g0;       // tiles of the pieces before
  int check0;   // values are looked over from this tile on
};

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(umma::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(umma::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void arrive_copies(uint64_t* bar) {  // when this thread's copies have landed
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(umma::smem_u32(bar)) : "memory");
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
__device__ __forceinline__ void mbar_arrive_many(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(umma::smem_u32(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(umma::smem_u32(bar)), "r"(bytes) : "memory");
}
// A box of 64 channels x some tokens of one head and page; zeros where the page is none.
__device__ __forceinline__ void load_box(const CUtensorMap* map, uint32_t dst, uint64_t* bar, int channel, int token,
                                         int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(channel), "r"(token), "r"(head), "r"(page), "r"(umma::smem_u32(bar))
      : "memory");
}
// A box of 64 channels of the queries: the item's heads of the row tile's tokens.
__device__ __forceinline__ void load_q(const CUtensorMap* map, uint32_t dst, uint64_t* bar, int channel, int head, int token) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(channel), "r"(head), "r"(token), "r"(umma::smem_u32(bar))
      : "memory");
}
// One lane of the warp, always the same (what it does stays in uniform registers).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void f2unpack(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 32 columns of this thread's lane, without a wait.
__device__ __forceinline__ void tmem_issue32(uint32_t at, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_issue16(uint32_t at, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(at));
}
__device__ __forceinline__ void landed16(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}
__device__ __forceinline__ void tmem_put8(uint32_t at, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// The values are there from here on: no use of them moves above.
__device__ __forceinline__ void landed32(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 8 columns of this thread's lane, there and back.
__device__ __forceinline__ void tmem_get8(uint32_t at, float (&o)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void tmem_set8(uint32_t at, const float (&o)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\ttcgen05.wait::st.sync.aligned;" ::"r"(at),
               "f"(o[0]), "f"(o[1]), "f"(o[2]), "f"(o[3]), "f"(o[4]), "f"(o[5]), "f"(o[6]), "f"(o[7])
               : "memory");
}

// A place of the ring and its phase.
template <int U>
struct At {
  int slot;
  uint32_t phase;
  __device__ __forceinline__ void step(int n) {
    slot += n;
    if (slot >= U) slot -= U, phase ^= 1;
  }
  __device__ __forceinline__ At plus(int n) const {
    At y = *this;
    y.step(n);
    return y;
  }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
chunk_umma_kernel(const Plan p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                  const __grid_constant__ CUtensorMap q_map) {
  constexpr int D = C::D, NQ = C::NQ, TK = C::TK, KU = C::KU, VU = C::VU, DV = C::DV, DK = C::DK, NK = C::NK, NV = C::NV;
  constexpr int NT = C::THREADS, SOFT = C::SOFT;
  constexpr bool TMA = C::TMA;
  constexpr int KFULL = TMA ? 1 : 32 + 1, VFULL = TMA ? 2 : 32 + 2;  // arrivals of a full unit
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ uint64_t b_kfull[NK], b_kempty[NK], b_vfull[NV], b_vempty[NV], b_qfull[NQ], b_qfree[NQ], b_s[2], b_sfree[2], b_p[2], b_o[2], b_look[kCheckRing], b_check[kCheckRing],
      b_pfull[kPieces], b_pempty[kPieces], b_drain;
  __shared__ UPiece s_piece[kPieces];
  __shared__ uint4 s_valid[kValidRing];  // live keys of a tile; a ring of tiles
  __shared__ uint4 s_wild[kCheckRing];   // keys of a looked-over tile with values that are not finite
  __shared__ WalkShared s_walk;
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const lin_kv_cache_t& c = p.c;
  const lin_attn_chunk_args_t& a = p.a;
  if (tid == 0) {
    for (int i = 0; i < NK; ++i) umma::mbar_init(&b_kfull[i], KFULL), umma::mbar_init(&b_kempty[i], NQ);
    for (int i = 0; i < NV; ++i) umma::mbar_init(&b_vfull[i], VFULL), umma::mbar_init(&b_vempty[i], NQ);
    for (int i = 0; i < NQ; ++i) umma::mbar_init(&b_qfull[i], p.q_box ? 1 : 64), umma::mbar_init(&b_qfree[i], 1);
    for (int i = 0; i < 2; ++i) umma::mbar_init(&b_s[i], 2), umma::mbar_init(&b_sfree[i], 4), umma::mbar_init(&b_p[i], 4), umma::mbar_init(&b_o[i], 1);
    for (int i = 0; i < kCheckRing; ++i) umma::mbar_init(&b_look[i], (TMA ? 1 : 32) * VU), umma::mbar_init(&b_check[i], 2);
    for (int i = 0; i < kPieces; ++i) umma::mbar_init(&b_pfull[i], 1), umma::mbar_init(&b_pempty[i], SOFT + 2 + 2 + 2);
    umma::mbar_init(&b_drain, 2);
    umma::mbar_fence_init();
    s_dead = 0;
  }
  Walk w;
  const bool tickets_on = one_by_one(p);
  if (!tickets_on) {
    if (!walk_begin<NT>(p, w, s_walk)) return;
  } else if (blockIdx.x == 0) {
#pragma unroll 1
    for (int r = tid; r < a.batch; r += NT) request(p, r, true);
  }
  // pieces handed out ahead: the next alone where another CTA could take it
  const int pieces = tickets_on ? 1 : kPieces;
  if (warp == SOFT + 2) umma::tmem_alloc(&s_tmem, C::TMEM);
  umma::fence_before_sync();
  __syncthreads();
  umma::fence_after_sync();
  const uint32_t tmem = s_tmem, t_o = tmem + C::T_O;
  unsigned char* const vbuf = smem + NK * C::KB;
  unsigned char* const qbuf = smem + C::RING;
  unsigned char* const stage = qbuf + NQ * C::QT;

  // A warp whose wait runs out waits for nothing more and goes to the end, and so do the
  // others in their turn. Called by whole warps, and the same for all lanes. (A look at a
  // barrier takes 45 cycles, a wait that may sleep 200 even where the phase is over.)
  bool gone = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (gone || __all_sync(~0u, mbar_test(bar, parity))) return;
    uint32_t left = kWaitTries;
#pragma unroll 1
    while (!__all_sync(~0u, umma::mbar_try_wait(bar, parity)))
      if (--left == 0) {
        gone = true;
        break;
      }
  };
  int at_piece = 0;
  uint32_t piece_phase = 0;
  // The next piece, by a whole warp, NULL at the end; what is needed of it is copied
  // before it is given back.
  auto take = [&]() -> const UPiece* {
    wait(&b_pfull[at_piece], piece_phase);
    if (gone || s_piece[at_piece].x.r < 0) return nullptr;
    return &s_piece[at_piece];
  };
  auto give_back = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&b_pempty[at_piece]);
    if (++at_piece == pieces) at_piece = 0, piece_phase ^= 1;
  };

  if (warp < SOFT) {
    // ---- softmax ------------------------------------------------------------------------
    if constexpr (NQ == 2)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int st = warp >> 2;  // row tile
    const int row = st * 128 + (tid & 127);
    const uint32_t t_lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t to = t_o + t_lane + st * D;
    const uint64_t scale2 = f2pack(p.scale_log2, p.scale_log2);
    uint32_t ct = 0, chk = 0;  // tiles, looked-over tiles so far
    // The product of tile t has ended. (A barrier for each buffer: when S of tile t is
    // there, the product of t - 2 has ended, and that of t - 1 need not have.)
    auto wait_o = [&](uint32_t t) { wait(&b_o[NQ == 2 ? st : t & 1], (NQ == 2 ? t : t >> 1) & 1); };
#pragma unroll 1
    while (const UPiece* piece = take()) {
      const UPiece y = *piece;
      give_back();
      const Piece& x = y.x;
      const int tok = token_of(p, row), head = row - tok * p.bheads;
      const bool mine = tok < x.tokens && head < x.heads;
      const int sees = mine ? max(0, x.pos + tok + 1) : 0;
      const int all_see = max(0, x.pos + token_of(p, st * 128) + 1);  // what every row of the tile sees
      const int nt = st == 0 ? y.nt[0] : y.nt[1];
      float4* const acc = reinterpret_cast<float4*>(p.part) + int64_t(x.part) * (D / 4) * p.rows + row;  // sums of earlier runs
      float cut = -INFINITY, z = 0.0f, l = 0.0f, z_acc = 0.0f;
      bool has_acc = false, unset = true;
      // looked-over tiles that are not this row tile's
      const int first_chk = max(x.t0, y.check0), chk_before = chk;
#pragma unroll 1
      for (int i = 0; i < nt && !gone; ++i) {
        const int tile = x.t0 + i, key0 = tile * TK;
        const int buf = NQ == 2 ? st : ct & 1;
        const uint32_t ts = tmem + t_lane + buf * TK;
        wait(&b_s[buf], (NQ == 2 ? ct : ct >> 1) & 1);
        umma::fence_after_sync();
        const uint4 valid = s_valid[(y.g0 + i) & (kValidRing - 1)];
        const bool first = i % kRun == 0;
        if (first && i > 0) {  // a run's end: its sums to the workspace
          wait_o(ct - 1);
          umma::fence_after_sync();
          const float f = has_acc ? attn::exp2_fast(z - z_acc) : 0.0f;
#pragma unroll 1
          for (int d = 0; d < D; d += 8) {
            float o[8];
            tmem_get8(to + d, o);
#pragma unroll
            for (int k = 0; k < 8; k += 4) {
              float4* m = acc + int64_t((d + k) / 4) * p.rows;
              const float4 was = i == kRun ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *m;
              *m = make_float4(fmaf(was.x, f, o[k]), fmaf(was.y, f, o[k + 1]), fmaf(was.z, f, o[k + 2]), fmaf(was.w, f, o[k + 3]));
            }
          }
          z_acc = z, has_acc = cut != -INFINITY;
        }
        const bool masked = key0 + TK > all_see || (valid.x & valid.y & valid.z & valid.w) != ~0u;
        float s[TK];
#pragma unroll
        for (int k = 0; k + 32 <= TK; k += 32) tmem_issue32(ts + k, s + k);
        if (TK % 32) tmem_issue16(ts + TK / 32 * 32, s + TK / 32 * 32);
        tmem_loaded();
#pragma unroll
        for (int k = 0; k + 32 <= TK; k += 32) landed32(s + k);
        if (TK % 32) landed16(s + TK / 32 * 32);
        if (C::APART) {  // the next scores may come
          umma::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b_sfree[st]);
        }
        if (p.negate) {
#pragma unroll
          for (int k = 0; k < TK; ++k) s[k] = -s[k];
        }
        if (masked) {
          const uint32_t live[4] = {valid.x, valid.y, valid.z, valid.w};
#pragma unroll
          for (int x = 0; x < TK; x += 32) {
            const int n = sees - key0 - x;
            const uint32_t vis = n <= 0 ? 0u : n >= 32 ? live[x / 32] : live[x / 32] & ((1u << n) - 1u);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (x + k < TK && !((vis >> k) & 1u)) s[x + k] = -INFINITY;
          }
        }
        uint32_t pk[TK / 2];
        float sum = 0.0f;
        // Looked up beforehand while some row of the warp has no reference (which moves no
        // other row's: sum is not made yet), and after the weights where a sum says so. A NaN
        // in a row's sum is there to stay, and wants no look.
        bool told = false;  // the look-up has seen the sums
#pragma unroll 1
        for (bool look_up = unset;; look_up = told = true) {
          if (look_up) {  // the reference, and what follows from its move
            float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int k = 4; k + 8 <= TK; k += 8)
#pragma unroll
              for (int x = 0; x < 4; ++x) top[x] = max3(top[x], s[k + x], s[k + 4 + x]);
#pragma unroll
            for (int x = 0; x < 4; ++x) top[x] = fmaxf(top[x], s[TK - 4 + x]);
            const float mx = fmaxf(max3(top[0], top[1], top[2]), top[3]);
            float f = 1.0f;
            // (a row goes by its own scores alone, whatever made its warp look)
            if (mx > cut && (cut == -INFINITY || sum > kMostSum)) {
              const float y0 = -mx * p.scale_log2;
              f = cut == -INFINITY ? 0.0f : attn::exp2_fast(y0 - z);
              z = y0, cut = mx, l *= f;
            }
            if (!first && __any_sync(~0u, f != 1.0f)) {
              wait_o(ct - 1);  // the last product has ended
              umma::fence_after_sync();
#pragma unroll 1
              for (int d = 0; d < D; d += 8) {
                float o[8];
                tmem_get8(to + d, o);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] *= f;
                tmem_set8(to + d, o);
              }
            }
            // a row that has seen nothing yet, and will see something
            unset = __any_sync(~0u, cut == -INFINITY && l == l && sees > key0 + TK);
          }
          const uint64_t z2 = f2pack(z, z);
          uint64_t add[2] = {0, 0};
#pragma unroll
          for (int k = 0; k < TK / 2; ++k) {
            float e0, e1;
            f2unpack(ffma2(f2pack(s[2 * k], s[2 * k + 1]), scale2, z2), e0, e1);
            e0 = attn::exp2_fast(e0), e1 = attn::exp2_fast(e1);
            add[k & 1] = fadd2(add[k & 1], f2pack(e0, e1));
            pk[k] = pack_bf16(e0, e1);
          }
          sum = mine ? f2sum(fadd2(add[0], add[1])) : 0.0f;
          if (told || !__any_sync(~0u, sum > kMostSum)) break;
        }
        l += sum;
        if (tile >= y.check0) {
          wait(&b_check[chk & (kCheckRing - 1)], (chk / kCheckRing) & 1);
          if (gone) break;  // s_wild may hold anything
          const uint4 wv = s_wild[chk & (kCheckRing - 1)];
          ++chk;
          if (wv.x | wv.y | wv.z | wv.w) {
            if (!first) wait_o(ct - 1);
            umma::fence_after_sync();
            const uint32_t wild[4] = {wv.x, wv.y, wv.z, wv.w};
            const char* vb = static_cast<const char*>(c.v) + a.layer * c.layer_stride + x.hk * c.head_stride;
#pragma unroll 1
            for (int d = 0; d < D; d += 8) {
              float o[8];
              tmem_get8(to + d, o);
              if (first) {  // the product adds to these, as it does not start from 0
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = 0.0f;
              }
#pragma unroll 1
              for (int g = 0; g < 4; ++g) {
                uint32_t left = g == 0 ? wild[0] : g == 1 ? wild[1] : g == 2 ? wild[2] : wild[3];
                for (; left; left &= left - 1) {
                  const int t = key0 + 32 * g + __ffs(left) - 1;
                  if (t >= sees) break;
                  const int pg = page_of(p, t), id = a.page_table[x.r * a.page_table_stride + pg];
                  if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(c.num_pages)) continue;  // (its values were 0)
                  const char* v = vb + id * c.page_stride + (t - pg * c.page_size) * c.token_stride + d * 2;
#pragma unroll
                  for (int k = 0; k < 8; ++k) {
                    const float e = bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(v)[k]);
                    if (!isfinite(e)) o[k] += e;
                  }
                }
              }
              __syncwarp();
              tmem_set8(to + d, o);
            }
          }
        }
        if (C::APART && ct > 0) wait_o(ct - 1);  // the last weights have been used
        umma::fence_after_sync();
#pragma unroll
        for (int k = 0; k < TK / 2; k += 8) tmem_put8(tmem + t_lane + C::T_P + buf * C::P_STEP + k, pk + k);
        tmem_stored();
        umma::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_p[buf]);
        ++ct;
      }
      if (gone) break;
      // the piece's looked-over tiles, those of the other row tile too
      chk = chk_before + max(0, x.t0 + y.n - first_chk);
      // ---- the piece's end ------------------------------------------------------------
      if (nt > 0) wait_o(ct - 1);
      if (gone) break;
      umma::fence_after_sync();
      const float fa = has_acc ? attn::exp2_fast(z - z_acc) : 0.0f;
      const float fo = !x.whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
      unsigned char* const rows = stage + warp * 4096;  // 32 rows of 64 outputs, swizzled
      // the rows that this lane writes 16 bytes of: 4 at a time, 128 bytes of each
      uint16_t* to_row[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = st * 128 + (warp & 3) * 32 + k * 4 + lane / 8, t = token_of(p, r), h = r - t * p.bheads;
        to_row[k] = x.whole && t < x.tokens && h < x.heads
                        ? static_cast<uint16_t*>(a.out) + (int64_t(x.row0 + t) * a.num_q_heads + x.head0 + h) * D + (lane & 7) * 8
                        : nullptr;
      }
#pragma unroll 1
      for (int d = 0; d < D; d += 64) {
        float o[64];
        if (nt > 0) {
          tmem_issue32(to + d, o);
          tmem_issue32(to + d + 32, o + 32);
          tmem_loaded();
          landed32(o);
          landed32(o + 32);
        } else {
#pragma unroll
          for (int k = 0; k < 64; ++k) o[k] = 0.0f;
        }
        if (has_acc) {
#pragma unroll
          for (int k = 0; k < 64; k += 4) {
            const float4 was = acc[int64_t((d + k) / 4) * p.rows];
            o[k] = fmaf(was.x, fa, o[k]), o[k + 1] = fmaf(was.y, fa, o[k + 1]);
            o[k + 2] = fmaf(was.z, fa, o[k + 2]), o[k + 3] = fmaf(was.w, fa, o[k + 3]);
          }
        }
        if (!x.whole) {  // rows of all lanes side by side
#pragma unroll
          for (int k = 0; k < 64; k += 4)
            acc[int64_t((d + k) / 4) * p.rows] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        } else {
#pragma unroll
          for (int k = 0; k < 64; k += 8)
            *reinterpret_cast<uint4*>(rows + lane * 128 + ((k / 8 ^ (lane & 7)) << 4)) =
                make_uint4(pack_bf16(o[k] * fo, o[k + 1] * fo), pack_bf16(o[k + 2] * fo, o[k + 3] * fo),
                           pack_bf16(o[k + 4] * fo, o[k + 5] * fo), pack_bf16(o[k + 6] * fo, o[k + 7] * fo));
          __syncwarp();
          uint4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int q = k * 4 + lane / 8;
            v[k] = *reinterpret_cast<const uint4*>(rows + q * 128 + (((lane & 7) ^ (q & 7)) << 4));
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (to_row[k]) *reinterpret_cast<uint4*>(to_row[k] + d) = v[k];
          __syncwarp();
        }
      }
      if (mine && !x.whole)
        p.part_ml[int64_t(x.part) * p.rows + row] = make_float2(cut == -INFINITY ? cut : -z, l);
      __syncwarp();
    }
  } else {
    if constexpr (NQ == 2)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 128;");
    if (warp < SOFT + 2) {
      // ---- loads of K (first warp) and V --------------------------------------------------
      const bool is_v = warp == SOFT + 1;
      At<NK> rk{0, 0};
      At<NV> rv{0, 0};
      uint32_t chk = 0;
#pragma unroll 1
      while (const UPiece* piece = take()) {
        const int n = piece->n, g0 = piece->g0, keys = piece->x.keys, hk = piece->x.hk, look0 = piece->check0 - piece->x.t0;
        const int32_t* table = a.page_table + piece->x.r * a.page_table_stride;
        int key0 = piece->x.t0 * TK;
        give_back();
        // (TMA) lane b has box b of a tile
        int key = key0 + lane * p.box, id = -1;
        auto look = [&](int k) { return lane * p.box < TK && k < keys ? table[page_of(p, k)] : -1; };
        if (TMA && n > 0) id = look(key);
#pragma unroll 1
        for (int i = 0; i < n && !gone; ++i) {
          uint32_t valid = 0;  // of keys 32 lane and on, in lanes 0 to 3; 1 past the tile
          const uint32_t past = 32 * lane >= TK ? ~0u : 32 * lane + 32 > TK ? ~0u << (TK & 31) : 0u;
          bool live = false;
          int in_page = 0, page = 0;
          int64_t off[4];      // (no TMA) of keys lane, lane + 32, ...
          if constexpr (TMA) {
            live = static_cast<uint32_t>(id) < static_cast<uint32_t>(c.num_pages);
            if (!is_v && lane * p.box < TK && key < keys && !live) report(a.status, LIN_ST_BAD_PAGE);
            in_page = key - page_of(p, key) * c.page_size;
            const uint32_t some = __ballot_sync(~0u, live);
            const uint32_t whole = p.box == 32 ? ~0u : (1u << p.box) - 1u;
#pragma unroll 1
            for (int b = 0; b < 32; b += p.box)
              if ((some >> ((32 * lane + b) / p.box & 31)) & 1u) valid |= whole << b;
            const int left = keys - key0 - 32 * lane;
            if (left < 32) valid = left <= 0 ? 0u : valid & ((1u << left) - 1u);
            valid |= past;
            page = live ? id : c.num_pages;  // (past the last: zeros)
            key += TK;
            id = look(key);
          } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const int k = key0 + 32 * h + lane;
              const int pg = page_of(p, k), at = k < keys ? table[pg] : -1;
              const bool ok = static_cast<uint32_t>(at) < static_cast<uint32_t>(c.num_pages);
              if (!is_v && k < keys && !ok) report(a.status, LIN_ST_BAD_PAGE);
              off[h] = ok ? at * c.page_stride + (k - pg * c.page_size) * c.token_stride : 0;
              const uint32_t some = __ballot_sync(~0u, ok);
              if (lane == h) valid = some | past;
            }
          }
          key0 += TK;
          // 16-byte copies of a unit's rows, `chunks` to each, from channel ch0 on
          auto copies = [&](const void* base, uint32_t dst, int chunks, int ch0) {
            const char* src = static_cast<const char*>(base) + a.layer * c.layer_stride + hk * c.head_stride + ch0 * 2;
            const int step = 32 / chunks, ch = lane % chunks;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const uint32_t ok = __shfl_sync(~0u, valid, h);
#pragma unroll 4
              for (int x = 0; x < 32 && 32 * h + x < TK; x += step) {
                const int row = x + lane / chunks;
                const int64_t o = __shfl_sync(~0u, off[h], row);
                attn::cp16(dst + umma::rp_offset(32 * h + row, ch * 8, TK), src + o + ch * 16, (ok >> row) & 1u);
              }
            }
          };
          if (!is_v) {
#pragma unroll 1
            for (int j = 0; j < KU; ++j) {
              wait(&b_kempty[rk.slot], rk.phase ^ 1);
              if (j == 0 && lane < 4) reinterpret_cast<uint32_t*>(&s_valid[(g0 + i) & (kValidRing - 1)])[lane] = valid;
              __syncwarp();
              const uint32_t dst = umma::smem_u32(smem) + rk.slot * C::KB;
              if constexpr (TMA) {
                if (lane == 0) mbar_expect(&b_kfull[rk.slot], C::KB);  // and passes on s_valid
                __syncwarp();
#pragma unroll
                for (int h = 0; h < DK / 64; ++h)
                  if (lane * p.box < TK)
                    load_box(&k_map, dst + h * (TK * 128) + lane * p.box * 128, &b_kfull[rk.slot], j * DK + h * 64, in_page, hk, page);
              } else {
                copies(c.k, dst, DK / 8, j * DK);
                arrive_copies(&b_kfull[rk.slot]);  // when they have landed: nobody waits here
                if (lane == 0) mbar_arrive(&b_kfull[rk.slot]);
              }
              rk.step(1);
            }
          } else {
            // values that are looked over go to their barrier, and are full after that
            const bool looked = i >= look0;
            uint64_t* const to_look = &b_look[chk & (kCheckRing - 1)];
            if (looked) ++chk;
#pragma unroll 1
            for (int j = 0; j < VU; ++j) {
              wait(&b_vempty[rv.slot], rv.phase ^ 1);
              const uint32_t dst = umma::smem_u32(vbuf) + rv.slot * C::VB;
              uint64_t* const bar = looked ? to_look : &b_vfull[rv.slot];
              if constexpr (TMA) {
                if (lane == 0) {
                  mbar_expect(bar, C::VB);
                  if (!looked) mbar_arrive(bar);
                }
                __syncwarp();
#pragma unroll
                for (int h = 0; h < DV / 64; ++h)
                  if (lane * p.box < TK)
                    load_box(&v_map, dst + h * (TK * 128) + lane * p.box * 128, bar, j * DV + h * 64, in_page, hk, page);
              } else {
                copies(c.v, dst, DV / 8, j * DV);
                arrive_copies(bar);
                if (!looked && lane == 0) mbar_arrive_many(bar, 2);
              }
              rv.step(1);
            }
          }
        }
        if (gone) break;
      }
      if (gone) {  // copies in flight land before the block ends
        auto land = [&](uint64_t* bar, uint32_t parity) {
          for (uint32_t i = 0; i < kWaitTries >> 8 && !umma::mbar_try_wait(bar, parity); ++i) {
          }
        };
        for (int j = 0; !is_v && j < NK; ++j) land(&b_kfull[j], j < rk.slot ? rk.phase : rk.phase ^ 1);
        for (int j = 0; is_v && j < NV; ++j) land(&b_vfull[j], j < rv.slot ? rv.phase : rv.phase ^ 1);
        for (uint32_t j = 0; is_v && j < kCheckRing && j < chk; ++j) land(&b_look[(chk - 1 - j) & (kCheckRing - 1)], ((chk - 1 - j) / kCheckRing) & 1);
      }
      attn::cp_wait_all();
    } else if (warp < SOFT + 4) {
      // ---- products ----------------------------------------------------------------------
      constexpr uint32_t id_s = umma::idesc_f16(128, TK, true, false, false);
      constexpr uint32_t id_o = umma::idesc_f16(128, DV, true, false, true);
      const uint64_t q_desc = umma::desc_kmajor(umma::smem_u32(qbuf), 128, 0);
      const uint64_t k_desc = umma::desc_kmajor(umma::smem_u32(smem), TK, 0);
      const uint64_t v_desc = umma::desc_mnmajor(umma::smem_u32(vbuf), TK, 0);
      const int me = warp - SOFT - 2;                // NQ 2: the row tile; NQ 1: S, or P V
      const int st = NQ == 2 ? me : 0;
      At<NK> rk{0, 0};
      At<NV> rv{0, 0};
      uint32_t ct = 0, cs = 0, qn = 0, chk = 0;
      // (whole warps wait, and one lane issues)
      // all of a tile's K is there
      auto wait_k = [&]() {
#pragma unroll
        for (int j = 0; j < KU; ++j) wait(&b_kfull[rk.plus(j).slot], rk.plus(j).phase);
        if (!TMA) umma::fence_smem_to_async();
      };
      // S of the next tile of K into buffer buf; left out: the tile is passed by
      auto make_s = [&](int buf, bool use, bool last) {
#pragma unroll 1
        for (int j = 0; j < KU; ++j) {
          if (NQ == 1) {  // a unit at a time; else wait_k() has waited
            wait(&b_kfull[rk.slot], rk.phase);
            if (!TMA) umma::fence_smem_to_async();
          }
          if (use) {
            umma::fence_after_sync();
            if (elect_one()) {
              const uint64_t kd = k_desc + rk.slot * (C::KB >> 4), qd = q_desc + ((st * C::QT + j * (DK / 64 * 128 * 128)) >> 4);
#pragma unroll
              for (int k = 0; k < DK; k += 16)
                umma::mma_f16(tmem + buf * TK, qd + ((k / 64 * (128 * 128) + k % 64 * 2) >> 4), kd + ((k / 64 * (TK * 128) + k % 64 * 2) >> 4), id_s, j > 0 || k > 0);
              if (j == KU - 1) {
                umma::mma_commit(&b_s[buf]);
                if (last) umma::mma_commit(&b_qfree[st]);
                mbar_arrive(&b_s[buf]);  // passes on what the loader wrote besides the tile
              }
              umma::mma_commit(&b_kempty[rk.slot]);
            }
            __syncwarp();
          } else if (lane == 0) {
            mbar_arrive(&b_kempty[rk.slot]);
          }
          rk.step(1);
        }
      };
      // O += P V of the next tile of V
      auto make_o = [&](int buf, bool use, bool fresh, bool looked) {
#pragma unroll
        for (int j = 0; j < VU; ++j) wait(&b_vfull[rv.plus(j).slot], rv.plus(j).phase);
        if (looked) {  // (its values are full once they are looked over)
          const uint4 wv = s_wild[chk++ & (kCheckRing - 1)];
          if (wv.x | wv.y | wv.z | wv.w) fresh = false;
        }
        if (!TMA) umma::fence_smem_to_async();
        if (use) {
          wait(&b_p[buf], (NQ == 2 ? ct : ct >> 1) & 1);
          umma::fence_after_sync();
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < VU; ++j) {
              const uint64_t vd = v_desc + ((rv.plus(j).slot * C::VB) >> 4);
#pragma unroll
              for (int k = 0; k < TK; k += 16)
                mma_ts(t_o + st * D + j * DV, tmem + C::T_P + buf * C::P_STEP + k / 2, vd + (k * 128 >> 4), id_o, k > 0 || !fresh);
            }
            umma::mma_commit(&b_o[buf]);
#pragma unroll
            for (int j = 0; j < VU; ++j) umma::mma_commit(&b_vempty[rv.plus(j).slot]);
          }
          __syncwarp();
        } else if (lane == 0) {
#pragma unroll
          for (int j = 0; j < VU; ++j) mbar_arrive(&b_vempty[rv.plus(j).slot]);
        }
        rv.step(VU);
      };
      auto wait_q = [&]() {
        wait(&b_qfull[st], qn++ & 1);
        umma::fence_smem_to_async();
      };
#pragma unroll 1
      while (const UPiece* piece = take()) {
        const int n = piece->n, nt = st == 0 ? piece->nt[0] : piece->nt[1], look0 = piece->check0 - piece->x.t0;
        give_back();
        if (nt > 0 && (NQ == 2 || me == 0)) wait_q();
        if constexpr (NQ == 2) {
#pragma unroll 1
          for (int i = -1; i < n && !gone; ++i) {  // S of tile i + 1, P V of tile i
            if (i + 1 < n) {
              const bool use = i + 1 < nt;
              wait_k();
              if (use && cs > 0) wait(&b_sfree[st], (cs - 1) & 1);  // the last scores are in registers
              if (use) ++cs;
              make_s(st, use, i + 2 == nt);
            }
            if (i >= 0) make_o(st, i < nt, i % kRun == 0, i >= look0);
            if (i >= 0 && i < nt) ++ct;
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < n && !gone; ++i) {
            const int buf = ct & 1;
            if (me == 0) {
              wait(&b_o[buf], (ct >> 1 & 1) ^ 1);  // the weights that lie there have been used
              make_s(buf, true, i + 1 == n);
            } else {
              make_o(buf, true, i % kRun == 0, i >= look0);
            }
            ++ct;
          }
        }
        if (gone) break;
      }
      // products in flight end before tensor memory is given back
      if (elect_one()) umma::mma_commit(&b_drain);
      __syncwarp();
      for (uint32_t i = 0; i < kWaitTries && !umma::mbar_try_wait(&b_drain, 0); ++i) {
      }
    } else if (warp == SOFT + 4) {
      // ---- pieces -------------------------------------------------------------------------
      UPiece y;
      Tickets tickets;
      int g = 0;
      if (pieces == 1) tickets.begin(p);
#pragma unroll 1
      do {
        wait(&b_pempty[at_piece], piece_phase ^ 1);
        if (gone) break;
        if (pieces == 1)
          y.x = tickets.next(p);
        else if (lane == 0)
          y.x = walk_next(p, w);
        if (lane == 0) {
          const Piece& x = y.x;
          y.n = 0, y.g0 = g, y.check0 = INT_MAX;
          y.nt[0] = y.nt[1] = 0;
          if (x.r >= 0) {
#pragma unroll
            for (int st = 0; st < NQ; ++st) {
              if (st * 128 >= x.tokens * p.bheads) continue;
              const int last = min(x.tokens - 1, token_of(p, st * 128 + 127));
              const int keys = max(0, x.pos + last + 1);
              y.nt[st] = max(0, min(x.t1, (keys + TK - 1) / TK) - x.t0);
              y.n = max(y.n, y.nt[st]);
            }
            if (x.keys > max(0, x.pos + 1)) y.check0 = max(0, x.pos + 1) / TK;
            // TMA brings what lies behind the last key in its box
            if (TMA && x.keys % p.box) y.check0 = min(y.check0, x.keys / TK);
            g += y.n;
          }
          s_piece[at_piece] = y;
          mbar_arrive(&b_pfull[at_piece]);
        }
        if (++at_piece == pieces) at_piece = 0, piece_phase ^= 1;
        y.x.r = __shfl_sync(~0u, y.x.r, 0);
      } while (y.x.r >= 0);
    } else if (warp < SOFT + 7) {
      // ---- queries, and a look at the values -------------------------------------------------
      constexpr int CPR = D / 8;
      const int me = tid - (SOFT + 5) * 32;
      At<NV> rv{0, 0};
      uint32_t qn[2] = {0, 0}, chk = 0;
#pragma unroll 1
      while (const UPiece* piece = take()) {
        const int n = piece->n, look0 = piece->check0 - piece->x.t0, tokens = piece->x.tokens, heads = piece->x.heads;
        const int nt[2] = {piece->nt[0], piece->nt[1]}, row0 = piece->x.row0, head0 = piece->x.head0;
        const char* const src = static_cast<const char*>(a.q) + int64_t(row0) * a.token_stride + int64_t(head0) * (D * 2);
        give_back();
#pragma unroll
        for (int st = 0; st < NQ; ++st) {
          if (nt[st] == 0) continue;
          wait(&b_qfree[st], (qn[st] & 1) ^ 1);
          if (gone) break;
          ++qn[st];
          const uint32_t dst = umma::smem_u32(qbuf) + st * C::QT;
          if (p.q_box) {  // (what other tokens' rows come with it, no output takes)
            if (me == 0) {
              mbar_expect(&b_qfull[st], C::QT);
#pragma unroll
              for (int d = 0; d < D; d += 64)
                load_q(&q_map, dst + d / 64 * (128 * 128), &b_qfull[st], d, head0, row0 + st * p.q_box);
            }
            continue;
          }
#pragma unroll 2
          for (int k = me; k < 128 * CPR; k += 64) {
            const int row = k / CPR, ch = k % CPR;
            const int t = token_of(p, st * 128 + row), h = st * 128 + row - t * p.bheads;
            const bool live = t < tokens && h < heads;
            attn::cp16(dst + umma::rp_offset(row, ch * 8, 128),
                       src + (live ? t * a.token_stride + h * (D * 2) + ch * 16 : 0), live);
          }
          arrive_copies(&b_qfull[st]);
        }
#pragma unroll 1
        for (int i = 0; i < n && !gone; ++i) {
          if (i >= look0) {
            // (a barrier of these tiles alone: the ring's may be many phases behind)
            wait(&b_look[chk & (kCheckRing - 1)], (chk / kCheckRing) & 1);
            if (gone) break;
            bool wild[2] = {false, false};
#pragma unroll
            for (int j = 0; j < VU; ++j) {
              unsigned char* const unit = vbuf + rv.plus(j).slot * C::VB;
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll 2
                for (int ch = 0; ch < DV / 8 && h * 64 + me < TK; ++ch) {
                  uint4* at = reinterpret_cast<uint4*>(unit + umma::rp_offset(h * 64 + me, ch * 8, TK));
                  const uint4 v = *at;
                  uint32_t e[4] = {v.x, v.y, v.z, v.w};
                  bool bad = false;
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    if ((e[k] & 0x7f80u) == 0x7f80u) e[k] &= 0xffff0000u, bad = true;
                    if ((e[k] & 0x7f800000u) == 0x7f800000u) e[k] &= 0x0000ffffu, bad = true;
                  }
                  if (bad) *at = make_uint4(e[0], e[1], e[2], e[3]), wild[h] = true;
                }
            }
            umma::fence_smem_to_async();
            __syncwarp();
            const uint32_t w0 = __ballot_sync(~0u, wild[0]), w1 = __ballot_sync(~0u, wild[1]);
            if (lane == 0) {
              uint32_t* to = reinterpret_cast<uint32_t*>(&s_wild[chk & (kCheckRing - 1)]) + (warp - SOFT - 5);
              to[0] = w0, to[2] = w1;
              mbar_arrive(&b_check[chk & (kCheckRing - 1)]);
#pragma unroll
              for (int j = 0; j < VU; ++j) mbar_arrive_many(&b_vfull[rv.plus(j).slot], VFULL / 2);
            }
            ++chk;
          }
          rv.step(VU);
        }
        if (gone) break;
      }
      if (gone && p.q_box)  // copies in flight land before the block ends
#pragma unroll
        for (int st = 0; st < NQ; ++st)
          for (uint32_t i = 0; qn[st] > 0 && i < kWaitTries >> 8 && !umma::mbar_try_wait(&b_qfull[st], (qn[st] - 1) & 1); ++i) {
          }
      attn::cp_wait_all();
    }
  }
  if (gone) s_dead = 1;
  umma::fence_before_sync();
  __syncthreads();
  if (warp == SOFT + 2) umma::tmem_dealloc(tmem, C::TMEM);
  if (s_dead) {
    // a wait ran out: what this range leaves unwritten counts as left out
    for (int x = tid; x < 2 * p.rows; x += NT) p.part_ml[2 * int64_t(blockIdx.x) * p.rows + x] = make_float2(-INFINITY, attn::kLeftOut);
    if (tid == 0) {
      p.split[blockIdx.x].parts = 0;
      report(a.status, LIN_ST_TIMEOUT);
    }
  }
}

template <class C>
cudaError_t launch_umma(const Plan& p, const Maps& m, cudaStream_t s) {
  auto kern = chunk_umma_kernel<C>;
  static bool ready[kMaxDevices];  // set twice at worst, to the same value
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev] = true;
  }
  kern<<<p.grid, C::THREADS, C::SMEM, s>>>(p, m.k, m.v, m.q);
  return cudaGetLastError();
}

template <int D, int NQ>
cudaError_t launch_umma_loads(const Plan& p, const Maps& m, cudaStream_t s) {
  return p.box ? launch_umma<UCfg<D, NQ, true>>(p, m, s) : launch_umma<UCfg<D, NQ, false>>(p, m, s);
}

template <int D>
cudaError_t launch_umma_tiles(const Plan& p, const Maps& m, cudaStream_t s) {
  if constexpr (D <= 128)
    if (p.rows == 256) return launch_umma_loads<D, 2>(p, m, s);
  return launch_umma_loads<D, 1>(p, m, s);
}

}  // namespace chunk
}  // namespace lin
