// Attention over caches on the tcgen05 tensor cores: bf16, head_dim 64, 128 or 256, for a call's parameters P
// (verify rows over a shared prefix and each request's own cache: AttnParams; new rows over a paged cache:
// PagedParams). Units, pieces and partials as in trunk.cuh.
//
// Per block of kBn positions: S = Q K^T (Q in TMEM, 128 rows x kBn), a row's softmax by one thread
// (TMEM lane = row, no shuffles), the weights as bf16 back into the columns of S, O += P V with P
// in TMEM too and V as it lies in the cache (rows of positions: the B operand is N-major).
//   * warp 0 loads K and V blocks by TMA (of a paged cache K, and warp 3 V); Q is gathered by the softmax
//     threads into TMEM, so that its 128 rows are not read from shared memory again for every block;
//   * warp 1 issues the MMAs: S of the blocks after i goes out before O of block i, so the tensor pipe works
//     on them while the softmax works on the others (two S buffers, or four);
//   * warps 4..7 and 8..11 do the softmax of the blocks in turns; warp 2 (and 3 where it loads nothing) watch
//     V (below). The reference a row's weights are taken against moves only when the row's maximum has grown
//     by more than 2^8 (the weights stay below 256 and their sum and O are fp32, so nothing is lost), which
//     makes rescaling O in TMEM rare.
// Weights are rounded to bf16 for the tensor cores (2^-9 of each weight, as the outputs are); their
// sum is taken in fp32 before that.
//
// A position that some row does not see has weight 0 in that row, and 0 times what lies there must
// be 0. In blocks where any running row's positions end, guard warps therefore look through V as
// it lands, ahead of the softmax: non-finite values that no row sees are cleared, and where a row
// does see one, that row's share of it is added by hand and the value cleared for the tensor cores.
//
// The code has to be short: an SM that runs five roles fetches all of them, and loops unrolled over a role's
// stages cost more in fetches than they saved (198 KB of code for both calls, now 120: 32 x 8 rows over 63,488
// positions 190 -> 176 us).
//
// 16 query heads on 4 KV heads of 256 dims, verify rows: 256 rows over 63,488 shared positions and 700 own ones
// each, 174 to 178 us with the join = 1.52 PFLOP/s (0.79 of cuBLAS); two rows of one request over its own
// 63,488: 49.5 us = 5.3 TB/s (0.77 of a copy), eight single rows over a shared 63,488 60 us = 5.0 TB/s: HBM
// while the blocks run, and some 16 us of launch, plan, first loads, partials and join around them. A paged
// cache: 2,048 rows over 61,440 positions 1,180 to 1,400 us by the clock that the power limit leaves, single calls
// the least (1.78 to 1.50 PFLOP/s, 0.92 of cuBLAS's burst to 0.88 of its long loop), 128 dims 700 to 760 and 64 dims
// 650 (half and a quarter of the work: a block's softmax is 128 x 64 exponentials whatever the head's size); 32
// requests of 8 rows over 15,360 each 287 us = 6.7 TB/s (0.99 of a copy); two rows over 63,488 55 us.
#pragma once

#include <math.h>

#include <cuda_bf16.h>

#include "trunk.cuh"

#include "tcgen05.cuh"

namespace spec {

constexpr int kTm = 128;
constexpr int kTcThreads = 12 * 32;  // producers and guards (three), MMA, eight softmax warps
constexpr int kRing = 16;  // pieces of a CTA that its roles are told of ahead (a paged cache's call)
struct PieceNote {
  int tile, head, blk0, blk1, slot, whole;  // tile -1: no more
};
template <int N>
struct Number {
  static constexpr int value = N;
};
constexpr int kGroupThreads = 128;  // a softmax group
template <typename P>
constexpr int kTcSmall = kPaged<P> ? 1536 : 512;  // bytes of barriers and flags
// Registers a thread: launched with 168 (64,512 in all); the first four warps give to the softmax's
// eight: 128 x 152 + 256 x 176 = 64,512. (104 and 200 spill in the guards: 214 us for 191.)
constexpr int kFewRegs = 152, kSoftRegs = 176;
// Bits that a row's maximum may grow by before its reference moves: 256 rows over 63,488 positions 260 us
// with 0, 192 with 8.
constexpr float kLazy = 8.f;

// A batch of products alone takes some 500 cycles more than the same products among others, so a block's way
// from its scores through its softmax to its product and the next scores in its place is long, and what
// hides it is blocks on their way: as many buffers of scores as tensor memory has room for.
template <int D, bool PAGED>
struct Shape {
  // Verify rows: K and V blocks of 16 or 32 KB. 128 dims in blocks of 64 positions took 168 us for 151 (256
  // rows over 63,488); 256 dims in blocks of 128 do not fit beside two buffers of S.
  static constexpr int kBn = D == 256 || PAGED ? 64 : 128;
  static constexpr int kBuf = D != 256 && PAGED ? 4 : 2;
  static constexpr int kTile = kBn * D * 2;
  static constexpr int kStages = PAGED ? (D == 256 ? 3 : D == 128 ? 6 : 8) : D == 64 ? 6 : 3;
  // The product with V starts on the first half of a block's weights. At 128 positions: 142 -> 128 us (256
  // rows of 128 dims over 63,488); at 64 the tensor pipe, in order, waits for the second half instead of
  // taking the other buffer's scores: 191 -> 211 us (of 256 dims).
  static constexpr bool kHalves = kBn == 128;
  static constexpr int kFixed = 2 * kStages * kTile;
  // TMEM columns: O, the S buffers, Q (two bf16 a column)
  static constexpr int kS = D, kQ = D + kBuf * kBn;
  static_assert(kQ + D / 2 <= 512, "TMEM");
  static_assert(kStages > kBuf, "K runs kBuf - 1 blocks ahead");
};

// A block of K or V in shared memory: for each panel of 64 dims rows of 128 bytes, eight positions to 1,024
// bytes (the swizzle's atom). A contiguous cache's box is [panel][position][64 dims], a page's [eight
// positions][panel][8][64]: then a page of any size lies in one piece, and its neighbour after it.
template <typename P, int D>
struct Place {
  static constexpr int kGroup = kPaged<P> ? D / 64 * 1024 : 1024;               // from eight positions to the next
  static constexpr int kPanel = kPaged<P> ? 1024 : Shape<D, false>::kBn * 128;  // from a panel to the next
  static __device__ __forceinline__ int at(int pos) { return (pos >> 3) * kGroup + (pos & 7) * 128; }
};

// A block of K or V at once, in the order of its map's box.
__device__ __forceinline__ void tma_load_block(void* dst, const CUtensorMap* map, int pos, int panel,
                                               int b, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%6, %2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(pos), "r"(panel), "r"(b), "r"(smem_u32(bar)), "r"(0)
      : "memory");
}

// B operand whose rows (K) are 128 bytes of N in the 128-byte swizzle: 8-row groups `group` bytes
// apart, the next 64 of N one panel on.
__device__ __forceinline__ uint64_t smem_desc_n_major(uint32_t saddr, uint32_t panel, uint32_t group) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((panel >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((group >> 4) & 0x3FFFu) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
// And whose rows (N) are 128 bytes of K, as smem_desc_sw128's.
__device__ __forceinline__ uint64_t smem_desc_k_major(uint32_t saddr, uint32_t group) {
  return smem_desc_sw128(saddr) + (static_cast<uint64_t>((group - 1024u) >> 4) << 32);
}

// A from TMEM (two bf16 of K per 32-bit column), B from shared memory.
__device__ __forceinline__ void tc_mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,"
      "%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t* r) {
  if constexpr (N == 16) {
    tmem_st16(taddr, r);
  } else {
#pragma unroll
    for (int j = 0; j < N / 32; ++j) tmem_st32(taddr + 32 * j, r + 32 * j);
  }
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 32 bytes at a time, a whole sector of memory: half the requests of 16-byte pieces a row apart.
__device__ __forceinline__ void load32(const void* p, uint32_t* r) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ bool odd_pair(uint32_t w) {  // an Inf or NaN in either half
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <int D, typename P, typename Req>
__device__ __forceinline__ const __nv_bfloat16* q_row(const P& p, const Req* req, const AttnPiece& a,
                                                      const AttnRow& r) {
  return static_cast<const __nv_bfloat16*>(p.q) + attn_q_row(p, req, r) * p.qs +
         static_cast<int64_t>(a.head * p.G + r.g) * D;
}

// Which of 32 positions of a block from c0 a row sees: those before `valid`, on pages that are there.
template <typename P>
__device__ __forceinline__ uint32_t seen_bits(const P& p, int valid, uint32_t lost, int c0) {
  const int n = min(max(valid - c0, 0), 32);
  uint32_t bits = n == 32 ? 0xffffffffu : (1u << n) - 1u;
  if (lost)
#pragma unroll 1
    for (int s = 0; s < 32; s += 8)  // a page has eight positions or more
      if (lost >> ((c0 + s) >> p.page_shift) & 1) bits &= ~(0xffu << s);
  return bits;
}

struct AttnMaps {
  CUtensorMap pk, pv, ok, ov;  // K and V of the prefix, of the own caches (the paged cache: ok and ov)
};

// A page's part of a block of K or V. A page's number past the last reads zeros.
__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, int panel, int eight, int page,
                                              uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(panel), "r"(eight), "r"(page), "r"(smem_u32(bar))
      : "memory");
}

template <typename P, int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ P p) {
  using Sh = Shape<D, kPaged<P>>;
  using Pl = Place<P, D>;
  constexpr int BN = Sh::kBn, NS = Sh::kStages, NB = Sh::kBuf;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sk = smem;
  uint8_t* sv = sk + NS * Sh::kTile;
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + Sh::kFixed);
  uint64_t* kdone = kfull + NS;   // the scores are there, and the stage is free
  uint64_t* vfull = kdone + NS;
  uint64_t* vdone = vfull + NS;   // O has the block, and the stage is free
  uint64_t* vok = vdone + NS;     // V has landed and been looked through
  // P (its first half, where there are halves) is written and V ok; its rest. One to a stage, as all of
  // these: an arrival for block i + NS cannot come before block i's product is complete, so no barrier
  // takes it for an earlier block's, and none runs through two phases while its waiter looks away.
  uint64_t* pready = vok + NS;
  uint64_t* prest = pready + NS;
  uint64_t* qready = prest + NS;
  uint64_t* meet = qready + 1;    // the softmax warps, [0] and [1] of a group, [2] all (verify rows)
  uint64_t* ofree = meet + 3;     // the piece's O has been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ofree + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* o_init = abort_flag + 1;      // [2] O holds something before the piece's first MMA on it
  volatile int* odd = abort_flag + 3;         // [NS][guards]: a row sees a non-finite V of the stage
  int* least_sm = const_cast<int*>(odd + 2 * NS);  // [2][4] per quarter of the rows
  // [2 NS] of a K block, which of its pages are not there. Written when the block's stage is free, which may
  // be before every warp has read an earlier block's word: two stages' worth.
  volatile uint32_t* gone = reinterpret_cast<volatile uint32_t*>(least_sm + 8);
  // [K, V][32] of the table's entries
  int* page_ring = const_cast<int*>(reinterpret_cast<volatile int*>(gone + 2 * NS));
  uint64_t* ring_full = reinterpret_cast<uint64_t*>(page_ring + 64);
  PieceNote* ring = reinterpret_cast<PieceNote*>(ring_full + kRing);
  static_assert(8 * (7 * NS + 5) + 4 * (12 + 2 * NS) +
                        (kPaged<P> ? 4 * (2 * NS + 64) + kRing * (8 + static_cast<int>(sizeof(PieceNote))) : 0) <=
                    kTcSmall<P>,
                "barriers and flags");
  float* row_m = reinterpret_cast<float*>(smem + Sh::kFixed + kTcSmall<P>);  // [2][128] each group's last reference
  float2* row_ml = reinterpret_cast<float2*>(row_m + 2 * kTm);       // [2][128] and sum, at a piece's end
  int32_t* cum = reinterpret_cast<int32_t*>(row_ml + 2 * kTm);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kdone[s], 1);
      mbar_init(&vfull[s], 1);
      mbar_init(&vdone[s], 1);
      mbar_init(&vok[s], kPaged<P> ? 1 : 2);
      mbar_init(&pready[s], kPaged<P> ? 5 : 6);
      mbar_init(&prest[s], 4);
    }
    mbar_init(qready, 8);
    mbar_init(&meet[0], 4);
    mbar_init(&meet[1], 4);
    mbar_init(&meet[2], 8);
    mbar_init(ofree, 8);
    if constexpr (kPaged<P>)
      for (int s = 0; s < kRing; ++s) mbar_init(&ring_full[s], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  pdl_wait();
  if constexpr (kPaged<P>) {
    pdl_trigger();  // the join's blocks come as these leave, and wait
    if (threadIdx.x == 0) paged_splits_clear(p);  // whatever becomes of the walk, the join finds no other call's
  }
  const auto* req = attn_plan(p, cum);  // ends with a block barrier
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  auto give_up = [&]() {
    atomicOr(&p.hdr->error, ERR_TC_WAIT);
    *abort_flag = 1;
  };
  AttnShares shares;
  AttnWalk walk;
  AttnPiece a;
  if (!kPaged<P> || warp == 0) {  // (paged: the others are told, below)
    shares = attn_shares(p, cum);
    if (!kPaged<P> && blockIdx.x == 0) attn_write_units(p, cum, shares);
    walk.start(p, cum, shares);
  }
  // The next piece. Of a paged cache the K producer's warp, which is ahead of the others by as many blocks as it
  // has stages, walks for all and leaves what it finds in a ring; a piece has a block at least, so that no role
  // is further behind than the ring is long: K(i) is loaded after the scores of block i - NS, those come after the
  // product of i - NS - NB, and that after the softmax.
  static_assert(!kPaged<P> || NS + NB + 2 <= kRing);
  int told = 0;
  auto tell = [&](bool more) {  // by one lane
    PieceNote& note = ring[told % kRing];
    note.tile = more ? a.tile : -1;
    note.head = a.head, note.blk0 = a.blk0, note.blk1 = a.blk1, note.slot = a.slot, note.whole = a.whole;
    mbar_arrive(&ring_full[told % kRing]);
  };
  auto next_piece = [&](bool one = false) {  // by a whole warp, or by one thread
    if constexpr (!kPaged<P>) {
      return walk.next(p, cum, shares, a);
    } else if (warp == 0) {
      const bool more = walk.next(p, cum, shares, a);
      if (lane == 0) {
        if (more) paged_split(p, cum, shares, walk, a);
        tell(more);
      }
      ++told;
      return more;
    } else {
      bool more = mbar_wait_bounded(&ring_full[told % kRing], (told / kRing) & 1);
      if (!more) give_up();
      const PieceNote note = ring[told % kRing];
      ++told;
      a.tile = note.tile, a.head = note.head, a.blk0 = note.blk0, a.blk1 = note.blk1, a.slot = note.slot;
      a.whole = note.whole != 0;
      more = more && note.tile >= 0;
      return one ? more : static_cast<bool>(__all_sync(0xffffffffu, more));
    }
  };

  if (warp < 4)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));

  constexpr int kGuards = kPaged<P> ? 1 : 2;
  if (warp == 0 || (warp == 3 && kPaged<P>)) {
    // ------------------------------------------------------------------ TMA producers
    // One elected thread waits and issues, as below. A wait and a copy take it 300 to 600 cycles.
    if constexpr (kPaged<P>) {
      // K by one warp and V by another: one for both was what a block took longest for (2,048 rows of 128
      // dims over 61,440 positions 1,004 us, 707 so). The other lanes help to the page table's entries.
      const bool leader = elect_one(), is_k = warp == 0;
      uint8_t* const tiles = is_k ? sk : sv;
      uint64_t* const full = is_k ? kfull : vfull;
      uint64_t* const done = is_k ? kdone : vdone;
      int gi = 0, s = 0, phase = 1, i = 0;  // the next block: its stage, the stage's phase, its number
      bool ok = true;
      bool more = true;
      while (__all_sync(0xffffffffu, ok && !*abort_flag) && (more = next_piece())) {
        const int panel = a.head * (D / 64), blk0 = a.blk0, blk1 = a.blk1;
        int left = blk1 - blk0;
        const int b = attn_tile_req(p, a.tile), ps = p.c.page_size;
        const CUtensorMap* map = is_k ? &maps.ok : &maps.ov;
        const int32_t* table = p.c.table + static_cast<int64_t>(b) * p.c.table_stride;
        const auto entry = [&](int j) { return j < p.c.max_pages ? __ldg(table + j) : -1; };
        int* const pages = page_ring + (is_k ? 0 : 32);
        int j = blk0 * BN / ps, at = blk0 * BN - j * ps;
        // entries 32 at a time, the next ones on their way
        int e = entry((j & ~31) + lane);
#pragma unroll 1
        for (int w = j & ~31; left > 0; w += 32) {
          __syncwarp();
          pages[lane] = static_cast<unsigned>(e) < static_cast<unsigned>(p.c.n_pages) ? e : p.c.n_pages;
          e = entry(w + 32 + lane);
          __syncwarp();
          if (leader) {
            // blocks of whole pages in pages of 8 to 32 positions, or a block and a part of a page
            const auto blocks = [&](auto number) {
              constexpr int PER = decltype(number)::value;
#pragma unroll 1
              while (left > 0 && j < w + 32) {
                int page[PER];
                uint32_t lost = 0;
#pragma unroll
                for (int m = 0; m < PER; ++m) {
                  page[m] = pages[j - w + m];
                  lost |= static_cast<uint32_t>(page[m] == p.c.n_pages) << m;
                }
                ok = i < NS || mbar_wait_bounded(&done[s], phase);
                if (!ok) break;
                if (is_k) {
                  gone[gi] = lost;  // seen with the block: the scores' wait for it comes before the softmax's for them
                  if (++gi == 2 * NS) gi = 0;
                }
                mbar_arrive_expect_tx(&full[s], Sh::kTile);
#pragma unroll
                for (int m = 0; m < PER; ++m)
                  tma_load_page(tiles + s * Sh::kTile + m * (Sh::kTile / PER), map, panel, at >> 3, page[m], &full[s]);
                at += BN;
                if (at >= ps) j += PER, at = 0;
                if (++s == NS) s = 0, phase ^= 1;
                ++i;
                --left;
              }
            };
            if (ps >= BN)
              blocks(Number<1>());
            else if (ps == 8)
              blocks(Number<BN / 8>());
            else if (ps == 16)
              blocks(Number<BN / 16>());
            else
              blocks(Number<BN / 32>());
          }
          left = __reduce_min_sync(0xffffffffu, leader ? (ok ? left : 0) : 0x7fffffff);
        }
      }
      if (is_k && more && lane == 0) tell(false);  // a wait ran out
      if (leader) {
        if (!ok) give_up();
        // Leave nothing in flight: the last loads of every stage have landed.
#pragma unroll 1
        for (int k = max(0, i - NS); k < i; ++k) mbar_wait_bounded(&full[k % NS], (k / NS) & 1);
      }
      __syncwarp();
    } else if (elect_one()) {
      int ks = 0, kp = 1, ki = 0, vs = 0, vp = 1, vi = 0;  // the next K and V blocks: stage, its phase, number
      bool ok = true;
      auto room = [&](uint64_t* empty, int s, int phase, int i) { return i < NS || mbar_wait_bounded(&empty[s], phase); };
      while (ok && !*abort_flag && next_piece()) {
        const int panel = a.head * (D / 64), blk1 = a.blk1;
        int left_k = blk1 - a.blk0, left_v = left_k;
        const bool pre = a.tile < p.npt;
        const int b = pre ? 0 : attn_tile_req(p, a.tile);
        const CUtensorMap* mk = pre ? &maps.pk : &maps.ok;
        const CUtensorMap* mv = pre ? &maps.pv : &maps.ov;
#pragma unroll 1
        while (left_v > 0) {
          const bool is_k = left_k > 0 && left_k > left_v - NB;  // K runs as far ahead as the MMAs take it
          ok = is_k ? room(kdone, ks, kp, ki) : room(vdone, vs, vp, vi);
          if (!ok) break;
          mbar_arrive_expect_tx(is_k ? &kfull[ks] : &vfull[vs], Sh::kTile);
          if (is_k) {
            tma_load_block(sk + ks * Sh::kTile, mk, (blk1 - left_k) * BN, panel, b, &kfull[ks]);
            if (++ks == NS) ks = 0, kp ^= 1;
            ++ki;
            --left_k;
          } else {
            tma_load_block(sv + vs * Sh::kTile, mv, (blk1 - left_v) * BN, panel, b, &vfull[vs]);
            if (++vs == NS) vs = 0, vp ^= 1;
            ++vi;
            --left_v;
          }
        }
      }
      if (!ok) give_up();
      // Leave nothing in flight: the last loads of every stage have landed.
#pragma unroll 1
      for (int j = max(0, ki - NS); j < ki; ++j) mbar_wait_bounded(&kfull[j % NS], (j / NS) & 1);
#pragma unroll 1
      for (int j = max(0, vi - NS); j < vi; ++j) mbar_wait_bounded(&vfull[j % NS], (j / NS) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    // One elected thread goes through all of it. Its time is part of every block's way, and there the compiler
    // keeps operands in uniform registers: 9 cycles an MMA, where a warp that elects a thread for each takes 15
    // alone and 37 beside the softmax's (four moves to uniform registers and a vote each).
    if (elect_one()) {
      constexpr uint32_t kIdS = tc_idesc(kTm, BN);
      constexpr uint32_t kIdO = tc_idesc(kTm, D) | (1u << 16);  // B is N-major
      const uint64_t kd0 = smem_desc_k_major(smem_u32(sk), Pl::kGroup);
      const uint64_t vd0 = smem_desc_n_major(smem_u32(sv), Pl::kPanel, Pl::kGroup);
      int ks = 0, kp = 0, kb = 0;             // of the next scores: stage, its phase, buffer
      int vs = 0, vp = 0, vb = 0, piece = 0;  // of the next product
      bool ok = true;
      auto scores = [&]() {
        if (!mbar_wait_bounded(&kfull[ks], kp)) return false;
        tc_fence_after();
        const uint64_t kd = desc_advance(kd0, ks * Sh::kTile);
        const uint32_t ds = tmem + Sh::kS + kb * BN;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ta(ds, tmem + Sh::kQ + kk * 8,
                    desc_advance(kd, (kk / 4) * Pl::kPanel + (kk % 4) * 32), kIdS, kk > 0);
        tc_commit(&kdone[ks]);
        if (++ks == NS) ks = 0, kp ^= 1;
        kb = kb + 1 == NB ? 0 : kb + 1;
        return true;
      };
#pragma unroll 1
      while (ok && !*abort_flag && next_piece(true)) {
        const int n = a.blk1 - a.blk0;
        ok = mbar_wait_bounded(qready, piece & 1);
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; ok && j < min(n, NB - 1); ++j) ok = scores();
#pragma unroll 1
        for (int j = 0; ok && j < n; ++j) {
          if (j + NB - 1 < n) ok = scores();
          ok = ok && mbar_wait_bounded(&pready[vs], vp);
          uint32_t acc0 = 1;
          if (j == 0) {
            if (piece > 0) ok = ok && mbar_wait_bounded(ofree, (piece - 1) & 1);
            acc0 = o_init[piece & 1] ? 1u : 0u;
          }
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = desc_advance(vd0, vs * Sh::kTile);
          const uint32_t ps = tmem + Sh::kS + vb * BN;
#pragma unroll
          for (int kk = 0; kk < BN / (Sh::kHalves ? 32 : 16); ++kk)
            tc_mma_ta(tmem, ps + kk * 8, desc_advance(vd, kk * 2 * Pl::kGroup), kIdO, kk > 0 ? 1u : acc0);
          if constexpr (Sh::kHalves) {
            ok = mbar_wait_bounded(&prest[vs], vp);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = BN / 32; kk < BN / 16; ++kk)
              tc_mma_ta(tmem, ps + kk * 8, desc_advance(vd, kk * 2 * Pl::kGroup), kIdO, 1u);
          }
          tc_commit(&vdone[vs]);
          if (++vs == NS) vs = 0, vp ^= 1;
          vb = vb + 1 == NB ? 0 : vb + 1;
        }
        ++piece;
      }
      if (!ok) give_up();
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------------ guards of V
    // In a block where some running row's positions end, non-finite values of positions that no
    // row sees are cleared; those that a row does see are reported to the softmax.
    const int gw = warp - 2;
    int it = 0;
    bool ok = true;
#pragma unroll 1
    while (ok && !__any_sync(0xffffffffu, *abort_flag) && next_piece()) {
      int least = 0x7fffffff, most = 0;  // positions every running row sees; positions any row sees
#pragma unroll 1
      for (int i = lane; i < kTm; i += 32) {
        const int lim = attn_row(p, req, a.tile, i).lim;
        most = max(most, lim);
        if (lim > 0) least = min(least, lim);
      }
      least = __reduce_min_sync(0xffffffffu, least);
      most = __reduce_max_sync(0xffffffffu, most);
      if constexpr (!kPaged<P>) {  // the next piece's queries, towards L2
        AttnWalk ahead = walk;
        AttnPiece nx;
        if (ahead.next(p, cum, shares, nx))
#pragma unroll 1
          for (int i = gw * 32 + lane; i < kTm; i += 32 * kGuards) {
            const AttnRow r = attn_row(p, req, nx.tile, i);
            if (r.lim <= 0) continue;
            const __nv_bfloat16* src = q_row<D>(p, req, nx, r);
#pragma unroll 1
            for (int d = 0; d < D; d += 64)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(src + d));
          }
      }
#pragma unroll 1
      const int blk1 = a.blk1;
#pragma unroll 1
      for (int blk = a.blk0; ok && blk < blk1; ++blk, ++it) {
        const int s = it % NS;
        ok = mbar_wait_warp(&vfull[s], (it / NS) & 1);
        bool seen = false;
        if (blk * BN + BN > least) {
          uint8_t* vt = sv + s * Sh::kTile;
          const int from = max(0, least - blk * BN);
          // The swizzle keeps a position's 128 bytes of a panel together. An exponent of all ones carries
          // into its half's top bit.
          const int run = (BN - from) * 8;
          uint32_t any = 0;
#pragma unroll 1
          for (int j = 0; j < D / 64; ++j) {
#pragma unroll 16
            for (int k = 0; k < BN * 8 / (32 * kGuards); ++k) {
              const int i = min((k * kGuards + gw) * 32 + lane, run - 1);
              const uint4 x = lds128(vt + j * Pl::kPanel + Pl::at(from + i / 8) + i % 8 * 16);
              any |= (x.x & 0x7f807f80u) + 0x00800080u;
              any |= (x.y & 0x7f807f80u) + 0x00800080u;
              any |= (x.z & 0x7f807f80u) + 0x00800080u;
              any |= (x.w & 0x7f807f80u) + 0x00800080u;
            }
          }
          if (__any_sync(0xffffffffu, any & 0x80008000u)) {
#pragma unroll 1
            for (int j = 0; j < D / 64; ++j)
#pragma unroll 1
              for (int i = gw * 32 + lane; i < run; i += 32 * kGuards) {
                uint4* at = reinterpret_cast<uint4*>(vt + j * Pl::kPanel + Pl::at(from + i / 8) + i % 8 * 16);
                const uint4 x = *at;
                if (odd_pair(x.x) || odd_pair(x.y) || odd_pair(x.z) || odd_pair(x.w)) {
                  if (blk * BN + from + i / 8 >= most)
                    *at = make_uint4(0u, 0u, 0u, 0u);
                  else
                    seen = true;
                }
              }
            fence_async_smem();
          }
        }
        seen = __any_sync(0xffffffffu, seen);
        if (lane == 0) {
          odd[kGuards * s + gw] = seen;
          mbar_arrive(&vok[s]);
          mbar_arrive(&pready[s]);
        }
      }
    }
    if (!ok && lane == 0) give_up();
  } else {
    // ------------------------------------------------------------------ softmax
    // Two groups of four warps, a thread to a row in each, take the blocks in turns: one is in its
    // exponentials while the other waits for scores or reads them. What a block needs of the one before
    // is the row's reference, which is known long before that one's weights.
    constexpr int DH = D / 2;
    const int quad = warp & 3, half = (warp - 4) >> 2, row = quad * 32 + lane, st = threadIdx.x & 127;
    const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const float scale = fmaxf(fabsf(p.scale_log2), 1e-45f);  // so that a masked score is -Inf whatever the scale
    int it = 0;
    // A wait that runs out ends all further waiting, not the walk: whatever happens, a softmax warp
    // goes through the same pieces as the others, which it meets at `meet` and at named barriers. Of verify rows
    // each walks for itself, all alike; of a paged cache each waits for the note of a piece with a limit of its
    // own, so they take the piece if all have its note and otherwise leave together (`agreed`).
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!ok || mbar_wait_warp(bar, parity)) return;
      if (lane == 0) give_up();
      __syncwarp();
      ok = false;
    };
    uint32_t met_all = 0, met_group = 0;
    auto bar_all = [&]() {  // a barrier of the softmax warps, with the limit of every wait
      __syncwarp();
      if (lane == 0) mbar_arrive(&meet[2]);
      wait(&meet[2], met_all++ & 1);
    };
    // Whether every softmax warp says so. A barrier without a limit, which ends: the warps come to it once a
    // piece and once after the last one, their waits before it have limits, and all go on as it says.
    auto agreed = [&](bool mine) {
      __syncwarp();
      uint32_t all;
      asm volatile(
          "{\n\t.reg .pred m, a;\n\tsetp.ne.u32 m, %1, 0;\n\tbar.red.and.pred a, 13, 256, m;\n\t"
          "selp.u32 %0, 1, 0, a;\n\t}"
          : "=r"(all)
          : "r"(static_cast<uint32_t>(mine))
          : "memory");
      return all != 0;
    };
    auto bar_group = [&]() {  // of the group's
      __syncwarp();
      if (lane == 0) mbar_arrive(&meet[half]);
      wait(&meet[half], met_group++ & 1);
    };
    // Q of a piece: this thread's half of its row into its TMEM lane; a negative scale goes into Q's signs
    int piece = 0, least = 0;
    AttnRow ar;
    auto fetch_q = [&](const AttnPiece& pc) {
      ar = attn_row(p, req, pc.tile, row);
      const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
      const __nv_bfloat16* src = q_row<D>(p, req, pc, ar);
      // (the paged call keeps more of the piece before: half of a long row at a time, or registers spill)
      constexpr int W = kPaged<P> && D == 256 ? DH / 4 : DH / 2;
      const uint32_t tq = trow + Sh::kQ + half * (DH / 2);
      // rows that do not run have read row 0's
      if (__all_sync(0xffffffffu, (reinterpret_cast<uintptr_t>(src) & 31u) == 0)) {
#pragma unroll
        for (int part = 0; part < DH / 2; part += W) {
          uint32_t w[W];
#pragma unroll
          for (int c = 0; c < W / 8; ++c) load32(src + half * DH + 2 * part + 16 * c, w + 8 * c);
#pragma unroll
          for (int c = 0; c < W; ++c) w[c] = ar.lim > 0 ? w[c] ^ flip : 0u;
          tmem_st<W>(tq + part, w);
        }
      } else {
        const uint16_t* from = reinterpret_cast<const uint16_t*>(src + half * DH);
#pragma unroll 1
        for (int part = 0; part < DH / 2; part += 16) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            w[c] = from[2 * (part + c)] | static_cast<uint32_t>(from[2 * (part + c) + 1]) << 16;
            w[c] = ar.lim > 0 ? w[c] ^ flip : 0u;
          }
          tmem_st16(tq + part, w);
        }
      }
      tmem_st_wait();
      const int lo = __reduce_min_sync(0xffffffffu, ar.lim > 0 ? ar.lim : 0x7fffffff);
      int* lsm = least_sm + 4 * (piece & 1);
      if (lane == 0 && half == 0) lsm[quad] = lo;
      if (st == 0 && half == 0) o_init[piece & 1] = 0;
      tc_fence_before();
    };
    auto load_q = [&](const AttnPiece& pc, bool more) {  // whether there is a piece
      if (more) fetch_q(pc);
      if constexpr (kPaged<P>)
        more = agreed(more);
      else if (more)
        bar_all();
      if (!more) return false;
      if (lane == 0) mbar_arrive(qready);
      const int* lsm = least_sm + 4 * (piece & 1);
      least = min(min(lsm[0], lsm[1]), min(lsm[2], lsm[3]));
      return true;
    };
    int lim = 0, slot = 0, tile = 0, head = 0;  // of the piece in work
    bool whole = false;
    float mg = -INFINITY, l = 0.f;  // of the group's blocks of it: the last reference, the sum
    auto output = [&]() {  // what the piece has come to
      const int lb = it - 1;
      wait(&vdone[lb % NS], (lb / NS) & 1);
      tc_fence_after();
      row_ml[half * kTm + row] = make_float2(mg, l);
      asm volatile("bar.sync %0, 64;" ::"r"(9 + quad) : "memory");
      const float2 other = row_ml[(half ^ 1) * kTm + row];
      // the reference never falls, so the greater one is the last one's
      const float m = fmaxf(mg, other.x), ref = m == -INFINITY ? 0.f : m;
      // in the groups' order, whichever of them asks
      const float w0 = half == 0 ? l * ex2(mg - ref) : other.y * ex2(other.x - ref);
      const float w1 = half == 0 ? other.y * ex2(other.x - ref) : l * ex2(mg - ref);
      const float sum = w0 + w1;
      if (whole) {
        // All that the row sees: its output itself. Nothing seen, or scores of -Inf alone: zero.
        const bool empty = m == -INFINITY && sum == sum;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const AttnRow out_row = attn_row(p, req, tile, row);
        const int64_t q_at = attn_q_row(p, req, out_row);
        const int q_head = head * p.G + out_row.g;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + q_at * p.os + static_cast<int64_t>(q_head) * D;
        if (p.lse && lim > 0 && half == 0)
          p.lse[q_at * (p.Hkv * p.G) + q_head] =
              empty ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
        if (__all_sync(0xffffffffu, (reinterpret_cast<uintptr_t>(dst) & 31u) == 0)) {
#pragma unroll 1
          for (int d = half * DH; d < half * DH + DH; d += 32) {
            float o[32];
            tmem_ld32(trow + d, o);
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              w[j] = empty ? 0u : bf16_pair(o[2 * j] * inv, o[2 * j + 1] * inv);
            if (lim > 0) {
              store32(dst + d, w);
              store32(dst + d + 16, w + 8);
            }
          }
        } else {
#pragma unroll 1
          for (int d = half * DH; d < half * DH + DH; d += 8) {
            float o[8];
            tmem_ld8(trow + d, o);
            if (lim > 0) {
#pragma unroll
              for (int j = 0; j < 8; ++j) dst[d + j] = __float2bfloat16_rn(empty ? 0.f : o[j] * inv);
            }
          }
        }
      } else {
        const int64_t at = static_cast<int64_t>(slot) * kTm + row;
        // The maxima pass over scores that are not numbers, the sum does not. The join takes a maximum of
        // -Inf for a row that saw nothing, so such a partial says NaN there.
        if (lim > 0 && half == 0) p.ml[at] = make_float2(sum != sum ? sum : m, sum);
#pragma unroll 1
        for (int d = half * DH; d < half * DH + DH; d += 32) {
          float o[32];
          tmem_ld32(trow + d, o);
          if (lim > 0) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) store32(p.o + at * D + d + j, o + j);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree);
    };
    bool more = next_piece();
    for (;;) {
      more = load_q(a, more);
      if (piece > 0) output();  // of the piece before, while this one's first scores are computed
      if (!more) break;
      lim = ar.lim, slot = a.slot, tile = a.tile, head = a.head;
      whole = kPaged<P> && a.whole;
      const int from_all = least, blk_end = a.blk1;
      const int n = blk_end - a.blk0, it0 = it;
      mg = -INFINITY, l = 0.f;
      it += (it & 1) ^ half;          // the first of them
#pragma unroll 1
      for (int blk = a.blk0 + it - it0; blk < blk_end; blk += 2, it += 2) {
        const bool first = it == it0, last = it + 1 == it0 + n;
        const int valid = min(BN, lim - blk * BN);  // positions of the block this row sees
        bool full = __all_sync(0xffffffffu, valid >= BN);
        float mo = -INFINITY;  // the reference after the block before, from the other group
        const auto others = [&]() {
          if (first) return;
          asm volatile("bar.sync %0, 64;" ::"r"(1 + 4 * (half ^ 1) + quad) : "memory");
          mo = row_m[(half ^ 1) * kTm + row];
        };
        if (kPaged<P>) others();  // while the scores are on their way (verify rows: registers spill)
        wait(&kdone[it % NS], (it / NS) & 1);
        uint32_t lost = 0;  // pages of the block that are not there
        if constexpr (kPaged<P>) {
          lost = gone[it % (2 * NS)];
          full = full && lost == 0;
        }
        tc_fence_after();
        const uint32_t ts = trow + Sh::kS + (it % NB) * BN;
        const auto mask = [&](float* x, int c0) {  // 32 scores
          if constexpr (kPaged<P>) {
            __syncwarp();  // (and with it a branch: a block that every row sees pays for no selects)
            const uint32_t bits = seen_bits(p, valid, lost, c0);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = bits >> j & 1 ? x[j] : -INFINITY;
            __syncwarp();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = c0 + j < valid ? x[j] : -INFINITY;
          }
        };
        float v[64], raw = -INFINITY;
#pragma unroll
        for (int c0 = 0; c0 < BN; c0 += 64) {
          tmem_ld64(ts + c0, v);
          if (!full) {
            mask(v, c0);
            mask(v + 32, c0 + 32);
          }
          float mx[4] = {raw, v[1], v[2], v[3]};
          mx[0] = max3(mx[0], v[0], v[4]);
#pragma unroll
          for (int j = 5; j + 1 < 64; j += 2) mx[(j / 2) & 3] = max3(mx[(j / 2) & 3], v[j], v[j + 1]);
          raw = max3(max3(mx[0], mx[1], v[63]), mx[2], mx[3]);
        }
        const float top = raw == -INFINITY ? -INFINITY : raw * scale;
        if (!kPaged<P>) others();
        const bool grow = top > mo + kLazy;  // from -Inf: at the first score
        const float m = grow ? top : mo;
        if (!last) {
          row_m[half * kTm + row] = m;
          asm volatile("bar.arrive %0, 64;" ::"r"(1 + 4 * half + quad) : "memory");
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const int sg = it % NS;
        bool by_hand = false;
        auto settle = [&]() {  // O as this block's product finds it; before its first weights are handed on
          const bool rescale = !first && __any_sync(0xffffffffu, grow);
          if (blk * BN + BN > from_all) {
            wait(&vok[sg], (it / NS) & 1);
            by_hand = odd[kGuards * sg] | odd[kGuards * sg + kGuards - 1];
          }
          if (rescale || by_hand) {
            // O of the blocks before is complete (the MMA of this one waits for this thread)
            if (!first)
              wait(&vdone[(it - 1) % NS], ((it - 1) / NS) & 1);
            else if (piece > 0)
              wait(ofree, (piece - 1) & 1);  // and the piece's before has been read
            tc_fence_after();
          }
          if (rescale) {
            const float c = grow ? ex2(mo - ref) : 1.f;  // ex2(-Inf) = 0
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
              float o[32];
              uint32_t u[32];
              tmem_ld32(trow + d, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(o[j] * c);
              tmem_st32(trow + d, u);
            }
          }
        };
        if (Sh::kHalves) settle();
        // A weight is 2^(scale s - ref): two at a time in packed arithmetic. A masked score is -Inf. Of 128
        // scores the last 32 stay in registers; the others are read again, before weights take their columns.
        unsigned long long sum[2] = {0ull, 0ull};
        const unsigned long long scale2 = pack2(__float_as_uint(scale), __float_as_uint(scale));
        const unsigned long long ref2 = pack2(__float_as_uint(-ref), __float_as_uint(-ref));
#pragma unroll
        for (int c0 = 0; c0 < BN; c0 += 32) {
          float again[32];
          const bool kept = BN == 64 || c0 + 32 == BN;
          if (!kept) {
            tmem_ld32(ts + c0, again);
            if (!full) mask(again, c0);
          }
          const float* x = kept ? v + (c0 & 32) : again;
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            unsigned long long y = ref2;
            ffma2_acc(y, pack2(__float_as_uint(x[j]), __float_as_uint(x[j + 1])), scale2);
            uint32_t lo, hi;
            asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(y));
            const float e0 = ex2(__uint_as_float(lo)), e1 = ex2(__uint_as_float(hi));
            asm("add.rn.f32x2 %0, %0, %1;"
                : "+l"(sum[(j / 2) & 1])
                : "l"(pack2(__float_as_uint(e0), __float_as_uint(e1))));
            w[j / 2] = bf16_pair(e0, e1);
          }
          tmem_st16(ts + c0 / 2, w);
          if (Sh::kHalves && c0 + 32 == BN / 2 && !by_hand) {  // the first half of the weights
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pready[sg]);
          }
        }
        if (!Sh::kHalves) settle();
        if (by_hand) {
          uint8_t* vt = sv + sg * Sh::kTile;
          const int from = max(0, from_all - blk * BN), nrow = BN - from;
          tmem_st_wait();
          // Some rows see non-finite values and some do not. Each row adds its own share of those
          // values to O (zero to begin with), then they are cleared for the tensor cores.
#pragma unroll 1
          for (int d = 0; d < D; d += 8) {
            float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (!first) tmem_ld8(trow + d, o);
#pragma unroll 1
            for (int pos = from; pos < BN; ++pos) {
              const uint4 x = *reinterpret_cast<const uint4*>(
                  vt + (d / 64) * Pl::kPanel + Pl::at(pos) + ((((d / 8) & 7) ^ (pos & 7)) << 4));
              uint32_t pw;  // this position's weight and its neighbour's
              asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\t"
                           "tcgen05.wait::ld.sync.aligned;"
                           : "=r"(pw)
                           : "r"(ts + pos / 2)
                           : "memory");
              if (pos < valid) {
                const uint32_t q4[4] = {x.x, x.y, x.z, x.w};
                const float e = __uint_as_float((pos & 1) ? (pw & 0xffff0000u) : (pw << 16));
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const float f =
                      __uint_as_float((j & 1) ? (q4[j / 2] & 0xffff0000u) : (q4[j / 2] << 16));
                  if (!(fabsf(f) < INFINITY)) o[j] += e * f;
                }
              }
              __syncwarp();
            }
            __syncwarp();
            asm volatile(
                "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                    trow + d),
                "r"(__float_as_uint(o[0])), "r"(__float_as_uint(o[1])), "r"(__float_as_uint(o[2])),
                "r"(__float_as_uint(o[3])), "r"(__float_as_uint(o[4])), "r"(__float_as_uint(o[5])),
                "r"(__float_as_uint(o[6])), "r"(__float_as_uint(o[7]))
                : "memory");
            tmem_st_wait();
          }
          bar_group();
#pragma unroll 1
          for (int i = st; i < nrow * (D / 8); i += kGroupThreads) {
            const int pos = from + i / (D / 8), ch = i % (D / 8);
            uint32_t* at = reinterpret_cast<uint32_t*>(vt + (ch / 8) * Pl::kPanel + Pl::at(pos) +
                                                       (((ch & 7) ^ (pos & 7)) << 4));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t x = at[j];
              if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
              if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
              at[j] = x;
            }
          }
          if (st == 0) o_init[piece & 1] = 1;
          fence_async_smem();
          bar_group();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (!Sh::kHalves || by_hand) mbar_arrive(&pready[sg]);
          if (Sh::kHalves) mbar_arrive(&prest[sg]);
        }
        l = (mg == m ? l : l * ex2(mg - ref)) + (sum2(sum[0]) + sum2(sum[1]));
        mg = m;
      }
      it = it0 + n;
      // every product with this piece's Q is complete: the next one's can take its place
      wait(&kdone[(it - 1) % NS], ((it - 1) / NS) & 1);
      ++piece;
      more = next_piece();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}


// Dynamic shared memory of a call, and its launch.
template <typename P, int D>
spec_status tc_launch(const P& p, const AttnMaps& m, int grid, cudaStream_t stream) {
  using Sh = Shape<D, kPaged<P>>;
  static SmemAllowance allowed;
  const int smem = Sh::kFixed + kTcSmall<P> + 24 * kTm + static_cast<int>(attn_plan_bytes(p)) + 1024;
  if (allow_dynamic_smem(attn_tc_kernel<P, D>, smem, allowed) != cudaSuccess) return SPEC_ERR_CUDA;
  return launch_pdl(attn_tc_kernel<P, D>, dim3(grid), dim3(kTcThreads), smem, stream, m, p) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // namespace spec
