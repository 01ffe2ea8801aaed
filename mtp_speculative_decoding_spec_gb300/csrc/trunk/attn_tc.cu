// Attention of the verify rows over a shared prefix and each request's own cache on the tcgen05
// tensor cores: bf16, head_dim 64, 128 or 256. Units, pieces and partials as in trunk.cuh.
//
// Per block of kBn positions: S = Q K^T (Q in TMEM, 128 rows x kBn), a row's softmax by one thread
// (TMEM lane = row, no shuffles), the weights as bf16 back into the columns of S, O += P V with P
// in TMEM too and V as it lies in the cache (rows of positions: the B operand is N-major).
//   * warp 0 loads K and V blocks by TMA; Q is gathered by the softmax threads into TMEM, so that
//     its 128 rows are not read from shared memory again for every block;
//   * warp 1 issues the MMAs: S of block i+1 goes out before O of block i, so the tensor pipe works
//     on one while the softmax works on the other (two S buffers);
//   * warps 4..7 and 8..11 do the softmax of the blocks in turns; warps 2 and 3 watch V (below). The
//     reference a row's weights are taken against moves only when the row's maximum has grown by more
//     than 2^8 (the weights stay below 256 and their sum and O are fp32, so nothing is lost), which makes
//     rescaling O in TMEM rare.
// Weights are rounded to bf16 for the tensor cores (2^-9 of each weight, as the outputs are); their
// sum is taken in fp32 before that.
//
// A position that some row does not see has weight 0 in that row, and 0 times what lies there must
// be 0. In blocks where any running row's positions end, two guard warps therefore look through V as
// it lands, ahead of the softmax: non-finite values that no row sees are cleared, and where a row
// does see one, that row's share of it is added by hand and the value cleared for the tensor cores.
//
// 16 query heads on 4 KV heads of 256 dims: 256 rows over 63,488 shared positions and 700 own ones each,
// 190 to 204 us with the join, by GPU and run = 1.42 to 1.32 PFLOP/s (0.73 to 0.68 of cuBLAS); a block of
// 64 positions takes about 1,450 cycles against 1,024 of the tensor pipe, the rest the way from a block's
// scores through its softmax to its second product, which two buffers of S hide in part. Two rows of one request over its own 63,488: 50.5
// us = 5.2 TB/s (0.76 of a copy), eight single rows over a shared 63,488 60 us = 5.0 TB/s: HBM while the
// blocks run, and some 18 us of launch, plan, first loads, partials and join around them.
#include <math.h>

#include <cuda_bf16.h>

#include "trunk.cuh"

#include "tcgen05.cuh"

namespace spec {
namespace {

constexpr int kTm = 128;
constexpr int kThreads = 12 * 32;  // producer, MMA and two guard warps, eight softmax warps
constexpr int kGroupThreads = 128;  // a softmax group
// Registers a thread: launched with 168 (64,512 in all); the first four warps give to the softmax's
// eight: 128 x 152 + 256 x 176 = 64,512. (104 and 200 spill in the guards: 214 us for 191.)
constexpr int kFewRegs = 152, kSoftRegs = 176;
// Bits that a row's maximum may grow by before its reference moves: 256 rows over 63,488 positions 260 us
// with 0, 192 with 8.
constexpr float kLazy = 8.f;

template <int D>
struct Shape {
  // K and V blocks of 16 or 32 KB. 128 dims in blocks of 64 positions took 168 us for 151 (256 rows over
  // 63,488); 256 dims in blocks of 128 do not fit beside two buffers of S.
  static constexpr int kBn = D == 256 ? 64 : 128;
  static constexpr int kStages = D == 64 ? 6 : 3;
  static constexpr int kTile = kBn * D * 2;
  // The product with V starts on the first half of a block's weights. At 128 positions: 142 -> 128 us (256
  // rows of 128 dims over 63,488); at 64 the tensor pipe, in order, waits for the second half instead of
  // taking the other buffer's scores: 191 -> 211 us (of 256 dims).
  static constexpr bool kHalves = kBn == 128;
  static constexpr int kPanel = kBn * 128;          // 64 dims of a block: rows of 128 bytes
  static constexpr int kFixed = 2 * kStages * kTile;
  // TMEM columns: O, two S buffers, Q (two bf16 a column)
  static constexpr int kS = D, kQ = D + 2 * kBn;
  static_assert(kQ + D / 2 <= 512, "TMEM");
};

// A block of K or V at once: [panel of 64 dims][position][64 dims], the order of its map's box. Called
// by a whole warp, one lane of which issues.
__device__ __forceinline__ void tma_load_block(void* dst, const CUtensorMap* map, int pos, int panel,
                                               int b, uint64_t* bar, uint32_t bytes) {
  asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%5], %6;\n\t"
        "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%7, %2, %3, %4}], [%5];\n\t}" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(pos), "r"(panel), "r"(b), "r"(smem_u32(bar)),
        "r"(bytes), "r"(0)
        : "memory");
}

// B operand whose rows (K) are 128 bytes of N in the 128-byte swizzle: 8-row groups 1,024 bytes
// apart, the next 64 of N one panel on.
__device__ __forceinline__ uint64_t smem_desc_n_major(uint32_t saddr, uint32_t panel) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((panel >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((1024u >> 4) & 0x3FFFu) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// A from TMEM (two bf16 of K per 32-bit column), B from shared memory. Called by a whole warp, one
// lane of which issues: the operands are the same in all lanes and stay in uniform registers.
__device__ __forceinline__ void tc_mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void tc_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
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
__device__ __forceinline__ bool odd_pair(uint32_t w) {  // an Inf or NaN in either half
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <int D>
__device__ __forceinline__ const __nv_bfloat16* q_row(const AttnParams& p, const AttnPiece& a,
                                                      const AttnRow& r) {
  return static_cast<const __nv_bfloat16*>(p.q) + (static_cast<int64_t>(r.b) * p.R + r.r) * p.qs +
         static_cast<int64_t>(a.head * p.G + r.g) * D;
}

struct AttnMaps {
  CUtensorMap pk, pv, ok, ov;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnParams p) {
  using Sh = Shape<D>;
  constexpr int BN = Sh::kBn, NS = Sh::kStages;
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
  uint64_t* meet = qready + 1;    // the softmax warps, [0] and [1] of a group, [2] all
  uint64_t* ofree = meet + 3;     // the piece's O has been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ofree + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* o_init = abort_flag + 1;      // [2] O holds something before the piece's first MMA on it
  volatile int* odd = abort_flag + 3;         // [NS][2]: a row sees a non-finite V of the stage
  int* least_sm = const_cast<int*>(odd + 2 * NS);  // [2][4] per quarter of the rows
  float* row_m = reinterpret_cast<float*>(smem + Sh::kFixed + 512);  // [2][128] each group's last reference
  float2* row_ml = reinterpret_cast<float2*>(row_m + 2 * kTm);       // [2][128] and sum, at a piece's end
  int32_t* cum = reinterpret_cast<int32_t*>(row_ml + 2 * kTm);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kdone[s], 1);
      mbar_init(&vfull[s], 1);
      mbar_init(&vdone[s], 1);
      mbar_init(&vok[s], 2);
      mbar_init(&pready[s], 6);
      mbar_init(&prest[s], 4);
    }
    mbar_init(qready, 8);
    mbar_init(&meet[0], 4);
    mbar_init(&meet[1], 4);
    mbar_init(&meet[2], 8);
    mbar_init(ofree, 8);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  pdl_wait();
  const AttnReq* req = attn_plan(p, cum);  // ends with a block barrier
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const AttnShares shares = attn_shares(p, cum);
  if (blockIdx.x == 0) attn_write_units(p, cum, shares);
  AttnWalk walk;
  walk.start(p, cum, shares);
  AttnPiece a;
  auto give_up = [&]() {
    atomicOr(&p.hdr->error, ERR_TC_WAIT);
    *abort_flag = 1;
  };

  if (warp < 4)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    int it = 0;  // V blocks; K runs one block ahead, as the MMAs take them
    bool ok = true;
    while (ok && !__any_sync(0xffffffffu, *abort_flag) && walk.next(p, cum, shares, a)) {
      const bool pre = a.tile < p.npt;
      const int b = pre ? 0 : (a.tile - p.npt) / p.nown, panel = a.head * (D / 64);
      auto load = [&](uint8_t* tiles, uint64_t* full, uint64_t* empty, const CUtensorMap* map, int i,
                      int blk) {
        const int s = i % NS;
        if (i >= NS && !mbar_wait_warp(&empty[s], ((i / NS) & 1) ^ 1))
          return false;
        tma_load_block(tiles + s * Sh::kTile, map, blk * BN, panel, b, &full[s], Sh::kTile);
        return true;
      };
      const CUtensorMap* mk = pre ? &maps.pk : &maps.ok;
      const CUtensorMap* mv = pre ? &maps.pv : &maps.ov;
      const int n = a.blk1 - a.blk0;
      ok = load(sk, kfull, kdone, mk, it, a.blk0);
      int j = 0;
      for (; ok && j < n; ++j) {
        if (j + 1 < n) ok = load(sk, kfull, kdone, mk, it + j + 1, a.blk0 + j + 1);
        ok = ok && load(sv, vfull, vdone, mv, it + j, a.blk0 + j);
      }
      it += j;
    }
    if (!ok && lane == 0) give_up();
    // Leave nothing in flight: the last loads of every stage have landed. Where a wait ran out, V's last
    // was not sent and one more of K's may have been; what was not sent costs a wait with its limit.
    for (int j = max(0, it - NS); j < it + !ok; ++j) mbar_wait_warp(&kfull[j % NS], (j / NS) & 1);
    for (int j = max(0, it - NS - !ok); j < it; ++j) mbar_wait_warp(&vfull[j % NS], (j / NS) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    {
      constexpr uint32_t kIdS = tc_idesc(kTm, BN);
      constexpr uint32_t kIdO = tc_idesc(kTm, D) | (1u << 16);  // B is N-major
      const uint64_t kd0 = smem_desc_sw128(smem_u32(sk));
      const uint64_t vd0 = smem_desc_n_major(smem_u32(sv), Sh::kPanel);
      int it = 0, piece = 0;
      bool ok = true;
      auto scores = [&](int i) {
        if (!mbar_wait_warp(&kfull[i % NS], (i / NS) & 1)) return false;
        tc_fence_after();
        const uint64_t kd = desc_advance(kd0, (i % NS) * Sh::kTile);
        const uint32_t ds = tmem + Sh::kS + (i & 1) * BN;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_ta(ds, tmem + Sh::kQ + kk * 8,
                    desc_advance(kd, (kk / 4) * Sh::kPanel + (kk % 4) * 32), kIdS, kk > 0);
        tc_commit_elect(&kdone[i % NS]);
        return true;
      };
      while (ok && !__any_sync(0xffffffffu, *abort_flag) && walk.next(p, cum, shares, a)) {
        const int n = a.blk1 - a.blk0;
        ok = mbar_wait_warp(qready, piece & 1);
        tc_fence_after();
        ok = ok && scores(it);
        for (int j = 0; ok && j < n; ++j) {
          const int i = it + j;
          if (j + 1 < n) ok = scores(i + 1);
          ok = ok && mbar_wait_warp(&pready[i % NS], (i / NS) & 1);
          if (j == 0 && piece > 0)
            ok = ok && mbar_wait_warp(ofree, (piece - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = desc_advance(vd0, (i % NS) * Sh::kTile);
          const uint32_t ps = tmem + Sh::kS + (i & 1) * BN;
          const uint32_t acc0 = j > 0 || o_init[piece & 1] ? 1u : 0u;
#pragma unroll
          for (int kk = 0; kk < BN / (Sh::kHalves ? 32 : 16); ++kk)
            tc_mma_ta(tmem, ps + kk * 8, desc_advance(vd, kk * 2048), kIdO, kk > 0 ? 1u : acc0);
          if constexpr (Sh::kHalves) {
            ok = mbar_wait_warp(&prest[i % NS], (i / NS) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = BN / 32; kk < BN / 16; ++kk)
              tc_mma_ta(tmem, ps + kk * 8, desc_advance(vd, kk * 2048), kIdO, 1u);
          }
          tc_commit_elect(&vdone[i % NS]);
        }
        it += n;
        ++piece;
      }
      if (!ok && lane == 0) give_up();
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------------ guards of V
    // In a block where some running row's positions end, non-finite values of positions that no
    // row sees are cleared; those that a row does see are reported to the softmax.
    const int gw = warp - 2;
    int it = 0;
    bool ok = true;
    while (ok && !__any_sync(0xffffffffu, *abort_flag) && walk.next(p, cum, shares, a)) {
      int least = 0x7fffffff, most = 0;  // positions every running row sees; positions any row sees
      for (int i = lane; i < kTm; i += 32) {
        const int lim = attn_row(p, req, a.tile, i).lim;
        most = max(most, lim);
        if (lim > 0) least = min(least, lim);
      }
      least = __reduce_min_sync(0xffffffffu, least);
      most = __reduce_max_sync(0xffffffffu, most);
      {  // the next piece's queries, towards L2
        AttnWalk ahead = walk;
        AttnPiece nx;
        if (ahead.next(p, cum, shares, nx))
          for (int i = gw * 32 + lane; i < kTm; i += 64) {
            const AttnRow r = attn_row(p, req, nx.tile, i);
            if (r.lim <= 0) continue;
            const __nv_bfloat16* src = q_row<D>(p, nx, r);
            for (int d = 0; d < D; d += 64)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(src + d));
          }
      }
      for (int blk = a.blk0; ok && blk < a.blk1; ++blk, ++it) {
        const int s = it % NS;
        ok = mbar_wait_warp(&vfull[s], (it / NS) & 1);
        bool seen = false;
        if (blk * BN + BN > least) {
          uint8_t* vt = sv + s * Sh::kTile;
          const int from = max(0, least - blk * BN);
          // The swizzle keeps a position's 128 bytes of a panel together, so each panel is one run of
          // 16-byte chunks. An exponent of all ones carries into its half's top bit.
          const int run = (BN - from) * 8;
          uint32_t any = 0;
#pragma unroll 1
          for (int j = 0; j < D / 64; ++j) {
            const uint8_t* base = vt + j * Sh::kPanel + from * 128;
#pragma unroll
            for (int k = 0; k < BN * 8 / 64; ++k) {
              const uint4 x = lds128(base + min(k * 64 + gw * 32 + lane, run - 1) * 16);
              any |= (x.x & 0x7f807f80u) + 0x00800080u;
              any |= (x.y & 0x7f807f80u) + 0x00800080u;
              any |= (x.z & 0x7f807f80u) + 0x00800080u;
              any |= (x.w & 0x7f807f80u) + 0x00800080u;
            }
          }
          if (__any_sync(0xffffffffu, any & 0x80008000u)) {
            for (int j = 0; j < D / 64; ++j)
              for (int i = gw * 32 + lane; i < run; i += 64) {
                uint4* at = reinterpret_cast<uint4*>(vt + j * Sh::kPanel + from * 128 + i * 16);
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
          odd[2 * s + gw] = seen;
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
    const float scale = fabsf(p.scale_log2);
    int it = 0;
    // A wait that runs out ends all further waiting, not the walk: whatever happens, a softmax warp
    // goes through the same pieces as the others, which it meets at `meet` and at named barriers.
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!ok || mbar_wait_warp(bar, parity)) return;
      if (lane == 0) give_up();
      ok = false;
    };
    uint32_t met_all = 0, met_group = 0;
    auto bar_all = [&]() {  // a barrier of the softmax warps, with the limit of every wait
      __syncwarp();
      if (lane == 0) mbar_arrive(&meet[2]);
      wait(&meet[2], met_all++ & 1);
    };
    auto bar_group = [&]() {  // of the group's
      __syncwarp();
      if (lane == 0) mbar_arrive(&meet[half]);
      wait(&meet[half], met_group++ & 1);
    };
    // Q of a piece: this thread's half of its row into its TMEM lane; a negative scale goes into Q's signs
    int piece = 0, least = 0;
    AttnRow ar;
    auto load_q = [&](const AttnPiece& pc) {
      ar = attn_row(p, req, pc.tile, row);
      const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
      const __nv_bfloat16* src = q_row<D>(p, pc, ar);
      uint32_t w[DH / 2];
      if (__all_sync(0xffffffffu, (reinterpret_cast<uintptr_t>(src) & 31u) == 0)) {
#pragma unroll
        for (int c = 0; c < DH / 16; ++c) load32(src + half * DH + 16 * c, w + 8 * c);
      } else {
        const uint16_t* from = reinterpret_cast<const uint16_t*>(src + half * DH);
#pragma unroll
        for (int c = 0; c < DH / 2; ++c) w[c] = from[2 * c] | static_cast<uint32_t>(from[2 * c + 1]) << 16;
      }
      // rows that do not run have read row 0's
#pragma unroll
      for (int c = 0; c < DH / 2; ++c) w[c] = ar.lim > 0 ? w[c] ^ flip : 0u;
      tmem_st<DH / 2>(trow + Sh::kQ + half * (DH / 2), w);
      tmem_st_wait();
      const int lo = __reduce_min_sync(0xffffffffu, ar.lim > 0 ? ar.lim : 0x7fffffff);
      int* lsm = least_sm + 4 * (piece & 1);
      if (lane == 0 && half == 0) lsm[quad] = lo;
      if (st == 0 && half == 0) o_init[piece & 1] = 0;
      tc_fence_before();
      bar_all();
      if (lane == 0) mbar_arrive(qready);
      least = min(min(lsm[0], lsm[1]), min(lsm[2], lsm[3]));
    };
    bool more = walk.next(p, cum, shares, a);
    if (more) load_q(a);
    while (more) {
      const int lim = ar.lim, from_all = least;
      const int64_t at = static_cast<int64_t>(a.slot) * kTm + row;
      const int blk_end = a.blk1;
      const int n = blk_end - a.blk0, it0 = it;
      float mg = -INFINITY, l = 0.f;  // of the group's blocks: the last reference, the sum
      it += (it & 1) ^ half;          // the first of them
      for (int blk = a.blk0 + it - it0; blk < blk_end; blk += 2, it += 2) {
        const bool first = it == it0, last = it + 1 == it0 + n;
        const int valid = min(BN, lim - blk * BN);  // positions of the block this row sees
        const bool full = __all_sync(0xffffffffu, valid >= BN);
        wait(&kdone[it % NS], (it / NS) & 1);
        tc_fence_after();
        const uint32_t ts = trow + Sh::kS + half * BN;
        float v[64], raw = -INFINITY;
#pragma unroll
        for (int c0 = 0; c0 < BN; c0 += 64) {
          tmem_ld64(ts + c0, v);
          if (!full) {
#pragma unroll
            for (int j = 0; j < 64; ++j) v[j] = c0 + j < valid ? v[j] : -INFINITY;
          }
          float mx[4] = {raw, v[1], v[2], v[3]};
          mx[0] = max3(mx[0], v[0], v[4]);
#pragma unroll
          for (int j = 5; j + 1 < 64; j += 2) mx[(j / 2) & 3] = max3(mx[(j / 2) & 3], v[j], v[j + 1]);
          raw = max3(max3(mx[0], mx[1], v[63]), mx[2], mx[3]);
        }
        const float top = raw == -INFINITY ? -INFINITY : raw * scale;
        float mo = -INFINITY;  // the reference after the block before, from the other group
        if (!first) {
          asm volatile("bar.sync %0, 64;" ::"r"(1 + 4 * (half ^ 1) + quad) : "memory");
          mo = row_m[(half ^ 1) * kTm + row];
        }
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
            by_hand = odd[2 * sg] | odd[2 * sg + 1];
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
        // A weight is 2^(scale s - ref): two at a time in packed arithmetic. Of 128 scores the last 32 stay
        // in registers; the others are read again, before weights take their columns.
        unsigned long long sum[2] = {0ull, 0ull};
        const unsigned long long scale2 = pack2(__float_as_uint(scale), __float_as_uint(scale));
        const unsigned long long ref2 = pack2(__float_as_uint(-ref), __float_as_uint(-ref));
#pragma unroll
        for (int c0 = 0; c0 < BN; c0 += 32) {
          float again[32];
          const bool kept = BN == 64 || c0 + 32 == BN;
          if (!kept) tmem_ld32(ts + c0, again);
          const float* x = kept ? v + (c0 & 32) : again;
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            unsigned long long y = ref2;
            ffma2_acc(y, pack2(__float_as_uint(x[j]), __float_as_uint(x[j + 1])), scale2);
            uint32_t lo, hi;
            asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(y));
            float e0 = ex2(__uint_as_float(lo)), e1 = ex2(__uint_as_float(hi));
            if (!full) {
              e0 = c0 + j < valid ? e0 : 0.f;
              e1 = c0 + j + 1 < valid ? e1 : 0.f;
            }
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
            for (int pos = from; pos < BN; ++pos) {
              const uint4 x = *reinterpret_cast<const uint4*>(
                  vt + (d / 64) * Sh::kPanel + pos * 128 + ((((d / 8) & 7) ^ (pos & 7)) << 4));
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
          for (int i = st; i < nrow * (D / 8); i += kGroupThreads) {
            const int pos = from + i / (D / 8), ch = i % (D / 8);
            uint32_t* at = reinterpret_cast<uint32_t*>(vt + (ch / 8) * Sh::kPanel + pos * 128 +
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
      // every product with this piece's Q is complete: the next one's can take its place, and its first
      // scores be computed, while this piece's output is written
      const int lb = it - 1;
      wait(&kdone[lb % NS], (lb / NS) & 1);
      ++piece;
      more = walk.next(p, cum, shares, a);
      if (more) load_q(a);
      // the piece's partial
      wait(&vdone[lb % NS], (lb / NS) & 1);
      tc_fence_after();
      row_ml[half * kTm + row] = make_float2(mg, l);
      asm volatile("bar.sync %0, 64;" ::"r"(9 + quad) : "memory");
      if (lim > 0 && half == 0) {
        const float2 other = row_ml[kTm + row];
        // the reference never falls, so the greater one is the last one's
        const float m = fmaxf(mg, other.x), ref = m == -INFINITY ? 0.f : m;
        const float sum = l * ex2(mg - ref) + other.y * ex2(other.x - ref);
        // The maxima pass over scores that are not numbers, the sum does not. The join takes a maximum of
        // -Inf for a row that saw nothing, so such a partial says NaN there.
        p.ml[at] = make_float2(sum != sum ? sum : m, sum);
      }
#pragma unroll 1
      for (int d = half * DH; d < half * DH + DH; d += 32) {
        float o[32];
        tmem_ld32(trow + d, o);
        if (lim > 0) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) store32(p.o + at * D + d + j, o + j);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
spec_status launch_tc(const AttnParams& p, int grid, EncodeTiledFn encode, cudaStream_t stream) {
  using Sh = Shape<D>;
  static SmemAllowance allowed;
  const int smem = Sh::kFixed + 512 + 24 * kTm + static_cast<int>(attn_plan_bytes(p.items, p.B)) + 1024;
  if (allow_dynamic_smem(attn_tc_kernel<D>, smem, allowed) != cudaSuccess) return SPEC_ERR_CUDA;
  AttnMaps m;
  // dims inside a 64-dim panel, positions, panels (64 dims on), requests
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(Sh::kBn), D / 64, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const auto map = [&](CUtensorMap* t, const uint8_t* base, int64_t positions, int64_t step, int64_t reqs,
                       int64_t req_step) {
    const cuuint64_t dim[4] = {64, static_cast<cuuint64_t>(positions),
                               static_cast<cuuint64_t>(p.Hkv) * (D / 64), static_cast<cuuint64_t>(reqs)};
    const cuuint64_t stride[3] = {static_cast<cuuint64_t>(step), 128, static_cast<cuuint64_t>(req_step)};
    return encode(t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint8_t*>(base), dim, stride, box,
                  es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const int64_t req = p.B > 1 ? p.kreq : p.krow;
  if (!map(&m.ok, p.kk, p.kcap, p.krow, p.B, req) || !map(&m.ov, p.kv, p.kcap, p.krow, p.B, req))
    return SPEC_ERR_CUDA;
  m.pk = m.ok;
  m.pv = m.ov;
  if (p.npt > 0 && (!map(&m.pk, p.pk, p.pcap, p.pstride, 1, p.pstride) ||
                    !map(&m.pv, p.pv, p.pcap, p.pstride, 1, p.pstride)))
    return SPEC_ERR_CUDA;
  return launch_pdl(attn_tc_kernel<D>, dim3(grid), dim3(kThreads), smem, stream, m, p) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // namespace

bool attn_tc_takes(int head_dim) { return head_dim == 64 || head_dim == 128 || head_dim == 256; }
int attn_tc_tm() { return kTm; }
int attn_tc_bn(int head_dim) { return head_dim == 256 ? Shape<256>::kBn : Shape<128>::kBn; }

spec_status attn_tc_launch(const AttnParams& p, int grid, EncodeTiledFn encode, cudaStream_t stream) {
  return p.D == 256   ? launch_tc<256>(p, grid, encode, stream)
         : p.D == 128 ? launch_tc<128>(p, grid, encode, stream)
                      : launch_tc<64>(p, grid, encode, stream);
}

}  // namespace spec
