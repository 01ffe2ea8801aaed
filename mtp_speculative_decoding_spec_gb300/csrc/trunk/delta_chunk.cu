// The gated delta rule over prompts by chunks of 64 tokens (bf16 inputs, rec_dk 128, rec_dv a multiple
// of 16). With G_i the running sum of the log decays in a chunk, S the state before it and
//   A_ij = beta_i e^(G_i - G_j) k_i.k_j (j < i),   T = (I + A)^-1 diag(beta),
// the chunk's updates, outputs and last state are
//   u = T (v - e^G (k S)),   o = scale (e^G (q S) + (e^(G_i - G_j) q_i.k_j)_(j <= i) u),
//   S' = e^G_last S + sum_j e^(G_last - G_j) k_j u_j^T.
// Two kernels. The first works all chunks out side by side: T and the scores of q against k, everything
// that does not need S. The second walks each head's chunks in turn, and is what the time goes to: a
// chain of three small products per chunk, each the next one's operand. Every column of S is a chain
// of its own, so a block takes 16 columns of one head (the least a matrix instruction takes) and
// there are rec_dv / 16 blocks a head; a block's four warps share out tokens and rows of S.
//
// The products run on the warp-level matrix instruction (m16n8k16, bf16 in, fp32 out), whose results
// are already in the registers that the next product is made from: at 16 columns a tcgen05 product
// would read its 128-row operand for 16 columns of result and cross tensor memory three times a
// chunk. S, u and T are fp32. q, k and v are bf16 as given; S, u, T enter products as sums of three
// bf16 (24 bits), with the product terms below 2^-24 left out, and sums are fp32: the state is as
// exact as fp32 arithmetic leaves it. Where only a bf16 output is made, two parts are enough.
#include <math.h>

#include <cuda_bf16.h>

#include "trunk.cuh"

namespace spec {
namespace {

constexpr int kC = 64;                 // tokens per chunk
constexpr int kDk = 128;
constexpr int kCols = 16;              // columns of S per block
constexpr int kPlane = kC * 128;       // a 64 x 64 bf16 matrix: rows of 128 bytes, swizzled
constexpr int kTBytes = 3 * kPlane;    // T in three parts
constexpr int kABytes = 2 * kPlane;    // scores in two parts
constexpr int kVecBytes = 1024;        // e^G [64], e^(G_last - G) [64], e^G_last
constexpr int kRec = kTBytes + kABytes + kVecBytes;  // one chunk and head of the workspace
constexpr int kTile = kC * kDk * 2;    // K or Q of a chunk: two panels of 64 dims

// Where 16-byte piece c (0..7) of row r lies in a run of swizzled 128-byte rows.
__device__ __forceinline__ int swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

__device__ __forceinline__ void ldm4(uint32_t a, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t a, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // an 8 x 8 matrix of 16-bit values
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// x, y as sums of N bf16 each, packed in pairs. A part that is not finite (x infinite or beyond bf16)
// leaves no finite rest, so what follows it is not a number, as x times anything summed with it is.
template <int N>
__device__ __forceinline__ void split(float x, float y, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i] = pack(x, y);
    x -= lo_of(w[i]);
    y -= hi_of(w[i]);
  }
}

struct Span {  // a chunk's request, first row and number of rows
  int b, row0, len;
};
__device__ __forceinline__ int cu_at(const DeltaParams& p, int b) {
  return static_cast<int>(max(static_cast<int64_t>(0),
                              min(static_cast<int64_t>(p.cu_rows[b]), p.rows)));
}
// Requests' chunks take slots of their own: request b's first is cu[b] / 64 + b, and as many follow as
// it has chunks.
__device__ __forceinline__ int first_slot(int cu, int b) { return cu / kC + b; }

// ------------------------------------------------------------------------- what needs no state
// One block per (slot, value head), 128 threads.
constexpr int kPrepThreads = 128;
constexpr int kLPitch = 68;  // floats between rows of A
constexpr int kPrepSmem = 2 * kTile + kABytes + kVecBytes + kC * kLPitch * 4 + 4 * kC * 4;

__global__ void __launch_bounds__(kPrepThreads)
    delta_prep_kernel(const __grid_constant__ DeltaParams p, uint8_t* rec) {
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* sk = smem;                              // K, Q; then the parts of T
  uint8_t* sq = smem + kTile;
  uint8_t* sa = smem + 2 * kTile;                  // scores, vectors
  float* vec = reinterpret_cast<float*>(sa + kABytes);
  float* L = reinterpret_cast<float*>(sa + kABytes + kVecBytes);
  float* ghi = L + kC * kLPitch;
  float* glo = ghi + kC;
  float* beta = glo + kC;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = blockIdx.x, h = blockIdx.y;
  if (tid == 0 && slot == 0 && h == 0) p.hdr->error = 0;
  int lo = 0, hi = p.B;  // the last request whose first slot is not past this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first_slot(cu_at(p, mid), mid) <= slot)
      lo = mid;
    else
      hi = mid;
  }
  const int c0 = cu_at(p, lo), c1 = max(c0, cu_at(p, lo + 1));
  const int row0 = c0 + (slot - first_slot(c0, lo)) * kC;
  const int len = min(kC, c1 - row0);
  if (len <= 0) return;  // the whole block
  const int kh = h / (p.H / p.Hk);
  {
    const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(p.k) + static_cast<int64_t>(kh) * kDk;
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q) + static_cast<int64_t>(kh) * kDk;
#pragma unroll 4
    for (int i = tid; i < kC * 16; i += kPrepThreads) {
      const int r = i >> 4, c = i & 15;
      uint4 k = make_uint4(0u, 0u, 0u, 0u), q = k;
      if (r < len) {
        k = __ldg(reinterpret_cast<const uint4*>(kp + (row0 + r) * p.ks) + c);
        q = __ldg(reinterpret_cast<const uint4*>(qp + (row0 + r) * p.qs) + c);
      }
      const int at = (c >> 3) * kPlane + swz(r, c & 7);
      *reinterpret_cast<uint4*>(sk + at) = k;
      *reinterpret_cast<uint4*>(sq + at) = q;
    }
  }
  if (warp == 0) {
    // Running sums in 64 bits, kept as two floats each: the difference of two of them is then as exact
    // as a float, however far they have run. A decay below e^-200 is 0 in fp32 either way.
    const int t0 = 2 * lane, t1 = t0 + 1;
    float g0 = t0 < len ? p.g[(static_cast<int64_t>(row0) + t0) * p.H + h] : 0.f;
    float g1 = t1 < len ? p.g[(static_cast<int64_t>(row0) + t1) * p.H + h] : 0.f;
    g0 = g0 < -200.f ? -200.f : g0;
    g1 = g1 < -200.f ? -200.f : g1;
    beta[t0] = t0 < len ? p.beta[(static_cast<int64_t>(row0) + t0) * p.H + h] : 0.f;
    beta[t1] = t1 < len ? p.beta[(static_cast<int64_t>(row0) + t1) * p.H + h] : 0.f;
    double s = static_cast<double>(g0) + g1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += x;
    }
    const double a = s - g1, last = __shfl_sync(0xffffffffu, s, 31);
    ghi[t0] = static_cast<float>(a);
    glo[t0] = static_cast<float>(a - ghi[t0]);
    ghi[t1] = static_cast<float>(s);
    glo[t1] = static_cast<float>(s - ghi[t1]);
    vec[t0] = expf(static_cast<float>(a));
    vec[t1] = expf(static_cast<float>(s));
    vec[kC + t0] = t0 < len ? expf(static_cast<float>(last - a)) : 0.f;
    vec[kC + t1] = t1 < len ? expf(static_cast<float>(last - s)) : 0.f;
    if (lane == 0) vec[2 * kC] = expf(static_cast<float>(last));
  }
  __syncthreads();
  // K K^T and Q K^T, lower triangle: warp w takes rows 16 w..16 w + 15, column tiles up to them
  {
    const uint32_t k32 = smem_u32(sk), q32 = smem_u32(sq);
    float kk[8][4] = {}, qk[8][4] = {};
    const int ar = warp * 16 + (lane & 15), ac = lane >> 4;                 // A: rows, halves of k
    const int br = (lane & 7) + ((lane >> 4) << 3), bc = (lane >> 3) & 1;   // B: two column tiles
#pragma unroll
    for (int s = 0; s < kDk / 16; ++s) {
      uint32_t ka[4], qa[4];
      const int pan = (s >> 2) * kPlane, c = (s & 3) * 2;
      ldm4(k32 + pan + swz(ar, c + ac), ka);
      ldm4(q32 + pan + swz(ar, c + ac), qa);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t <= warp) {
          uint32_t b[4];
          ldm4(k32 + pan + swz(t * 16 + br, c + bc), b);
          mma(kk[2 * t], ka, b[0], b[1]);
          mma(kk[2 * t + 1], ka, b[2], b[3]);
          mma(qk[2 * t], qa, b[0], b[1]);
          mma(qk[2 * t + 1], qa, b[2], b[3]);
        }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = warp * 16 + (lane >> 2) + 8 * half, j = t * 8 + 2 * (lane & 3);
        float l[2], a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float d = expf((ghi[i] - ghi[j + e]) + (glo[i] - glo[j + e]));
          l[e] = j + e < i ? beta[i] * d * kk[t][2 * half + e] : 0.f;
          a[e] = j + e <= i ? p.scale * d * qk[t][2 * half + e] : 0.f;
        }
        *reinterpret_cast<float2*>(L + i * kLPitch + j) = make_float2(l[0], l[1]);
        uint32_t w[2];
        split<2>(a[0], a[1], w);
        const int at = swz(i, t) + 4 * (lane & 3);
        *reinterpret_cast<uint32_t*>(sa + at) = w[0];
        *reinterpret_cast<uint32_t*>(sa + kPlane + at) = w[1];
      }
    }
  }
  __syncthreads();
  // (I + A)^-1 by forward substitution, a column to a thread in registers, rows above it zero
  if (warp < 2) {
    float t[kC];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      t[i] = i == tid ? 1.f : 0.f;
      if (i < 32 && warp == 1) continue;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < i; j += 4) {
        const float4 x = *reinterpret_cast<const float4*>(L + i * kLPitch + j);
        acc[0] = fmaf(x.x, t[j], acc[0]);
        if (j + 1 < i) acc[1] = fmaf(x.y, t[j + 1], acc[1]);
        if (j + 2 < i) acc[2] = fmaf(x.z, t[j + 2], acc[2]);
        if (j + 3 < i) acc[3] = fmaf(x.w, t[j + 3], acc[3]);
      }
      t[i] -= (acc[0] + acc[1]) + (acc[2] + acc[3]);
    }
    const float bt = beta[tid];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float x = t[i] * bt;
      __nv_bfloat16* at = reinterpret_cast<__nv_bfloat16*>(smem + swz(i, tid >> 3) + 2 * (tid & 7));
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        const __nv_bfloat16 v = __float2bfloat16_rn(x);
        at[s * (kPlane / 2)] = v;
        x -= __bfloat162float(v);
      }
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  if (tid == 0) {
    uint8_t* dst = rec + (static_cast<int64_t>(slot) * p.H + h) * kRec;
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                 "r"(smem_u32(smem)), "r"(kTBytes)
                 : "memory");
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst + kTBytes),
                 "r"(smem_u32(sa)), "r"(kABytes + kVecBytes)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
  }
}

// ------------------------------------------------------------------------- the chain of chunks
// Grid (rec_dv / 16, H, B), clusters of blocks of one head, which read the same K, Q, T and scores:
// each loads a share of them and multicasts it to all. Four compute warps and a producer warp.
constexpr int kChainThreads = 5 * 32;
constexpr int kStages = 2;
constexpr int kVTile = kC * kCols * 2;
constexpr int kStage = 2 * kTile + kRec + kVTile;  // K, Q, record, V
constexpr int kPieces = 8;                         // two panels of K, of Q, four quarters of the record
constexpr int kSPlane = kCols * 256;               // S^T: two panels of 16 rows of 128 bytes
constexpr int kUPlane = kCols * 128;               // 16 x 64
constexpr int kWork = 3 * kSPlane + 8 * kUPlane;   // S, r, u scaled for the state (3 each), u (2)
constexpr int kChainSmem = kStages * kStage + kWork + 256 + 1024;
static_assert(kRec % 64 == 0 && kStage % 128 == 0, "copies of whole 16-byte units");

struct ChainMaps {
  CUtensorMap k, q, v;  // [rows][columns], boxes of 64 x 64 (swizzled) and 16 x 64
};

// A box of 64 rows (a run of bytes) to this block, or to the same place in all blocks of the cluster, the
// bytes counted on each one's barrier.
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar,
                                        int cs, uint16_t mask) {
  if (cs > 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".multicast::cluster [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "h"(mask)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint32_t bar,
                                          int cs, uint16_t mask) {
  if (cs > 1)
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.multicast::cluster"
        " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(bar), "h"(mask)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void bar_compute() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__global__ void __launch_bounds__(kChainThreads, 1)
    delta_chain_kernel(const __grid_constant__ ChainMaps maps, const __grid_constant__ DeltaParams p,
                       const uint8_t* rec, int cs) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  // every swizzled tile starts at a multiple of 1,024 bytes: K and Q tiles and T and score planes do
  // (kStage is padded below), the work planes are 128-byte rows whose count is a multiple of 8
  uint8_t* work = smem + kStages * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(work + kWork);
  uint64_t* empty = full + kStages;    // this block's warps are done with the stage
  uint64_t* pempty = empty + kStages;  // all blocks of the cluster are
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, b = blockIdx.z, kh = h / (p.H / p.Hk);
  const int col0 = blockIdx.x * kCols, rank = blockIdx.x % cs;
  pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
      mbar_init(&pempty[s], cs);
    }
    fence_mbar_init();
  }
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  pdl_wait();
  const int c0 = cu_at(p, b), c1 = max(c0, cu_at(p, b + 1));
  const int n = (c1 - c0 + kC - 1) / kC;
  const int64_t elems = static_cast<int64_t>(p.layers) * p.H * p.dk * p.dv;
  const int64_t off = b * elems + (static_cast<int64_t>(p.layer) * p.H + h) * p.dk * p.dv + col0;

  if (warp == 4) {
    // ------------------------------------------------------------------ producer
    const uint8_t* base = rec + (static_cast<int64_t>(first_slot(c0, b)) * p.H + h) * kRec;
    const uint16_t mask = static_cast<uint16_t>((1u << cs) - 1);
    bool ok = true;
    int c = 0;
    for (; c < n; ++c) {
      const int s = c % kStages;
      const uint32_t parity = ((c / kStages) & 1) ^ 1;
      if (c >= kStages) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(&empty[s], parity));
        if (lane < cs) {
          uint32_t remote;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                       : "=r"(remote)
                       : "r"(smem_u32(&pempty[s])), "r"(lane));
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote)
                       : "memory");
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(&pempty[s], parity));
        if (!ok) break;
      }
      uint8_t* st = smem + s * kStage;
      if (lane == 0) {
        const int row = c0 + c * kC;
        const uint32_t bar = smem_u32(&full[s]);
        mbar_arrive_expect_tx(&full[s], kStage);
        tma_box(st + 2 * kTile + kRec, &maps.v, h * p.dv + col0, row, bar, 1, 0);
        for (int i = rank; i < kPieces; i += cs) {
          if (i < 4) {
            tma_box(st + (i >> 1) * kTile + (i & 1) * kPlane, i < 2 ? &maps.k : &maps.q,
                   kh * kDk + (i & 1) * 64, row, bar, cs, mask);
          } else {
            bulk_copy(st + 2 * kTile + (i - 4) * (kRec / 4),
                      base + static_cast<int64_t>(c) * p.H * kRec + (i - 4) * (kRec / 4), kRec / 4, bar,
                      cs, mask);
          }
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&p.hdr->error, ERR_TC_WAIT);
    for (int j = max(0, c - kStages); j < c; ++j)  // nothing is left in flight
      mbar_wait_bounded(&full[j % kStages], (j / kStages) & 1);
  } else {
    // ------------------------------------------------------------------ compute
    // S^T: this warp's rows of S are dims 32 w..32 w + 31; in registers, lane (g, q) of the fragment
    // has columns col0 + g and + 8 of dims 32 w + 8 t + 2 q and + 1
    const int g = lane >> 2, q = lane & 3;
    const uint32_t sp = smem_u32(work);                      // parts of S
    const uint32_t rp = sp + 3 * kSPlane;                    // of r
    const uint32_t up = rp + 3 * kUPlane;                    // of e^(G_last - G) u
    const uint32_t op = up + 3 * kUPlane;                    // of u
    uint8_t* sps = work;
    uint8_t* rps = sps + 3 * kSPlane;
    uint8_t* ups = rps + 3 * kUPlane;
    uint8_t* ops = ups + 3 * kUPlane;
    float S[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dim = 32 * warp + 8 * t + 2 * q + (e & 1), col = g + 8 * (e >> 1);
        S[t][e] = p.init ? p.init[off + static_cast<int64_t>(dim) * p.dv + col] : 0.f;
      }
    auto put_state = [&]() {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[3];
          split<3>(S[t][2 * half], S[t][2 * half + 1], w);
          // dim 32 w + 8 t: panel w / 2, 16-byte piece 4 (w & 1) + t
          const int at = (warp >> 1) * (kSPlane / 2) + swz(g + 8 * half, 4 * (warp & 1) + t) + 4 * q;
#pragma unroll
          for (int s = 0; s < 3; ++s) *reinterpret_cast<uint32_t*>(sps + s * kSPlane + at) = w[s];
        }
    };
    put_state();
    bar_compute();
    // token tiles of 8: this warp's are tl and tr; causality gives every warp the same work
    const int tl = warp, tr = 7 - warp;
    // lane's row and 16-byte piece of an A operand, and of B tiles of tokens tl (lanes 0-15) and tr
    const int ar = lane & 15, ac = lane >> 4;
    const int bt = (lane & 16 ? tr : tl) * 8 + (lane & 7), bc = (lane >> 3) & 1;
    bool ok = true;
    for (int c = 0; c < n; ++c) {
      const int s = c % kStages;
      if (ok && !mbar_wait_bounded(&full[s], (c / kStages) & 1)) {
        atomicOr(&p.hdr->error, ERR_TC_WAIT);
        ok = false;
      }
      uint8_t* st = smem + s * kStage;
      const uint32_t k32 = smem_u32(st), q32 = k32 + kTile, t32 = k32 + 2 * kTile, a32 = t32 + kTBytes;
      const float* eg = reinterpret_cast<const float*>(st + 2 * kTile + kTBytes + kABytes);
      const float* el = eg + kC;
      const uint8_t* sv = st + 2 * kTile + kRec;
      const int len = min(kC, c1 - c0 - c * kC);
      if (len < kC) {
        // rows past the request's end are another's: what they hold must not reach S even times 0
        for (int i = tid; i < (kC - len) * 16; i += 128) {
          const int r = len + (i >> 4), pc = i & 15;
          *reinterpret_cast<uint4*>(st + (pc >> 3) * kPlane + swz(r, pc & 7)) = make_uint4(0u, 0u, 0u, 0u);
        }
        bar_compute();
      }
      // k S and q S of the warp's tokens
      float xk[2][4] = {}, xq[2][4] = {};
#pragma unroll
      for (int i = 0; i < kDk / 16; ++i) {
        const int pan = i >> 2, pc = (i & 3) * 2;
        uint32_t a0[4], a1[4], a2[4], kb[4], qb[4];
        const uint32_t sa = sp + pan * (kSPlane / 2) + swz(ar, pc + ac);
        ldm4(sa, a0);
        ldm4(sa + kSPlane, a1);
        ldm4(sa + 2 * kSPlane, a2);
        const int bo = pan * kPlane + swz(bt, pc + bc);
        ldm4(k32 + bo, kb);
        ldm4(q32 + bo, qb);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          mma(xk[t], a2, kb[2 * t], kb[2 * t + 1]);
          mma(xk[t], a1, kb[2 * t], kb[2 * t + 1]);
          mma(xk[t], a0, kb[2 * t], kb[2 * t + 1]);
          mma(xq[t], a1, qb[2 * t], qb[2 * t + 1]);
          mma(xq[t], a0, qb[2 * t], qb[2 * t + 1]);
        }
      }
      // r = v - e^G (k S)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int tile = t ? tr : tl;
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // columns g, g + 8
          const uint32_t v = transpose8(
              *reinterpret_cast<const uint32_t*>(sv + (tile * 8 + g) * (kCols * 2) + 16 * half + 4 * q));
          const int tok = tile * 8 + 2 * q;
          const float r0 = tok < len ? fmaf(-eg[tok], xk[t][2 * half], lo_of(v)) : 0.f;
          const float r1 = tok + 1 < len ? fmaf(-eg[tok + 1], xk[t][2 * half + 1], hi_of(v)) : 0.f;
          uint32_t w[3];
          split<3>(r0, r1, w);
          const int at = swz(g + 8 * half, tile) + 4 * q;
#pragma unroll
          for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t*>(rps + i * kUPlane + at) = w[i];
        }
      }
      bar_compute();
      // u = T r
      float u[2][4] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i > tr / 2) break;  // tokens after the tile's
        uint32_t r[3][4], tb[3][4];
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          ldm4(rp + j * kUPlane + swz(ar, 2 * i + ac), r[j]);
          ldm4(t32 + j * kPlane + swz(bt, 2 * i + bc), tb[j]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t == 0 && i > tl / 2) continue;
          mma(u[t], r[0], tb[2][2 * t], tb[2][2 * t + 1]);
          mma(u[t], r[2], tb[0][2 * t], tb[0][2 * t + 1]);
          mma(u[t], r[1], tb[1][2 * t], tb[1][2 * t + 1]);
          mma(u[t], r[0], tb[1][2 * t], tb[1][2 * t + 1]);
          mma(u[t], r[1], tb[0][2 * t], tb[0][2 * t + 1]);
          mma(u[t], r[0], tb[0][2 * t], tb[0][2 * t + 1]);
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int tile = t ? tr : tl, tok = tile * 8 + 2 * q;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int at = swz(g + 8 * half, tile) + 4 * q;
          uint32_t w[3], x[2];
          split<3>(el[tok] * u[t][2 * half], el[tok + 1] * u[t][2 * half + 1], w);
          split<2>(u[t][2 * half], u[t][2 * half + 1], x);
#pragma unroll
          for (int i = 0; i < 3; ++i) *reinterpret_cast<uint32_t*>(ups + i * kUPlane + at) = w[i];
#pragma unroll
          for (int i = 0; i < 2; ++i) *reinterpret_cast<uint32_t*>(ops + i * kUPlane + at) = x[i];
        }
      }
      bar_compute();
      // S <- e^G_last S + sum over tokens; the sum in accumulators of its own, joined by one rounding
      {
        float d[4][4] = {};
        // B: K as it lies (tokens down, dims across), transposed on the way: dims 32 w.., 16 tokens
        const int kr = (lane & 7) + ((lane >> 3) & 1) * 8, kc = 4 * (warp & 1) + (lane >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a[3][4], k0[4], k1[4];
#pragma unroll
          for (int j = 0; j < 3; ++j) ldm4(up + j * kUPlane + swz(ar, 2 * i + ac), a[j]);
          const uint32_t kb = k32 + (warp >> 1) * kPlane;
          ldm4t(kb + swz(16 * i + kr, kc), k0);
          ldm4t(kb + swz(16 * i + kr, kc + 2), k1);
#pragma unroll
          for (int j = 2; j >= 0; --j) {
            mma(d[0], a[j], k0[0], k0[1]);
            mma(d[1], a[j], k0[2], k0[3]);
            mma(d[2], a[j], k1[0], k1[1]);
            mma(d[3], a[j], k1[2], k1[3]);
          }
        }
        const float all = eg[2 * kC];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[t][e] = fmaf(all, S[t][e], d[t][e]);
      }
      put_state();
      bar_compute();
      // o = scale e^G (q S) + scores u
      float o[2][4] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i > tr / 2) break;
        uint32_t x[2][4], ab[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          ldm4(op + j * kUPlane + swz(ar, 2 * i + ac), x[j]);
          ldm4(a32 + j * kPlane + swz(bt, 2 * i + bc), ab[j]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t == 0 && i > tl / 2) continue;
          mma(o[t], x[1], ab[0][2 * t], ab[0][2 * t + 1]);
          mma(o[t], x[0], ab[1][2 * t], ab[1][2 * t + 1]);
          mma(o[t], x[0], ab[0][2 * t], ab[0][2 * t + 1]);
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int tile = t ? tr : tl, tok = tile * 8 + 2 * q;
        const float e0 = p.scale * eg[tok], e1 = p.scale * eg[tok + 1];
        uint32_t w[2];
#pragma unroll
        for (int half = 0; half < 2; ++half)
          w[half] = transpose8(pack(fmaf(e0, xq[t][2 * half], o[t][2 * half]),
                                    fmaf(e1, xq[t][2 * half + 1], o[t][2 * half + 1])));
        if (tile * 8 + g < len) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                               (static_cast<int64_t>(c0) + c * kC + tile * 8 + g) * p.os +
                               static_cast<int64_t>(h) * p.dv + col0 + 2 * q;
          *reinterpret_cast<uint32_t*>(dst) = w[0];
          *reinterpret_cast<uint32_t*>(dst + 8) = w[1];
        }
      }
      if (len < kC) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
    float* live = p.live + off;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dim = 32 * warp + 8 * t + 2 * q + (e & 1), col = g + 8 * (e >> 1);
        live[static_cast<int64_t>(dim) * p.dv + col] = S[t][e];
      }
  }
  // the cluster's copies and arrivals come to this block's memory until all are done
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

}  // namespace

// Sizes alone: whether the workspace has to hold chunks, and how many bytes.
bool delta_chunk_sizes(int dk, int dv) { return dk == kDk && dv % kCols == 0; }
size_t delta_chunk_workspace(int64_t rows, int B, int H) {
  return sizeof(WsHeader) + static_cast<size_t>(rows / kC + B) * H * kRec;
}

// Below this many tokens a request (on average) a chunk's fixed work outweighs the row scan's.
bool delta_chunk_takes(const DeltaParams& p, spec_dtype dtype) {
  return dtype == SPEC_BF16 && delta_chunk_sizes(p.dk, p.dv) && p.vec_qk && p.vec_o &&
         (reinterpret_cast<uintptr_t>(p.v) & 15u) == 0 && p.vs % 8 == 0 && p.H <= 65535 &&
         p.B <= 65535 && p.rows >= kDeltaChunkRows * static_cast<int64_t>(p.B);
}

spec_status delta_chunk_launch(const DeltaParams& p, void* workspace, EncodeTiledFn encode,
                               cudaStream_t stream) {
  static SmemAllowance prep_allowed, chain_allowed;
  if (allow_dynamic_smem(delta_prep_kernel, kPrepSmem, prep_allowed) != cudaSuccess ||
      allow_dynamic_smem(delta_chain_kernel, kChainSmem, chain_allowed) != cudaSuccess)
    return SPEC_ERR_CUDA;
  uint8_t* rec = static_cast<uint8_t*>(workspace) + sizeof(WsHeader);
  const int64_t slots = p.rows / kC + p.B;
  if (slots > 0x7fffffff) return SPEC_ERR_UNSUPPORTED;
  if (launch_pdl(delta_prep_kernel, dim3(static_cast<unsigned>(slots), p.H), dim3(kPrepThreads),
                 kPrepSmem, stream, p, rec) != cudaSuccess)
    return SPEC_ERR_CUDA;
  ChainMaps m;
  const cuuint32_t es[2] = {1, 1};
  const auto map = [&](CUtensorMap* t, const void* base, int64_t cols, int64_t stride, int box_cols,
                       CUtensorMapSwizzle sw) {
    const cuuint64_t dim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(p.rows)};
    const cuuint64_t step[1] = {static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), kC};
    return encode(t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dim, step, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!map(&m.k, p.k, static_cast<int64_t>(p.Hk) * kDk, p.ks, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !map(&m.q, p.q, static_cast<int64_t>(p.Hk) * kDk, p.qs, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !map(&m.v, p.v, static_cast<int64_t>(p.H) * p.dv, p.vs, kCols, CU_TENSOR_MAP_SWIZZLE_NONE))
    return SPEC_ERR_CUDA;
  const int slices = p.dv / kCols;
  int cs = 8;
  while (slices % cs != 0) cs /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(slices, p.H, p.B);
  cfg.blockDim = dim3(kChainThreads);
  cfg.dynamicSmemBytes = kChainSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cs;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, delta_chain_kernel, m, p, static_cast<const uint8_t*>(rec), cs) ==
                 cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // namespace spec
