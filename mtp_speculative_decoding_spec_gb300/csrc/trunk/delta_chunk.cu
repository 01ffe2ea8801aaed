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
//
// What is not finite stays where the recurrence takes it. The matrices are triangular but a product's
// steps are not: a token's zeros above the diagonal meet up to 15 later tokens, and 0 times NaN is NaN.
// So r and u enter products with what is not finite in them taken out; u has it again for the state, and
// the outputs of a column are NaN from its first token with such a u on. Finding out takes a vote of each
// warp on r and on u: 472 us for 471 (below; with a branch of each thread's own 476 to 485).
//
// 16 heads of [128, 128], one prompt of 15,360 rows: 473 us, of which 75 the first kernel (0.25 GB, 3.3
// TB/s) and 1.65 us a chunk the second; 63,488 rows 1.93 ms. q, k, v and the outputs alone would take 38
// us: what bounds it is the chain's latency, some 3,300 cycles a chunk in which an SM's sub-core has one
// warp of the chain and one of the outputs, its matrix instructions (198 of 8.3 cycles) half the time.
#include <math.h>

#include <cuda_bf16.h>

#include "trunk.cuh"

namespace spec {
namespace {

constexpr int kC = 64;                 // tokens per chunk
constexpr int kDk = 128;
constexpr int kCols = 16;              // columns of S per block
constexpr int kPanel = kC * 128;       // 64 dims of K or Q: rows of 128 bytes, swizzled
constexpr int kTri = 32 * 64 + 32 * 128;  // 64 x 64 up to the diagonal: rows of 32, then of 64 columns
constexpr int kTBytes = 3 * kTri;      // T in three parts
constexpr int kABytes = 2 * kTri;      // scores in two parts
constexpr int kVecBytes = 640;         // e^G [64], e^(G_last - G) [64], e^G_last
constexpr int kRec = kTBytes + kABytes + kVecBytes;  // one chunk and head of the workspace
constexpr int kTile = kC * kDk * 2;    // K or Q of a chunk: two panels of 64 dims

// Where 16-byte piece c (0..7) of row r lies in a run of swizzled 128-byte rows.
__device__ __forceinline__ int swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// The same in a triangular matrix, whose first 32 rows have four pieces each.
__device__ __forceinline__ int tri(int r, int c) {
  return r < 32 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : 32 * 64 + swz(r - 32, c);
}

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
// The counterpart: a product's results, packed in pairs, to rows of shared memory.
__device__ __forceinline__ void stm4(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(r0), "r"(r1),
               "r"(r2), "r"(r3)
               : "memory");
}
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // an 8 x 8 matrix of 16-bit values
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
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

// An Inf or NaN among four pairs of bf16. An exponent of all ones carries into its half's top bit.
__device__ __forceinline__ bool any_odd(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const auto top = [](uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; };
  return ((top(a) | top(b) | top(c) | top(d)) & 0x80008000u) != 0;
}
// The elements of four pairs that are one (element e of pair i: bit 2 i + e), which are cleared in the
// N parts of each.
template <int N>
__device__ __forceinline__ uint32_t take_odd(uint32_t (&w)[4][N]) {
  uint32_t odd = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if ((w[i][0] >> (16 * e) & 0x7f80u) != 0x7f80u) continue;
      odd |= 1u << (2 * i + e);
#pragma unroll
      for (int k = 0; k < N; ++k) w[i][k] &= e ? 0xffffu : 0xffff0000u;
    }
  return odd;
}

__device__ __forceinline__ int cu_at(const DeltaParams& p, int b) {
  return static_cast<int>(max(static_cast<int64_t>(0),
                              min(static_cast<int64_t>(p.cu_rows[b]), p.rows)));
}
// Requests' chunks take slots of their own: request b's first is cu[b] / 64 + b, and as many follow as
// it has chunks.
__device__ __forceinline__ int first_slot(int cu, int b) { return cu / kC + b; }

// ------------------------------------------------------------------------- what needs no state
// One block per (slot, value head), 128 threads. (I + A)^-1 by blocks of 16: the diagonal blocks by
// forward substitution, a column to a thread, then twice
//   [[P, 0], [B, Q]]^-1 = [[P^-1, 0], [-Q^-1 B P^-1, Q^-1]]
// in fp32, the inverse taking the place of A. Of T and the scores only the 16 x 16 blocks up to the
// diagonal are made: the chain reads no others. Shared memory is used twice over (Q then A, K and the
// scores then T), so that four blocks fit on an SM: with so many small phases it is the other blocks
// that fill a phase's latencies.
constexpr int kPrepThreads = 128;
constexpr int kLPitch = 68;  // floats between rows of A
constexpr int kMPitch = 36;  // and of the 32 x 32 product in between
constexpr int kLBytes = kC * kLPitch * 4;
constexpr int kPrepSmem = kTile + kLBytes + kABytes + kVecBytes + 3 * kC * 4;
static_assert(2 * kTri <= kTile && kTri <= kABytes, "T's parts take the places of K and the scores");

// Sums of floats kept as two floats (hi + lo, Knuth's exact sum of two): as exact as 48 bits, in fp32
// operations alone (64-bit floating point runs at a small fraction of their rate here).
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add_two(Two a, Two b) {
  const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
  const float l = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
  const float hi = __fadd_rn(s, l);
  return Two{hi, __fsub_rn(l, __fsub_rn(hi, s))};
}
// e^x for x <= 0. The rounding of x log2(e) costs |x| 2^-24 of the result, which is itself e^-|x|: at
// most 2^-25 of 1 whatever x.
__device__ __forceinline__ float exp_neg(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

// c += A B of 16 x 16 blocks in shared memory, by a warp: lane has rows 2 (l / 4) and + 1, columns
// 4 (l % 4) to + 3. Lower: A is lower triangular, and what lies above its diagonal is not multiplied, so
// that a row of B that is not finite stays out of the rows before it.
template <bool Lower = false>
__device__ __forceinline__ void mul16(float (&c)[2][4], const float* A, int pa, const float* B, int pb,
                                      int lane) {
  const float* a0 = A + 2 * (lane >> 2) * pa;
  const float* b0 = B + 4 * (lane & 3);
#pragma unroll
  for (int k = 0; k < 16; k += 4) {
    const float4 x = *reinterpret_cast<const float4*>(a0 + k);
    const float4 y = *reinterpret_cast<const float4*>(a0 + pa + k);
    const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 b = *reinterpret_cast<const float4*>(b0 + (k + j) * pb);
      if (!Lower || k + j <= 2 * (lane >> 2)) {
        c[0][0] = fmaf(xs[j], b.x, c[0][0]), c[0][1] = fmaf(xs[j], b.y, c[0][1]);
        c[0][2] = fmaf(xs[j], b.z, c[0][2]), c[0][3] = fmaf(xs[j], b.w, c[0][3]);
      }
      if (!Lower || k + j <= 2 * (lane >> 2) + 1) {
        c[1][0] = fmaf(ys[j], b.x, c[1][0]), c[1][1] = fmaf(ys[j], b.y, c[1][1]);
        c[1][2] = fmaf(ys[j], b.z, c[1][2]), c[1][3] = fmaf(ys[j], b.w, c[1][3]);
      }
    }
  }
}
__device__ __forceinline__ void put16(const float (&c)[2][4], float sign, float* D, int pd, int lane) {
#pragma unroll
  for (int r = 0; r < 2; ++r)
    *reinterpret_cast<float4*>(D + (2 * (lane >> 2) + r) * pd + 4 * (lane & 3)) =
        make_float4(sign * c[r][0], sign * c[r][1], sign * c[r][2], sign * c[r][3]);
}

__global__ void __launch_bounds__(kPrepThreads, 4)
    delta_prep_kernel(const __grid_constant__ DeltaParams p, uint8_t* rec) {
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* sk = smem;                              // K; then M, then T's first two parts
  uint8_t* sq = smem + kTile;                      // Q; then A and its inverse
  uint8_t* sa = sq + kLBytes;                      // scores, vectors; then T's third part
  float* vec = reinterpret_cast<float*>(sa + kABytes);
  float* L = reinterpret_cast<float*>(sq);
  float* ghi = reinterpret_cast<float*>(sa + kABytes + kVecBytes);
  float* glo = ghi + kC;
  float* beta = glo + kC;
  float* M = reinterpret_cast<float*>(sk);
  uint8_t* dst;                                    // this chunk's and head's record
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
  dst = rec + (static_cast<int64_t>(slot) * p.H + h) * kRec;
  {
    const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(p.k) + static_cast<int64_t>(kh) * kDk;
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.q) + static_cast<int64_t>(kh) * kDk;
    const int t0 = 2 * lane, t1 = t0 + 1;
    float g0 = 0.f, g1 = 0.f, b0 = 0.f, b1 = 0.f;
    if (warp == 0) {
      const int64_t at = (static_cast<int64_t>(row0) + t0) * p.H + h;
      if (t0 < len) g0 = p.g[at], b0 = p.beta[at];
      if (t1 < len) g1 = p.g[at + p.H], b1 = p.beta[at + p.H];
    }
    uint4 k[8], q[8];  // all loads in flight at once
    const int c = tid & 15, r0 = tid >> 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + 8 * i;
      k[i] = q[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < len) {
        k[i] = __ldg(reinterpret_cast<const uint4*>(kp + (row0 + r) * p.ks) + c);
        q[i] = __ldg(reinterpret_cast<const uint4*>(qp + (row0 + r) * p.qs) + c);
      }
    }
    if (warp == 0) {
      // running sums of the log decays: the difference of two of them is as exact as a float, however
      // far they have run. A decay below e^-200 is 0 in fp32 either way.
      g0 = g0 < -200.f ? -200.f : g0;
      g1 = g1 < -200.f ? -200.f : g1;
      beta[t0] = b0;
      beta[t1] = b1;
      Two s = add_two(Two{g0, 0.f}, Two{g1, 0.f});
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Two x{__shfl_up_sync(0xffffffffu, s.hi, o), __shfl_up_sync(0xffffffffu, s.lo, o)};
        if (lane >= o) s = add_two(s, x);
      }
      const Two last{__shfl_sync(0xffffffffu, s.hi, 31), __shfl_sync(0xffffffffu, s.lo, 31)};
      const Two x{__shfl_up_sync(0xffffffffu, s.hi, 1), __shfl_up_sync(0xffffffffu, s.lo, 1)};
      const Two a = lane == 0 ? Two{g0, 0.f} : add_two(x, Two{g0, 0.f});
      ghi[t0] = a.hi, glo[t0] = a.lo;
      ghi[t1] = s.hi, glo[t1] = s.lo;
      vec[t0] = expf(a.hi);
      vec[t1] = expf(s.hi);
      vec[kC + t0] = t0 < len ? expf((last.hi - a.hi) + (last.lo - a.lo)) : 0.f;
      vec[kC + t1] = t1 < len ? expf((last.hi - s.hi) + (last.lo - s.lo)) : 0.f;
      if (lane == 0) vec[2 * kC] = expf(last.hi);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = (c >> 3) * kPanel + swz(r0 + 8 * i, c & 7);
      *reinterpret_cast<uint4*>(sk + at) = k[i];
      *reinterpret_cast<uint4*>(sq + at) = q[i];
    }
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
      const int pan = (s >> 2) * kPanel, c = (s & 3) * 2;
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
    __syncthreads();  // A takes Q's place
    float hi2[2], lo2[2], bt2[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = warp * 16 + (lane >> 2) + 8 * half;
      hi2[half] = ghi[i], lo2[half] = glo[i], bt2[half] = beta[i];
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t > 2 * warp + 1) break;
      const int j = t * 8 + 2 * (lane & 3);
      const float2 hj = *reinterpret_cast<const float2*>(ghi + j);
      const float2 lj = *reinterpret_cast<const float2*>(glo + j);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = warp * 16 + (lane >> 2) + 8 * half;
        const float d[2] = {exp_neg((hi2[half] - hj.x) + (lo2[half] - lj.x)),
                            exp_neg((hi2[half] - hj.y) + (lo2[half] - lj.y))};
        float l[2], a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[e] = j + e < i ? bt2[half] * d[e] * kk[t][2 * half + e] : 0.f;
          a[e] = j + e <= i ? p.scale * d[e] * qk[t][2 * half + e] : 0.f;
        }
        *reinterpret_cast<float2*>(L + i * kLPitch + j) = make_float2(l[0], l[1]);
        uint32_t w[2];
        split<2>(a[0], a[1], w);
        const int at = tri(i, t) + 4 * (lane & 3);
        *reinterpret_cast<uint32_t*>(sa + at) = w[0];
        *reinterpret_cast<uint32_t*>(sa + kTri + at) = w[1];
      }
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  if (tid == 0) {  // scores and vectors leave while T is worked out
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst + kTBytes),
                 "r"(smem_u32(sa)), "r"(kABytes + kVecBytes)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  if (warp < 2) {  // diagonal blocks: thread 16 b + c has column c of block b
    const int blk = tid >> 4, c = tid & 15;
    float* D = L + blk * 16 * (kLPitch + 1);
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float acc[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < i; ++j) acc[j & 1] = fmaf(D[i * kLPitch + j], t[j], acc[j & 1]);
      t[i] = (i == c ? 1.f : 0.f) - (acc[0] + acc[1]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) D[i * kLPitch + c] = t[i];
  }
  __syncthreads();
  auto block = [&](int i, int j) { return L + i * 16 * kLPitch + j * 16; };
  if (warp < 2) {  // the two blocks next to the diagonal in the 32 x 32 blocks
    const int i = 2 * warp + 1;
    float c[2][4] = {};
    mul16(c, block(i, i - 1), kLPitch, block(i - 1, i - 1), kLPitch, lane);
    __syncwarp();
    put16(c, 1.f, M + warp * 16 * kMPitch, kMPitch, lane);
    __syncwarp();
    float d[2][4] = {};
    mul16<true>(d, block(i, i), kLPitch, M + warp * 16 * kMPitch, kMPitch, lane);
    put16(d, -1.f, block(i, i - 1), kLPitch, lane);
  }
  __syncthreads();
  {  // the lower left 32 x 32: a 16 x 16 block to a warp
    const int bi = warp >> 1, bj = warp & 1;
    float c[2][4] = {};
    for (int k = bj; k < 2; ++k) mul16(c, block(2 + bi, k), kLPitch, block(k, bj), kLPitch, lane);
    put16(c, 1.f, M + bi * 16 * kMPitch + bj * 16, kMPitch, lane);
    __syncthreads();
    float d[2][4] = {};
    if (bi > 0) mul16(d, block(3, 2), kLPitch, M + bj * 16, kMPitch, lane);
    mul16<true>(d, block(2 + bi, 2 + bi), kLPitch, M + bi * 16 * kMPitch + bj * 16, kMPitch, lane);
    put16(d, -1.f, block(2 + bi, bj), kLPitch, lane);
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the scores are out
  __syncthreads();
  // T = (I + A)^-1 diag(beta) in three parts, a pair of columns of each block to a thread
#pragma unroll
  for (int bi = 0; bi < 4; ++bi)
#pragma unroll
    for (int bj = 0; bj <= bi; ++bj) {
      const int r = 16 * bi + (tid >> 3), j = 16 * bj + 2 * (tid & 7);
      const float2 x = *reinterpret_cast<const float2*>(L + r * kLPitch + j);
      const float2 bt = *reinterpret_cast<const float2*>(beta + j);
      uint32_t w[3];
      split<3>(j <= r ? x.x * bt.x : 0.f, j < r ? x.y * bt.y : 0.f, w);
      const int at = tri(r, j >> 3) + 2 * (j & 7);
      *reinterpret_cast<uint32_t*>(sk + at) = w[0];
      *reinterpret_cast<uint32_t*>(sk + kTri + at) = w[1];
      *reinterpret_cast<uint32_t*>(sa + at) = w[2];
    }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  if (tid == 0) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                 "r"(smem_u32(sk)), "r"(2 * kTri)
                 : "memory");
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst + 2 * kTri),
                 "r"(smem_u32(sa)), "r"(kTri)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
  }
}

// ------------------------------------------------------------------------- the chain of chunks
// Grid (rec_dv / 16, H, B). Warps 0-3 carry the chain (k S, u, S), warps 4-7 make the outputs beside it
// (q S, scores times u), warps 8 and 9 load for them. A head's blocks read the same K, Q, T and scores at
// about the same time, from L2 all but once (clusters of 2 and 4 with multicast copies took the same
// time, of 8 885 us against 488: too few of those fit at once).
//   chain   k S -> r -> | u | S' -> |      | three barriers of the four warps a chunk
//   output  q S    ...    scores u, store
// A warp of the chain has two tiles of eight tokens (w and 7 - w: the same work under causality) and a
// quarter of S's rows. What a phase multiplies by (K, T) is read into registers before the barrier
// that its other operand waits for. Warp 10 waits for the chain's stages in its place: even over, a
// wait for a copy costs a warp 100 to 250 cycles, a named barrier 25 (488 -> 472 us). (S kept in registers
// as the next chunk's operand, its four partial products meeting in shared memory instead, moves fewer
// bytes but took 2.16 us a chunk.)
constexpr int kChainThreads = 12 * 32;  // three groups of four warps; the last one does nothing
// Registers a thread: launched with 168 (64,512 in all), then shared out again by group, 63,488 in use.
constexpr int kChainRegs = 224, kOutRegs = 168, kLoadRegs = 104;
constexpr int kCStages = 3, kOStages = 3;
constexpr int kSortMost = 256;  // requests that are put in order (their lengths lie in the place of S)
constexpr int kVTile = kC * kCols * 2;
// Beside K (Q), whose tiles start on 1,024 bytes: T, vectors, V for the chain, scores and vectors for
// the outputs.
constexpr int kCRest = kTBytes + kVecBytes + kVTile;
constexpr int kORest = kABytes + kVecBytes;
constexpr int kSPlane = kCols * 256;               // S^T: two panels of 16 rows of 128 bytes
constexpr int kUPlane = kCols * 128;               // 16 x 64
constexpr int kWork = 3 * kSPlane + 8 * kUPlane;   // S, r, u scaled for the state (3 each), u (2)
constexpr int kChainSmem =
    kCStages * (kTile + kCRest) + kOStages * (kTile + kORest) + kWork + 128 + 64 + 1024;
static_assert(kCRest % 128 == 0 && kORest % 128 == 0, "swizzled tiles start on 128 bytes");
static_assert(kChainSmem <= 227 * 1024, "shared memory of an SM");

struct ChainMaps {
  CUtensorMap k, q, v;  // [rows][columns], boxes of 64 x 64 (swizzled) and 16 x 64
};

__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Barriers between the groups of warps. Both go through the same chunks whatever happens, so each
// side's turn always comes.
enum : int { kBarChain = 1, kBarState = 2, kBarQs = 3, kBarU = 4, kBarUsed = 5, kBarStage = 6 };
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__global__ void __launch_bounds__(kChainThreads, 1)
    delta_chain_kernel(const __grid_constant__ ChainMaps maps, const __grid_constant__ DeltaParams p,
                       const uint8_t* rec) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sq = smem + kCStages * kTile;        // after the tiles of K
  uint8_t* crest = sq + kOStages * kTile;
  uint8_t* orest = crest + kCStages * kCRest;
  uint8_t* sps = orest + kOStages * kORest;     // parts of S
  uint8_t* rps = sps + 3 * kSPlane;             // of r
  uint8_t* ups = rps + 3 * kUPlane;             // of e^(G_last - G) u
  uint8_t* ops = ups + 3 * kUPlane;             // of u
  uint64_t* cfull = reinterpret_cast<uint64_t*>(sps + kWork);
  uint64_t* cempty = cfull + kCStages;
  uint64_t* ofull = cempty + kCStages;
  uint64_t* oempty = ofull + kOStages;
  int* odd_from = reinterpret_cast<int*>(sps + kWork + 128);  // [16] a column's first token with an odd u
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, kh = h / (p.H / p.Hk);
  const int col0 = blockIdx.x * kCols;
  if (tid == 0) {
    for (int s = 0; s < kCStages; ++s) {
      mbar_init(&cfull[s], 1);
      mbar_init(&cempty[s], 4);
    }
    for (int s = 0; s < kOStages; ++s) {
      mbar_init(&ofull[s], 1);
      mbar_init(&oempty[s], 4);
    }
    fence_mbar_init();
  }
  if (tid < kCols) odd_from[tid] = kC;
  __syncthreads();
  pdl_wait();
  // The longest request first: blocks are dealt out in order, and what starts last should be short (prompts
  // of 0, 1, 77, 1,000 and 2,311 rows: 124 us, 134 in the order given).
  int b = blockIdx.z;
  if (p.B > 1 && p.B <= kSortMost) {
    int* lens = reinterpret_cast<int*>(sps);
    int* pick = lens + kSortMost;
    for (int i = tid; i < p.B; i += kChainThreads) lens[i] = cu_at(p, i + 1) - cu_at(p, i);
    __syncthreads();
    for (int i = tid; i < p.B; i += kChainThreads) {
      int before = 0;
      for (int j = 0; j < p.B; ++j) before += lens[j] > lens[i] || (lens[j] == lens[i] && j < i);
      if (before == static_cast<int>(blockIdx.z)) *pick = i;
    }
    __syncthreads();
    b = __shfl_sync(0xffffffffu, *pick, 0);
    __syncthreads();  // the place is used otherwise from here on
  }
  const int c0 = cu_at(p, b), c1 = max(c0, cu_at(p, b + 1));
  const int n = (c1 - c0 + kC - 1) / kC;
  const int64_t elems = static_cast<int64_t>(p.layers) * p.H * p.dk * p.dv;
  const int64_t off = b * elems + (static_cast<int64_t>(p.layer) * p.H + h) * p.dk * p.dv + col0;
  // fragment coordinates: lane (g, q); an A operand's row and 16-byte piece; B tiles of tokens tl (lanes
  // 0-15) and tr
  const int g = lane >> 2, q = lane & 3, w4 = warp & 3, tl = w4, tr = 7 - w4;
  const int ar = lane & 15, ac = lane >> 4;
  const int bt = (lane & 16 ? tr : tl) * 8 + (lane & 7), bc = (lane >> 3) & 1;
  const uint32_t sp = smem_u32(sps), rp = smem_u32(rps), up = smem_u32(ups), op = smem_u32(ops);
  // and of a triangular matrix's step i (tile tl has steps 0 and 1 only: anything in its place past them)
  auto tri_at = [&](int i) { return tri(bt, bt < 32 ? (2 * i + bc) & 3 : 2 * i + bc); };
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {  // gives up waiting for good, not the walk
    if (ok && !mbar_wait_bounded(bar, parity)) {
      atomicOr(&p.hdr->error, ERR_TC_WAIT);
      ok = false;
    }
    ok = __all_sync(0xffffffffu, ok);
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    // ------------------------------------------------------------------ loads, for the chain and the outputs
    const bool chain = warp == 8;
    const int stages = chain ? kCStages : kOStages;
    uint64_t* full = chain ? cfull : ofull;
    uint64_t* empty = chain ? cempty : oempty;
    const uint8_t* base = rec + (static_cast<int64_t>(first_slot(c0, b)) * p.H + h) * kRec;
    if (warp == 10)
      for (int c = 0; c < n; ++c) {
        wait(&cfull[c % kCStages], (c / kCStages) & 1);
        bar_sync(kBarStage, 160);
      }
    int c = 0;
    for (; c < n && warp < 10; ++c) {
      const int s = c % stages;
      if (c >= stages) wait(&empty[s], ((c / stages) & 1) ^ 1);
      if (!ok) break;
      if (lane == 0) {
        const int row = c0 + c * kC;
        const uint8_t* r = base + static_cast<int64_t>(c) * p.H * kRec;
        const uint32_t bar = smem_u32(&full[s]);
        uint8_t* st = (chain ? smem : sq) + s * kTile;
        uint8_t* rest = chain ? crest + s * kCRest : orest + s * kORest;
        mbar_arrive_expect_tx(&full[s], kTile + (chain ? kCRest : kORest));
        for (int i = 0; i < 2; ++i)
          tma_box(st + i * kPanel, chain ? &maps.k : &maps.q, kh * kDk + i * 64, row, bar);
        if (chain) {
          bulk_copy(rest, r, kTBytes, bar);
          bulk_copy(rest + kTBytes, r + kTBytes + kABytes, kVecBytes, bar);
          tma_box(rest + kTBytes + kVecBytes, &maps.v, h * p.dv + col0, row, bar);
        } else {
          bulk_copy(rest, r + kTBytes, kABytes + kVecBytes, bar);
        }
      }
    }
    ok = true;
    for (int j = max(0, c - stages); j < c; ++j) {  // nothing is left in flight
      wait(&full[j % stages], (j / stages) & 1);
    }
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOutRegs));
    // ------------------------------------------------------------------ outputs
    for (int c = 0; c < n; ++c) {
      const int s = c % kOStages;
      wait(&ofull[s], (c / kOStages) & 1);
      const uint8_t* rest = orest + s * kORest;
      const uint32_t q32 = smem_u32(sq + s * kTile), a32 = smem_u32(rest);
      const float* eg = reinterpret_cast<const float*>(rest + kABytes);
      const int len = min(kC, c1 - c0 - c * kC);
      uint32_t qb[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) ldm4(q32 + (i >> 2) * kPanel + swz(bt, (i & 3) * 2 + bc), qb[i]);
      bar_sync(kBarState, 256);
      float x[2][2][4] = {};  // [part][tile]
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t a[2][4];
        const uint32_t sa = sp + (i >> 2) * (kSPlane / 2) + swz(ar, (i & 3) * 2 + ac);
        ldm4(sa, a[0]);
        ldm4(sa + kSPlane, a[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int t = 0; t < 2; ++t) mma(x[j][t], a[j], qb[i][2 * t], qb[i][2 * t + 1]);
      }
      bar_arrive(kBarQs, 256);
      uint32_t ab[4][2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i <= tr / 2) {
          ldm4(a32 + tri_at(i), ab[i][0]);
          ldm4(a32 + kTri + tri_at(i), ab[i][1]);
        }
      bar_sync(kBarU, 256);
      float o[3][2][4] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i > tr / 2) break;
        uint32_t u[2][4];
        ldm4(op + swz(ar, 2 * i + ac), u[0]);
        ldm4(op + kUPlane + swz(ar, 2 * i + ac), u[1]);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t == 0 && i > tl / 2) continue;
          mma(o[0][t], u[0], ab[i][0][2 * t], ab[i][0][2 * t + 1]);
          mma(o[1][t], u[1], ab[i][0][2 * t], ab[i][0][2 * t + 1]);
          mma(o[2][t], u[0], ab[i][1][2 * t], ab[i][1][2 * t + 1]);
        }
      }
      // The chain lowers these before kBarU alone, and once a column has an odd u all its later ones are.
      const int from[2] = {odd_from[g], odd_from[g + 8]};
      const bool odd = __any_sync(0xffffffffu, min(from[0], from[1]) < kC);
      bar_arrive(kBarUsed, 256);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int tile = t ? tr : tl, tok = tile * 8 + 2 * q;
        const float e[2] = {p.scale * eg[tok], p.scale * eg[tok + 1]};
        float y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          y[k] = fmaf(e[k & 1], x[0][t][k] + x[1][t][k], o[0][t][k] + (o[1][t][k] + o[2][t][k]));
        if (odd) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (tok + (k & 1) >= from[k >> 1]) y[k] = NAN;
          __syncwarp();
        }
        const uint32_t w0 = transpose8(pack(y[0], y[1])), w1 = transpose8(pack(y[2], y[3]));
        if (tile * 8 + g < len) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                               (static_cast<int64_t>(c0) + c * kC + tile * 8 + g) * p.os +
                               static_cast<int64_t>(h) * p.dv + col0 + 2 * q;
          *reinterpret_cast<uint32_t*>(dst) = w0;
          *reinterpret_cast<uint32_t*>(dst + 8) = w1;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&oempty[s]);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChainRegs));
    // ------------------------------------------------------------------ chain
    // S^T: this warp's rows of S are dims 32 w..32 w + 31; lane (g, q) has columns col0 + g and + 8 of dims
    // 32 w + 8 t + 2 q and + 1
    float S[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dim = 32 * warp + 8 * t + 2 * q + (e & 1), col = g + 8 * (e >> 1);
        S[t][e] = p.init ? p.init[off + static_cast<int64_t>(dim) * p.dv + col] : 0.f;
      }
    // where a lane's row of four stored matrices lies: columns g and g + 8 (lane / 8, odd), and of two
    // pieces of 8 dims or tiles of tokens
    const int mr = (lane & 7) + (lane & 8), mh = lane >> 4;
    const uint32_t s_at = sp + (warp >> 1) * (kSPlane / 2) + swz(mr, 4 * (warp & 1) + mh);
    const uint32_t u_at = swz(mr, mh ? tr : tl);
    auto put_state = [&]() {
#pragma unroll
      for (int t = 0; t < 4; t += 2) {  // dims 32 w + 8 t: panel w / 2, 16-byte piece 4 (w & 1) + t
        uint32_t w[4][3];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          split<3>(S[t + (i >> 1)][2 * (i & 1)], S[t + (i >> 1)][2 * (i & 1) + 1], w[i]);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          stm4((s_at ^ (t << 4)) + k * kSPlane, w[0][k], w[1][k], w[2][k], w[3][k]);
      }
    };
    // What a chunk's first phase takes from its stage: K is read between the last products of the chunk
    // before, as the registers of its other form come free
    uint32_t kb[8][4];
    float v[2][4], ge[2][2];
    int len = 0;
    auto open_stage = [&](int c) {
      len = min(kC, c1 - c0 - c * kC);
      if (len < kC) {
        uint8_t* st = smem + (c % kCStages) * kTile;
        // rows past the request's end are another's: what they hold must not reach S even times 0
        for (int i = tid; i < (kC - len) * 16; i += 128) {
          const int r = len + (i >> 4), pc = i & 15;
          *reinterpret_cast<uint4*>(st + (pc >> 3) * kPanel + swz(r, pc & 7)) = make_uint4(0u, 0u, 0u, 0u);
        }
        bar_sync(kBarChain, 128);
      }
    };
    auto load_k = [&](int c, int i) {
      ldm4(smem_u32(smem + (c % kCStages) * kTile) + (i >> 2) * kPanel + swz(bt, (i & 3) * 2 + bc), kb[i]);
    };
    auto load_rest = [&](int c) {
      const uint8_t* rest = crest + (c % kCStages) * kCRest;
      const float* eg = reinterpret_cast<const float*>(rest + kTBytes);
      const uint8_t* sv = rest + kTBytes + kVecBytes;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int tile = t ? tr : tl, tok = tile * 8 + 2 * q;
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // columns g, g + 8
          const uint32_t x = transpose8(
              *reinterpret_cast<const uint32_t*>(sv + (tile * 8 + g) * (kCols * 2) + 16 * half + 4 * q));
          v[t][2 * half] = lo_of(x);
          v[t][2 * half + 1] = hi_of(x);
        }
        ge[t][0] = -eg[tok], ge[t][1] = -eg[tok + 1];
      }
    };
    if (n > 0) {
      bar_sync(kBarStage, 160);
      open_stage(0);
#pragma unroll
      for (int i = 0; i < 8; ++i) load_k(0, i);
      load_rest(0);
      put_state();
    }
    for (int c = 0; c < n; ++c) {
      const int s = c % kCStages;
      const uint8_t* rest = crest + s * kCRest;
      const uint32_t k32 = smem_u32(smem + s * kTile), t32 = smem_u32(rest);
      const float* eg = reinterpret_cast<const float*>(rest + kTBytes);
      bar_sync(kBarChain, 128);  // the parts of S are there
      // k S of the warp's tokens, the parts of S in sums of their own
      float x[3][2][4] = {};
      {
        uint32_t a[2][3][4];
        auto load = [&](int i) {
          const uint32_t sa = sp + (i >> 2) * (kSPlane / 2) + swz(ar, (i & 3) * 2 + ac);
#pragma unroll
          for (int j = 0; j < 3; ++j) ldm4(sa + j * kSPlane, a[i & 1][j]);
        };
        load(0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i + 1 < 8) load(i + 1);
#pragma unroll
          for (int j = 0; j < 3; ++j)
#pragma unroll
            for (int t = 0; t < 2; ++t) mma(x[j][t], a[i & 1][j], kb[i][2 * t], kb[i][2 * t + 1]);
        }
      }
      bar_arrive(kBarState, 256);  // the outputs' turn at S, when the chain is past its own
      uint32_t tb[4][3][4];  // the first three here, the last one beside the products of the others
      auto load_t = [&](int i) {
#pragma unroll
        for (int j = 0; j < 3; ++j) ldm4(t32 + j * kTri + tri_at(i), tb[i][j]);
      };
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i <= tr / 2) load_t(i);
      // r = v - e^G (k S)
      float u[3][2][4] = {};
      {
        uint32_t w[4][3];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = i >> 1, tok = (t ? tr : tl) * 8 + 2 * q;
          float r[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = 2 * (i & 1) + e;
            r[e] = tok + e < len ? fmaf(ge[t][e], x[0][t][k] + (x[1][t][k] + x[2][t][k]), v[t][k]) : 0.f;
          }
          split<3>(r[0], r[1], w[i]);
        }
        // the sum that u begins with: 0, or NaN where r is odd, which is then taken out of the products
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[2][i >> 1][2 * (i & 1)] = 0.f * lo_of(w[i][0]);
          u[2][i >> 1][2 * (i & 1) + 1] = 0.f * hi_of(w[i][0]);
        }
        if (__any_sync(0xffffffffu, any_odd(w[0][0], w[1][0], w[2][0], w[3][0]))) {
          take_odd<3>(w);
          __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) stm4(rp + u_at + k * kUPlane, w[0][k], w[1][k], w[2][k], w[3][k]);
      }
      bar_sync(kBarChain, 128);
      // u = T r, the terms by size in sums of their own
      uint32_t ra[2][3][4];
      auto load_r = [&](int i) {
#pragma unroll
        for (int j = 0; j < 3; ++j) ldm4(rp + j * kUPlane + swz(ar, 2 * i + ac), ra[i & 1][j]);
      };
      load_r(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i > tr / 2) break;  // tokens after the tile's
        if (i + 1 < 4 && i + 1 <= tr / 2) load_r(i + 1);
        if (i == 1 && tr / 2 == 3) load_t(3);
        const uint32_t(&r)[3][4] = ra[i & 1];
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // T_k r_0, then what is 2^-8 and 2^-16 of it
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == 0 && i > tl / 2) continue;
            const uint32_t(&b0)[4] = tb[i][0], (&b1)[4] = tb[i][1], (&b2)[4] = tb[i][2];
            if (k == 0) {
              mma(u[0][t], r[0], b0[2 * t], b0[2 * t + 1]);
              mma(u[1][t], r[1], b0[2 * t], b0[2 * t + 1]);
              mma(u[2][t], r[2], b0[2 * t], b0[2 * t + 1]);
            } else {
              mma(u[1][t], r[0], b1[2 * t], b1[2 * t + 1]);
              mma(u[2][t], r[1], b1[2 * t], b1[2 * t + 1]);
              mma(u[2][t], r[0], b2[2 * t], b2[2 * t + 1]);
            }
          }
        }
      }
      // for S': K as it lies (tokens down, dims across), transposed on the way: this warp's dims
      uint32_t kt[4][8];
      {
        const int kr = (lane & 7) + ((lane >> 3) & 1) * 8, kc = 4 * (warp & 1) + (lane >> 4);
        const uint32_t k0 = k32 + (warp >> 1) * kPanel;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ldm4t(k0 + swz(16 * i + kr, kc), kt[i]);
          ldm4t(k0 + swz(16 * i + kr, kc + 2), kt[i] + 4);
        }
      }
      const float all = eg[2 * kC];
      float le[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int tok = (t ? tr : tl) * 8 + 2 * q;
        le[t][0] = eg[kC + tok], le[t][1] = eg[kC + tok + 1];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&cempty[s]);  // everything of the stage is in registers
      if (c > 0) bar_sync(kBarUsed, 256);
      {
        uint32_t w[4][3], z[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = i >> 1, k = 2 * (i & 1);
          const float y0 = u[0][t][k] + (u[1][t][k] + u[2][t][k]);
          const float y1 = u[0][t][k + 1] + (u[1][t][k + 1] + u[2][t][k + 1]);
          split<3>(le[t][0] * y0, le[t][1] * y1, w[i]);
          split<2>(y0, y1, z[i]);
        }
        if (__any_sync(0xffffffffu, any_odd(z[0][0], z[1][0], z[2][0], z[3][0]))) {
          const uint32_t m = take_odd<2>(z);
#pragma unroll
          for (int i = 0; i < 8; ++i)  // bit 2 (2 tile + half) + token
            if (m >> i & 1) {
              w[i >> 1][0] |= i & 1 ? 0x7fc00000u : 0x7fc0u;  // and so is the state from here on
              atomicMin(&odd_from[g + 8 * (i >> 1 & 1)], (i >> 2 ? tr : tl) * 8 + 2 * q + (i & 1));
            }
          __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) stm4(up + u_at + k * kUPlane, w[0][k], w[1][k], w[2][k], w[3][k]);
#pragma unroll
        for (int k = 0; k < 2; ++k) stm4(op + u_at + k * kUPlane, z[0][k], z[1][k], z[2][k], z[3][k]);
      }
      bar_arrive(kBarU, 256);
      if (c + 1 < n) {
        bar_sync(kBarStage, 160);
        open_stage(c + 1);
      } else {
        bar_sync(kBarChain, 128);
      }
      // S <- e^G_last S + sum over tokens; the sum in accumulators of its own, joined by one rounding
      float d[4][4] = {};
      {
        uint32_t a[2][3][4];
        auto load_u = [&](int i) {
#pragma unroll
          for (int j = 0; j < 3; ++j) ldm4(up + j * kUPlane + swz(ar, 2 * i + ac), a[i & 1][j]);
        };
        load_u(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i + 1 < 4) load_u(i + 1);
#pragma unroll
          for (int j = 2; j >= 0; --j)
#pragma unroll
            for (int t = 0; t < 4; ++t) mma(d[t], a[i & 1][j], kt[i][2 * t], kt[i][2 * t + 1]);
          if (c + 1 < n) {
            load_k(c + 1, 2 * i);
            load_k(c + 1, 2 * i + 1);
          }
        }
      }
      if (c + 1 < n) load_rest(c + 1);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[t][e] = fmaf(all, S[t][e], d[t][e]);
      bar_sync(kBarQs, 256);  // q S has been taken of the state before
      if (c + 1 < n) put_state();
    }
    float* live = p.live + off;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dim = 32 * warp + 8 * t + 2 * q + (e & 1), col = g + 8 * (e >> 1);
        live[static_cast<int64_t>(dim) * p.dv + col] = S[t][e];
      }
    if (n > 0) bar_sync(kBarUsed, 256);  // the outputs' last turn
  }
}

}  // namespace

// Sizes alone: whether the workspace has to hold chunks, and how many bytes.
bool delta_chunk_sizes(int dk, int dv) { return dk == kDk && dv % kCols == 0; }
size_t delta_chunk_workspace(int64_t rows, int B, int H) {
  return sizeof(WsHeader) + static_cast<size_t>(rows / kC + B) * H * kRec;
}

// With fewer tokens a request (on average) the row scan takes the call: a chunk costs the same however
// few of its rows there are, and a block an SM at a time. 16 heads of [128, 128], scan and chunks: one
// request of 16 rows 8.7 and 12.2 us, of 32 15.3 and 12.2, of 64 28.4 and 12.5; eight of 32 26.0 and
// 44.6, of 64 48.8 and 45.6; 32 of 16 44.5 and 156, of 32 80.0 and 157, of 64 151 and 160. One request of
// 15,360 7,549 and 488: with the limit any lower or higher, the worse of its two sides costs more, since
// the host does not know whether the rows are spread evenly. Where they are not it can be far off: one
// prompt of 1,000 rows takes 39 us alone, 156 among 30 single tokens (a block an SM for each of them) and
// 509 among 32, which is the scan's side.
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
  return launch_pdl(delta_chain_kernel, dim3(p.dv / kCols, p.H, p.B), dim3(kChainThreads), kChainSmem, stream,
                    m, p, static_cast<const uint8_t*>(rec)) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // namespace spec
