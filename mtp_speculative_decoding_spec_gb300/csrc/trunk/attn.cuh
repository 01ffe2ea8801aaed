// Attention over caches on the CUDA cores (fp32, and bf16 head sizes that the tensor-core kernel does not
// take) and the kernel that joins partial results, for a call's parameters P: verify rows over a shared
// prefix and each request's own cache (AttnParams), new rows over a paged cache (PagedParams).
//
//   o = sum_p exp(s_p) v_p / sum_p exp(s_p),  s_p = scale q.k_p
//
// A partial over a range of positions is (m, l, O) with m the range's largest score, l = sum
// exp(s - m) and O = sum exp(s - m) v; partials of ranges join as m = max m_i, l = sum e^(m_i-m) l_i,
// O = sum e^(m_i-m) O_i. Scores are kept in the log2 domain (scale log2(e) folded in once).
#pragma once

#include <math.h>

#include <cuda_bf16.h>

#include "trunk.cuh"

namespace spec {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Four elements of shared memory (aligned to their size), as floats.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u),
                     __uint_as_float(a.y << 16), __uint_as_float(a.y & 0xffff0000u));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

constexpr int kSimtTm = 16;       // rows per tile
constexpr int kSimtBn = 32;       // positions per block: a lane's
constexpr int kSimtThreads = 256;
constexpr int kMaxD = 256;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kPad = 16;          // bytes after a row of Q, K, V: rows start 16 bytes apart in the banks
constexpr int kPsPitch = kSimtTm + 4;  // floats between positions' weights

// 256 threads over a tile of 16 rows and blocks of 32 positions, the next block's K and V on their way to
// the other of two buffers (as many buffers as fit were slower, 249 us for 222). Scores: a warp takes four
// rows and half of the dims, a lane a position, so that a piece of K read serves four rows. The halves meet in shared memory, and four warps do the softmax of
// four rows each. Values: a thread takes four consecutive dims of one, two or four rows. A block in which
// some row's positions end takes only the positions a row sees, one by one, so what a masked position
// holds reaches no row. fp32, 4 rows of 16 heads on 4 KV heads of 256 dims over 50,000 positions: 190 us = 2.2
// TB/s, 17 TFLOP/s; bound by shared memory (a piece of K serves four rows, one of V four) and the three
// barriers a block. Two rows of 64 dims over 258 positions 8.0 us with the join: two launches' latency.
// Over pages 10 to 16 TFLOP/s with full tiles (a table's entry for each piece): 2,048 rows over 61,440 of 16 heads on
// 4 of 256 fp32 dims 157 ms, of 96 bf16 dims 81, two and a half and two times what products in torch take (58, 40);
// 32 requests of 1 to 8 fp32 rows over 2,000 400 us, two rows over 63,488 337.
template <typename P, typename T>
__global__ void __launch_bounds__(kSimtThreads, 1) attn_simt_kernel(const __grid_constant__ P p) {
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_wait();
  if constexpr (kPaged<P>) pdl_trigger();  // the join's blocks come as these leave, and wait
  const int D = p.D, ld = D + kPad / 4, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pitch = D * static_cast<int>(sizeof(T)) + kPad, tile_bytes = kSimtBn * pitch;
  uint8_t* kv = smem;                                    // [2][K, V][32][pitch]
  float* qs = reinterpret_cast<float*>(smem + 4 * tile_bytes);  // [16][ld]
  float* ps = qs + kSimtTm * ld;                         // [32][20]
  float* part = ps + kSimtBn * kPsPitch;                 // [16][32] scores over the upper dims
  float* row_m = part + kSimtTm * kSimtBn;               // running max, the old scale's factor, sum
  float* row_c = row_m + kSimtTm;
  float* row_l = row_c + kSimtTm;
  int* row_lim = reinterpret_cast<int*>(row_l + kSimtTm);
  int* row_h = row_lim + kSimtTm;                        // its query head
  int64_t* row_q = reinterpret_cast<int64_t*>(row_h + kSimtTm);  // the row of the queries
  int32_t* cum = reinterpret_cast<int32_t*>(row_q + kSimtTm);
  const auto* req = attn_plan(p, cum);
  const AttnShares shares = attn_shares(p, cum);
  if (!kPaged<P> && blockIdx.x == 0) attn_write_units(p, cum, shares);
  AttnWalk walk;
  walk.start(p, cum, shares);
  AttnPiece a;
  // scores: this warp's rows and dims
  const int sr = (warp & 3) * 4, sd = (warp >> 2) * (D / 2);
  // values: this thread's four dims of `rpt` (1, 2 or 4) rows from r0; the fewer the dims, the fewer the rows
  const int nd = D / 4, ng = min(kSimtTm, kSimtThreads / nd);
  const int rpt = ng >= 16 ? 1 : ng >= 8 ? 2 : 4;
  const int d0 = (tid % nd) * 4, r0 = tid / nd * rpt;
  const bool holds = r0 < kSimtTm;
  if constexpr (kPaged<P>)
    if (tid == 0) paged_splits_clear(p);
  while (walk.next(p, cum, shares, a)) {
    if constexpr (kPaged<P>)
      if (tid == 0) paged_split(p, cum, shares, walk, a);
    const int head = a.head, slot = a.slot;
    __syncthreads();  // the previous piece's shared memory is no longer read
    if (tid < kSimtTm) {
      const AttnRow ar = attn_row(p, req, a.tile, tid);
      row_lim[tid] = ar.lim;
      row_q[tid] = attn_q_row(p, req, ar);
      row_h[tid] = head * p.G + ar.g;
      row_m[tid] = -INFINITY;
      row_l[tid] = 0.f;
    }
    const bool pre = a.tile < p.npt;
    const int b = pre ? 0 : attn_tile_req(p, a.tile);
    const int64_t step = pre ? p.pstride : p.krow;
    const int64_t hoff = static_cast<int64_t>(head) * D * sizeof(T);
    const uint8_t* kbase = (pre ? p.pk : p.kk + static_cast<int64_t>(b) * p.kreq) + hoff;
    const uint8_t* vbase = (pre ? p.pv : p.kv + static_cast<int64_t>(b) * p.kreq) + hoff;
    __syncthreads();
    int most = 0, least = 0x7fffffff;  // positions any row sees; positions every running row sees
    for (int r = 0; r < kSimtTm; ++r) {
      most = max(most, row_lim[r]);
      if (row_lim[r] > 0) least = min(least, row_lim[r]);
    }
    const int chunks = D * static_cast<int>(sizeof(T)) / 16;
    auto fetch = [&](int blk, int buf) {  // positions that some row sees; the others' places hold anything
      uint8_t* k = kv + 2 * buf * tile_bytes;
      const int p0 = blk * kSimtBn, np = min(kSimtBn, most - p0);
      for (int i = tid; i < np * chunks; i += kSimtThreads) {
        const int r = i / chunks, c = (i - r * chunks) * 16;
        if constexpr (kPaged<P>) {
          const int64_t at = paged_offset(p, b, p0 + r);
          if (at >= 0) {
            copy_async16(k + r * pitch + c, p.c.k + at + hoff + c);
            copy_async16(k + tile_bytes + r * pitch + c, p.c.v + at + hoff + c);
          } else {  // a page that is not there: its scores are masked, its values 0
            *reinterpret_cast<uint4*>(k + r * pitch + c) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(k + tile_bytes + r * pitch + c) = make_uint4(0u, 0u, 0u, 0u);
          }
        } else {
          copy_async16(k + r * pitch + c, kbase + (p0 + r) * step + c);
          copy_async16(k + tile_bytes + r * pitch + c, vbase + (p0 + r) * step + c);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(a.blk0, 0);
    {  // 16 threads a row
      const int r = tid >> 4;
      const T* src = static_cast<const T*>(p.q) + row_q[r] * p.qs + static_cast<int64_t>(row_h[r]) * D;
      const bool runs = row_lim[r] > 0;
      for (int d = tid & 15; d < D; d += 16) qs[r * ld + d] = runs ? to_f(src[d]) : 0.f;
    }
    float acc[4][4] = {};
    for (int blk = a.blk0; blk < a.blk1; ++blk) {
      const int p0 = blk * kSimtBn, buf = (blk - a.blk0) & 1;
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();  // this block is here, and the other buffer no longer read
      if (blk + 1 < a.blk1) fetch(blk + 1, buf ^ 1);
      const T* ks = reinterpret_cast<const T*>(kv + 2 * buf * tile_bytes + lane * pitch) + sd;
      const T* vs = reinterpret_cast<const T*>(kv + (2 * buf + 1) * tile_bytes);
      float4 w[4] = {};  // four sums a score, every fourth dim in one
#pragma unroll 2
      for (int d = 0; d < D / 2; d += 4) {
        const float4 y = load4(ks + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = load4(qs + (sr + i) * ld + sd + d);
          w[i].x = fmaf(x.x, y.x, w[i].x), w[i].y = fmaf(x.y, y.y, w[i].y);
          w[i].z = fmaf(x.z, y.z, w[i].z), w[i].w = fmaf(x.w, y.w, w[i].w);
        }
      }
      float z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = (w[i].x + w[i].y) + (w[i].z + w[i].w);
      if (warp >= 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) part[(sr + i) * kSimtBn + lane] = z[i];
      }
      __syncthreads();
      if (warp < 4) {
        bool there = p0 + lane < most;
        if constexpr (kPaged<P>) there = there && paged_offset(p, b, p0 + lane) >= 0;
        float e[4], m[4], l[4], old[4];  // four rows side by side
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = sr + i;
          old[i] = row_m[r];
          e[i] = there && p0 + lane < row_lim[r] ? (z[i] + part[r * kSimtBn + lane]) * p.scale_log2 : -INFINITY;
          m[i] = max_nan(e[i], old[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int i = 0; i < 4; ++i) m[i] = max_nan(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float ref = m[i] == -INFINITY ? 0.f : m[i];  // nothing seen yet: every weight is 0
          e[i] = there && p0 + lane < row_lim[sr + i] ? exp2f(e[i] - ref) : 0.f;
          l[i] = e[i];
          old[i] = exp2f(old[i] - ref);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int i = 0; i < 4; ++i) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
        if (lane == 0) {  // every lane is past its reading
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            row_c[sr + i] = old[i];
            row_l[sr + i] = row_l[sr + i] * old[i] + l[i];
            row_m[sr + i] = m[i];
          }
        }
        *reinterpret_cast<float4*>(ps + lane * kPsPitch + sr) = make_float4(e[0], e[1], e[2], e[3]);
      }
      __syncthreads();
      if (holds) {
        // a block's sum by itself, joined to the blocks' before by one operation: the error of a long sum
        // then grows with the square roots of 32 and of the blocks, not of all positions
        float sum[4][4] = {};
        const int np = min(kSimtBn, most - p0);
        const int all = max(0, min(np, least - p0));  // positions that every running row sees
        auto add = [&](int i, float x, const float4& v) {
          sum[i][0] = fmaf(x, v.x, sum[i][0]);
          sum[i][1] = fmaf(x, v.y, sum[i][1]);
          sum[i][2] = fmaf(x, v.z, sum[i][2]);
          sum[i][3] = fmaf(x, v.w, sum[i][3]);
        };
        const char* vp = reinterpret_cast<const char*>(vs + d0);
        if (rpt == 4) {
#pragma unroll 4
          for (int t = 0; t < all; ++t) {
            const float4 v = load4(reinterpret_cast<const T*>(vp + t * pitch));
            const float4 x = load4(ps + t * kPsPitch + r0);
            add(0, x.x, v);
            add(1, x.y, v);
            add(2, x.z, v);
            add(3, x.w, v);
          }
        } else {
#pragma unroll 4
          for (int t = 0; t < all; ++t) {
            const float4 v = load4(reinterpret_cast<const T*>(vp + t * pitch));
            add(0, ps[t * kPsPitch + r0], v);
            if (rpt == 2) add(1, ps[t * kPsPitch + r0 + 1], v);
          }
        }
        for (int t = all; t < np; ++t) {
          const float4 v = load4(reinterpret_cast<const T*>(vp + t * pitch));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < rpt && p0 + t < row_lim[r0 + i]) add(i, ps[t * kPsPitch + r0 + i], v);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i >= rpt) break;
          const float c = row_c[r0 + i];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(acc[i][j], c, sum[i][j]);
        }
      }
    }
    __syncthreads();
    if (kPaged<P> && a.whole) {  // all that the rows see: no partial, the rows themselves
      if (holds) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + i;
          if (i >= rpt || row_lim[r] <= 0) continue;
          const float m = row_m[r], l = row_l[r], inv = l == 0.f ? 0.f : 1.f / l;
          T* dst = static_cast<T*>(p.out) + row_q[r] * p.os + static_cast<int64_t>(row_h[r]) * D + d0;
#pragma unroll
          for (int j = 0; j < 4; ++j) from_f(dst + j, m == -INFINITY ? 0.f : acc[i][j] * inv);
          if (p.lse && d0 == 0)
            p.lse[row_q[r] * (p.Hkv * p.G) + row_h[r]] = m == -INFINITY ? -INFINITY : (m + log2f(l)) * kLn2;
        }
      }
      continue;
    }
    if (tid < kSimtTm)
      p.ml[static_cast<int64_t>(slot) * kSimtTm + tid] = make_float2(row_m[tid], row_l[tid]);
    if (holds) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < rpt && row_lim[r0 + i] > 0)
          *reinterpret_cast<float4*>(p.o + (static_cast<int64_t>(slot) * kSimtTm + r0 + i) * D + d0) =
              make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    }
  }
}

template <typename P, typename T>
cudaError_t simt_launch(const P& p, int grid, cudaStream_t stream) {
  static SmemAllowance allowed;
  const int tiles = 4 * kSimtBn * (p.D * static_cast<int>(sizeof(T)) + kPad);
  const int floats = kSimtTm * (p.D + kPad / 4) + kSimtBn * kPsPitch + kSimtTm * kSimtBn + 3 * kSimtTm;
  const int smem = tiles + 4 * (floats + 4 * kSimtTm) + static_cast<int>(attn_plan_bytes(p));
  const cudaError_t e = allow_dynamic_smem(attn_simt_kernel<P, T>, smem, allowed);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_simt_kernel<P, T>, dim3(grid), dim3(kSimtThreads), smem, stream, p);
}

}  // namespace spec
