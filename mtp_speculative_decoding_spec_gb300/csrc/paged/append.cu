// New rows of queries, keys and values on their way to attention: each head normed, its first dims rotated
// by its position, keys and values written to their pages, in one pass.
//
//   y = w x / sqrt(mean(x^2) + eps);   y_a' = s (y_a cos t - y_b sin t),  y_b' = s (y_b cos t + y_a sin t)
//   t = pos * f_i
//
// The angle. pos * f in fp32 is off by 2e-3 at a position of 60,000, and fp64 is slow here. But cos and sin
// need the product in turns only, modulo 1: F = f / (2 pi) as a fraction of 64 bits (24 bits of f times 128
// bits of 1 / (2 pi), once per thread), so that F * pos modulo 2^64 is the angle's fraction of a turn with
// 2^-64 * pos of error, by integer multiplication. Its upper 32 bits, as a signed number of half turns, go
// to sincospif.
//
// A lane holds eight dims of a head, so a head is D / 8 lanes and a warp has 32 / (D / 8) heads at once. A
// row's angles are formed once, a lane each, and handed round through shared memory. What the arithmetic has
// to do then is kept short, since it and not the memory would be the bound: with the weights taken into cos
// and sin, an output is (x / rms) wc + (x' / rms) ws with x' the pair's other end, whose bits come from the
// lane that has it before anything is done to them (two bf16 a shuffle), in packed fp32.
//
// HBM bounds it where there are many rows: a prompt of 15,360 rows of 16 + 2 x 4 heads of 256 dims, a quarter
// rotated, with norms, 65 us = 5.8 TB/s of bytes read and written (0.86 of a copy). A few thousand are a round of
// the warps that fit at once and part of another: 3,389 rows of 16 + 2 x 8 heads of 128, all rotated, on 2,432 warps
// 13.4 us, and 11.3 with all of it in L2. Latency where there are few: 32 x 8 rows 4.7, one request of two 2.7 (in a
// graph).
#include <cuda_bf16.h>

#include "paged.cuh"

namespace spec {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
// Of an SM, to deal out few rows: 4, 8, 16, 32, 64: 32 requests of 8 rows 5.4, 5.1, 5.2, 5.4, 8.2 us in a graph, 128
// of them 8.3, 9.3, 7.8, 9.1, 11.6, prompts of 3,389 rows in all 11.3, 11.3, 11.3, 12.2, 15.7.
constexpr int kAppendWarps = 16;

enum : int { ROT_NONE = 0, ROT_SIDE = 1, ROT_HALF = 2, ROT_HALF_ODD = 3 };

// Blocks an SM, which bounds the registers: 15,360 bf16 rows 72 us with three, 65 with four (fp32's registers, and
// those of pairs that end inside a lane, do not fit so).
template <typename T, int ROT, int STEP>
constexpr int kMinBlocks = ROT == ROT_HALF_ODD ? 1 : sizeof(T) == 2 && STEP ? 4 : 3;
// Heads of a lane side by side. Two and four: 15,360 bf16 rows of 16 + 2 x 4 heads of 256 dims 81 and 65 us; where
// a warp has fewer than two fours of a row's queries (or keys) none is on its way while another is worked on: 8,000
// rows of 16 + 2 x 8 heads of 64 dims 12.9 and 15.7, 32 x 8 rows of the first 4.7 and 5.2. fp32, one and two:
// 15,360 rows 141 and 127.
constexpr int kBatchMany = 4, kBatchFew = 2;

template <typename T>
struct Eight;  // eight elements as they lie in memory
template <>
struct Eight<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ Eight from(int lane, int width, bool any) const {  // another lane's, or zeros
    Eight o;
    o.w.x = __shfl_sync(0xffffffffu, w.x, lane, width), o.w.y = __shfl_sync(0xffffffffu, w.y, lane, width);
    o.w.z = __shfl_sync(0xffffffffu, w.z, lane, width), o.w.w = __shfl_sync(0xffffffffu, w.w, lane, width);
    if (!any) o.w = make_uint4(0u, 0u, 0u, 0u);
    return o;
  }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(a[j] << 16);
      x[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float* x) {
    uint32_t a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
      a[j] = *reinterpret_cast<const uint32_t*>(&v);
    }
    w = make_uint4(a[0], a[1], a[2], a[3]);
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool whole) {
    if (whole) {
      w = __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
      const uint16_t* s = reinterpret_cast<const uint16_t*>(p);
      uint32_t a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = s[2 * j] | static_cast<uint32_t>(s[2 * j + 1]) << 16;
      w = make_uint4(a[0], a[1], a[2], a[3]);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, bool whole) const {
    if (whole) {
      *reinterpret_cast<uint4*>(p) = w;
    } else {
      uint16_t* d = reinterpret_cast<uint16_t*>(p);
      const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = static_cast<uint16_t>(a[j / 2] >> (16 * (j & 1)));
    }
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ Eight from(int lane, int width, bool any) const {
    float x[8];
    get(x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = __shfl_sync(0xffffffffu, x[j], lane, width);
      if (!any) x[j] = 0.f;
    }
    Eight o;
    o.set(x);
    return o;
  }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float* x) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ __forceinline__ void load(const float* p, bool whole) {
    if (whole) {
      a = __ldcs(reinterpret_cast<const float4*>(p));
      b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    } else {
      a = make_float4(p[0], p[1], p[2], p[3]);
      b = make_float4(p[4], p[5], p[6], p[7]);
    }
  }
  __device__ __forceinline__ void store(float* p, bool whole) const {
    if (whole) {
      *reinterpret_cast<float4*>(p) = a;
      *(reinterpret_cast<float4*>(p) + 1) = b;
    } else {
      p[0] = a.x, p[1] = a.y, p[2] = a.z, p[3] = a.w;
      p[4] = b.x, p[5] = b.y, p[6] = b.z, p[7] = b.w;
    }
  }
};

// f / (2 pi) modulo 1 as a fraction of 64 bits; f finite, |f| < 2^24.
__device__ __forceinline__ uint64_t turns_of(float f) {
  const uint32_t u = __float_as_uint(f);
  const int e = static_cast<int>((u >> 23) & 255u);
  const uint64_t m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int right = 150 - max(e, 1);  // f = m 2^-right; 0..149 for |f| < 2^24
  // m times 1 / (2 pi) as a fraction of 128 bits: 152 bits, of which those from 2^-64 up remain
  constexpr uint64_t c1 = 0x28be60db9391054aull, c0 = 0x7f09d5f47d4d3770ull;
  const uint64_t carry = __umul64hi(m, c0);
  const uint64_t mid = m * c1 + carry;
  const uint64_t top = __umul64hi(m, c1) + (mid < carry);
  const uint64_t t = right >= 128 || right < 0 ? 0
                     : right >= 64 ? top >> (right - 64)
                     : right > 0   ? (mid >> right) | (top << (64 - right))
                                   : mid;
  return (u >> 31) ? 0 - t : t;
}

__device__ __forceinline__ unsigned long long pair(float a, float b) {
  return pack2(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Eight consecutive floats of shared memory (32-byte aligned).
__device__ __forceinline__ void lds8(const float* p, float* x) {
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    const float4 v = *reinterpret_cast<const float4*>(p + j);
    x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
  }
}

// WHOLE: rows of q, k, v and q_out are whole 16-byte vectors (element by element 15,360 rows take 161 us for 65).
// STEP: elements that a warp's heads take, 0 where D is no power of two and the host's number counts (73 us for 65).
template <typename T, int ROT, bool WHOLE, int STEP, int kBatch>
__global__ void __launch_bounds__(kThreads, kMinBlocks<T, ROT, STEP>)
    append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ __align__(32) float weights[2][256];       // of queries and keys
  __shared__ __align__(32) float2 trig[kWarps][128];    // cos and sin of a warp's row
  __shared__ uint64_t freq[128];                        // turns a position
  pdl_wait();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int tph = p.tph, at = lane & (tph - 1), sub = lane / tph, heads = 32 / tph;
  const int D = p.D, e0 = 8 * at, half = p.rot / 2, step = STEP ? STEP : heads * D;
  const bool holds = e0 < D;
  for (int d = threadIdx.x; d < D; d += kThreads) {
    weights[0][d] = p.q_norm ? p.q_norm[d] : 1.f;
    weights[1][d] = p.k_norm ? p.k_norm[d] : 1.f;
  }
  if (ROT != ROT_NONE && threadIdx.x < half) freq[threadIdx.x] = turns_of(p.inv_freq[threadIdx.x]);
  __syncthreads();
  const float inv_d = 1.f / static_cast<float>(D);
  // with pairs half of rot_dim apart: the lane that has the other ends, whether there are any
  const bool low = e0 < half, turned = ROT == ROT_HALF && e0 < p.rot;
  const int other = !turned ? at : low ? at + half / 8 : at - half / 8;
  const auto angle = [&](int e) { return trig[wid][ROT == ROT_SIDE ? e >> 1 : e < half ? e : e - half]; };
  // this block's turns of a row: queries' cq, then keys' ck, then values' ck
  const int i0 = blockIdx.y * p.per_task, i1 = min(p.iters, i0 + p.per_task);
  const int q1 = min(i1, p.cq), k0 = max(0, i0 - p.cq), k1 = min(i1 - p.cq, p.ck);
  const int v0 = max(0, i0 - p.cq - p.ck), v1 = i1 - p.cq - p.ck;

  // kBatch of a row's heads, from turn a on, at the lane's dims; turn n is there where a + n < a1 and its head
  // < nh. What is not there is computed on all the same (straight code: the heads' shuffles overlap), but a
  // lane's registers reach no lane of another head, and it is not stored.
  Eight<T> x[kBatch];
  auto fetch = [&](const T* src, int a, int a1, int nh) {
#pragma unroll
    for (int n = 0; n < kBatch; ++n)
      if (a + n < a1 && holds && (a + n) * heads + sub < nh) x[n].load(src + (a + n) * step, WHOLE);
  };
  auto write = [&](const Eight<T>* y, T* dst, int a, int a1, int nh, bool whole) {
#pragma unroll
    for (int n = 0; n < kBatch; ++n)
      if (a + n < a1 && holds && (a + n) * heads + sub < nh) y[n].store(dst + (a + n) * step, whole);
  };
  unsigned long long wc[4], ws[4];
  auto turn_weights = [&](const float* weight) {  // out_j = y_j wc_j + y'_j ws_j, y and y' without weights
    float w[8], v[8], cs[16];
    lds8(weight + e0, w);
    if constexpr (ROT == ROT_SIDE || ROT == ROT_HALF) {
      const bool on = e0 < p.rot;
      const int first = !on ? 0 : ROT == ROT_SIDE ? e0 / 2 : low ? e0 : e0 - half;
      const float* from = reinterpret_cast<const float*>(trig[wid] + first);
      lds8(from, cs);
      if (ROT == ROT_HALF) lds8(from + 8, cs + 8);
      // a dim that is not turned takes nothing of another, whose weight need not be finite
      if (ROT == ROT_SIDE || on) {
        lds8(weight + (ROT == ROT_SIDE ? e0 : low ? e0 + half : e0 - half), v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
      }
      float c[8], s[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool there = ROT == ROT_SIDE ? e0 + j < p.rot : on;
        c[j] = there ? cs[ROT == ROT_SIDE ? j & ~1 : 2 * j] : 1.f;
        s[j] = there ? cs[ROT == ROT_SIDE ? j | 1 : 2 * j + 1] : 0.f;
        if (ROT == ROT_SIDE && !there) v[j ^ 1] = 0.f;  // pairs are turned both or neither
        if (ROT == ROT_SIDE ? (j & 1) == 0 : low) s[j] = -s[j];
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        wc[j / 2] = pair(w[j] * c[j], w[j + 1] * c[j + 1]);
        ws[j / 2] = ROT == ROT_SIDE ? pair(v[j + 1] * s[j], v[j] * s[j + 1]) : pair(v[j] * s[j], v[j + 1] * s[j + 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j += 2) wc[j / 2] = pair(w[j], w[j + 1]);
    }
  };
  // The heads in x; `next` fetches the ones after them into x once their bits are taken.
  auto work = [&](Eight<T>* out, bool norm, auto&& next) {
    Eight<T> mine[kBatch], far[kBatch];
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      mine[n] = x[n];
      // (with a norm a lane that is not turned may have its own bits there: they are finite, or its output is
      // NaN as it is)
      if (ROT == ROT_HALF) far[n] = x[n].from(other, tph, norm || turned);
    }
    next();
    unsigned long long y2[kBatch][4];
    float inv[kBatch];
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      float y[8];
      mine[n].get(y);
#pragma unroll
      for (int j = 0; j < 4; ++j) y2[n][j] = STEP || holds ? pair(y[2 * j], y[2 * j + 1]) : 0ull;
    }
    if (norm) {
#pragma unroll
      for (int n = 0; n < kBatch; ++n) {
        unsigned long long sq = mul2(y2[n][0], y2[n][0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) ffma2_acc(sq, y2[n][j], y2[n][j]);
        inv[n] = sum2(sq);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < tph) {
#pragma unroll
          for (int n = 0; n < kBatch; ++n) inv[n] += __shfl_xor_sync(0xffffffffu, inv[n], o);
        }
#pragma unroll
      for (int n = 0; n < kBatch; ++n) inv[n] = rsqrtf(fmaf(inv[n], inv_d, p.eps));
    }
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      unsigned long long o2[4];
      const unsigned long long inv2 = pair(inv[n], inv[n]);
      float z[8];
      if (ROT == ROT_HALF) far[n].get(z);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        unsigned long long z2 = ROT == ROT_HALF ? pair(z[2 * j], z[2 * j + 1]) : 0ull;
        if (norm) {
          y2[n][j] = mul2(y2[n][j], inv2);
          if (ROT == ROT_HALF) z2 = mul2(z2, inv2);
        }
        if (ROT == ROT_SIDE && e0 + 2 * j < p.rot) z2 = y2[n][j] << 32 | y2[n][j] >> 32;
        o2[j] = mul2(y2[n][j], wc[j]);
        if (ROT == ROT_SIDE || ROT == ROT_HALF) ffma2_acc(o2[j], z2, ws[j]);
      }
      float y[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[2 * j] = __uint_as_float(static_cast<uint32_t>(o2[j]));
        y[2 * j + 1] = __uint_as_float(static_cast<uint32_t>(o2[j] >> 32));
      }
      if constexpr (ROT == ROT_HALF_ODD) {
        // half of rot_dim no multiple of eight: element j's other end is element (j +- half) & 7 of the lane
        // that far on or back
        float up[8], down[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) up[j] = down[j] = y[j];
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
          if (half & o) {
            float a[8], b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = up[(j + o) & 7], b[j] = down[(j - o) & 7];
#pragma unroll
            for (int j = 0; j < 8; ++j) up[j] = a[j], down[j] = b[j];
          }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a = __shfl_sync(0xffffffffu, up[j], at + ((j + half) >> 3), tph);
          const float b = __shfl_sync(0xffffffffu, down[j], at + ((j - half) >> 3), tph);
          if (e0 + j < p.rot) {
            const float2 cs = angle(e0 + j);
            y[j] = fmaf(e0 + j < half ? -a : b, cs.y, y[j] * cs.x);
          }
        }
      }
      out[n].set(y);
    }
  };

  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kWarps + wid;
  const auto one_row = [&](int64_t row) {
    const T* const q = static_cast<const T*>(p.q) + row * p.qs + sub * D + e0;
    const T* const k = static_cast<const T*>(p.k) + row * p.ks + sub * D + e0;
    const T* const v = static_cast<const T*>(p.v) + row * p.vs + sub * D + e0;
    if (i0 < q1)
      fetch(q, i0, q1, p.nq);
    else if (k0 < k1)
      fetch(k, k0, k1, p.nk);
    else
      fetch(v, v0, v1, p.nk);
    const int b = paged_request_of(p.cu_rows, p.B, row);
    if (b >= p.B) return;  // nobody's
    const PagedRows pr = paged_rows(p.cu_rows, p.n_rows, p.rows, b);
    const int64_t r = row - pr.start;
    if (r < 0 || r >= pr.runs) return;
    const int64_t P = paged_len(p.c, b), pos = P + r;
    // where the row's keys and values go, in bytes from the layer's first page
    const int64_t page_at = p.nk > 0 && pos < static_cast<int64_t>(p.c.max_pages) * p.c.page_size
                                ? paged_offset(p.c, b, static_cast<int>(pos))
                                : -1;
    if constexpr (ROT != ROT_NONE) {
      const uint64_t turn = static_cast<uint64_t>(p.pos ? p.pos[b] : P) + static_cast<uint64_t>(r);
#pragma unroll 1
      for (int n = lane; n < half; n += 32) {
        const uint32_t part = static_cast<uint32_t>((freq[n] * turn) >> 32);
        float sn, cs;
        sincospif(static_cast<float>(static_cast<int32_t>(part)) * 0x1p-31f, &sn, &cs);
        trig[wid][n] = make_float2(cs * p.rot_scale, sn * p.rot_scale);
      }
      __syncwarp();
    }
    T* const out = static_cast<T*>(p.q_out) + row * p.qos + sub * D + e0;
    if (i0 < q1) {
      turn_weights(weights[0]);
#pragma unroll 1
      for (int a = i0; a < q1; a += kBatch) {
        Eight<T> y[kBatch];
        work(y, p.q_norm != nullptr, [&] {
          if (a + kBatch < q1)
            fetch(q, a + kBatch, q1, p.nq);
          else if (k0 < k1)
            fetch(k, k0, k1, p.nk);
        });
        write(y, out, a, q1, p.nq, WHOLE);
      }
    }
    T* const kp = reinterpret_cast<T*>(p.c.k + page_at) + sub * D + e0;
    T* const vp = reinterpret_cast<T*>(p.c.v + page_at) + sub * D + e0;
    if (k0 < k1) {
      turn_weights(weights[1]);
#pragma unroll 1
      for (int a = k0; a < k1; a += kBatch) {
        Eight<T> y[kBatch];
        work(y, p.k_norm != nullptr, [&] {
          if (a + kBatch < k1)
            fetch(k, a + kBatch, k1, p.nk);
          else if (v0 < v1)
            fetch(v, v0, v1, p.nk);
        });
        if (page_at >= 0) write(y, kp, a, k1, p.nk, true);
      }
    }
#pragma unroll 1
    for (int a = v0; a < v1; a += kBatch) {
      Eight<T> y[kBatch];
#pragma unroll
      for (int n = 0; n < kBatch; ++n) y[n] = x[n];
      if (a + kBatch < v1) fetch(v, a + kBatch, v1, p.nk);
      if (page_at >= 0) write(y, vp, a, v1, p.nk, true);
    }
  };
  if (warp < p.rows) one_row(warp);

  if (p.status) {  // a warp to a request: the pages of its rows
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t b = blockIdx.y == 0 ? warp : p.B; b < p.B; b += warps) {
      const int n = paged_rows(p.cu_rows, p.n_rows, p.rows, static_cast<int>(b)).runs;
      const int64_t P = paged_len(p.c, static_cast<int>(b));
      const int64_t cap = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
      bool bad = n > 0 && P + n > cap;
      if (n > 0 && P < cap) {
        const int j1 = static_cast<int>((min(P + n, cap) - 1) / p.c.page_size);
        for (int j = static_cast<int>(P / p.c.page_size) + lane; j <= j1; j += 32) {
          const int g = p.c.table[b * p.c.table_stride + j];
          bad = bad || g < 0 || g >= p.c.n_pages;
        }
      }
      bad = __any_sync(0xffffffffu, bad && p.nk > 0);
      if (lane == 0) p.status[b] = bad ? SPEC_REQ_KV_OVERFLOW : SPEC_REQ_OK;
    }
  }
}

template <typename T, int ROT, bool WHOLE, int STEP>
cudaError_t launch_batch(const AppendParams& p, dim3 grid, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2)
    if (min(max(p.cq, p.ck), p.per_task) >= 2 * kBatchMany)
      return launch_pdl(append_kernel<T, ROT, WHOLE, STEP, kBatchMany>, grid, dim3(kThreads), 0, stream, p);
  return launch_pdl(append_kernel<T, ROT, WHOLE, STEP, kBatchFew>, grid, dim3(kThreads), 0, stream, p);
}

template <typename T, int ROT>
cudaError_t launch_rot(const AppendParams& p, dim3 grid, cudaStream_t stream) {
  const bool pow2 = p.tph * 8 == p.D;  // 32 lanes of eight dims are whole heads then
  return !p.whole ? launch_batch<T, ROT, false, 0>(p, grid, stream)
         : pow2   ? launch_batch<T, ROT, true, 256>(p, grid, stream)
                  : launch_batch<T, ROT, true, 0>(p, grid, stream);
}

template <typename T>
cudaError_t launch(const AppendParams& p, bool interleaved, dim3 grid, cudaStream_t stream) {
  if (p.rot == 0) return launch_rot<T, ROT_NONE>(p, grid, stream);
  if (interleaved) return launch_rot<T, ROT_SIDE>(p, grid, stream);
  return p.rot % 16 == 0 ? launch_rot<T, ROT_HALF>(p, grid, stream) : launch_rot<T, ROT_HALF_ODD>(p, grid, stream);
}

}  // namespace

cudaError_t append_launch(AppendParams& p, spec_dtype dtype, bool interleaved, int sms, cudaStream_t stream) {
  p.tph = 1;
  while (p.tph * 8 < p.D) p.tph *= 2;
  const int heads = 32 / p.tph;
  p.cq = (p.nq + heads - 1) / heads;
  p.ck = (p.nk + heads - 1) / heads;
  p.iters = p.cq + 2 * p.ck;
  // A warp takes some of a row's heads where there are few rows, so that they spread over the SMs, and a whole
  // row where there are many, which then forms its angles once (two rows to a warp: 70 us for 67).
  const int64_t warps = static_cast<int64_t>(sms) * kAppendWarps;
  const int64_t per = (p.rows * p.iters + warps - 1) / warps;
  p.per_task = static_cast<int>(max(int64_t(1), min(per, static_cast<int64_t>(p.iters))));
  // (so a row has no more parts than there are such warps, which a grid's y holds; no rows: the status alone)
  const int parts = p.rows > 0 ? max(1, (p.iters + p.per_task - 1) / p.per_task) : 1;
  const int64_t blocks = max(int64_t(1), (p.rows + kWarps - 1) / kWarps);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(parts));
  return dtype == SPEC_BF16 ? launch<__nv_bfloat16>(p, interleaved, grid, stream)
                            : launch<float>(p, interleaved, grid, stream);
}

}  // namespace spec
