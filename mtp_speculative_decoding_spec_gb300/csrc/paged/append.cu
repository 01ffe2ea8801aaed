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
// A lane holds eight dims of a head, so a head is D / 8 lanes and a warp has 32 / (D / 8) heads at once. The
// dims of a lane are the same in all heads, so a row's cos and sin are formed once and stay in registers
// while the warp goes over the row's heads, four loads in flight.
#include <cuda_bf16.h>

#include "paged.cuh"

namespace spec {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 4;   // heads of a lane in flight

enum : int { ROT_NONE = 0, ROT_SIDE = 1, ROT_HALF = 2, ROT_HALF_ODD = 3 };

template <typename T>
struct Eight;  // eight elements as they lie in memory
template <>
struct Eight<__nv_bfloat16> {
  uint4 w;
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

template <typename T, int ROT>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int tph = p.tph, at = lane & (tph - 1), sub = lane / tph, heads = 32 / tph;
  const int D = p.D, e0 = 8 * at, half = p.rot / 2;
  const bool holds = e0 < D;
  // this lane's weights and frequencies; element j is turned where bit j of `turns` is set
  float wq[8], wk[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    wq[j] = p.q_norm && holds ? p.q_norm[e0 + j] : 1.f;
    wk[j] = p.k_norm && holds ? p.k_norm[e0 + j] : 1.f;
  }
  constexpr int NF = ROT == ROT_NONE ? 1 : ROT == ROT_SIDE ? 4 : 8;
  uint64_t F[NF];
  uint32_t turns = 0, low = 0;  // low: the element is its pair's first
  if constexpr (ROT == ROT_SIDE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      F[j] = 0;
      if (e0 + 2 * j < p.rot) {
        F[j] = turns_of(p.inv_freq[(e0 >> 1) + j]);
        turns |= 3u << (2 * j);
      }
    }
  } else if constexpr (ROT != ROT_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      F[j] = 0;
      if (e0 + j < p.rot) {
        const bool first = e0 + j < half;
        F[j] = turns_of(p.inv_freq[e0 + j - (first ? 0 : half)]);
        turns |= 1u << j;
        low |= static_cast<uint32_t>(first) << j;
      }
    }
  }
  const int nheads = p.nq + 2 * p.nk;
  const float inv_d = 1.f / static_cast<float>(D);
  const T* qb = static_cast<const T*>(p.q);
  const T* kb = static_cast<const T*>(p.k);
  const T* vb = static_cast<const T*>(p.v);

  int64_t last_row = -1;
  bool runs = false;
  int64_t page_at = -1;  // where the row's keys and values go, in bytes from the layer's first page
  float c[NF], s[NF];
  const int64_t t1 = min(p.tasks, (warp + 1) * p.tasks_warp);
  for (int64_t t = warp * p.tasks_warp; t < t1; ++t) {
    const int64_t row = t / p.tasks_row;
    const int i0 = static_cast<int>(t - row * p.tasks_row) * p.per_task, i1 = min(p.iters, i0 + p.per_task);
    Eight<T> x[kBatch];
    auto fetch = [&](int i) {
#pragma unroll
      for (int n = 0; n < kBatch; ++n) {
        const int h = (i + n) * heads + sub;
        if (i + n >= i1 || h >= nheads || !holds) continue;
        const T* src = h < p.nq ? qb + row * p.qs + static_cast<int64_t>(h) * D
                       : h < p.nq + p.nk
                           ? kb + row * p.ks + static_cast<int64_t>(h - p.nq) * D
                           : vb + row * p.vs + static_cast<int64_t>(h - p.nq - p.nk) * D;
        x[n].load(src + e0, p.vec_in);
      }
    };
    fetch(i0);
    if (row != last_row) {
      last_row = row;
      const int b = paged_request_of(p.cu_rows, p.B, row);
      runs = false;
      if (b < p.B) {
        const PagedRows pr = paged_rows(p.cu_rows, p.n_rows, p.rows, b);
        const int64_t r = row - pr.start;
        runs = r >= 0 && r < pr.runs;
        if (runs) {
          const int64_t P = max(static_cast<int64_t>(0), p.c.kv_len[b]), pos = P + r;
          const int64_t turn = p.pos ? p.pos[b] + r : pos;
          page_at = p.nk > 0 && pos < static_cast<int64_t>(p.c.max_pages) * p.c.page_size
                        ? paged_offset(p.c, b, static_cast<int>(pos))
                        : -1;
          if constexpr (ROT != ROT_NONE) {
#pragma unroll
            for (int j = 0; j < NF; ++j) {
              const uint32_t part = static_cast<uint32_t>((F[j] * static_cast<uint64_t>(turn)) >> 32);
              float sn, cs;
              sincospif(static_cast<float>(static_cast<int32_t>(part)) * 0x1p-31f, &sn, &cs);
              c[j] = cs * p.rot_scale;
              s[j] = sn * p.rot_scale;
              if (ROT != ROT_SIDE && (low >> j & 1)) s[j] = -s[j];
            }
          }
        }
      }
    }
    if (!runs) continue;  // the whole warp
    for (int i = i0; i < i1; i += kBatch) {
      if (i > i0) fetch(i);
#pragma unroll
      for (int n = 0; n < kBatch; ++n) {
        if (i + n >= i1) break;  // the whole warp
        const int h = (i + n) * heads + sub;
        const bool is_q = h < p.nq, is_k = !is_q && h < p.nq + p.nk, live = h < nheads && holds;
        if (__any_sync(0xffffffffu, is_q || is_k)) {
          float y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = 0.f;
          if (live) x[n].get(y);
          const bool norm = is_q ? p.q_norm != nullptr : p.k_norm != nullptr;
          if (__any_sync(0xffffffffu, norm)) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(y[j], y[j], sum);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
              if (o < tph) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = __frsqrt_rn(fmaf(sum, inv_d, p.eps));
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (norm) y[j] *= inv * (is_q ? wq[j] : wk[j]);
          }
          if constexpr (ROT == ROT_SIDE) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float a = y[2 * j], b = y[2 * j + 1];
              if (turns >> (2 * j) & 1) {
                y[2 * j] = a * c[j] - b * s[j];
                y[2 * j + 1] = b * c[j] + a * s[j];
              }
            }
          } else if constexpr (ROT == ROT_HALF) {  // half a multiple of 8: eight pairs' other ends in one lane
            const int from = e0 < half ? at + half / 8 : at - half / 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float o = __shfl_sync(0xffffffffu, y[j], from, tph);
              if (turns >> j & 1) y[j] = fmaf(o, s[j], y[j] * c[j]);
            }
          } else if constexpr (ROT == ROT_HALF_ODD) {
            // element j's other end is element (j +- half) & 7 of the lane that far on or back
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
              if (turns >> j & 1) y[j] = fmaf(low >> j & 1 ? a : b, s[j], y[j] * c[j]);
            }
          }
          if (is_q || is_k) x[n].set(y);
        }
        if (!live) continue;
        if (is_q) {
          x[n].store(static_cast<T*>(p.q_out) + row * p.qos + static_cast<int64_t>(h) * D + e0, p.vec_out);
        } else if (page_at >= 0) {
          uint8_t* pages = is_k ? p.c.k : p.c.v;
          const int kh = h - p.nq - (is_k ? 0 : p.nk);
          x[n].store(reinterpret_cast<T*>(pages + page_at) + static_cast<int64_t>(kh) * D + e0, true);
        }
      }
    }
  }

  if (p.status) {  // a warp to a request: the pages of its rows
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    for (int64_t b = warp; b < p.B; b += warps) {
      const int n = paged_rows(p.cu_rows, p.n_rows, p.rows, static_cast<int>(b)).runs;
      const int64_t P = max(static_cast<int64_t>(0), p.c.kv_len[b]);
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

template <typename T>
cudaError_t launch(const AppendParams& p, bool interleaved, unsigned grid, cudaStream_t stream) {
  const int half = p.rot / 2;
  if (p.rot == 0) return launch_pdl(append_kernel<T, ROT_NONE>, dim3(grid), dim3(kThreads), 0, stream, p);
  if (interleaved) return launch_pdl(append_kernel<T, ROT_SIDE>, dim3(grid), dim3(kThreads), 0, stream, p);
  if (half % 8 == 0) return launch_pdl(append_kernel<T, ROT_HALF>, dim3(grid), dim3(kThreads), 0, stream, p);
  return launch_pdl(append_kernel<T, ROT_HALF_ODD>, dim3(grid), dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t append_launch(AppendParams& p, spec_dtype dtype, bool interleaved, int sms, cudaStream_t stream) {
  p.tph = 1;
  while (p.tph * 8 < p.D) p.tph *= 2;
  const int heads = 32 / p.tph;
  p.iters = (p.nq + 2 * p.nk + heads - 1) / heads;
  // A warp takes a row's heads four at a time where there are few rows, so that they spread over the SMs,
  // and whole rows where there are many, which then form their angles once.
  const int64_t warps = static_cast<int64_t>(sms) * 16;
  const int64_t per = (p.rows * p.iters + warps - 1) / warps;
  p.per_task = static_cast<int>(max(int64_t(1), min(per, static_cast<int64_t>(p.iters))));
  p.tasks_row = (p.iters + p.per_task - 1) / p.per_task;
  p.tasks = p.rows * p.tasks_row;
  p.tasks_warp = max(int64_t(1), (p.tasks + warps - 1) / warps);
  const int64_t used = max(int64_t(1), (p.tasks + p.tasks_warp - 1) / p.tasks_warp);
  const unsigned grid = static_cast<unsigned>((used + kThreads / 32 - 1) / (kThreads / 32));
  return dtype == SPEC_BF16 ? launch<__nv_bfloat16>(p, interleaved, grid, stream)
                            : launch<float>(p, interleaved, grid, stream);
}

}  // namespace spec
