// Attention of new rows over a paged cache: the CUDA-core kernel of trunk/attn.cuh for it, and the kernel that
// joins the partial results of both kernels.
#include "paged.cuh"

#include "trunk/attn.cuh"

namespace spec {
namespace {

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kInFlight = 4;  // partials of a warp

__device__ __forceinline__ void store4(float* p, const float* v) {
  if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    p[0] = v[0], p[1] = v[1], p[2] = v[2], p[3] = v[3];
  }
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  if ((reinterpret_cast<uintptr_t>(p) & 7u) == 0) {
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    p[0] = a.x, p[1] = a.y, p[2] = b.x, p[3] = b.y;
  }
}

// Every row of every unit that more than one CTA has part of, from its partials in the positions' order: a
// warp to a row, or eight where there are fewer rows than blocks. Most units of a prompt are whole, so what
// there is to do is found from the CTAs' notes (PagedSplit), not from the rows: a warp to each row and head
// of 2,311 rows of 16 heads took 30 us. (The last CTA to come to a unit joining it in the attention kernel
// saved this launch and took 18 us more at two rows over 63,488 positions: code that each SM fetches anew.)
// And rows that requests own and do not run become zero.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedParams p, int ctas) {
  __shared__ int first[2 * kPagedMaxCtas + 1];  // of the rows before each unit's
  __shared__ int4 notes[2 * kPagedMaxCtas];
  __shared__ int sums[kJoinWarps];
  __shared__ float sm_m[kJoinWarps], sm_l[kJoinWarps];
  __shared__ __align__(16) float sm_o[kJoinWarps][kMaxD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, Hq = p.Hkv * p.G;
  pdl_wait();
  const auto rows_of = [&](int b) { return paged_rows(p.cu_rows, p.n_rows, p.rows, b); };
  PagedRows own = {0, 0, 0};  // the request whose rows this block fills up first, below
  if (static_cast<int>(blockIdx.x) < p.B) own = rows_of(blockIdx.x);
  constexpr int kEach = 2 * kPagedMaxCtas / kJoinThreads;
  int n[kEach], sum = 0;  // a thread's units, and the rows of them and of those before
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int i = threadIdx.x * kEach + j;
    n[j] = 0;
    if (i < 2 * ctas) {
      notes[i] = __ldcg(reinterpret_cast<const int4*>(p.splits + i));
      n[j] = paged_split_of(notes[i]).count;
    }
    sum += n[j];
  }
  int before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  if (lane == 31) sums[warp] = before;
  before -= sum;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  if (total > 0) {
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int i = threadIdx.x * kEach + j;
      if (i <= 2 * ctas) first[i] = before;
      before += n[j];
    }
    __syncthreads();
  }
  const bool few = total <= static_cast<int>(gridDim.x);
  const int nw = few ? kJoinWarps : 1, w0 = few ? warp : 0;
  const int nv = p.D / 4;
#pragma unroll 1
  for (int t = few ? blockIdx.x : blockIdx.x * kJoinWarps + warp; t < total; t += gridDim.x * (kJoinWarps / nw)) {
    int lo = 0, hi = 2 * ctas;  // first[lo] <= t < first[hi]
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const PagedSplit u = paged_split_of(notes[lo]);
    const int at = t - first[lo], c0 = lo >> 1, part = 2 * (lo & 1);
    float m = -INFINITY, l = 0.f;
    float acc[2][4] = {};
#pragma unroll 1
    for (int i0 = w0; i0 < u.n; i0 += kInFlight * nw) {
      float2 mlv[kInFlight];
      float4 ov[kInFlight][2];
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) {
        const int i = i0 + nw * j;
        mlv[j] = make_float2(-INFINITY, 0.f);
        ov[j][0] = ov[j][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < u.n) {
          const int64_t s = static_cast<int64_t>(4 * (c0 + i * u.step) + part + (i == 0)) * p.tm + at;
          mlv[j] = __ldcg(p.ml + s);
          const float4* o = reinterpret_cast<const float4*>(p.o + s * p.D);
          if (lane < nv) ov[j][0] = __ldcg(o + lane);
          if (lane + 32 < nv) ov[j][1] = __ldcg(o + lane + 32);
        }
      }
      float top = m;
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) top = (top != top || mlv[j].x != mlv[j].x) ? NAN : fmaxf(top, mlv[j].x);
      const float ref = top == -INFINITY ? 0.f : top;
      const float c = exp2f(m - ref);
      m = top;
      l *= c;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[h][d] *= c;
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) {
        const float w = exp2f(mlv[j].x - ref);
        l = fmaf(w, mlv[j].y, l);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          acc[h][0] = fmaf(w, ov[j][h].x, acc[h][0]);
          acc[h][1] = fmaf(w, ov[j][h].y, acc[h][1]);
          acc[h][2] = fmaf(w, ov[j][h].z, acc[h][2]);
          acc[h][3] = fmaf(w, ov[j][h].w, acc[h][3]);
        }
      }
    }
    if (few) {  // the warps' parts, in their order
      if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < nv)
          *reinterpret_cast<float4*>(&sm_o[warp][(lane + 32 * h) * 4]) =
              make_float4(acc[h][0], acc[h][1], acc[h][2], acc[h][3]);
      __syncthreads();
      if (warp == 0) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) top = (top != top || sm_m[w] != sm_m[w]) ? NAN : fmaxf(top, sm_m[w]);
        const float ref = top == -INFINITY ? 0.f : top;
        m = top;
        l = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int d = 0; d < 4; ++d) acc[h][d] = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
          const float c = exp2f(sm_m[w] - ref);
          l = fmaf(c, sm_l[w], l);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (lane + 32 * h < nv) {
              const float4 o = *reinterpret_cast<const float4*>(&sm_o[w][(lane + 32 * h) * 4]);
              acc[h][0] = fmaf(c, o.x, acc[h][0]), acc[h][1] = fmaf(c, o.y, acc[h][1]);
              acc[h][2] = fmaf(c, o.z, acc[h][2]), acc[h][3] = fmaf(c, o.w, acc[h][3]);
            }
        }
      }
    }
    if (!few || warp == 0) {
      const bool empty = m == -INFINITY;  // nothing seen, or scores of -Inf alone: zero
      const float inv = empty || l == 0.f ? 0.f : 1.f / l;
      const int x = u.tile * p.tm + at, r = x / p.G;
      const int64_t row = static_cast<int64_t>(u.start) + r;
      const int qh = u.head * p.G + x - r * p.G;
      T* dst = static_cast<T*>(p.out) + row * p.os + static_cast<int64_t>(qh) * p.D;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (lane + 32 * h < nv) {
          float v[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) v[d] = empty ? 0.f : acc[h][d] * inv;
          store4(dst + (lane + 32 * h) * 4, v);
        }
      if (p.lse && lane == 0) p.lse[row * Hq + qh] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
    }
    if (few) __syncthreads();  // the parts are no longer read
  }
#pragma unroll 1
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const PagedRows r = b == static_cast<int>(blockIdx.x) ? own : rows_of(b);
#pragma unroll 1
    for (int i = r.runs; i < r.owned; ++i) {
      const int64_t row = r.start + i;
      const float zero[4] = {0.f, 0.f, 0.f, 0.f};
      for (int d = threadIdx.x * 4; d < Hq * p.D; d += kJoinThreads * 4)
        store4(static_cast<T*>(p.out) + row * p.os + d, zero);
      if (p.lse)
        for (int h = threadIdx.x; h < Hq; h += kJoinThreads) p.lse[row * Hq + h] = -INFINITY;
    }
  }
}

}  // namespace

cudaError_t paged_simt_launch(const PagedParams& p, spec_dtype dtype, int grid, cudaStream_t stream) {
  return dtype == SPEC_BF16 ? simt_launch<PagedParams, __nv_bfloat16>(p, grid, stream)
                            : simt_launch<PagedParams, float>(p, grid, stream);
}

cudaError_t paged_join_launch(const PagedParams& p, spec_dtype dtype, int grid, cudaStream_t stream) {
  // Blocks for each CTA of the attention: 2, 3, 4, 6: 1,000 rows beside 31 single tokens 122.7, 111.6, 111.3, 110.8
  // us, a call with nothing to join 12.8, 13.2, 13.7, 14.9.
  // And no more than rows and heads (8 and 32 of them: 12.8 and 55.7 us with all blocks, 12.0 and 54.8).
  const int64_t rows = p.rows * p.Hkv * p.G;
  const dim3 g(static_cast<unsigned>(max(int64_t(1), min(int64_t(3) * grid, rows)))), t(kJoinThreads);
  return dtype == SPEC_BF16 ? launch_pdl(paged_join_kernel<__nv_bfloat16>, g, t, 0, stream, p, grid)
                            : launch_pdl(paged_join_kernel<float>, g, t, 0, stream, p, grid);
}

}  // namespace spec
