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
// And rows that requests own and do not run become zero (Fill): by the blocks of their request, or by all, a warp
// to a row. Of a request of 8,192 rows (16 heads of 256 dims over 1,000 positions) that runs three, a call by one
// block 1,232 us, by all 27; 32 requests of 1 to 8 rows 36.2 by theirs (38.1 by one each), 38.7 by all.
enum class Fill { kNone, kBlocks, kWarps };
constexpr int kFillRows = 8, kFillRequests = 64;  // of a request in the mean, and requests, for kBlocks
template <typename T, Fill FILL>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedParams p, int ctas) {
  __shared__ int first[2 * kPagedMaxCtas + 1];  // of the rows before each unit's
  __shared__ int4 notes[2 * kPagedMaxCtas];
  __shared__ int sums[kJoinWarps];
  __shared__ float sm_m[kJoinWarps], sm_l[kJoinWarps];
  __shared__ __align__(16) float sm_o[kJoinWarps][kMaxD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, Hq = p.Hkv * p.G;
  pdl_wait();
  const auto rows_of = [&](int b) { return paged_rows(p.cu_rows, p.n_rows, p.rows, b); };
  // (here, so that what they wait for comes with the notes)
  int row = 0, end = 0;  // this block's rows to clear, every parts-th
  if (const int part = blockIdx.x / p.B; FILL == Fill::kBlocks && part < static_cast<int>(gridDim.x) / p.B) {
    const PagedRows own = rows_of(blockIdx.x - part * p.B);
    row = own.start + own.runs + part, end = own.start + own.owned;
  }
  const auto idles = [&](int64_t at) {  // by a warp
    const int b = paged_request_of(p.cu_rows, p.B, at);
    if (b >= p.B) return false;
    const PagedRows r = rows_of(b);
    return at - r.start >= r.runs;
  };
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kJoinWarps + warp;
  bool idle = false;
  if (FILL == Fill::kWarps && row0 < p.rows) idle = idles(row0);
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
  const auto clear = [&](int64_t row, int i, int n) {  // by n threads, of which this is i
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t d = i * 4; d < static_cast<int64_t>(Hq) * p.D; d += n * 4)
      store4(static_cast<T*>(p.out) + row * p.os + d, zero);
    if (p.lse)
      for (int h = i; h < Hq; h += n) p.lse[row * Hq + h] = -INFINITY;
  };
  if constexpr (FILL == Fill::kBlocks) {
#pragma unroll 1
    for (const int parts = gridDim.x / p.B; row < end; row += parts) clear(row, threadIdx.x, kJoinThreads);
  }
  if constexpr (FILL == Fill::kWarps) {
#pragma unroll 1
    for (int64_t t = row0; t < p.rows;) {
      if (idle) clear(t, lane, 32);
      t += static_cast<int64_t>(gridDim.x) * kJoinWarps;
      if (t < p.rows) idle = idles(t);
    }
  }
}

template <typename T>
cudaError_t launch_join(const PagedParams& p, dim3 g, int ctas, cudaStream_t stream) {
  const dim3 t(kJoinThreads);
  if (!p.n_rows) return launch_pdl(paged_join_kernel<T, Fill::kNone>, g, t, 0, stream, p, ctas);
  // a block to a request at least, and not so many rows that one request's could be the most of the time
  if (p.B <= kFillRequests && static_cast<int>(g.x) >= p.B && p.rows <= int64_t(kFillRows) * p.B)
    return launch_pdl(paged_join_kernel<T, Fill::kBlocks>, g, t, 0, stream, p, ctas);
  return launch_pdl(paged_join_kernel<T, Fill::kWarps>, g, t, 0, stream, p, ctas);
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
  const dim3 g(static_cast<unsigned>(max(int64_t(1), min(int64_t(3) * grid, rows))));
  return dtype == SPEC_BF16 ? launch_join<__nv_bfloat16>(p, g, grid, stream) : launch_join<float>(p, g, grid, stream);
}

}  // namespace spec
