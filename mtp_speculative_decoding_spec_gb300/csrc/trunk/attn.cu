// Attention of the verify rows over a shared prefix and each request's own cache: the CUDA-core kernel of
// attn.cuh for it, and the kernel that joins the partial results of both kernels.
#include "attn.cuh"

namespace spec {
namespace {

// One output row (verify row, query head) by NW warps: the partials of its prefix unit and then of its
// own unit, warp w taking every NW-th of them, joined in that order. Many rows have few partials
// each and get one warp a row (four rows to a block); few rows have many, and get eight warps. The whole
// call, 16 query heads of 256 dims over a prefix of 15,360, one warp and eight: 8 verify rows 28.9 and 22.2
// us, 32 32.8 and 30.2, 40 32.7 and 32.8, 48 32.7 and 33.5, 64 33.6 and 36.0, 128 42.6 and 51.9.
// A partial of weight 0, from a row that saw nothing there or scores of -Inf alone, is added like any:
// its output is 0, or what is not finite among the values of positions that the row does see.
constexpr int kJoinMost = 4;  // partials in flight per warp

template <typename T, int NW>
__global__ void __launch_bounds__(NW == 1 ? 128 : 32 * NW)
    attn_join_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float sm_m[NW], sm_l[NW];
  __shared__ float sm_o[NW == 1 ? 1 : NW][NW == 1 ? 1 : kMaxD];
  const int lane = threadIdx.x & 31, warp = NW == 1 ? 0 : threadIdx.x >> 5;
  const int Hq = p.Hkv * p.G;
  const int64_t id = NW == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t row = id / Hq;
  if (row >= static_cast<int64_t>(p.B) * p.R) return;  // whole warps, and only where NW is 1
  const int qh = static_cast<int>(id - row * Hq);
  const int head = qh / p.G, g = qh - head * p.G;
  const int b = static_cast<int>(row / p.R), r = static_cast<int>(row) - b * p.R;
  const int s = (b * p.R + r) * p.G + g, x = r * p.G + g;
  pdl_wait();
  const AttnReq rq = attn_req(p, b);
  int2 u0 = make_int2(0, 0);
  const int t0 = s / p.tm;
  if (p.npt > 0) u0 = __ldcg(p.units + t0 / p.grp * p.Hkv + head);
  int2 u1 = __ldcg(p.units + (p.npi + b * p.nown + x / p.tm) * p.Hkv + head);
  u0.x += t0 % p.grp;
  if (rq.prefix == 0) u0.y = 0;
  if (r >= rq.rows) u0.y = u1.y = 0;
  const int at0 = s % p.tm, at1 = x % p.tm, ntot = u0.y + u1.y;
  float m = -INFINITY, l = 0.f;
  float acc[2][4] = {};
  const int nv = p.D / 4;
  for (int i0 = warp; i0 < ntot; i0 += kJoinMost * NW) {
    float2 mlv[kJoinMost];
    float4 ov[kJoinMost][2];
#pragma unroll
    for (int j = 0; j < kJoinMost; ++j) {
      const int i = i0 + NW * j;
      mlv[j] = make_float2(-INFINITY, 0.f);
      ov[j][0] = ov[j][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < ntot) {
        const bool pre = i < u0.y;
        const int64_t t = static_cast<int64_t>(pre ? u0.x + i * p.grp : u1.x + i - u0.y) * p.tm +
                          (pre ? at0 : at1);
        mlv[j] = __ldcg(p.ml + t);
        const float4* o = reinterpret_cast<const float4*>(p.o + t * p.D);
        if (lane < nv) ov[j][0] = __ldcg(o + lane);
        if (lane + 32 < nv) ov[j][1] = __ldcg(o + lane + 32);
      }
    }
    float top = m;
#pragma unroll
    for (int j = 0; j < kJoinMost; ++j)
      top = (top != top || mlv[j].x != mlv[j].x) ? NAN : fmaxf(top, mlv[j].x);
    const float ref = top == -INFINITY ? 0.f : top;
    const float c = exp2f(m - ref);
    m = top;
    l *= c;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int d = 0; d < 4; ++d) acc[h][d] *= c;
#pragma unroll
    for (int j = 0; j < kJoinMost; ++j) {
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
  T* dst = static_cast<T*>(p.out) + row * p.os + static_cast<int64_t>(qh) * p.D;
  if constexpr (NW == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const bool empty = m == -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (lane + 32 * h < nv) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const float v = empty ? 0.f : acc[h][d] * inv;
          if constexpr (sizeof(T) == 2)
            dst[(lane + 32 * h) * 4 + d] = __float2bfloat16_rn(v);
          else
            dst[(lane + 32 * h) * 4 + d] = v;
        }
      }
    if (p.lse && lane == 0) p.lse[row * Hq + qh] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
    return;
  }
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
  float top = -INFINITY;
#pragma unroll
  for (int w = 0; w < NW; ++w) top = (top != top || sm_m[w] != sm_m[w]) ? NAN : fmaxf(top, sm_m[w]);
  const float ref = top == -INFINITY ? 0.f : top;
  float wt[NW], tot = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    wt[w] = exp2f(sm_m[w] - ref);
    tot = fmaf(wt[w], sm_l[w], tot);
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  for (int d = threadIdx.x; d < p.D; d += 32 * NW) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v = fmaf(wt[w], sm_o[w][d], v);
    v = top == -INFINITY ? 0.f : v * inv;
    if constexpr (sizeof(T) == 2)
      dst[d] = __float2bfloat16_rn(v);
    else
      dst[d] = v;
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[row * Hq + qh] = top == -INFINITY ? -INFINITY : (top + log2f(tot)) * kLn2;
}

}  // namespace

int attn_simt_tm() { return kSimtTm; }
int attn_simt_bn() { return kSimtBn; }

cudaError_t attn_simt_launch(const AttnParams& p, spec_dtype dtype, int grid, cudaStream_t stream) {
  return dtype == SPEC_BF16 ? simt_launch<AttnParams, __nv_bfloat16>(p, grid, stream)
                            : simt_launch<AttnParams, float>(p, grid, stream);
}

cudaError_t attn_join_launch(const AttnParams& p, spec_dtype dtype, int sms, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.B) * p.R * p.Hkv * p.G;
  if (rows > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const bool many = rows >= 4 * static_cast<int64_t>(sms);  // both sides measured at the kernel
  const dim3 g(static_cast<unsigned>(many ? (rows + 3) / 4 : rows)), t(many ? 128 : 256);
  if (dtype == SPEC_BF16)
    return many ? launch_pdl(attn_join_kernel<__nv_bfloat16, 1>, g, t, 0, stream, p)
                : launch_pdl(attn_join_kernel<__nv_bfloat16, 8>, g, t, 0, stream, p);
  return many ? launch_pdl(attn_join_kernel<float, 1>, g, t, 0, stream, p)
              : launch_pdl(attn_join_kernel<float, 8>, g, t, 0, stream, p);
}

}  // namespace spec
