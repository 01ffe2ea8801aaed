// The gated delta rule of a recurrent layer, row by row: the recurrence that a verify pass runs
// over its 1..8 rows, and the state that the commit keeps or drops.
//
//   S~ = a S,  u = beta (v - S~^T k),  S' = S~ + k u^T,  o = scale S'^T q     (a = exp(log_decay))
//
// The update is the commit's own step S <- fl(fl(a S) + fl(b c^T)) with b = k and c = u, each
// operation rounded separately, so a state replayed from (a, k, u) has the snapshots' bytes
// (DS4Server issue #98, section "Implementation": only the accepted rows are committed or replayed).
//
// Every column of S is a recurrence of its own (u_j needs column j alone), so a warp owns a tile
// of 4 LV columns and all dk rows in registers: LV lanes side by side hold four columns each,
// 32 / LV groups of lanes hold NI consecutive rows each. A row costs two dot products per column,
// taken together over S~ (o = scale (S~^T q + (k.q) u)), one butterfly over the groups, and
// the rank-one update; no block barrier. Rows come in groups of eight through the warp's own piece of
// shared memory, the next group's copies in flight while one is computed: a verify pass waits for
// memory once, not once a row. Bound by the state's bytes when there are many requests (read once, one
// write per snapshot), by the latency of the row chain when there are few. 16 heads of [128, 128], bf16
// rows: 32 requests x up to 8 rows, snapshots 40.5 us = 5.4 TB/s (0.80 of a copy's 6.79); replay, which
// moves a third of that, 26.5 us = 2.7 TB/s, two and a half turns of the warps that fit, each load,
// row chain and store one after another; 1 x 8 rows, index 6.4 us. (Turns of one set of warps, the next
// tile's state copied ahead to shared memory: replay 34.5 us, snapshots 45.0.)
#include <math.h>

#include <cuda_bf16.h>

#include "trunk.cuh"

namespace spec {
namespace {

using f2 = unsigned long long;  // two fp32 lanes

__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 pair(float x, float y) {
  return pack2(__float_as_uint(x), __float_as_uint(y));
}
__device__ __forceinline__ float2 unpair(f2 v) {
  uint32_t x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(v));
  return make_float2(__uint_as_float(x), __uint_as_float(y));
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// N consecutive elements: whole vectors where the caller says they are aligned and present, else
// one at a time, zero from `have` on.
template <typename T, int N>
struct Raw {
  static constexpr int kBytes = N * static_cast<int>(sizeof(T));
  alignas(kBytes < 16 ? kBytes : 16) T e[N];
  __device__ __forceinline__ void shared(const T* p) {  // aligned to its own size, at most 16 bytes
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4*>(e)[i] = reinterpret_cast<const uint4*>(p)[i];
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(e) = *reinterpret_cast<const uint32_t*>(p);
    } else {
      e[0] = p[0];
    }
  }
  __device__ __forceinline__ void store_shared(T* p) const {  // neighbours' values begin where these end
    static_assert(sizeof(Raw) == kBytes && (kBytes == 8 || kBytes == 16), "one aligned store of just this");
    if constexpr (kBytes == 16)
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(e);
    else
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(e);
  }
  __device__ __forceinline__ void load(const T* p, bool vec, int have) {
    if (vec && have >= N) {
      if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
          reinterpret_cast<uint4*>(e)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
      } else if constexpr (kBytes == 8) {
        *reinterpret_cast<uint2*>(e) = __ldg(reinterpret_cast<const uint2*>(p));
      } else if constexpr (kBytes == 4) {
        *reinterpret_cast<uint32_t*>(e) = __ldg(reinterpret_cast<const uint32_t*>(p));
      } else {
        e[0] = p[0];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = i < have ? p[i] : from_f<T>(0.f);
    }
  }
};

constexpr int kGroup = 8;  // rows staged at once

// A warp's shared memory: q and k of a group (one or two of them in flight), v, decay and beta.
template <typename T, int NI, int LV>
struct Staged {
  static constexpr int kP = 32 / LV * NI;  // dk, filled up to the lanes' rows
  static constexpr int kQk = kGroup * kP * static_cast<int>(sizeof(T));
  static constexpr int kV = kGroup * 4 * LV * static_cast<int>(sizeof(T));
  static constexpr int bytes(int bufs) { return 2 * bufs * kQk + kV + 2 * kGroup * 4; }
};

// One warp to a block: no warp needs another, and warps that end make room one by one. Blocks an SM: as
// many as the state's registers allow. With many requests it is the warps in flight that count (32
// requests x 8 rows of [128, 128]: replay 32.1 us with eight, 26.5 with eleven; snapshots 47.4 and 40.6).
// Of the tiles with fewer rows a lane, more than 16 do not help (1 x 8 rows, index: 6.4 us, 7.6 with 24).
template <typename T, int NI>
constexpr int kScanBlocks = NI >= 16 ? (sizeof(T) == 2 ? 11 : 10) : 16;

template <typename T, int NI, int LV>
__global__ void __launch_bounds__(32, kScanBlocks<T, NI>)
    delta_scan_kernel(const __grid_constant__ DeltaParams p, int bufs) {
  using St = Staged<T, NI, LV>;
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_wait();
  if (p.hdr && blockIdx.x == 0 && threadIdx.x == 0) p.hdr->error = 0;  // no wait here can set it
  const int lane = threadIdx.x;
  const int tiles = (p.dv + 4 * LV - 1) / (4 * LV);
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
  const int h = bh % p.H, b = bh / p.H;
  const int kh = h / (p.H / p.Hk);
  const int col = tile * 4 * LV + (lane % LV) * 4;
  const int i0 = (lane / LV) * NI;
  const bool lead = lane < LV;  // the lanes that write rows of dv values
  const bool on = col < p.dv;
  const int have = min(NI, max(0, p.dk - i0));
  const bool prefill = p.mode == DELTA_PREFILL;

  // the request's rows
  int64_t row0;
  int n, R;
  if (prefill) {
    const int64_t lo = max(static_cast<int64_t>(0),
                           min(static_cast<int64_t>(p.cu_rows[b]), p.rows));
    const int64_t hi = max(lo, min(static_cast<int64_t>(p.cu_rows[b + 1]), p.rows));
    row0 = lo;
    R = n = static_cast<int>(hi - lo);
  } else {
    row0 = static_cast<int64_t>(b) * p.R;
    R = p.R;
    n = p.n_rows ? max(0, min(p.n_rows[b], p.R)) : p.R;
  }
  int slot = 0;
  if (p.mode == SPEC_COMMIT_INDEX) {
    slot = p.live_slot[b];
    if (slot < 0 || slot >= p.n_slots) {  // no live state: no row runs
      slot = 0;
      n = 0;
    }
  }
  // the first group's rows and the state, all in flight together
  uint8_t* sv = smem + 2 * bufs * St::kQk;
  float* sa = reinterpret_cast<float*>(sv + St::kV);
  float* sb = sa + kGroup;
  const T* qp = static_cast<const T*>(p.q) + row0 * p.qs + static_cast<int64_t>(kh) * p.dk;
  const T* kp = static_cast<const T*>(p.k) + row0 * p.ks + static_cast<int64_t>(kh) * p.dk;
  const T* vp = static_cast<const T*>(p.v) + row0 * p.vs + static_cast<int64_t>(h) * p.dv;
  T* op = static_cast<T*>(p.out) + row0 * p.os + static_cast<int64_t>(h) * p.dv + col;
  Raw<T, 4> vn;  // row lane / LV of the group (in the first 8 LV lanes)
  float gn = 0.f, bn = 0.f;
  auto fetch = [&](int r0, int buf) {
    constexpr int kE = 16 / static_cast<int>(sizeof(T));
    T* sq = reinterpret_cast<T*>(smem + 2 * buf * St::kQk);
    T* sk = sq + kGroup * St::kP;
    if (p.vec_qk) {
      for (int i = lane; i < kGroup * St::kP / kE; i += 32) {
        const int r = i / (St::kP / kE), d = (i % (St::kP / kE)) * kE;
        if (r0 + r < n && d < p.dk) {
          copy_async16(sq + r * St::kP + d, qp + (r0 + r) * p.qs + d);
          copy_async16(sk + r * St::kP + d, kp + (r0 + r) * p.ks + d);
        } else {
          *reinterpret_cast<uint4*>(sq + r * St::kP + d) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(sk + r * St::kP + d) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    } else {
      for (int i = lane; i < kGroup * St::kP; i += 32) {
        const int r = i / St::kP, d = i % St::kP;
        const bool there = r0 + r < n && d < p.dk;
        sq[i] = there ? qp[(r0 + r) * p.qs + d] : from_f<T>(0.f);
        sk[i] = there ? kp[(r0 + r) * p.ks + d] : from_f<T>(0.f);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    const int r = r0 + lane / LV;
    vn.load(vp + r * p.vs + col, p.vec_v, lane < kGroup * LV && r < n && on ? 4 : 0);
    if (lane < kGroup && r0 + lane < n) {
      gn = __ldg(p.g + (row0 + r0 + lane) * p.H + h);
      bn = __ldg(p.beta + (row0 + r0 + lane) * p.H + h);
    }
  };
  if (n > 0) fetch(0, 0);
  // its state: elements of a request's state (or of a slot), of this layer and head in it
  const int64_t elems = static_cast<int64_t>(p.layers) * p.H * p.dk * p.dv;
  const int64_t off = (static_cast<int64_t>(p.layer) * p.H + h) * p.dk * p.dv +
                      static_cast<int64_t>(i0) * p.dv + col;
  const float* src = prefill ? (p.init ? p.init + b * elems + off : nullptr)
                     : p.mode == SPEC_COMMIT_INDEX
                         ? p.slots + (static_cast<int64_t>(b) * p.n_slots + slot) * elems + off
                         : p.live + b * elems + off;
  f2 s[NI][2];
#pragma unroll
  for (int ii = 0; ii < NI; ++ii) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on && ii < have && src) x = *reinterpret_cast<const float4*>(src + static_cast<int64_t>(ii) * p.dv);
    s[ii][0] = pair(x.x, x.y);
    s[ii][1] = pair(x.z, x.w);
  }
  auto store_state = [&](float* dst) {
#pragma unroll
    for (int ii = 0; ii < NI; ++ii) {
      const float2 x = unpair(s[ii][0]), y = unpair(s[ii][1]);
      if (on && ii < have)
        __stcs(reinterpret_cast<float4*>(dst + static_cast<int64_t>(ii) * p.dv),
               make_float4(x.x, x.y, y.x, y.y));
    }
  };
  float* slots = p.slots + static_cast<int64_t>(b) * p.n_slots * elems + off;
  if (p.mode == SPEC_COMMIT_SNAPSHOT || p.mode == SPEC_COMMIT_REPLAY)  // slot 0: before the cycle
    store_state(slots);

  int to = slot;
  for (int r0 = 0; r0 < n; r0 += kGroup) {
    const int buf = bufs == 2 ? (r0 / kGroup) & 1 : 0;
    if (lane < kGroup * LV) vn.store_shared(reinterpret_cast<T*>(sv) + lane * 4);
    if (lane < kGroup) {
      sa[lane] = expf(gn);
      sb[lane] = bn;
    }
    if (r0 + kGroup < n) {  // only with two buffers
      fetch(r0 + kGroup, buf ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    const T* sq = reinterpret_cast<const T*>(smem + 2 * buf * St::kQk) + i0;
    const T* sk = sq + kGroup * St::kP;
    const int rows = min(kGroup, n - r0);
    for (int r = 0; r < rows; ++r) {
      Raw<T, NI> qr, kr;
      Raw<T, 4> vr;
      qr.shared(sq + r * St::kP);
      kr.shared(sk + r * St::kP);
      vr.shared(reinterpret_cast<const T*>(sv) + (r * LV + lane % LV) * 4);
      const float a = sa[r], beta = sb[r];
      const f2 a2 = pair(a, a);
      f2 ks0 = 0, ks1 = 0, qs0 = 0, qs1 = 0;
      float qk = 0.f;
#pragma unroll
      for (int ii = 0; ii < NI; ++ii) {
        const float kf = to_f(kr.e[ii]), qf = to_f(qr.e[ii]);
        const f2 k2 = pair(kf, kf), q2 = pair(qf, qf);
        s[ii][0] = mul2(s[ii][0], a2);
        s[ii][1] = mul2(s[ii][1], a2);
        ffma2_acc(ks0, k2, s[ii][0]);
        ffma2_acc(ks1, k2, s[ii][1]);
        ffma2_acc(qs0, q2, s[ii][0]);
        ffma2_acc(qs1, q2, s[ii][1]);
        qk = fmaf(kf, qf, qk);
      }
#pragma unroll
      for (int o = LV; o < 32; o <<= 1) {
        ks0 = add2(ks0, __shfl_xor_sync(0xffffffffu, ks0, o));
        ks1 = add2(ks1, __shfl_xor_sync(0xffffffffu, ks1, o));
        qs0 = add2(qs0, __shfl_xor_sync(0xffffffffu, qs0, o));
        qs1 = add2(qs1, __shfl_xor_sync(0xffffffffu, qs1, o));
        qk += __shfl_xor_sync(0xffffffffu, qk, o);
      }
      const float2 ka = unpair(ks0), kb = unpair(ks1), qa = unpair(qs0), qb = unpair(qs1);
      float u[4];
      u[0] = beta * (to_f(vr.e[0]) - ka.x);
      u[1] = beta * (to_f(vr.e[1]) - ka.y);
      u[2] = beta * (to_f(vr.e[2]) - kb.x);
      u[3] = beta * (to_f(vr.e[3]) - kb.y);
      if (lead && on) {
        T* dst = op + static_cast<int64_t>(r0 + r) * p.os;
        alignas(16) T o4[4];
        o4[0] = from_f<T>(p.scale * fmaf(qk, u[0], qa.x));
        o4[1] = from_f<T>(p.scale * fmaf(qk, u[1], qa.y));
        o4[2] = from_f<T>(p.scale * fmaf(qk, u[2], qb.x));
        o4[3] = from_f<T>(p.scale * fmaf(qk, u[3], qb.y));
        if (p.vec_o) {
          if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(o4);
          else
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(o4);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[j] = o4[j];
        }
      }
      __syncwarp();  // so that the key is read anew: held since the dot products it would cost registers
      kr.shared(sk + r * St::kP);
#pragma unroll
      for (int ii = 0; ii < NI; ++ii) {
        const float kf = to_f(kr.e[ii]);
        // scalar products: a packed product and sum come out fused, which rounds once only
        s[ii][0] = add2(s[ii][0], pair(__fmul_rn(kf, u[0]), __fmul_rn(kf, u[1])));
        s[ii][1] = add2(s[ii][1], pair(__fmul_rn(kf, u[2]), __fmul_rn(kf, u[3])));
      }
      if (p.mode == SPEC_COMMIT_SNAPSHOT || p.mode == SPEC_COMMIT_INDEX) {
        if (++to == p.n_slots) to = 0;
        store_state(slots + to * elems);
      } else if (p.mode == SPEC_COMMIT_REPLAY) {
        const int64_t lh =
            ((static_cast<int64_t>(b) * (p.n_slots - 1) + r0 + r) * p.layers + p.layer) * p.H + h;
        if (lead && on)
          *reinterpret_cast<float4*>(p.step_c + lh * p.dv + col) = make_float4(u[0], u[1], u[2], u[3]);
        if (tile == 0 && lane % LV == 0) {
#pragma unroll
          for (int ii = 0; ii < NI; ++ii)
            if (ii < have) p.step_b[lh * p.dk + i0 + ii] = to_f(kr.e[ii]);
          if (lane == 0) p.step_a[lh] = a;
        }
      }
    }
    __syncwarp();  // the group's rows are read
  }
  if (prefill) {
    store_state(p.live + b * elems + off);
  } else if (lead && on) {  // rows the request does not run
    for (int r = n; r < R; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) op[static_cast<int64_t>(r) * p.os + j] = from_f<T>(0.f);
  }
}

template <typename T, int NI, int LV>
cudaError_t launch_scan(const DeltaParams& p, cudaStream_t stream) {
  static SmemAllowance allowed;
  const int64_t tiles = (p.dv + 4 * LV - 1) / (4 * LV);
  const int64_t blocks = tiles * p.H * p.B;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int bufs = p.mode == DELTA_PREFILL ? 2 : 1;
  const int smem = Staged<T, NI, LV>::bytes(bufs);
  const cudaError_t e = allow_dynamic_smem(delta_scan_kernel<T, NI, LV>, smem, allowed);
  if (e != cudaSuccess) return e;
  return launch_pdl(delta_scan_kernel<T, NI, LV>, dim3(static_cast<unsigned>(blocks)), dim3(32), smem,
                    stream, p, bufs);
}

template <typename T>
cudaError_t scan_of(const DeltaParams& p, int sms, cudaStream_t stream) {
  // Tiles of 8 columns instead of 16 while 16-column tiles would not give every SM two warps: the row chain
  // is half as long for the same work in total. 16 heads of [128, 128] x 8 rows, index, tiles of 8 and of
  // 16 columns: one request 6.4 and 8.8 us, two 7.5 and 8.9, three 9.4 and 9.0, four 10.5 and 9.6; 32
  // requests, replay, 32.8 and 26.5. A lane's rows follow rec_dk, so that no registers hold nothing.
  const int64_t warps = static_cast<int64_t>((p.dv + 15) / 16) * p.H * p.B;
  if (warps < 2 * sms && p.dk <= 128) {
    if (p.dk <= 16) return launch_scan<T, 1, 2>(p, stream);
    if (p.dk <= 64) return launch_scan<T, 4, 2>(p, stream);
    return launch_scan<T, 8, 2>(p, stream);
  }
  if (p.dk <= 16) return launch_scan<T, 2, 4>(p, stream);
  if (p.dk <= 64) return launch_scan<T, 8, 4>(p, stream);
  if (p.dk <= 128) return launch_scan<T, 16, 4>(p, stream);
  return launch_scan<T, 16, 2>(p, stream);  // 256 rows: a warp's registers hold 8 columns
}

}  // namespace

cudaError_t delta_scan_launch(const DeltaParams& p, spec_dtype dtype, int sms,
                              cudaStream_t stream) {
  return dtype == SPEC_BF16 ? scan_of<__nv_bfloat16>(p, sms, stream) : scan_of<float>(p, sms, stream);
}

}  // namespace spec
