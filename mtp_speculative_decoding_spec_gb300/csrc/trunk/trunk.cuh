// Launch parameters of the trunk's token mixers: the gated delta rule and attention over a shared
// prefix (the files of this folder).
#pragma once

#include "host.cuh"
#include "params.cuh"

namespace spec {

enum : int { DELTA_PREFILL = 3 };  // beside the SPEC_COMMIT_* modes of a verify pass

struct DeltaParams {
  int B, R, H, Hk, dk, dv, layer, layers, n_slots;
  int mode;                 // SPEC_COMMIT_* or DELTA_PREFILL
  const void *q, *k, *v;
  int64_t qs, ks, vs, os;   // elements between rows
  const float *g, *beta;    // [rows][H]
  float scale;
  void* out;
  int vec_qk, vec_v, vec_o; // the rows of q and k, of v, of out are whole aligned vectors
  const int32_t* n_rows;    // [B] or null (a verify pass)
  const int32_t* cu_rows;   // [B + 1] (prefill)
  int64_t rows;             // rows of the inputs (prefill)
  const float* init;        // state before the rows (prefill; null: zeros)
  float* live;
  float* slots;
  const int32_t* live_slot;
  float *step_a, *step_b, *step_c;
  WsHeader* hdr;            // prefill: the workspace's, its error word cleared by each call
};

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// A bounded wait by a whole warp, whose branches stay uniform: 38 cycles when the phase is over, 105 when
// each lane decides for itself.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t n = 1;; ++n) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((n & 63u) == 0 && __any_sync(0xffffffffu, globaltimer_ns() - t0 > 2000000000ull)) return false;
  }
}

cudaError_t delta_scan_launch(const DeltaParams& p, spec_dtype dtype, int sms, cudaStream_t stream);

constexpr int kDeltaChunkRows = 32;
bool delta_chunk_sizes(int dk, int dv);
size_t delta_chunk_workspace(int64_t rows, int B, int H);
bool delta_chunk_takes(const DeltaParams& p, spec_dtype dtype);
spec_status delta_chunk_launch(const DeltaParams& p, void* workspace, EncodeTiledFn encode,
                               cudaStream_t stream);

// Attention of verify rows over a shared prefix and each request's own cache. The work is cut into
// units: a tile of `tm` rows and a KV head over the positions of one region. Prefix tiles hold the
// rows of all requests stacked (s = (b R + r) G + g), own tiles the R G rows of one request. A unit
// is cut into blocks of `bn` positions; the blocks of all units in a row are dealt out evenly to
// the grid, and each (CTA, unit) that meet leave one partial (max, sum, unnormalised output) in a
// slot of their own. Item = a tile of rows for all KV heads: prefix tiles first, then own tiles.
// With `grp` > 1, prefix items are `grp` tiles each and are dealt to groups of as many neighbouring
// CTAs, a tile to a CTA, before the own items are dealt to single CTAs: a group walks the same
// positions at the same pace, so the prefix comes from HBM once and from L2 for the others. `over`
// is what starting a prefix unit and an own unit costs, in blocks: it counts in the dealing as if the unit
// began with that many blocks more (a prefix tile has four times the rows of queries and partials here).
struct AttnParams {
  int B, R, G, Hkv, D;
  int tm, bn;
  int npt, npi, nown, items;  // prefix tiles and items, own tiles per request, npi + B * nown
  int grp, over[2];
  const void* q;
  int64_t qs;
  void* out;
  int64_t os;
  float scale_log2;         // scale * log2(e)
  const uint8_t *pk, *pv;   // prefix
  int64_t pcap, pstride;    // positions, bytes between positions
  const int64_t* prefix_len;
  const uint8_t *kk, *kv;   // own caches (of request 0, this layer)
  int64_t kreq, kcap, krow; // bytes between requests, positions, bytes between positions
  const int64_t* kv_len;
  const int32_t* n_rows;
  float* lse;
  WsHeader* hdr;
  int2* units;              // [items * Hkv]: each unit's first slot and number of partials
  float2* ml;               // [slots][tm]: running max (log2 domain) and sum
  float* o;                 // [slots][tm][D]
};

constexpr int kAttnMaxItems = 8192;  // four bytes each in shared memory, beside what a block holds
constexpr int64_t kAttnMaxPos = (int64_t(1) << 31) - 256;  // a block past the last one still has an int
// See `over`; own / prefix units at 0 / 0, 6 / 6, 6 / 10 and 4 / 10, us: 32 x 8 rows with 700 own positions each
// over a prefix of 2,000 (100 own) 34.0, 33.8, 31.3, 30.6; of 15,360 87.9, 77.0, 75.5, 72.2; of 63,488 195.7,
// 190.1, 189.0, 190.7; 64 rows over 63,488 76.0, 73.1, 70.3, 70.7; two rows over their own 63,488 52.5, 50.6,
// 50.4, 51.2.
constexpr int kAttnOver = 6, kAttnOverPre = 10;
// On CUDA cores (blocks of 32 positions): 1 to 4 81-84 us, 6 87 (4 x 8 fp32 rows of 12 heads of 128 dims over
// 3,000 shared and 2,000 own positions).
constexpr int kAttnSimtOver = 2;
// The most of `grp`. 256 rows (8 tiles) over 63,488 positions, groups of 1, 4 and 8: 211, 194 and 192 us;
// 40 rows of 4 heads (2 tiles) singly and in pairs: 104 and 68 us.
constexpr int kAttnGroup = 16;

// Of request b: the rows that run, the positions of the prefix it sees and of its own cache before them.
struct AttnReq {
  int rows, prefix, base;
};
__device__ __forceinline__ AttnReq attn_req(const AttnParams& p, int b) {
  const int64_t base = p.kv_len[b], prefix = p.prefix_len ? p.prefix_len[b] : p.pcap;
  AttnReq r;
  r.rows = p.n_rows ? max(0, min(p.n_rows[b], p.R)) : p.R;
  r.prefix = static_cast<int>(max(static_cast<int64_t>(0), min(prefix, p.pcap)));
  r.base = static_cast<int>(max(static_cast<int64_t>(0), min(base, p.kcap)));
  return r;
}
__device__ __forceinline__ int attn_own(const AttnParams& p, const AttnReq& r, int rows) {
  return min(r.base + rows, static_cast<int>(p.kcap));
}
__host__ __device__ constexpr size_t attn_plan_bytes(int items, int B) {
  return sizeof(int32_t) * (items + 1) + sizeof(AttnReq) * B;
}

// cum[0..items] in shared memory: cost of one KV head before each item, in blocks; after it the
// requests' numbers. By the whole block (a barrier at the end). Every CTA works it out for itself from
// the lengths on the device, so no launch comes before and no host reads them.
__device__ __forceinline__ AttnReq* attn_plan(const AttnParams& p, int32_t* cum) {
  const int tid = threadIdx.x, nt = blockDim.x, per = p.R * p.G;
  AttnReq* req = reinterpret_cast<AttnReq*>(cum + p.items + 1);
  const auto cost = [&p](int n, int own) { return n > 0 ? (n + p.bn - 1) / p.bn + p.over[own] : 0; };
  for (int b = tid; b < p.B; b += nt) {
    const AttnReq r = attn_req(p, b);
    req[b] = r;
    const int c = r.rows > 0 ? cost(attn_own(p, r, r.rows), 1) : 0;
    for (int j = 0; j < p.nown; ++j) cum[p.npi + b * p.nown + j + 1] = c;
  }
  __syncthreads();
  for (int i = tid >> 5; i < p.npi; i += nt >> 5) {  // a warp to an item
    const int span = p.tm * p.grp;
    const int b0 = i * span / per, b1 = min(p.B - 1, ((i + 1) * span - 1) / per);
    int n = 0;
    for (int b = b0 + (tid & 31); b <= b1; b += 32)
      if (req[b].rows > 0) n = max(n, req[b].prefix);
    n = __reduce_max_sync(0xffffffffu, n);
    if ((tid & 31) == 0) cum[i + 1] = cost(n, 0);
  }
  if (tid == 0) cum[0] = 0;
  __syncthreads();
  if (tid < 32) {
    int base = 0;
    for (int i0 = 1; i0 <= p.items; i0 += 32) {
      const int i = i0 + tid;
      int v = i <= p.items ? cum[i] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (tid >= o) v += x;
      }
      v += base;
      if (i <= p.items) cum[i] = v;
      base = __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  return req;
}

// How the costs are dealt out: the groups' part [0, wp), `sp` to each group, and the rest up to w: `s1`
// to each of the `in` CTAs in groups, `s2` to each of the others, which have that much more room; where
// the second part's units and slots begin.
struct AttnShares {
  int64_t wp, w, sp, s1, s2;
  int in, u1, base1;
  __device__ __forceinline__ int64_t single_at(int cta) const {  // where a CTA's part of the rest begins
    return cta < in ? s1 * cta : s1 * in + s2 * (cta - in);
  }
  __device__ __forceinline__ int single_cta(int64_t x) const {  // which CTA has place x of the rest
    return static_cast<int>(x < s1 * in ? x / s1 : in + (x - s1 * in) / s2);
  }
  // With so many groups: the shares, and what the CTA with the most then has. A second unit's start
  // comes on top where the groups' CTAs take some of the rest too.
  __device__ __forceinline__ int64_t split(const AttnParams& p, int groups, int grid) {
    in = groups * p.grp;
    sp = (wp + groups - 1) / groups;
    const int64_t rest = w - wp, more = rest - sp * (grid - in);
    s1 = more > 0 ? (more + grid - 1) / grid : 0;
    s2 = more > 0 ? s1 + sp : in < grid ? (rest + grid - in - 1) / (grid - in) : 0;
    return s1 > 0 ? sp + s1 + p.over[1] : max(sp, s2);
  }
};
__device__ __forceinline__ AttnShares attn_shares(const AttnParams& p, const int32_t* cum) {
  AttnShares s;
  const int grid = gridDim.x;
  s.w = static_cast<int64_t>(cum[p.items]) * p.Hkv;
  s.wp = s.sp = 0;
  s.in = 0;
  int groups = 0;
  if (p.grp > 1) {
    // as many groups as the prefix is of the work, so that a CTA has one kind of work, or one more
    s.wp = static_cast<int64_t>(cum[p.npi]) * p.Hkv;
    const int64_t all = s.wp * p.grp + s.w - s.wp;
    const int most = grid / p.grp;
    groups = all > 0 ? max(1, static_cast<int>(s.wp * grid / all)) : 1;
    const int64_t fewer = s.split(p, groups, grid);
    if (groups < most) {
      AttnShares more = s;
      if (more.split(p, groups + 1, grid) < fewer) {
        s = more;
        ++groups;
      }
    }
  } else {
    s.s1 = s.s2 = (s.w + grid - 1) / grid;
  }
  s.u1 = p.grp > 1 ? p.npi * p.Hkv : 0;
  s.base1 = p.grp * (groups + s.u1);
  return s;
}

// Each unit's first slot and number of partials (the slots of a group's tile lie `grp` apart), for the
// join; by CTA 0 of the kernel that computes them.
__device__ __forceinline__ void attn_write_units(const AttnParams& p, const int32_t* cum,
                                                 const AttnShares& s) {
  for (int u = threadIdx.x; u < p.items * p.Hkv; u += blockDim.x) {
    const int item = u / p.Hkv, head = u - item * p.Hkv;
    const int cost = cum[item + 1] - cum[item];
    int2 v = make_int2(0, 0);
    if (cost > 0) {
      const int64_t x = static_cast<int64_t>(cum[item]) * p.Hkv + static_cast<int64_t>(head) * cost;
      const int64_t first = x + p.over[item >= p.npi], last = x + cost - 1;  // places of its first and last block
      if (u < s.u1) {
        const int c0 = static_cast<int>(first / s.sp);
        v = make_int2(p.grp * (c0 + u), static_cast<int>(last / s.sp) - c0 + 1);
      } else {
        const int c0 = s.single_cta(first - s.wp);
        v = make_int2(s.base1 + c0 + u - s.u1, s.single_cta(last - s.wp) - c0 + 1);
      }
    }
    p.units[u] = v;
  }
}

// A CTA's piece of one unit: its tile of rows (prefix tiles, then own tiles), KV head, blocks and slot.
struct AttnPiece {
  int tile, head, blk0, blk1, slot;
};

// One piece after another of a CTA's shares. Only the start of a share is looked for; from there on the
// next unit follows.
struct AttnWalk {
  int64_t left;        // costs of the share still to walk
  int item, head, at;  // the unit, and where in its costs
  bool group;          // the groups' part is being walked
  __device__ __forceinline__ void seek(const AttnParams& p, const int32_t* cum, int64_t x, int64_t x1) {
    left = x1 - x;
    if (left <= 0) return;
    int lo = 0, hi = p.items;  // cum[lo] Hkv <= x < cum[hi] Hkv
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (static_cast<int64_t>(cum[mid]) * p.Hkv <= x)
        lo = mid;
      else
        hi = mid;
    }
    const int64_t rel = x - static_cast<int64_t>(cum[lo]) * p.Hkv;
    item = lo;
    head = static_cast<int>(rel / (cum[lo + 1] - cum[lo]));
    at = static_cast<int>(rel - static_cast<int64_t>(head) * (cum[lo + 1] - cum[lo]));
  }
  __device__ __forceinline__ void start(const AttnParams& p, const int32_t* cum, const AttnShares& s) {
    group = static_cast<int>(blockIdx.x) < s.in;
    if (group) {
      const int64_t x = s.sp * (blockIdx.x / p.grp);
      seek(p, cum, x, min(s.wp, x + s.sp));
    } else {
      single(p, cum, s);
    }
  }
  __device__ __forceinline__ void single(const AttnParams& p, const int32_t* cum, const AttnShares& s) {
    group = false;
    const int cta = blockIdx.x;
    const int64_t x = s.wp + s.single_at(cta);
    seek(p, cum, x, min(s.w, s.wp + s.single_at(cta + 1)));
  }
  __device__ __forceinline__ bool next(const AttnParams& p, const int32_t* cum, const AttnShares& s,
                                       AttnPiece& a) {
    for (;;) {
      if (left <= 0) {
        if (!group) return false;
        single(p, cum, s);
        continue;
      }
      const int cost = cum[item + 1] - cum[item];
      if (at >= cost) {  // the next unit, past items without positions
        at = 0;
        if (++head == p.Hkv || cost == 0) {
          head = 0;
          ++item;
        }
        continue;
      }
      const int v0 = at, v1 = static_cast<int>(min(static_cast<int64_t>(cost), v0 + left));
      at = v1;
      left -= v1 - v0;
      const int over = p.over[item >= p.npi];
      a.blk0 = max(0, v0 - over);
      a.blk1 = max(0, v1 - over);
      if (a.blk0 == a.blk1) continue;
      a.head = head;
      const int u = item * p.Hkv + head;
      if (group) {
        const int at_group = static_cast<int>(blockIdx.x) / p.grp, rank = blockIdx.x - at_group * p.grp;
        a.tile = item * p.grp + rank;
        if (a.tile >= p.npt) continue;  // the last group of tiles is not full
        a.slot = p.grp * (at_group + u) + rank;
      } else {
        a.tile = item < p.npi ? item : item - p.npi + p.npt;
        a.slot = s.base1 + static_cast<int>(blockIdx.x) + u - s.u1;
      }
      return true;
    }
  }
};

// Row i of a tile: its request, row and query head in the group, and the positions it sees (0: it
// does not run, or there is no such row).
struct AttnRow {
  int b, r, g, lim;
};
__device__ __forceinline__ AttnRow attn_row(const AttnParams& p, const AttnReq* req, int tile, int i) {
  AttnRow a;
  a.b = a.r = a.g = a.lim = 0;
  const int per = p.R * p.G;
  if (tile < p.npt) {
    const int s = tile * p.tm + i;
    if (s >= p.B * per) return a;
    a.b = s / per;
    const int x = s - a.b * per;
    a.r = x / p.G;
    a.g = x - a.r * p.G;
    if (a.r < req[a.b].rows) a.lim = req[a.b].prefix;
  } else {
    const int own = tile - p.npt;
    a.b = own / p.nown;
    const int x = (own - a.b * p.nown) * p.tm + i;
    if (x >= per) return a;
    a.r = x / p.G;
    a.g = x - a.r * p.G;
    if (a.r < req[a.b].rows) a.lim = attn_own(p, req[a.b], a.r + 1);
  }
  return a;
}

cudaError_t attn_simt_launch(const AttnParams& p, spec_dtype dtype, int grid, cudaStream_t stream);
cudaError_t attn_join_launch(const AttnParams& p, spec_dtype dtype, int sms, cudaStream_t stream);
int attn_simt_tm();
int attn_simt_bn();
// Head sizes of the tensor-core kernel, bf16 alone. On the CUDA cores two rows over 63,488 positions of 256
// dims take 206 us for 51, 32 rows of 64 dims over 15,360 224 for 20; two rows of 64 dims over 258 8.4 for
// 9.7, which is not worth a limit on lengths that the host does not know.
bool attn_tc_takes(int head_dim);
spec_status attn_tc_launch(const AttnParams& p, int grid, EncodeTiledFn encode, cudaStream_t stream);
int attn_tc_tm();
int attn_tc_bn(int head_dim);

}  // namespace spec
