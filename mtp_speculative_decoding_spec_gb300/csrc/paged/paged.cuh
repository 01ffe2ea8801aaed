// Launch parameters of the paged KV cache's calls, and what attention's kernels (trunk/attn.cuh,
// trunk/attn_tc.cuh) ask of them.
#pragma once

#include <cuda_bf16.h>

#include "trunk/trunk.cuh"

namespace spec {

constexpr int kPagedMaxB = 512, kPagedMaxHeads = 65536;
constexpr int kPagedMaxTiles = 4096, kPagedSimtMaxTiles = 12288;  // four bytes each in shared memory

// One layer of a paged cache.
struct PagedLayer {
  uint8_t *k, *v;
  int64_t page_stride, table_stride;
  const int32_t* table;
  int64_t* kv_len;
  int row_bytes, page_size, n_pages, max_pages;
};

// The positions in the cache before the call's rows: none where negative, and so few that no position of a row
// overflows (past the table all are alike).
__device__ __forceinline__ int64_t paged_len(const PagedLayer& c, int b) {
  return max(static_cast<int64_t>(0), min(c.kv_len[b], static_cast<int64_t>(1) << 62));
}

// Bytes from the layer's first page to a position of request b, or -1 where its page is not there.
__device__ __forceinline__ int64_t paged_offset(const PagedLayer& c, int b, int pos) {
  const int j = pos / c.page_size;
  if (j >= c.max_pages) return -1;
  const int g = __ldg(c.table + b * c.table_stride + j);
  if (g < 0 || g >= c.n_pages) return -1;
  return g * c.page_stride + static_cast<int64_t>(pos - j * c.page_size) * c.row_bytes;
}

// How many of the requests' ends cu[1..B] lie at or before a row: the request of a row that has one. By a
// whole warp; B at most 1,024.
__device__ __forceinline__ int paged_request_of(const int32_t* cu, int B, int64_t row) {
  const int lane = threadIdx.x & 31;
  int first = 0;
  if (B > 32) {
    const int i = 32 * (lane + 1);
    first = 32 * __popc(__ballot_sync(0xffffffffu, i <= B && cu[min(i, B)] <= row));
  }
  const int i = first + lane + 1;
  return first + __popc(__ballot_sync(0xffffffffu, i <= B && cu[min(i, B)] <= row));
}

// Request b's rows: where they begin, how many it owns and how many of them run.
struct PagedRows {
  int start, owned, runs;
};
__device__ __forceinline__ PagedRows paged_rows(const int32_t* cu, const int32_t* n_rows, int64_t rows, int b) {
  const int total = static_cast<int>(rows);
  PagedRows r;
  r.start = max(0, min(cu[b], total));
  r.owned = max(r.start, min(cu[b + 1], total)) - r.start;
  r.runs = n_rows ? max(0, min(n_rows[b], r.owned)) : r.owned;
  return r;
}

constexpr int kPagedMaxCtas = 512;

// Tiles of a request that walk the same positions side by side (152 SMs are 19 eights), and above how many
// positions that its rows see in the mean. 2,048 rows of 16 heads on 4 of 256 dims over 61,440 positions, groups of
// 1, 4, 8, 16: 1,469, 1,231, 1,192, 1,197 us. With groups and without: 512 rows over 20,000 four times 259 and 338
// us (128 dims), 463 and 636 (256); 2,048 over 9,000 143 and 157; prompts of 49,152 from their start 7,588 and 8,658,
// 13,067 and 15,569; of 16,384 904 and 798, 1,386 and 1,401; of 8,192 273 and 219, 395 and 389; 4,096 rows over 6,000
// 219 and 210: from the start tiles see so much less than a group's last one, and groups take no whole units.
constexpr int kPagedGroup = 8, kPagedGroupMin = 8192;

// `over` on the tensor cores (trunk.cuh), for grouped tiles (4 to 16: no difference) and single ones. All units
// cut, 6, 9, 12, 16, 20: prompts of 1,000 and 2,311 rows among shorter ones 70.7, 65.7, 65.3, 63.7, 65.4 us, 32
// requests of 8 rows over 15,360 positions 309.5, 312.0, 311.2, 313.5, 316.6.
constexpr int kPagedOver = 12;
// On the tensor cores, what the busiest CTA may have above an equal share, in blocks, before units are cut instead.
// Where there is a CTA for every unit: what a cut costs, and where a request has no more than a tile and 128 dims
// or more the share's so-many-th part, since then HBM is the limit and fewer CTAs draw as much. 32 requests of 8
// rows over 1,000, 4,000 and 15,360 positions of 256 dims whole and cut: 31, 87, 288 and 36, 94, 309 us; 128 dims
// over 15,360 158 and 169; 64 dims, which HBM does not limit, 132 and 119; two rows over 2,000 35 and 16. Where a
// CTA has several: also the start and the partials of the units that it would have parts of, and the join. Prompts
// of 1,000 and 2,311 rows among shorter ones of 128 dims 54 and 64, 2,311 alone 42 and 53, 64 requests of 8 rows
// over 4,000 of 256 dims 140 and 149; 4,000 rows over 2,000 (28 above the share) 117 and 133. With 20, 32, 40
// allowed the last 135, 117, 117; working it out for nothing costs 2 us. On the CUDA cores nothing is gained (32
// fp32 requests over 500 positions: 121 both).
constexpr int kPagedUnitOne = 8, kPagedUnitPart = 4, kPagedUnitMore = 32;
// Of so many items (each finds its place by looking at all others), and so many units a CTA, whose cuts are the
// smaller part then.
constexpr int kPagedSort = 256, kPagedRounds = 16;

struct AppendParams {
  PagedLayer c;
  int B, D;
  int nq, nk;            // query heads, and key heads, that are processed (values: as many as keys)
  int64_t rows;
  const int32_t *cu_rows, *n_rows;
  const void *q, *k, *v;
  void* q_out;
  int64_t qs, ks, vs, qos;
  int whole;             // rows of q, k, v and q_out are whole 16-byte vectors
  const float *q_norm, *k_norm;
  float eps;
  int rot;
  const float* inv_freq;
  float rot_scale;
  const int64_t* pos;
  int32_t* status;
  int tph;               // lanes of a head
  int cq, ck, iters;     // turns of a warp over a row's query heads, its key heads (its values'), all
  int per_task;          // of which a warp takes so many
};
cudaError_t append_launch(AppendParams& p, spec_dtype dtype, bool interleaved, int sms, cudaStream_t stream);

struct PagedCommitParams {
  PagedLayer c;
  int64_t layer_stride;
  int layers;
  const spec_accept_out* acc;
  const int32_t* k;
  int32_t* status;
};
cudaError_t paged_commit_launch(const PagedCommitParams& p, int B, cudaStream_t stream);

// Attention of new rows over a paged cache. A request's rows times the query heads of a KV head, stacked
// (x = r G + g), are cut into tiles; a unit is a tile and a KV head over the positions that its last row
// sees. Requests of many tiles over many positions have them in groups of `grp`, as a shared prefix has.
// Of AttnParams npt, npi, nown and items are not used but for `items`, the most tiles that there can be; a
// tile's number is its place in the request and the request.
struct PagedReq {
  int start, rows, base;  // first row, rows that run, positions before them
  int g0, s0;             // its first item of `grp` tiles, its first item of a single tile
};
struct PagedSplit;
struct PagedParams : AttnParams {
  PagedLayer c;
  const int32_t* cu_rows;
  int64_t rows;
  int tm_shift, bn_shift;    // log2 of tm and bn
  int unit_more, unit_part;  // attn_by_units (-1: never; part 0: none)
  int group_min;          // mean positions above which a request's tiles are grouped
  int page_shift;         // tensor cores: positions (log2) of a block's part on one page, 31 where that is all
  PagedSplit* splits;     // [2 CTAs]
};
template <>
inline constexpr bool kPaged<PagedParams> = true;

__device__ __forceinline__ int64_t paged_offset(const PagedParams& p, int b, int pos) {
  return paged_offset(p.c, b, pos);
}

// cum[0..items], then the counts of grouped and of all items and what the busiest CTA has with whole units (0: not
// worked out), then the requests, then the items by cost, where they are few.
__host__ __device__ inline size_t attn_plan_bytes(const PagedParams& p) {
  return sizeof(int32_t) * (p.items + 4) + sizeof(PagedReq) * p.B + sizeof(uint16_t) * kPagedSort;
}
__device__ __forceinline__ int attn_group_items(const PagedParams& p, const int32_t* cum) {
  return cum[p.items + 1];
}
__device__ __forceinline__ int attn_items(const PagedParams& p, const int32_t* cum) { return cum[p.items + 2]; }
__device__ __forceinline__ const PagedReq* paged_reqs(const PagedParams& p, const int32_t* cum) {
  return reinterpret_cast<const PagedReq*>(cum + p.items + 4);
}
__device__ __forceinline__ uint16_t* paged_order(const PagedParams& p, const int32_t* cum) {
  return reinterpret_cast<uint16_t*>(const_cast<PagedReq*>(paged_reqs(p, cum)) + p.B);
}
__device__ __forceinline__ int paged_tiles(const PagedParams& p, int rows) {
  return (rows * p.G + p.tm - 1) >> p.tm_shift;
}
__device__ __forceinline__ int paged_groups(const PagedParams& p, int rows, int base) {
  const int n = paged_tiles(p, rows);
  return p.grp > 1 && n >= p.grp && static_cast<int64_t>(base) + rows / 2 > p.group_min ? n / kPagedGroup : 0;
}
__device__ __forceinline__ int64_t attn_div(const PagedParams&, int64_t x, int64_t y) {  // all below 2^31
  return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
}
__device__ __forceinline__ int attn_part(const PagedParams&, int64_t x, int64_t all, int grid) {
  const float part = static_cast<float>(x) / static_cast<float>(all) * static_cast<float>(grid);
  return min(grid, static_cast<int>(part + 0.01f));
}
// Whole units to a CTA, where the busiest one then has no more than `unit_more` above an equal share: no unit is cut
// and the join has nothing to do.
__device__ __forceinline__ bool attn_by_units(const PagedParams& p, const int32_t* cum, int64_t share) {
  const int worst = cum[p.items + 3], items = attn_items(p, cum);
  if (worst == 0) return false;
  int64_t more = p.unit_more;
  if (items * p.Hkv <= static_cast<int>(gridDim.x))
    more = kPagedUnitOne + (p.unit_part > 0 && items <= p.B ? share / p.unit_part : 0);
  return worst <= share + more;
}
// What a request's tile sees: up to its last row's position.
__device__ __forceinline__ int paged_sees(const PagedParams& p, const PagedReq& r, int tile) {
  const int last = min(r.rows, (((tile + 1) << p.tm_shift) - 1) / p.G + 1);
  return static_cast<int>(min(p.kcap, static_cast<int64_t>(r.base) + last));
}

// The unit, the costliest first, that a CTA takes in a round.
__device__ __forceinline__ int paged_unit(int round, int cta, int grid) {
  return round * grid + (round & 1 ? grid - 1 - cta : cta);
}
// As for AttnParams: by the whole block, in shared memory, a barrier at the end. Requests whose tiles would
// be more than there can be (cu_rows not as documented) have none.
static __device__ __noinline__ const PagedReq* attn_plan(const PagedParams& p, int32_t* cum) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
  PagedReq* req = const_cast<PagedReq*>(paged_reqs(p, cum));
#pragma unroll 1
  for (int b = tid; b < p.B; b += nt) {
    const PagedRows r = paged_rows(p.cu_rows, p.n_rows, p.rows, b);
    req[b].start = r.start;
    req[b].rows = r.runs;
    req[b].base = static_cast<int>(max(static_cast<int64_t>(0), min(p.kv_len[b], p.kcap)));
  }
  __syncthreads();
  if (tid < 32) {
    int all = 0, groups = 0, singles = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      int n = b < p.B ? paged_tiles(p, req[b].rows) : 0, at = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += x;
      }
      if (all + at > p.items) n = 0;
      all = min(p.items + 1, all + __shfl_sync(0xffffffffu, at, 31));
      if (b < p.B && n == 0) req[b].rows = 0;
      const int g = b < p.B ? paged_groups(p, req[b].rows, req[b].base) : 0;
      int cg = g, cs = n - g * p.grp;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, cg, o), y = __shfl_up_sync(0xffffffffu, cs, o);
        if (lane >= o) {
          cg += x;
          cs += y;
        }
      }
      if (b < p.B) {
        req[b].g0 = groups + cg - g;
        req[b].s0 = singles + cs - (n - g * p.grp);
      }
      groups += __shfl_sync(0xffffffffu, cg, 31);
      singles += __shfl_sync(0xffffffffu, cs, 31);
    }
#pragma unroll 1
    for (int b = lane; b < p.B; b += 32) req[b].s0 += groups;
    if (lane == 0) {
      cum[0] = 0;
      cum[p.items + 1] = groups;
      cum[p.items + 2] = groups + singles;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int b = tid >> 5; b < p.B; b += nt >> 5) {  // a warp to a request
    const PagedReq r = req[b];
    const int n = paged_tiles(p, r.rows), ng = paged_groups(p, r.rows, r.base);
#pragma unroll 1
    for (int i = lane; i < ng; i += 32)
      cum[r.g0 + i + 1] = (paged_sees(p, r, (i + 1) * p.grp - 1) + p.bn - 1 >> p.bn_shift) + p.over[0];
#pragma unroll 1
    for (int t = ng * p.grp + lane; t < n; t += 32)
      cum[r.s0 + t - ng * p.grp + 1] = (paged_sees(p, r, t) + p.bn - 1 >> p.bn_shift) + p.over[1];
  }
  __syncthreads();
  if (tid < 32) {
    const int items = cum[p.items + 2];
    int base = 0, most = 0, least = 0x7fffffff;
#pragma unroll 1
    for (int i0 = 1; i0 <= items; i0 += 32) {
      const int i = i0 + lane;
      int v = i <= items ? cum[i] : 0;
      most = max(most, v);
      if (i <= items) least = min(least, v);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      v += base;
      if (i <= items) cum[i] = v;
      base = __shfl_sync(0xffffffffu, v, 31);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) {
      // 0: whole units are not for this call; 1: that is to be worked out, below
      const int64_t units = static_cast<int64_t>(items) * p.Hkv, grid = gridDim.x;
      int worst = 0;
      if (p.unit_more >= 0 && cum[p.items + 1] == 0 && items > 0) {
        if (units <= grid) {
          worst = most;
        } else if (items <= kPagedSort && units <= kPagedRounds * grid) {
          const int64_t rounds = attn_div(p, units + grid - 1, grid);
          const int64_t share = attn_div(p, static_cast<int64_t>(base) * p.Hkv + grid - 1, grid);
          worst = rounds * least <= share + p.unit_more;
        }
      }
      cum[p.items + 3] = worst;
    }
  }
  __syncthreads();
  // Whole units, the costliest first, dealt out forth and back over the grid: what the busiest CTA has then.
  if (cum[p.items + 3] == 1) {
    const int items = cum[p.items + 2], grid = gridDim.x;
    uint16_t* order = paged_order(p, cum);
#pragma unroll 1
    for (int i = tid; i < items; i += nt) {
      const int cost = cum[i + 1] - cum[i];
      int rank = 0, from = 0;
#pragma unroll 4
      for (int j = 0; j < items; ++j) {
        const int to = cum[j + 1], other = to - from;
        from = to;
        rank += other > cost || (other == cost && j < i);
      }
      order[rank] = static_cast<uint16_t>(i);
    }
    __syncthreads();
    int worst = 0;
#pragma unroll 1
    for (int cta = tid; cta < grid; cta += nt) {
      int sum = 0;
#pragma unroll 1
      for (int round = 0; round * grid < items * p.Hkv; ++round) {
        const int u = paged_unit(round, cta, grid);
        if (u >= items * p.Hkv) continue;
        const int item = order[u / p.Hkv];
        sum += cum[item + 1] - cum[item];
      }
      worst = max(worst, sum);
    }
    worst = __reduce_max_sync(0xffffffffu, worst);
    if (lane == 0) atomicMax(cum + p.items + 3, worst);
    __syncthreads();
  }
  return req;
}

constexpr int kTileReqBits = 9;
static_assert(kPagedMaxB <= 1 << kTileReqBits);
__device__ __forceinline__ int attn_tile_req(const PagedParams&, int tile) {
  return tile & ((1 << kTileReqBits) - 1);
}
// The request of an item: the last whose first one (of its kind) is not after it and that has any there.
__device__ __forceinline__ int attn_single_tile(const PagedParams& p, const int32_t* cum, int item) {
  const PagedReq* req = paged_reqs(p, cum);
  int lo = 0, hi = p.B;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (req[mid].s0 <= item)
      lo = mid;
    else
      hi = mid;
  }
  const int t = item - req[lo].s0 + paged_groups(p, req[lo].rows, req[lo].base) * p.grp;
  return t << kTileReqBits | lo;
}
__device__ __forceinline__ int attn_group_tile(const PagedParams& p, const int32_t* cum, int item, int rank) {
  const PagedReq* req = paged_reqs(p, cum);
  int lo = 0, hi = p.B;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (req[mid].g0 <= item)
      lo = mid;
    else
      hi = mid;
  }
  return ((item - req[lo].g0) * p.grp + rank) << kTileReqBits | lo;
}
// The next whole unit of a CTA (attn_by_units); `round` of them lie behind it.
__device__ __forceinline__ bool attn_next_unit(const PagedParams& p, const int32_t* cum, int& round, AttnPiece& a) {
  const int grid = gridDim.x, units = attn_items(p, cum) * p.Hkv;
#pragma unroll 1
  while (round * grid < units) {
    const int u = paged_unit(round++, blockIdx.x, grid);
    if (u >= units) continue;
    const int rank = u / p.Hkv, item = units > grid ? paged_order(p, cum)[rank] : rank;
    a.blk0 = 0;
    a.blk1 = cum[item + 1] - cum[item] - p.over[1];
    if (a.blk1 <= 0) continue;
    a.whole = true;
    a.head = u - rank * p.Hkv;
    a.tile = attn_single_tile(p, cum, item);
    a.slot = 0;
    return true;
  }
  return false;
}
__device__ __forceinline__ AttnRow attn_row(const PagedParams& p, const PagedReq* req, int tile, int i) {
  AttnRow a;
  a.b = attn_tile_req(p, tile);
  const int x = ((tile >> kTileReqBits) << p.tm_shift) + i;
  a.r = x / p.G;
  a.g = x - a.r * p.G;
  a.lim = a.r < req[a.b].rows
              ? static_cast<int>(min(p.kcap, static_cast<int64_t>(req[a.b].base) + a.r + 1))
              : 0;
  if (a.lim == 0) a.r = a.g = 0;
  return a;
}
__device__ __forceinline__ int64_t attn_q_row(const PagedParams&, const PagedReq* req, const AttnRow& r) {
  return static_cast<int64_t>(req[r.b].start) + r.r;
}

// Only units that more than one CTA has leave partials, and of those a CTA has at most the end of one
// (its first piece) and the start of another (its last) in each part of the dealing: four slots a CTA.
__device__ __forceinline__ int attn_slot(const PagedParams&, const AttnShares& s, int u, int cta, int blk0) {
  return 4 * cta + (u < s.u1 ? 0 : 2) + (blk0 == 0);
}

// What the join has to know of a unit that begins in a CTA's share and ends in another's, in 16 bytes: its
// number of partials and the CTAs from one to the next, its request's first row, its place among the request's
// tiles, its head and its number of rows (x = r G + g). A CTA writes its two (of the groups' part and of the
// rest), by one thread: clear() first, then every piece.
struct PagedSplit {
  uint16_t n, step;
  int start, tile;
  uint16_t head, count;
};
static_assert(sizeof(PagedSplit) == 16 && kPagedMaxCtas < 65536 && kPagedMaxHeads <= 65536);
__device__ __forceinline__ int4 paged_split_bits(const PagedSplit& s) {
  return make_int4(s.n | static_cast<int>(static_cast<uint32_t>(s.step) << 16), s.start, s.tile,
                   s.head | static_cast<int>(static_cast<uint32_t>(s.count) << 16));
}
__device__ __forceinline__ PagedSplit paged_split_of(const int4& v) {
  PagedSplit s;
  s.n = static_cast<uint16_t>(v.x), s.step = static_cast<uint16_t>(static_cast<uint32_t>(v.x) >> 16);
  s.start = v.y, s.tile = v.z;
  s.head = static_cast<uint16_t>(v.w), s.count = static_cast<uint16_t>(static_cast<uint32_t>(v.w) >> 16);
  return s;
}
__device__ __forceinline__ void paged_splits_clear(const PagedParams& p) {
  for (int i = 0; i < 2; ++i) *reinterpret_cast<int4*>(p.splits + 2 * blockIdx.x + i) = make_int4(0, 0, 0, 0);
}
__device__ __forceinline__ void paged_split(const PagedParams& p, const int32_t* cum, const AttnShares& s,
                                            const AttnWalk& walk, const AttnPiece& a) {
  if (a.whole || a.blk0 > 0) return;
  const int cta = blockIdx.x, cost = cum[walk.item + 1] - cum[walk.item];
  // the place of its last block
  const int64_t last = static_cast<int64_t>(cum[walk.item]) * p.Hkv + static_cast<int64_t>(a.head + 1) * cost - 1;
  const bool group = walk.item * p.Hkv + a.head < s.u1;
  const int n = group ? static_cast<int>(attn_div(p, last, s.sp)) - cta / p.grp + 1
                      : s.single_cta(p, last - s.wp) - cta + 1;
  const PagedReq& r = paged_reqs(p, cum)[attn_tile_req(p, a.tile)];
  PagedSplit out;
  out.n = static_cast<uint16_t>(n), out.step = static_cast<uint16_t>(group ? p.grp : 1);
  out.start = r.start, out.tile = a.tile >> kTileReqBits;
  out.head = static_cast<uint16_t>(a.head), out.count = static_cast<uint16_t>(min(p.tm, r.rows * p.G - out.tile * p.tm));
  *reinterpret_cast<int4*>(p.splits + 2 * cta + !group) = paged_split_bits(out);
}

cudaError_t paged_simt_launch(const PagedParams& p, spec_dtype dtype, int grid, cudaStream_t stream);
cudaError_t paged_join_launch(const PagedParams& p, spec_dtype dtype, int grid, cudaStream_t stream);
int paged_tc_bn();
// Page sizes of the tensor-core kernel: a block of its positions is whole pages or lies on one, and a page has
// at least the eight rows of the operands' swizzle.
inline bool paged_tc_takes(int head_dim, int page_size) {
  return attn_tc_takes(head_dim) && page_size % 8 == 0 &&
         (page_size % paged_tc_bn() == 0 || paged_tc_bn() % page_size == 0);
}
spec_status paged_tc_launch(const PagedParams& p, int grid, EncodeTiledFn encode, cudaStream_t stream);

}  // namespace spec
