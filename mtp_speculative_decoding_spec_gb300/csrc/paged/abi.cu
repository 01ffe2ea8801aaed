// extern "C" entry points of the paged KV cache: argument validation, workspace layout, launch
// configuration. As everywhere, a call validates on the host and then enqueues on the caller's stream.
#include <stdint.h>
#include <string.h>

#include "paged.cuh"

namespace spec {
namespace {

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The cache's sizes. Products are of numbers checked before: nothing overflows.
spec_status cache_check(int32_t B, const spec_paged_cache* c) {
  if (B < 1 || !c) return SPEC_ERR_INVALID;
  if (c->dtype != SPEC_BF16 && c->dtype != SPEC_F32) return SPEC_ERR_INVALID;
  if (c->layers < 1 || c->kv_heads < 1 || c->head_dim < 8 || c->head_dim % 8 != 0 || c->page_size < 1 ||
      c->n_pages < 1 || c->max_pages < 1 || c->table_stride < c->max_pages)
    return SPEC_ERR_INVALID;
  if (B > kPagedMaxB || c->head_dim > 256 || c->kv_heads > kPagedMaxHeads || c->layers > 65536)
    return SPEC_ERR_UNSUPPORTED;
  if (c->n_pages >= (int64_t(1) << 31) || static_cast<int64_t>(c->max_pages) * c->page_size > kAttnMaxPos)
    return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

// And its pointers and strides; the given layer of it.
spec_status cache_layer(int32_t B, const spec_paged_cache* c, int32_t layer, PagedLayer& L) {
  const spec_status s = cache_check(B, c);
  if (s != SPEC_OK) return s;
  if (layer < 0 || layer >= c->layers) return SPEC_ERR_INVALID;
  if (!c->k_pages || !c->v_pages || !aligned16(c->k_pages) || !aligned16(c->v_pages) || !c->page_table ||
      !aligned_to(c->page_table, 4) || !c->kv_len || !aligned_to(c->kv_len, 8))
    return SPEC_ERR_INVALID;
  const int64_t row = static_cast<int64_t>(c->kv_heads) * c->head_dim * (c->dtype == SPEC_BF16 ? 2 : 4);
  const int64_t page = row * c->page_size;  // below 2^26 * 2^31
  if (c->page_stride % 16 != 0 || c->layer_stride % 16 != 0 || c->page_stride < 0 || c->layer_stride < 0)
    return SPEC_ERR_INVALID;
  if (c->page_stride >= (int64_t(1) << 62) / c->n_pages || c->layer_stride >= (int64_t(1) << 62) / c->layers)
    return SPEC_ERR_UNSUPPORTED;  // an offset fits 64 bits
  const int64_t pages = (c->n_pages - 1) * c->page_stride + page, layers = (c->layers - 1) * c->layer_stride + page;
  if (c->n_pages > 1 && c->page_stride < page) return SPEC_ERR_INVALID;
  // layers of whole pools, or a page's layers together
  if (c->layers > 1 && c->layer_stride < pages &&
      (c->layer_stride < page || (c->n_pages > 1 && c->page_stride < layers)))
    return SPEC_ERR_INVALID;
  L.k = static_cast<uint8_t*>(c->k_pages) + layer * c->layer_stride;
  L.v = static_cast<uint8_t*>(c->v_pages) + layer * c->layer_stride;
  L.page_stride = c->page_stride;
  L.table_stride = c->table_stride;
  L.table = c->page_table;
  L.kv_len = c->kv_len;
  L.row_bytes = static_cast<int>(row);
  L.page_size = c->page_size;
  L.n_pages = static_cast<int>(c->n_pages);
  L.max_pages = c->max_pages;
  return SPEC_OK;
}

bool rows_ok(const int32_t* cu_rows, int64_t rows, const int32_t* n_rows) {
  return cu_rows && aligned_to(cu_rows, 4) && aligned_to(n_rows, 4) && rows >= 0 && rows < (int64_t(1) << 31);
}

// Attention: the tile sizes of the kernel that takes the call, and the workspace's layout.
struct PagedPlan {
  int tc, tm, bn, tiles, grid;
  size_t ml, o, total;
};

spec_status plan_check(int32_t B, int64_t rows, const spec_paged_cache* c, const spec_paged_attn_desc* d,
                       PagedPlan& w) {
  const spec_status s = cache_check(B, c);
  if (s != SPEC_OK) return s;
  if (!d || d->q_heads < 1 || d->q_heads % c->kv_heads != 0 || rows < 0 || rows >= (int64_t(1) << 31))
    return SPEC_ERR_INVALID;
  const int64_t G = d->q_heads / c->kv_heads;
  if (G > 64) return SPEC_ERR_UNSUPPORTED;
  w.tc = c->dtype == SPEC_BF16 && paged_tc_takes(c->head_dim, c->page_size) &&
         c->page_stride < (int64_t(1) << 40);  // a tensor map's strides
  w.tm = w.tc ? attn_tc_tm() : attn_simt_tm();
  w.bn = w.tc ? paged_tc_bn() : attn_simt_bn();
  const int64_t tiles = rows * G / w.tm + B;  // each request's last tile may not be full
  if (tiles > (w.tc ? kPagedMaxTiles : kPagedSimtMaxTiles)) return SPEC_ERR_UNSUPPORTED;
  const int64_t cap = static_cast<int64_t>(c->max_pages) * c->page_size;
  // the dealing counts blocks of all heads in 31 bits, grid - 1 more when it rounds up
  if (tiles * (cap / w.bn + 1 + kPagedOver) >= ((int64_t(1) << 31) - 1024) / c->kv_heads) return SPEC_ERR_UNSUPPORTED;
  w.tiles = static_cast<int>(tiles);
  return SPEC_OK;
}

spec_status plan_of(int32_t B, int64_t rows, const spec_paged_cache* c, const spec_paged_attn_desc* d,
                    PagedPlan& w) {
  const spec_status s = plan_check(B, rows, c, d, w);
  if (s != SPEC_OK) return s;
  const DevAttr a = dev_attr();
  if (a.sms <= 0) return SPEC_ERR_CUDA;
  w.grid = min(a.sms, kPagedMaxCtas);
  const size_t slots = 4 * static_cast<size_t>(w.grid);
  w.ml = sizeof(WsHeader) + align_up(2 * w.grid * sizeof(PagedSplit), 256);
  w.o = w.ml + align_up(slots * w.tm * sizeof(float2), 256);
  w.total = w.o + align_up(slots * w.tm * c->head_dim * sizeof(float), 256);
  return SPEC_OK;
}

}  // namespace
}  // namespace spec

extern "C" {

using namespace spec;

spec_status spec_paged_append(int32_t B, const int32_t* cu_rows, int64_t rows,
                              const spec_paged_cache* c, int32_t layer, const spec_append_desc* d,
                              const int32_t* n_rows, int32_t* status, spec_stream_t stream) {
  AppendParams p;
  memset(&p, 0, sizeof(p));
  const spec_status s = cache_layer(B, c, layer, p.c);
  if (s != SPEC_OK) return s;
  if (!d || !rows_ok(cu_rows, rows, n_rows) || !aligned_to(status, 4) || d->q_heads < 0) return SPEC_ERR_INVALID;
  if (d->q_heads > 65536) return SPEC_ERR_UNSUPPORTED;
  if ((d->k == nullptr) != (d->v == nullptr)) return SPEC_ERR_INVALID;
  const size_t e = c->dtype == SPEC_BF16 ? 2 : 4;
  const int64_t wq = static_cast<int64_t>(d->q_heads) * c->head_dim;
  const int64_t wk = static_cast<int64_t>(c->kv_heads) * c->head_dim;
  if (rows > 0 && d->q_heads > 0 &&
      (!d->q || !d->q_out || d->q_stride < wq || d->q_out_stride < wq || !aligned_to(d->q, e) ||
       !aligned_to(d->q_out, e)))
    return SPEC_ERR_INVALID;
  if (d->k && (d->k_stride < wk || d->v_stride < wk || !aligned_to(d->k, e) || !aligned_to(d->v, e)))
    return SPEC_ERR_INVALID;
  if (d->rot_dim < 0 || d->rot_dim % 2 != 0 || d->rot_dim > c->head_dim || (d->rot_dim > 0 && !d->inv_freq) ||
      !aligned_to(d->inv_freq, 4) || !aligned_to(d->q_norm, 4) || !aligned_to(d->k_norm, 4) ||
      !aligned_to(d->pos, 8) || !(d->norm_eps >= 0.f))
    return SPEC_ERR_INVALID;
  if ((rows == 0 || (d->q_heads == 0 && !d->k)) && !status) return SPEC_OK;
  const DevAttr a = dev_attr();
  if (a.sms <= 0) return SPEC_ERR_CUDA;
  p.B = B;
  p.D = c->head_dim;
  p.nq = d->q_heads;
  p.nk = d->k ? c->kv_heads : 0;
  p.rows = rows;
  p.cu_rows = cu_rows;
  p.n_rows = n_rows;
  p.q = d->q;
  p.k = d->k;
  p.v = d->v;
  p.q_out = d->q_out;
  p.qs = d->q_stride;
  p.ks = d->k_stride;
  p.vs = d->v_stride;
  p.qos = d->q_out_stride;
  const auto whole = [e](const void* x, int64_t stride) { return aligned16(x) && stride * e % 16 == 0; };
  p.whole = (p.nq == 0 || (whole(d->q, d->q_stride) && whole(d->q_out, d->q_out_stride))) &&
            (p.nk == 0 || (whole(d->k, d->k_stride) && whole(d->v, d->v_stride)));
  p.q_norm = d->q_norm;
  p.k_norm = d->k_norm;
  p.eps = d->norm_eps;
  p.rot = d->rot_dim;
  p.inv_freq = d->inv_freq;
  p.rot_scale = d->rot_scale;
  p.pos = d->pos;
  p.status = status;
  return append_launch(p, c->dtype, d->rot_interleaved != 0, a.sms, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

size_t spec_paged_attention_workspace_bytes(int32_t B, int64_t rows, const spec_paged_cache* c,
                                            const spec_paged_attn_desc* d) {
  PagedPlan w;
  return plan_of(B, rows, c, d, w) == SPEC_OK ? w.total : 0;
}

spec_status spec_paged_attention(int32_t B, const int32_t* cu_rows, int64_t rows,
                                 const spec_paged_cache* c, int32_t layer,
                                 const spec_paged_attn_desc* d, const int32_t* n_rows, void* workspace,
                                 size_t workspace_bytes, spec_stream_t stream) {
  PagedParams p;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  spec_status s = cache_layer(B, c, layer, p.c);
  if (s != SPEC_OK) return s;
  PagedPlan w;
  s = plan_check(B, rows, c, d, w);
  if (s != SPEC_OK) return s;
  const size_t e = c->dtype == SPEC_BF16 ? 2 : 4;
  const int64_t width = static_cast<int64_t>(d->q_heads) * c->head_dim;
  if (!rows_ok(cu_rows, rows, n_rows) || !workspace || !aligned_to(workspace, 256)) return SPEC_ERR_INVALID;
  if (rows > 0 && (!d->q || !d->out || d->q_stride < width || d->out_stride < width || !aligned_to(d->q, e) ||
                   !aligned_to(d->out, e) || !aligned_to(d->lse, 4)))
    return SPEC_ERR_INVALID;
  s = plan_of(B, rows, c, d, w);
  if (s != SPEC_OK) return s;
  if (workspace_bytes < w.total) return SPEC_ERR_INVALID;
  if (rows == 0) return SPEC_OK;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.B = B;
  p.G = d->q_heads / c->kv_heads;
  p.Hkv = c->kv_heads;
  p.D = c->head_dim;
  p.tm = w.tm;
  p.bn = w.bn;
  while (1 << p.tm_shift < p.tm) ++p.tm_shift;
  while (1 << p.bn_shift < p.bn) ++p.bn_shift;
  p.items = w.tiles;
  p.grp = w.tc && w.grid >= kPagedGroup ? kPagedGroup : 1;
  p.group_min = kPagedGroupMin;
  for (p.page_shift = 0; w.tc && p.page_shift < 31 && (1 << p.page_shift) < c->page_size; ++p.page_shift) {
  }
  if (c->page_size >= w.bn) p.page_shift = 31;
  p.unit_more = w.tc ? kPagedUnitMore : -1;
  p.unit_part = w.tc && c->head_dim >= 128 ? kPagedUnitPart : 0;
  p.over[0] = p.over[1] = w.tc ? kPagedOver : kAttnSimtOver;
  p.q = d->q;
  p.qs = d->q_stride;
  p.out = d->out;
  p.os = d->out_stride;
  p.scale_log2 = d->scale * 1.4426950408889634f;
  p.kcap = static_cast<int64_t>(c->max_pages) * c->page_size;
  p.kv_len = c->kv_len;
  p.n_rows = n_rows;
  p.lse = d->lse;
  p.cu_rows = cu_rows;
  p.rows = rows;
  p.hdr = static_cast<WsHeader*>(workspace);
  p.splits = reinterpret_cast<PagedSplit*>(ws + sizeof(WsHeader));
  p.ml = reinterpret_cast<float2*>(ws + w.ml);
  p.o = reinterpret_cast<float*>(ws + w.o);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (w.tc) {
    EncodeTiledFn encode = encode_tiled();
    if (!encode) return SPEC_ERR_CUDA;
    s = paged_tc_launch(p, w.grid, encode, cs);
    if (s != SPEC_OK) return s;
  } else if (paged_simt_launch(p, c->dtype, w.grid, cs) != cudaSuccess) {
    return SPEC_ERR_CUDA;
  }
  return paged_join_launch(p, c->dtype, w.grid, cs) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_paged_commit(int32_t B, const spec_paged_cache* c, const spec_accept_out* acc,
                              const int32_t* k, int32_t* commit_status, spec_stream_t stream) {
  PagedCommitParams p;
  memset(&p, 0, sizeof(p));
  const spec_status s = cache_layer(B, c, 0, p.c);
  if (s != SPEC_OK) return s;
  if (!k || !aligned_to(k, 4) || !aligned_to(acc, 8) || !aligned_to(commit_status, 4)) return SPEC_ERR_INVALID;
  p.layer_stride = c->layer_stride;
  p.layers = c->layers;
  p.acc = acc;
  p.k = k;
  p.status = commit_status;
  return paged_commit_launch(p, B, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? SPEC_OK
                                                                                          : SPEC_ERR_CUDA;
}

}  // extern "C"
