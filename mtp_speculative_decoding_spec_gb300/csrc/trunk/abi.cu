// extern "C" entry points of the trunk's token mixers (the gated delta rule, attention over a shared
// prefix): argument validation, workspace layout, launch configuration. As everywhere, a call validates
// on the host and then enqueues on the caller's stream.
#include <stdint.h>
#include <string.h>

#include "trunk.cuh"

namespace spec {
namespace {

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Elements of one request's recurrent state, or 0 if the sizes are not valid.
int64_t rec_elems(const spec_state_desc* st) {
  if (!st || st->rec_layers < 1 || st->rec_heads < 1 || st->rec_dk < 1 || st->rec_dv < 4 ||
      st->rec_dv % 4 != 0)
    return 0;
  const int64_t e = static_cast<int64_t>(st->rec_layers) * st->rec_heads;
  if (e >= (int64_t(1) << 31)) return 0;
  const int64_t hd = static_cast<int64_t>(st->rec_dk) * st->rec_dv;
  if (hd >= (int64_t(1) << 31) || e * hd >= (int64_t(1) << 33)) return 0;
  return e * hd;
}

// Checks shared by both calls, and the parameters they give. Without rows no pointer to them is needed.
spec_status delta_params(const spec_state_desc* st, int32_t layer, const spec_delta_desc* d, bool any_rows,
                         DeltaParams& p) {
  memset(&p, 0, sizeof(p));
  if (!d || rec_elems(st) == 0 || layer < 0 || layer >= st->rec_layers) return SPEC_ERR_INVALID;
  if (d->dtype != SPEC_BF16 && d->dtype != SPEC_F32) return SPEC_ERR_INVALID;
  if (any_rows && (!d->q || !d->k || !d->v || !d->log_decay || !d->beta || !d->out))
    return SPEC_ERR_INVALID;
  if (d->key_heads < 1 || st->rec_heads % d->key_heads != 0) return SPEC_ERR_INVALID;
  const size_t e = d->dtype == SPEC_BF16 ? 2 : 4;
  const int64_t wqk = static_cast<int64_t>(d->key_heads) * st->rec_dk;
  const int64_t wv = static_cast<int64_t>(st->rec_heads) * st->rec_dv;
  if (d->q_stride < wqk || d->k_stride < wqk || d->v_stride < wv || d->out_stride < wv)
    return SPEC_ERR_INVALID;
  if (!aligned_to(d->q, e) || !aligned_to(d->k, e) || !aligned_to(d->v, e) ||
      !aligned_to(d->out, e) || !aligned_to(d->log_decay, 4) || !aligned_to(d->beta, 4))
    return SPEC_ERR_INVALID;
  if (st->rec_dk > 256) return SPEC_ERR_UNSUPPORTED;
  p.H = st->rec_heads;
  p.Hk = d->key_heads;
  p.dk = st->rec_dk;
  p.dv = st->rec_dv;
  p.layer = layer;
  p.layers = st->rec_layers;
  p.q = d->q;
  p.k = d->k;
  p.v = d->v;
  p.qs = d->q_stride;
  p.ks = d->k_stride;
  p.vs = d->v_stride;
  p.os = d->out_stride;
  p.g = d->log_decay;
  p.beta = d->beta;
  p.scale = d->scale;
  p.out = d->out;
  const auto whole = [e](const void* x, int64_t stride, size_t a) {
    return aligned_to(x, a) && (static_cast<size_t>(stride) * e) % a == 0;
  };
  p.vec_qk = whole(d->q, d->q_stride, 16) && whole(d->k, d->k_stride, 16) && (p.dk * e) % 16 == 0;
  p.vec_v = whole(d->v, d->v_stride, 4 * e);  // dv is a multiple of 4
  p.vec_o = whole(d->out, d->out_stride, 4 * e);
  p.live = st->rec_live;
  return SPEC_OK;
}

// Attention: the tile sizes of the kernel that takes the call, and the workspace's layout.
struct AttnPlan {
  int tc, tm, bn, npt, npi, grp, nown, items, grid;
  size_t units, ml, o, total;
};

spec_status attn_check(int32_t B, int32_t R, const spec_state_desc* st, const spec_attn_desc* d) {
  if (B < 1 || R < 1 || R > kMaxRows || !st || !d) return SPEC_ERR_INVALID;
  if (d->dtype != SPEC_BF16 && d->dtype != SPEC_F32) return SPEC_ERR_INVALID;
  if (d->kv_heads < 1 || d->q_heads < 1 || d->q_heads % d->kv_heads != 0 || d->head_dim < 8 ||
      d->head_dim % 8 != 0)
    return SPEC_ERR_INVALID;
  const int64_t e = d->dtype == SPEC_BF16 ? 2 : 4;
  if (st->kv_layers < 1 || st->kv_capacity < 1 ||
      st->kv_row_bytes != d->kv_heads * static_cast<int64_t>(d->head_dim) * e)
    return SPEC_ERR_INVALID;
  if ((d->prefix_k == nullptr) != (d->prefix_v == nullptr)) return SPEC_ERR_INVALID;
  if (d->prefix_k && d->prefix_capacity < 0) return SPEC_ERR_INVALID;
  if (B > 1024 || d->head_dim > 256 || d->q_heads / d->kv_heads > 64 || d->kv_heads > 65536)
    return SPEC_ERR_UNSUPPORTED;
  if (st->kv_capacity > kAttnMaxPos || (d->prefix_k && d->prefix_capacity > kAttnMaxPos))
    return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

spec_status attn_plan_of(int32_t B, int32_t R, const spec_state_desc* st, const spec_attn_desc* d,
                         AttnPlan& w) {
  const spec_status s = attn_check(B, R, st, d);
  if (s != SPEC_OK) return s;
  w.tc = d->dtype == SPEC_BF16 && attn_tc_takes(d->head_dim);
  w.tm = w.tc ? attn_tc_tm() : attn_simt_tm();
  w.bn = w.tc ? attn_tc_bn(d->head_dim) : attn_simt_bn();
  const int64_t G = d->q_heads / d->kv_heads, per = R * G;
  const bool prefix = d->prefix_k && d->prefix_capacity > 0;
  const int64_t npt = prefix ? (B * per + w.tm - 1) / w.tm : 0;
  const int64_t nown = (per + w.tm - 1) / w.tm;
  const int64_t sets = (npt + kAttnGroup - 1) / kAttnGroup;
  w.grp = w.tc && npt >= 2 ? static_cast<int>((npt + sets - 1) / sets) : 1;
  const int64_t npi = (npt + w.grp - 1) / w.grp;
  const int64_t items = npi + B * nown;
  const int64_t blocks = npi * ((prefix ? d->prefix_capacity : 0) / w.bn + 1 + kAttnOverPre) +
                         B * nown * (st->kv_capacity / w.bn + 1 + kAttnOver);
  if (items > kAttnMaxItems || blocks >= (int64_t(1) << 31)) return SPEC_ERR_UNSUPPORTED;
  const DevAttr a = dev_attr();
  if (a.sms <= 0) return SPEC_ERR_CUDA;
  w.npt = static_cast<int>(npt);
  w.npi = static_cast<int>(npi);
  w.nown = static_cast<int>(nown);
  w.items = static_cast<int>(items);
  w.grid = a.sms;
  const size_t slots = 2 * static_cast<size_t>(w.grid) +
                       static_cast<size_t>(npi * w.grp + items - npi) * d->kv_heads;
  w.units = sizeof(WsHeader);
  w.ml = w.units + align_up(sizeof(int2) * static_cast<size_t>(items) * d->kv_heads, 256);
  w.o = w.ml + align_up(slots * w.tm * sizeof(float2), 256);
  w.total = w.o + align_up(slots * w.tm * d->head_dim * sizeof(float), 256);
  return SPEC_OK;
}

}  // namespace
}  // namespace spec

extern "C" {

using namespace spec;

spec_status spec_delta_rows(int32_t B, int32_t R, const spec_state_desc* st, int32_t layer,
                            int32_t mode, const spec_delta_desc* d, const int32_t* n_rows,
                            spec_stream_t stream) {
  if (B < 1 || R < 1 || R > kMaxRows) return SPEC_ERR_INVALID;
  DeltaParams p;
  const spec_status s = delta_params(st, layer, d, true, p);
  if (s != SPEC_OK) return s;
  if (mode != SPEC_COMMIT_SNAPSHOT && mode != SPEC_COMMIT_REPLAY && mode != SPEC_COMMIT_INDEX)
    return SPEC_ERR_INVALID;
  if (st->n_slots < R + 1 || !st->rec_slots || !aligned16(st->rec_slots)) return SPEC_ERR_INVALID;
  if (mode == SPEC_COMMIT_INDEX ? !st->live_slot : (!st->rec_live || !aligned16(st->rec_live)))
    return SPEC_ERR_INVALID;
  if (mode == SPEC_COMMIT_REPLAY &&
      (!st->step_a || !st->step_b || !st->step_c || !aligned16(st->step_c)))
    return SPEC_ERR_INVALID;
  const DevAttr a = dev_attr();
  if (a.sms <= 0) return SPEC_ERR_CUDA;
  p.B = B;
  p.R = R;
  p.mode = mode;
  p.n_slots = st->n_slots;
  p.n_rows = n_rows;
  p.slots = const_cast<float*>(st->rec_slots);  // the forward pass fills what the commit reads
  p.live_slot = st->live_slot;
  p.step_a = const_cast<float*>(st->step_a);
  p.step_b = const_cast<float*>(st->step_b);
  p.step_c = const_cast<float*>(st->step_c);
  const cudaError_t e = delta_scan_launch(p, d->dtype, a.sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

size_t spec_delta_prefill_workspace_bytes(int64_t rows, int32_t B, const spec_state_desc* st) {
  if (rows < 0 || B < 1 || rec_elems(st) == 0) return 0;
  return delta_chunk_sizes(st->rec_dk, st->rec_dv) ? delta_chunk_workspace(rows, B, st->rec_heads)
                                                   : sizeof(WsHeader);
}

spec_status spec_delta_prefill(int32_t B, const int32_t* cu_rows, int64_t rows,
                               const spec_state_desc* st, int32_t layer, const spec_delta_desc* d,
                               const float* rec_init, void* workspace, size_t workspace_bytes,
                               spec_stream_t stream) {
  if (B < 1 || !cu_rows || rows < 0 || rows >= (int64_t(1) << 31)) return SPEC_ERR_INVALID;
  DeltaParams p;
  const spec_status s = delta_params(st, layer, d, rows > 0, p);
  if (s != SPEC_OK) return s;
  if (!st->rec_live || !aligned16(st->rec_live) || !aligned16(rec_init)) return SPEC_ERR_INVALID;
  p.B = B;
  p.mode = DELTA_PREFILL;
  p.cu_rows = cu_rows;
  p.rows = rows;
  p.init = rec_init;
  p.hdr = static_cast<WsHeader*>(workspace);
  const bool chunks = delta_chunk_takes(p, d->dtype);  // the row scan uses the header alone
  if (!workspace || !aligned_to(workspace, 256) ||
      workspace_bytes < (chunks ? delta_chunk_workspace(rows, B, p.H) : sizeof(WsHeader)))
    return SPEC_ERR_INVALID;
  const DevAttr a = dev_attr();
  if (a.sms <= 0) return SPEC_ERR_CUDA;
  if (chunks) {
    EncodeTiledFn encode = encode_tiled();
    if (!encode) return SPEC_ERR_CUDA;
    return delta_chunk_launch(p, workspace, encode, reinterpret_cast<cudaStream_t>(stream));
  }
  const cudaError_t e = delta_scan_launch(p, d->dtype, a.sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

size_t spec_prefix_attention_workspace_bytes(int32_t B, int32_t R, const spec_state_desc* st,
                                             const spec_attn_desc* d) {
  AttnPlan w;
  return attn_plan_of(B, R, st, d, w) == SPEC_OK ? w.total : 0;
}

spec_status spec_prefix_attention(int32_t B, int32_t R, const spec_state_desc* st, int32_t layer,
                                  const spec_attn_desc* d, const int32_t* n_rows, void* workspace,
                                  size_t workspace_bytes, spec_stream_t stream) {
  spec_status s = attn_check(B, R, st, d);
  if (s != SPEC_OK) return s;
  const int64_t e = d->dtype == SPEC_BF16 ? 2 : 4;
  const int64_t width = static_cast<int64_t>(d->q_heads) * d->head_dim;
  if (layer < 0 || layer >= st->kv_layers || !st->kv || !aligned16(st->kv) || !st->kv_len ||
      st->kv_row_bytes % 16 != 0 || st->kv_request_stride % 16 != 0)
    return SPEC_ERR_INVALID;
  if (B > 1 && st->kv_request_stride < 2 * st->kv_layers * st->kv_capacity * st->kv_row_bytes)
    return SPEC_ERR_INVALID;
  if (!d->q || !d->out || d->q_stride < width || d->out_stride < width || !aligned_to(d->q, e) ||
      !aligned_to(d->out, e))
    return SPEC_ERR_INVALID;
  if (d->prefix_k && (!aligned16(d->prefix_k) || !aligned16(d->prefix_v) ||
                      d->prefix_stride < static_cast<int64_t>(d->kv_heads) * d->head_dim ||
                      d->prefix_stride * e % 16 != 0))
    return SPEC_ERR_INVALID;
  AttnPlan w;
  s = attn_plan_of(B, R, st, d, w);
  if (s != SPEC_OK) return s;
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < w.total) return SPEC_ERR_INVALID;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AttnParams p;
  memset(&p, 0, sizeof(p));
  p.B = B;
  p.R = R;
  p.G = d->q_heads / d->kv_heads;
  p.Hkv = d->kv_heads;
  p.D = d->head_dim;
  p.tm = w.tm;
  p.bn = w.bn;
  p.npt = w.npt;
  p.npi = w.npi;
  p.grp = w.grp;
  p.over[0] = w.tc ? kAttnOverPre : kAttnSimtOver;
  p.over[1] = w.tc ? kAttnOver : kAttnSimtOver;
  p.nown = w.nown;
  p.items = w.items;
  p.q = d->q;
  p.qs = d->q_stride;
  p.out = d->out;
  p.os = d->out_stride;
  p.scale_log2 = d->scale * 1.4426950408889634f;
  p.pk = static_cast<const uint8_t*>(d->prefix_k);
  p.pv = static_cast<const uint8_t*>(d->prefix_v);
  p.pcap = d->prefix_k ? d->prefix_capacity : 0;
  p.pstride = d->prefix_stride * e;
  p.prefix_len = d->prefix_len;
  p.kk = static_cast<const uint8_t*>(st->kv) +
         2 * static_cast<int64_t>(layer) * st->kv_capacity * st->kv_row_bytes;
  p.kv = p.kk + st->kv_capacity * st->kv_row_bytes;
  p.kreq = st->kv_request_stride;
  p.kcap = st->kv_capacity;
  p.krow = st->kv_row_bytes;
  p.kv_len = st->kv_len;
  p.n_rows = n_rows;
  p.lse = d->lse;
  p.hdr = static_cast<WsHeader*>(workspace);
  p.units = reinterpret_cast<int2*>(ws + w.units);
  p.ml = reinterpret_cast<float2*>(ws + w.ml);
  p.o = reinterpret_cast<float*>(ws + w.o);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (w.tc) {
    EncodeTiledFn encode = encode_tiled();
    if (!encode) return SPEC_ERR_CUDA;
    s = attn_tc_launch(p, w.grid, encode, cs);
    if (s != SPEC_OK) return s;
  } else if (attn_simt_launch(p, d->dtype, w.grid, cs) != cudaSuccess) {
    return SPEC_ERR_CUDA;
  }
  return attn_join_launch(p, d->dtype, w.grid, cs) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
