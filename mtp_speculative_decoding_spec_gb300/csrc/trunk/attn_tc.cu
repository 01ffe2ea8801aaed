// Attention of the verify rows over a shared prefix and each request's own cache: the tensor-core kernel of
// attn_tc.cuh for it.
#include "attn_tc.cuh"

namespace spec {
namespace {

template <int D>
spec_status launch_tc(const AttnParams& p, int grid, EncodeTiledFn encode, cudaStream_t stream) {
  using Sh = Shape<D, false>;
  AttnMaps m;
  // dims inside a 64-dim panel, positions, panels (64 dims on), requests
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(Sh::kBn), D / 64, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const auto map = [&](CUtensorMap* t, const uint8_t* base, int64_t positions, int64_t step, int64_t reqs,
                       int64_t req_step) {
    const cuuint64_t dim[4] = {64, static_cast<cuuint64_t>(positions),
                               static_cast<cuuint64_t>(p.Hkv) * (D / 64), static_cast<cuuint64_t>(reqs)};
    const cuuint64_t stride[3] = {static_cast<cuuint64_t>(step), 128, static_cast<cuuint64_t>(req_step)};
    return encode(t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint8_t*>(base), dim, stride, box,
                  es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const int64_t req = p.B > 1 ? p.kreq : p.krow;
  if (!map(&m.ok, p.kk, p.kcap, p.krow, p.B, req) || !map(&m.ov, p.kv, p.kcap, p.krow, p.B, req))
    return SPEC_ERR_CUDA;
  m.pk = m.ok;
  m.pv = m.ov;
  if (p.npt > 0 && (!map(&m.pk, p.pk, p.pcap, p.pstride, 1, p.pstride) ||
                    !map(&m.pv, p.pv, p.pcap, p.pstride, 1, p.pstride)))
    return SPEC_ERR_CUDA;
  return tc_launch<AttnParams, D>(p, m, grid, stream);
}

}  // namespace

bool attn_tc_takes(int head_dim) { return head_dim == 64 || head_dim == 128 || head_dim == 256; }
int attn_tc_tm() { return kTm; }
int attn_tc_bn(int head_dim) { return head_dim == 256 ? Shape<256, false>::kBn : Shape<128, false>::kBn; }

spec_status attn_tc_launch(const AttnParams& p, int grid, EncodeTiledFn encode, cudaStream_t stream) {
  return p.D == 256   ? launch_tc<256>(p, grid, encode, stream)
         : p.D == 128 ? launch_tc<128>(p, grid, encode, stream)
                      : launch_tc<64>(p, grid, encode, stream);
}

}  // namespace spec
