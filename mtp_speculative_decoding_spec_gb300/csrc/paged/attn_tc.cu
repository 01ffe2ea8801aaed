// Attention of new rows over a paged cache: the tensor-core kernel of trunk/attn_tc.cuh for it.
#include "trunk/attn_tc.cuh"

#include "paged.cuh"

namespace spec {
namespace {

template <int D>
spec_status launch_tc(const PagedParams& p, int grid, EncodeTiledFn encode, cudaStream_t stream) {
  constexpr int BN = Shape<D>::kBn;
  const bool one = p.c.page_size >= BN;  // a block lies on one page
  AttnMaps m;
  // dims inside a 64-dim panel, positions of a page, panels (64 dims on), pages
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(one ? BN : p.c.page_size), one ? D / 64u : 1u, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const cuuint64_t dim[4] = {64, static_cast<cuuint64_t>(p.c.page_size),
                             static_cast<cuuint64_t>(p.Hkv) * (D / 64), static_cast<cuuint64_t>(p.c.n_pages)};
  const int64_t page = p.c.n_pages > 1 ? p.c.page_stride : static_cast<int64_t>(p.c.row_bytes) * p.c.page_size;
  const cuuint64_t stride[3] = {static_cast<cuuint64_t>(p.c.row_bytes), 128, static_cast<cuuint64_t>(page)};
  const auto map = [&](CUtensorMap* t, uint8_t* base) {
    return encode(t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dim, stride, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!map(&m.ok, p.c.k) || !map(&m.ov, p.c.v)) return SPEC_ERR_CUDA;
  m.pk = m.ok;
  m.pv = m.ov;
  return tc_launch<PagedParams, D>(p, m, grid, stream);
}

}  // namespace

spec_status paged_tc_launch(const PagedParams& p, int grid, EncodeTiledFn encode, cudaStream_t stream) {
  return p.D == 256   ? launch_tc<256>(p, grid, encode, stream)
         : p.D == 128 ? launch_tc<128>(p, grid, encode, stream)
                      : launch_tc<64>(p, grid, encode, stream);
}

}  // namespace spec
