// Attention of new rows over a paged cache: the tensor-core kernel of trunk/attn_tc.cuh for it.
#include "paged.cuh"

#include "trunk/attn_tc.cuh"

namespace spec {
namespace {

template <int D>
spec_status launch_tc(const PagedParams& p, int grid, EncodeTiledFn encode, cudaStream_t stream) {
  constexpr int BN = Shape<D, true>::kBn;
  AttnMaps m;
  // dims inside a 64-dim panel, eight positions, panels (64 dims on), eights of a page, pages
  const cuuint32_t box[5] = {64, 8, D / 64, static_cast<cuuint32_t>(min(p.c.page_size, BN) / 8), 1};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  const cuuint64_t dim[5] = {64, 8, static_cast<cuuint64_t>(p.Hkv) * (D / 64),
                             static_cast<cuuint64_t>(p.c.page_size / 8), static_cast<cuuint64_t>(p.c.n_pages)};
  const cuuint64_t row = static_cast<cuuint64_t>(p.c.row_bytes);
  const cuuint64_t page = p.c.n_pages > 1 ? static_cast<cuuint64_t>(p.c.page_stride) : row * p.c.page_size;
  const cuuint64_t stride[4] = {row, 128, 8 * row, page};
  const auto map = [&](CUtensorMap* t, uint8_t* base) {
    return encode(t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, base, dim, stride, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!map(&m.ok, p.c.k) || !map(&m.ov, p.c.v)) return SPEC_ERR_CUDA;
  m.pk = m.ok;
  m.pv = m.ov;
  return tc_launch<PagedParams, D>(p, m, grid, stream);
}

}  // namespace

int paged_tc_bn() { return Shape<256, true>::kBn; }  // of all head sizes
static_assert(Shape<128, true>::kBn == Shape<256, true>::kBn && Shape<64, true>::kBn == Shape<256, true>::kBn);

spec_status paged_tc_launch(const PagedParams& p, int grid, EncodeTiledFn encode, cudaStream_t stream) {
  return p.D == 256   ? launch_tc<256>(p, grid, encode, stream)
         : p.D == 128 ? launch_tc<128>(p, grid, encode, stream)
                      : launch_tc<64>(p, grid, encode, stream);
}

}  // namespace spec
