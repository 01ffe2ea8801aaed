// Attention of new rows over a paged cache: the CUDA-core kernel and the join of trunk/attn.cuh for it.
#include "trunk/attn.cuh"

#include "paged.cuh"

namespace spec {

cudaError_t paged_simt_launch(const PagedParams& p, spec_dtype dtype, int grid, cudaStream_t stream) {
  return dtype == SPEC_BF16 ? simt_launch<PagedParams, __nv_bfloat16>(p, grid, stream)
                            : simt_launch<PagedParams, float>(p, grid, stream);
}

cudaError_t paged_join_launch(const PagedParams& p, spec_dtype dtype, int sms, cudaStream_t stream) {
  return join_launch(p, p.rows, dtype, sms, stream);
}

}  // namespace spec
