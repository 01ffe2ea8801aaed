// Attention of the verify rows over a shared prefix and each request's own cache: the CUDA-core kernel and
// the join of attn.cuh for it.
#include "attn.cuh"

namespace spec {

int attn_simt_tm() { return kSimtTm; }
int attn_simt_bn() { return kSimtBn; }

cudaError_t attn_simt_launch(const AttnParams& p, spec_dtype dtype, int grid, cudaStream_t stream) {
  return dtype == SPEC_BF16 ? simt_launch<AttnParams, __nv_bfloat16>(p, grid, stream)
                            : simt_launch<AttnParams, float>(p, grid, stream);
}

cudaError_t attn_join_launch(const AttnParams& p, spec_dtype dtype, int sms, cudaStream_t stream) {
  return join_launch(p, static_cast<int64_t>(p.B) * p.R, dtype, sms, stream);
}

}  // namespace spec
