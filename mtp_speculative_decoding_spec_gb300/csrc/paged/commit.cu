// Commit of the verify rows of a paged KV cache: the rows that are not kept become zero on their pages, in
// every layer, and the lengths move, all by what the acceptance left in device memory.
#include "paged.cuh"

namespace spec {
namespace {

// A cluster of blocks per request, so that no block reads the length after one of them has moved it. A
// verify pass of 32 requests drops some 100 rows of 4 KB a layer: launch and three dependent loads (k and
// acc, the table, then the stores) are the time, not the bytes.
__global__ void __launch_bounds__(256) paged_commit_kernel(const __grid_constant__ PagedCommitParams p) {
  pdl_wait();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int64_t P = max(static_cast<int64_t>(0), p.c.kv_len[b]);
  const int64_t cap = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
  const int k = p.k[b];
  int64_t len = P, lo = 0, hi = 0;  // the new length, and the positions to clear
  bool bad = k < 0 || (p.acc && k >= kMaxRows), over = false;
  if (!bad) {
    const int m = !p.acc ? k : p.acc[b].status != SPEC_REQ_OK ? 0 : max(0, min(p.acc[b].n_emit, k + 1));
    const int64_t end = P + k + (p.acc ? 1 : 0);
    len = lo = P + m;
    over = end > cap;
    hi = min(end, cap);
  }
  const int vecs = p.c.row_bytes / 16;
  const int64_t n = hi > lo ? (hi - lo) * 2 * p.layers * vecs : 0;
  for (int64_t i = blockIdx.x * blockDim.x + tid; i < n; i += gridDim.x * blockDim.x) {
    const int64_t row = i / vecs;
    const int within = static_cast<int>(i - row * vecs);
    const int pos = static_cast<int>(lo + row / (2 * p.layers)), plane = static_cast<int>(row % (2 * p.layers));
    const int64_t at = paged_offset(p.c, b, pos);
    if (at < 0) continue;
    uint8_t* pages = plane & 1 ? p.c.v : p.c.k;
    reinterpret_cast<uint4*>(pages + (plane >> 1) * p.layer_stride + at)[within] = make_uint4(0u, 0u, 0u, 0u);
  }
  // every block has read the length
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  if (blockIdx.x == 0 && tid == 0) {
    if (!bad) p.c.kv_len[b] = len;
    if (p.status) p.status[b] = bad ? SPEC_REQ_BAD_K : over ? SPEC_REQ_KV_OVERFLOW : SPEC_REQ_OK;
  }
}

}  // namespace

cudaError_t paged_commit_launch(const PagedCommitParams& p, int B, cudaStream_t stream) {
  // the blocks of a request: one for as many bytes as its 256 threads store in two turns, at most eight
  const int64_t most = static_cast<int64_t>(kMaxRows - 1) * 2 * p.layers * p.c.row_bytes;
  const unsigned blocks = p.acc && most > 2 * 256 * 16 ? (most > 8 * 256 * 16 ? 8 : 4) : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, B);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, paged_commit_kernel, p);
}

}  // namespace spec
