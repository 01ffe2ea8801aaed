// Commit of the verify rows of a paged KV cache: the rows that are not kept become zero on their pages, in
// every layer, and the lengths move, all by what the acceptance left in device memory.
#include "paged.cuh"

namespace spec {
namespace {

// A cluster of blocks per request, so that no block reads the length after one of them has moved it; the rows
// of all layers are dealt to its warps, without a division or a table's entry for each vector (32 requests of
// 8 rows, 12 layers of 4 KB, in a graph: 7.6 us for 4.8). A verify pass drops some 3 MB at most: launch and three
// dependent loads (k and acc, the table, then the stores) are the time, not the bytes (0.4 us). Clusters of 1, 2,
// 4, 8: 8.4, 6.3, 5.2, 4.8 us there, one request of one small layer 2.3 with all.
constexpr unsigned kCommitBlocks = 8;
__global__ void __launch_bounds__(256) paged_commit_kernel(const __grid_constant__ PagedCommitParams p) {
  pdl_wait();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int64_t P = paged_len(p.c, b);
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
  // At most eight positions (m >= 0 of k + 1 <= 8): a lane finds one's place, and a warp clears a row of K or V.
  const int vecs = p.c.row_bytes / 16, lane = tid & 31, planes = 2 * p.layers;
  const int n = static_cast<int>(max(hi - lo, static_cast<int64_t>(0)));
  const int64_t place = lane < n ? paged_offset(p.c, b, static_cast<int>(lo) + lane) : -1;
  for (int u = (blockIdx.x * blockDim.x + tid) >> 5; u < n * planes; u += gridDim.x * (blockDim.x >> 5)) {
    const int row = u / planes, plane = u - row * planes;
    const int64_t at = __shfl_sync(0xffffffffu, place, row);
    if (at < 0) continue;
    uint4* to = reinterpret_cast<uint4*>((plane & 1 ? p.c.v : p.c.k) + (plane >> 1) * p.layer_stride + at);
    for (int i = lane; i < vecs; i += 32) to[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  // every block has read the length (the stores above are some lanes': the barrier takes whole warps)
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  if (blockIdx.x == 0 && tid == 0) {
    if (!bad) p.c.kv_len[b] = len;
    if (p.status) p.status[b] = bad ? SPEC_REQ_BAD_K : over ? SPEC_REQ_KV_OVERFLOW : SPEC_REQ_OK;
  }
}

}  // namespace

cudaError_t paged_commit_launch(const PagedCommitParams& p, int B, cudaStream_t stream) {
  const unsigned blocks = p.acc ? kCommitBlocks : 1;
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
