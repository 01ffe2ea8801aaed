// Host helpers shared by the entry points: device attributes, the tensor-map encoder, checks.
#pragma once

#include <stdint.h>

#include <atomic>

#include <cuda.h>
#include <cuda_runtime.h>

#include "spec.h"

namespace spec {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled from the CUDA driver API, fetched through the runtime (no -lcuda).
inline EncodeTiledFn lookup_encode_tiled() {
  void* ptr = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                       &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    return reinterpret_cast<EncodeTiledFn>(ptr);
  return nullptr;
}

inline EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = lookup_encode_tiled();  // looked up once, by the first caller
  return fn;
}

struct DevAttr {
  int sms = 0;
  int smem_optin = 0;
};

// Per-device attributes, queried on first use. Calls may come from several host threads: the
// cache is atomic (sms is published last, so a non-zero sms implies smem_optin is set).
inline DevAttr dev_attr() {
  struct Slot {
    std::atomic<int> sms{0};
    std::atomic<int> smem_optin{0};
  };
  static Slot cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DevAttr{};
  DevAttr a;
  a.sms = cache[dev].sms.load(std::memory_order_acquire);
  if (a.sms != 0) {
    a.smem_optin = cache[dev].smem_optin.load(std::memory_order_relaxed);
    return a;
  }
  if (cudaDeviceGetAttribute(&a.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&a.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
          cudaSuccess)
    return DevAttr{};
  cache[dev].smem_optin.store(a.smem_optin, std::memory_order_relaxed);
  cache[dev].sms.store(a.sms, std::memory_order_release);
  return a;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace spec
