// Host-side launch helpers shared by the translation units that hold kernels:
// the tensor-map encoder, launches with programmatic stream serialization and
// the once-per-device shared-memory limit.
#pragma once

#include <atomic>
#include <mutex>
#include <utility>

#include <cuda.h>
#include <cuda_runtime.h>

#include "dora_internal.h"

namespace dora {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// Launch with programmatic stream serialization so the kernel's prologue can
// overlap the previous kernel's tail (see pdl_wait / pdl_trigger).
template <class... KArgs, class... Args>
inline cudaError_t launch_pdl_if(bool early, void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                 cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  // Under the kernel profiler each launch is timed on its own: no early start.
  attr[0].val.programmaticStreamSerializationAllowed = (early && !profiling_on()) ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

template <class... KArgs, class... Args>
inline cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                              Args&&... args) {
  return launch_pdl_if(true, kern, grid, block, smem, st, std::forward<Args>(args)...);
}

// Raise the kernel's dynamic shared-memory limit once per device; `done` is
// the caller's own flag word (one per kernel instantiation).
template <class Kern>
inline cudaError_t set_smem_once(std::atomic<unsigned long long>& done, Kern kern, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load() & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

}  // namespace dora
