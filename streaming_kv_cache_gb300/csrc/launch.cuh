// Host-side helpers of the tensor-core launches.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>

namespace skv {

PFN_cuTensorMapEncodeTiled_v12000 tmap_encode_fn();

// SM count of the current device, asked once (threads that race store the same value)
int sm_count();

// Opt in to `bytes` of dynamic shared memory, once per device and variant of
// the kernels of one signature.
template <typename K>
cudaError_t set_smem_once(K kernel, int bytes, int variant) {
  static std::atomic<int> done[64][32];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev][variant].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev][variant].store(1, std::memory_order_relaxed);
  return e;
}

inline bool encode_3d(CUtensorMap* m, bool f16, const void* base, const cuuint64_t (&dims)[3],
                      const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3]) {
  auto fn = tmap_encode_fn();
  const cuuint32_t es[3] = {1, 1, 1};
  return fn && fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace skv
