// attn_res_tensor_host.cuh -- host side shared by the launches of the
// tensor-core kernels.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace attn_res_host {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline cudaError_t encode_tiled(EncodeTiled* out) {
  static std::atomic<void*> found{nullptr};
  void* f = found.load(std::memory_order_acquire);
  if (f == nullptr) {
    cudaDriverEntryPointQueryResult state;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                     cudaEnableDefault, &state);
    if (e != cudaSuccess) return e;
    if (state != cudaDriverEntryPointSuccess || f == nullptr) return cudaErrorNotSupported;
    found.store(f, std::memory_order_release);
  }
  *out = reinterpret_cast<EncodeTiled>(f);
  return cudaSuccess;
}

// Tensor map of rows of `cols` elements, `row_bytes` apart: boxes of box_cols x
// box_rows; elements past the row's end and rows past the last read as 0.
inline cudaError_t map_2d(CUtensorMapDataType type, const void* at, int64_t cols, int64_t rows, int64_t row_bytes,
                          uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle, CUtensorMap* map) {
  EncodeTiled enc;
  cudaError_t e = encode_tiled(&enc);
  if (e != cudaSuccess) return e;
  const cuuint64_t dim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t stride[1] = {(cuuint64_t)row_bytes};
  const cuuint32_t box[2] = {box_cols, box_rows};
  const cuuint32_t one[2] = {1, 1};
  const CUresult r = enc(map, type, 2, const_cast<void*>(at), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The dynamic shared memory above 48 KB is opt-in, per function and device.
template <class Kern>
cudaError_t allow_smem(Kern kern, uint32_t bytes, int device, std::atomic<uint64_t>& enabled) {
  const uint64_t bit = 1ull << device;
  if (!(enabled.load(std::memory_order_acquire) & bit)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    enabled.fetch_or(bit, std::memory_order_acq_rel);
  }
  return cudaSuccess;
}

}  // namespace attn_res_host
