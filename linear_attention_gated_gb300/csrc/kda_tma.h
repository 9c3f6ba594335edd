// kda_tma.h -- host side of the tiled copies: a map of [tokens, heads, 128] BF16 tensors, copied in
// boxes of 64 elements by `rows` tokens of one head in the 128-byte swizzle, and one of states.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace kda {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The CUDA driver's encoder, looked up once (the runtime is linked statically and the driver not at all).
inline EncodeTiled encode_tiled() {
  static const EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return f;
}

// Strides in elements, multiples of 8; base 16-byte aligned. Tokens past the end read as zeros.
inline cudaError_t token_map(CUtensorMap* map, const void* base, int64_t heads, int64_t tokens, int64_t head_stride,
                             int64_t token_stride, uint32_t rows) {
  const EncodeTiled f = encode_tiled();
  if (!f) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {128, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)token_stride * 2};
  const cuuint32_t box[3] = {64, 1, rows}, step[3] = {1, 1, 1};
  const CUresult r = f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// States [slots, heads, 128, 128], BF16 or FP32, in boxes of 128 bytes (64 or 32 columns) by 128 rows in the 128-byte swizzle.
inline cudaError_t state_map(CUtensorMap* map, const void* base, bool bf16, int64_t heads, int64_t slots) {
  const EncodeTiled f = encode_tiled();
  if (!f) return cudaErrorNotSupported;
  const cuuint64_t es = bf16 ? 2 : 4;
  const cuuint64_t dims[4] = {128, 128, (cuuint64_t)heads, (cuuint64_t)slots};
  const cuuint64_t strides[3] = {128 * es, 128 * 128 * es, (cuuint64_t)heads * 128 * 128 * es};
  const cuuint32_t box[4] = {(cuuint32_t)(128 / es), 128, 1, 1}, step[4] = {1, 1, 1, 1};
  const CUresult r = f(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<void*>(base), dims,
                       strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace kda
