// Host-side encoding of TMA tensor maps through the driver entry point
// (the runtime library does not export cuTensorMapEncodeTiled itself).
#include <mutex>

#include <cudaTypedefs.h>

#include "kernels.h"

namespace v4kv {

namespace {
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;
}  // namespace

cudaError_t encode_cols_u8(CUtensorMap* map, const void* base, uint64_t rows, uint32_t row_bytes,
                           uint32_t box_bytes, uint32_t box_rows) {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) return cudaErrorNotSupported;
  if ((reinterpret_cast<uintptr_t>(base) & 15) || row_bytes % 16 || box_bytes % 16 ||
      box_bytes > 128 || rows == 0)
    return cudaErrorInvalidValue;
  const cuuint64_t dims[2] = {row_bytes, rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_bytes, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t encode_rows_u8(CUtensorMap* map, const void* base, uint64_t rows, uint32_t row_bytes,
                           uint32_t box_rows) {
  return encode_cols_u8(map, base, rows, row_bytes, row_bytes, box_rows);
}

}  // namespace v4kv
