// tmap.cu -- tensor maps (TMA descriptors) of row-major matrices, 128-byte swizzle.
#include <cudaTypedefs.h>

#include "internal.h"

namespace moe {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

bool encode(CUtensorMap* tm, CUtensorMapDataType type, uint64_t es, const void* ptr, uint64_t inner,
            uint64_t outer, uint32_t box_in, uint32_t box_out, uint64_t pitch,
            CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {pitch ? pitch : inner * es};
  cuuint32_t box[2] = {box_in, box_out};
  cuuint32_t estr[2] = {1, 1};
  return fn(tm, type, 2, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool encode_2d(CUtensorMap* tm, const void* ptr, uint64_t inner, uint64_t outer, uint32_t box_in,
               uint32_t box_out, bool f32, uint64_t pitch) {
  return encode(tm, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f32 ? 4 : 2, ptr,
                inner, outer, box_in, box_out, pitch);
}

bool encode_2d_narrow(CUtensorMap* tm, const void* ptr, uint64_t inner, uint64_t outer, uint32_t box_out) {
  return encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, inner, outer, 32, box_out, 0, CU_TENSOR_MAP_SWIZZLE_64B);
}

bool encode_column_blocks(CUtensorMap* tm, const void* ptr, uint64_t cols, uint64_t rows, uint32_t blocks) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {64, rows, cols / 64};
  cuuint64_t strides[2] = {cols * 2, 128};
  cuuint32_t box[3] = {64, 64, blocks};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_2d_bytes(CUtensorMap* tm, const void* ptr, uint64_t inner, uint64_t outer, uint32_t box_in, uint32_t box_out) {
  return encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, ptr, inner, outer, box_in, box_out, 0);
}

}  // namespace moe
