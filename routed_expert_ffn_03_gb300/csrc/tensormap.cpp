// tensormap.cpp - tensor maps for TMA loads, through the driver's encoder (found at run time, so the
// library needs no link against libcuda).
#include "grouped.h"

namespace moe {

bool tensor_map(CUtensorMap* m, const void* base, size_t elem, int rank, const uint64_t* dims, const uint64_t* strides,
                const uint32_t* box) {
  if ((uintptr_t)base % 16) return false;
  for (int i = 0; i < rank; ++i)
    if (dims[i] < 1 || dims[i] > 0xffffffffull || (i + 1 < rank && (strides[i] % 16 || strides[i] >= (1ull << 40)))) return false;
  if (!m) return true;
  typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return (Encode)f;
  }();
  if (!encode) return false;
  cuuint64_t d[5], st[4];
  cuuint32_t b[5], es[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    es[i] = 1;
  }
  for (int i = 0; i + 1 < rank; ++i) st[i] = strides[i];
  return encode(m, elem == 4   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                   : elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                               : CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), d, st, b, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
