// Tensor maps of the kernels on uncompressed weights.  The driver's encoder is looked up at
// run time, so that the library links against the CUDA runtime alone.
#include "dense.cuh"

namespace sesg {

namespace {
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}
}  // namespace

cudaError_t dense_map(CUtensorMap* m, const void* base, int bf16, uint64_t cols, uint64_t rows, uint64_t row_stride,
                      uint64_t z, uint64_t z_stride, uint32_t box_rows) {
  const EncodeFn fn = encoder();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {cols, rows, z};
  const cuuint64_t strides[2] = {row_stride * 2, z_stride * 2};
  const cuuint32_t box[3] = {(cuuint32_t)kDnChunk, box_rows, 1};
  const cuuint32_t step[3] = {1, 1, 1};
  const CUresult r =
      fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, z ? 3 : 2,
         const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace sesg
