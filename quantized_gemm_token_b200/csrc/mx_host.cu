// mx_host.cu -- tensor maps of the microscaled kernels.
#include <cudaTypedefs.h>

#include <mutex>

#include "mx.h"

namespace dq {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_once;
cudaError_t g_err = cudaSuccess;

void resolve() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  g_err = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
  if (g_err == cudaSuccess && q == cudaDriverEntryPointSuccess && fn != nullptr)
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  else if (g_err == cudaSuccess)
    g_err = cudaErrorNotSupported;
}

dq_status encode(CUtensorMap* map, CUtensorMapDataType type, uint32_t rank, const void* base, const cuuint64_t* dims,
                 const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle sw) {
  std::call_once(g_once, resolve);
  if (g_encode == nullptr) return cuda_fail(g_err);
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_encode(map, type, rank, const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DQ_OK : cuda_fail(static_cast<cudaError_t>(r));
}

}  // namespace

dq_status make_tmap_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t outer,
                       uint64_t stride_bytes, uint32_t box_inner, uint32_t box_outer, int swizzle_bytes) {
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {stride_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  return encode(map, type, 2, base, dims, strides, box,
                swizzle_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE);
}

dq_status make_tmap_chunks(CUtensorMap* map, const void* base, uint64_t rows, uint64_t chunks, uint64_t stride_bytes,
                           uint32_t box_rows, uint32_t box_chunks) {
  const cuuint64_t dims[3] = {64, rows, chunks};
  const cuuint64_t strides[2] = {stride_bytes, 128};
  const cuuint32_t box[3] = {64, box_rows, box_chunks};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace dq
