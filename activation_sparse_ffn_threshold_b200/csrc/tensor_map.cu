// tensor_map.cu -- host side of the TMA descriptors (the driver's encoder is looked up at
// run time, so the library needs no link against the driver).
#include <cuda_runtime.h>

#include "umma.cuh"

namespace sfnn {
namespace {

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// The encoder needs a current context; a thread that has made no runtime call that binds one
// (an autograd worker) has none.  cudaSetDevice on the thread's own device binds it.
bool bind_context() {
  thread_local int bound = -1;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev != bound) {
    if (cudaSetDevice(dev) != cudaSuccess) return false;
    bound = dev;
  }
  return true;
}

}  // namespace

bool make_tensor_map(CUtensorMap *out, const void *base, int esize, int64_t rows, int64_t cols, int64_t ld,
                     int box_rows, int box_cols, bool swizzle) {
  const EncodeFn fn = encoder();
  if (!fn || !bind_context()) return false;
  const CUtensorMapDataType dt = esize == 2   ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                                 : esize == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                              : CU_TENSOR_MAP_DATA_TYPE_UINT32;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * esize};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  const cuuint32_t step[2] = {1, 1};
  return fn(out, dt, 2, const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sfnn
