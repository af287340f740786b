// Tensor maps (TMA descriptors) over the latent rows of queries and cache.
#include <cuda.h>

#include "decode.h"

namespace mla {

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

typedef CUresult (*GetContextFn)(CUcontext*);

void* entry_point(const char* name) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  return cudaGetDriverEntryPoint(name, &p, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess
             ? p : nullptr;
}

struct Driver {
  EncodeTiledFn encode = reinterpret_cast<EncodeTiledFn>(entry_point("cuTensorMapEncodeTiled"));
  GetContextFn get_context = reinterpret_cast<GetContextFn>(entry_point("cuCtxGetCurrent"));
};

// The encoding fails in a host thread that has no context yet, as a thread has none before its
// first runtime call that needs one (a query of the device does not): it gets the device's own,
// as such a call would have given it.
bool have_context(const Driver& d) {
  CUcontext c = nullptr;
  if (d.get_context(&c) == CUDA_SUCCESS && c != nullptr) return true;
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
}

}  // namespace

bool encode_rows(CUtensorMap* m, const void* base, uint64_t rows, uint32_t width, uint32_t box_rows) {
  static const Driver driver;
  if (driver.encode == nullptr || driver.get_context == nullptr || !have_context(driver)) return false;
  cuuint64_t dims[2] = {width, rows};
  cuuint64_t strides[1] = {width * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t es[2] = {1, 1};
  return driver.encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mla
