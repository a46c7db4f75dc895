// opq_host.h — host helpers shared by the library's translation units (defined in opq_capi.cu
// and opq_fp8.cu; not exported).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "opq.h"

#define OPQ_INTERNAL __attribute__((visibility("hidden")))

namespace opqhost {

// records the error for opq_last_cuda_error and returns OPQ_ERR_CUDA
OPQ_INTERNAL opq_status cuda_fail(int code);
// every pointer non-null, then 16-byte aligned, then device-accessible
OPQ_INTERNAL opq_status check_ptrs(std::initializer_list<const void *> ptrs);
// every pointer device-accessible (no alignment asked)
OPQ_INTERNAL opq_status check_device(std::initializer_list<const void *> ptrs);

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
OPQ_INTERNAL EncodeTiledFn encode_fn();

// opq_fp8.cu keeps its own copies of the device error word and the wait limit (device symbols
// belong to their translation unit): read-and-clear, set and read
OPQ_INTERNAL cudaError_t fp8_device_error(uint32_t *err);
OPQ_INTERNAL cudaError_t fp8_set_wait_limit(uint64_t ns);
OPQ_INTERNAL cudaError_t fp8_get_wait_limit(uint64_t *ns);

}  // namespace opqhost
