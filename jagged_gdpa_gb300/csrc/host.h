// Host helpers shared by the entry points (defined in api.cu).
#pragma once

#include <cuda.h>

namespace jg {

int host_sm_count();                       // SMs of the current device, 0 on failure
unsigned long long host_wait_limit_ns();   // limit of one internal device wait

// cuTensorMapEncodeTiled, or nullptr without a driver.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn host_encode_fn();

}  // namespace jg
