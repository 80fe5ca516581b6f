// Host helpers shared by the entry points (defined in api.cu).
#pragma once

#include <cuda.h>

#include <cstdint>

#include "../../include/jgdpa.h"

namespace jg {

int host_sm_count();                       // SMs of the current device, 0 on failure
unsigned long long host_wait_limit_ns();   // limit of one internal device wait

// cuTensorMapEncodeTiled, or nullptr without a driver.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn host_encode_fn();

// Paged caches (defined in cache_api.cu).
constexpr int64_t kMaxTokens = INT32_MAX - 1024;  // so that a tile's last key is an int32, too
int page_shift_of(int32_t page_size);  // log2 of an accepted page size (a power of two, 16 to 1024 tokens), or -1
jgdpa_status check_cache(const void* k_cache, const void* v_cache, int64_t k_page_stride, int64_t v_page_stride,
                         int32_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim);

}  // namespace jg
