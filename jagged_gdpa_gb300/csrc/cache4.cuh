// The paged cache held in 4 bits: parameters and layout (cache4.cu,
// cache4_fwd.cu, step_api.cu).
//
// A page holds page_size tokens of every key/value head, head by head: codes
// [kv_heads][page_size][D / 2] bytes, two columns a byte, the even one in the low
// bits, and scales [kv_heads][page_size][2] bf16, a step s and a middle z for each token's
// head.  A code c stands for z + s (c - 8).  Head by head, so that the tokens
// that one head of the attention reads lie side by side (a token's 64 bytes of D =
// 128 by themselves would be a quarter of the 256 that DRAM fetches best).
#pragma once

#include <cuda_bf16.h>

#include "cache.cuh"

namespace jg {

// Query rows per item of the attention kernel, and its CTAs per SM with 8 nq of
// them: as many as registers allow (D = 128: 157 to 160 a thread with one set of columns, 226 to
// 241 with two, whose 84 KB of shared memory a third CTA would not find either; D = 64: 114 to 125
// and 165 to 168; D = 32: 91 to 96 and 141 to 160).
constexpr int kCache4Rows = 16;
constexpr int kCache4MinRange = 5;  // the least length of a CTA's range on the line of items
__host__ __device__ constexpr int cache4_ctas(int d, int nq) { return d == 128 ? 4 - nq : nq == 2 ? 3 : d == 64 ? 4 : 5; }
inline int cache4_columns(int64_t rows) { return rows <= 8 ? 1 : 2; }

struct Cache4 {  // K or V
  uint8_t* codes;
  __nv_bfloat16* scales;
  int64_t code_stride, scale_stride;  // bytes, elements from one page to the next
};

struct Cache4FwdParams {
  CacheFwdParams f;  // (without its tensor maps and pointers to K and V)
  Cache4 k, v;
};

struct Cache4RowsParams {  // rows [heads][D] to or from their slots
  const __nv_bfloat16* in[2];  // K and V rows
  __nv_bfloat16* out[2];
  int64_t stride[2];           // elements from one row to the next
  Cache4 cache[2];
  const int32_t* slots;
  int32_t rows, heads, page_shift, slot_end;
};

}  // namespace jg
