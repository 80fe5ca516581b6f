// Parameters of the norm and rotation kernels (rotate.cu, step_api.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace jg {

// One tensor of a call: rows of `heads` vectors each.
struct RotateJob {
  const __nv_bfloat16* x;   // input rows (backward without norm: not read)
  const __nv_bfloat16* dy;  // backward: gradient of the output
  __nv_bfloat16* y;         // output, or the input's gradient
  int64_t x_stride, dy_stride, y_stride;  // elements from one row to the next
  const float* weight;      // [D] or nullptr (1)
  const int32_t* offsets;   // [batch + 1]: segments of rows
  const int32_t* positions; // [rows], or nullptr: by the offsets
  const int32_t* slots;     // [rows]: rows go to these slots of a cache at y, or nullptr
  int64_t page_stride;      // elements from one page of that cache to the next
  int32_t rows, heads, batch;
  int32_t copy;             // as it is, neither norm nor rotation
  int64_t unit0;            // its first unit of the call's
};

struct RotateParams {
  RotateJob job[3];
  int64_t units;            // of all jobs
  const float* inv_freq;    // [pairs]
  int32_t jobs, pairs;
  int32_t run;              // vectors that a group of lanes takes after one another
  float eps;
  const int32_t* kv_lens;   // [batch]: the rows are their requests' last tokens; nullptr: positions from 0
  const int32_t* depths;    // [rows] or nullptr: places after the context instead of the row's own
  int32_t page_shift, slot_end;
  float* partial;           // backward: [grid][2][D] sums of the weights' gradients
  float* dweight[2];        // [D] each or nullptr
  int* status;              // or nullptr
};

}  // namespace jg
