// Parameters of the verification of drafted tokens (verify.cu, step_api.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace jg {

constexpr int kVerifyMaxTokens = 1024;  // rows of a request

struct VerifyParams {
  const void* target;       // probabilities [total][vocab], fp32 or bf16
  const void* draft;        // the same of the draft, or nullptr
  int64_t target_stride, draft_stride;
  const int32_t* tokens;    // [total]
  const int32_t* parents;   // [total] or nullptr: chains
  const float* uniforms;    // [total]
  const int32_t* q_off;     // [batch + 1]
  const int32_t* kv_lens;   // [batch] or nullptr
  const int32_t* slots;     // [total] or nullptr
  int32_t total, batch, vocab;
  int32_t* accepted;        // [batch]
  int32_t* next;            // [batch]
  int32_t* places;          // [total]
  int32_t* keep_lens;       // [batch] or nullptr
  int32_t* keep_slots;      // [total] or nullptr
  int* status;              // or nullptr
};

}  // namespace jg
