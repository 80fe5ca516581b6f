// Entry points around the attention calls: norms with rotation, rotated cache
// writes, verification of drafted tokens, the cache held in 4 bits.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/jgdpa.h"
#include "act.cuh"
#include "cache.cuh"
#include "cache4.cuh"
#include "host.h"
#include "rotate.cuh"
#include "verify.cuh"

namespace jg {
cudaError_t launch_rotate(const RotateParams& p, int head_dim, bool norm, bool pairs, int sms, cudaStream_t stream);
cudaError_t launch_rotate_back(const RotateParams& p, int head_dim, bool norm, bool pairs, int sms, cudaStream_t stream);
size_t rotate_back_partial_bytes(int head_dim, int sms);
cudaError_t launch_verify(const VerifyParams& p, bool target_half, bool draft_half, int sms, cudaStream_t stream);
cudaError_t launch_cache4_rows(const Cache4RowsParams& p, int head_dim, bool append, int sms, cudaStream_t stream);
template <int D>
cudaError_t launch_cache4_fwd_d(const Cache4FwdParams& p, int act, int grid, cudaStream_t stream);
template <int D>
cudaError_t launch_cache_join_d(const CacheFwdParams& p, int act, int n_ctas, int tile_rows, cudaStream_t stream);
}  // namespace jg

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxStride = int64_t{1} << 39;
constexpr int32_t kMaxBatch = 1 << 30;  // (its offsets are searched and counted in 32 bits)
size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool head_dim_ok(int32_t d) { return d == 32 || d == 64 || d == 128; }

#define JG_CUDA(x)                                 \
  do {                                             \
    if ((x) != cudaSuccess) return JGDPA_ERR_CUDA; \
  } while (0)
#define JG_CHECK(x)                              \
  do {                                           \
    const jgdpa_status st_ = (x);                \
    if (st_ != JGDPA_OK) return st_;             \
  } while (0)

// An optional workspace for the status word alone.
jgdpa_status check_status(void* workspace, size_t bytes, size_t need) {
  if (workspace == nullptr) return JGDPA_OK;
  if (bytes < need) return JGDPA_ERR_WORKSPACE_TOO_SMALL;
  return aligned(workspace, kAlign) ? JGDPA_OK : JGDPA_ERR_MISALIGNED;
}

// Rows [heads][head_dim], stride elements apart.
jgdpa_status check_rows(const void* x, int64_t stride, int64_t rows, int32_t heads, int32_t head_dim) {
  if (rows == 0) return JGDPA_OK;
  if (x == nullptr || stride < static_cast<int64_t>(heads) * head_dim) return JGDPA_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || stride % 8) return JGDPA_ERR_MISALIGNED;
  return stride < kMaxStride ? JGDPA_OK : JGDPA_ERR_UNSUPPORTED;
}

// What the calls with a rotation share.
jgdpa_status check_rotation(const float* inv_freq, int32_t pairs, int32_t interleaved, int32_t norm, float eps,
                            int32_t head_dim, const float* q_weight, const float* k_weight) {
  if (pairs < 1 || (interleaved != 0 && interleaved != 1) || (norm != 0 && norm != 1)) return JGDPA_ERR_INVALID_ARGUMENT;
  if (!head_dim_ok(head_dim)) return JGDPA_ERR_UNSUPPORTED;
  if (pairs > head_dim / 2 || inv_freq == nullptr) return JGDPA_ERR_INVALID_ARGUMENT;
  if (!interleaved && pairs % 8) return JGDPA_ERR_UNSUPPORTED;
  if (norm ? !(std::isfinite(eps) && eps >= 0.f) : (q_weight != nullptr || k_weight != nullptr))
    return JGDPA_ERR_INVALID_ARGUMENT;
  if (!aligned(inv_freq, 4) || !aligned(q_weight, 4) || !aligned(k_weight, 4)) return JGDPA_ERR_MISALIGNED;
  return JGDPA_OK;
}

jgdpa_status check_segments(int64_t rows, int32_t heads, int32_t batch, const int32_t* offsets, const int32_t* positions) {
  if (rows < 0 || batch < 0 || heads < 0 || (rows > 0 && heads < 1)) return JGDPA_ERR_INVALID_ARGUMENT;
  if (rows > INT32_MAX || rows * std::max<int64_t>(heads, 1) > INT32_MAX || batch > kMaxBatch) return JGDPA_ERR_UNSUPPORTED;
  if (rows > 0 && offsets == nullptr && positions == nullptr) return JGDPA_ERR_INVALID_ARGUMENT;
  if (!aligned(offsets, 4) || !aligned(positions, 4)) return JGDPA_ERR_MISALIGNED;
  return JGDPA_OK;
}

jg::RotateJob rotate_job(const void* x, int64_t x_stride, void* y, int64_t y_stride, int64_t rows, int32_t heads,
                         const int32_t* offsets, const int32_t* positions, int32_t batch, const float* weight) {
  jg::RotateJob j{};
  j.x = static_cast<const __nv_bfloat16*>(x);
  j.x_stride = x_stride;
  j.y = static_cast<__nv_bfloat16*>(y);
  j.y_stride = y_stride;
  j.rows = static_cast<int32_t>(rows);
  j.heads = heads;
  j.batch = batch;
  j.offsets = offsets;
  j.positions = positions;
  j.weight = weight;
  return j;
}

// The status word starts at 0; kernels write it only where something is wrong.
jgdpa_status start_status(int** status, void* workspace, cudaStream_t stream) {
  *status = static_cast<int*>(workspace);
  if (workspace != nullptr) JG_CUDA(cudaMemsetAsync(workspace, 0, sizeof(int), stream));
  return JGDPA_OK;
}

jgdpa_status check_cache4(const void* codes, const void* scales, int64_t code_stride, int64_t scale_stride,
                          int32_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim) {
  if (num_pages < 1 || page_size < 1 || kv_heads < 1) return JGDPA_ERR_INVALID_ARGUMENT;
  if (!head_dim_ok(head_dim) || jg::page_shift_of(page_size) < 0 || kv_heads > 65535 ||
      static_cast<int64_t>(num_pages) * page_size > jg::kMaxTokens)
    return JGDPA_ERR_UNSUPPORTED;
  if (codes == nullptr || scales == nullptr) return JGDPA_ERR_INVALID_ARGUMENT;
  const int64_t tokens = static_cast<int64_t>(page_size) * kv_heads;
  if (code_stride < tokens * (head_dim / 2) || scale_stride < tokens * 2) return JGDPA_ERR_INVALID_ARGUMENT;
  if (code_stride >= kMaxStride || scale_stride >= kMaxStride) return JGDPA_ERR_UNSUPPORTED;
  if (!aligned(codes, 16) || !aligned(scales, 16) || code_stride % 16 || scale_stride % 8) return JGDPA_ERR_MISALIGNED;
  return JGDPA_OK;
}
jg::Cache4 cache4(const void* codes, const void* scales, int64_t code_stride, int64_t scale_stride) {
  return {static_cast<uint8_t*>(const_cast<void*>(codes)), static_cast<__nv_bfloat16*>(const_cast<void*>(scales)),
          code_stride, scale_stride};
}

jgdpa_status cache4_rows(bool append, const void* k_in, const void* v_in, void* k_out, void* v_out, int64_t k_stride,
                         int64_t v_stride, const int32_t* slots, int32_t rows, jg::Cache4 k, jg::Cache4 v,
                         int32_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim, cudaStream_t stream) {
  if (rows < 0) return JGDPA_ERR_INVALID_ARGUMENT;
  JG_CHECK(check_cache4(k.codes, k.scales, k.code_stride, k.scale_stride, num_pages, page_size, kv_heads, head_dim));
  JG_CHECK(check_cache4(v.codes, v.scales, v.code_stride, v.scale_stride, num_pages, page_size, kv_heads, head_dim));
  if (rows == 0) return JGDPA_OK;
  JG_CHECK(check_rows(append ? k_in : k_out, k_stride, rows, kv_heads, head_dim));
  JG_CHECK(check_rows(append ? v_in : v_out, v_stride, rows, kv_heads, head_dim));
  if (slots == nullptr) return JGDPA_ERR_INVALID_ARGUMENT;
  if (!aligned(slots, 4)) return JGDPA_ERR_MISALIGNED;
  if (static_cast<int64_t>(rows) * kv_heads > INT32_MAX) return JGDPA_ERR_UNSUPPORTED;
  const int sms = jg::host_sm_count();
  if (sms <= 0) return JGDPA_ERR_CUDA;
  jg::Cache4RowsParams p{};
  p.in[0] = static_cast<const __nv_bfloat16*>(k_in);
  p.in[1] = static_cast<const __nv_bfloat16*>(v_in);
  p.out[0] = static_cast<__nv_bfloat16*>(k_out);
  p.out[1] = static_cast<__nv_bfloat16*>(v_out);
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.cache[0] = k;
  p.cache[1] = v;
  p.slots = slots;
  p.rows = rows;
  p.heads = kv_heads;
  p.page_shift = jg::page_shift_of(page_size);
  p.slot_end = num_pages * page_size;
  JG_CUDA(jg::launch_cache4_rows(p, head_dim, append, sms, stream));
  return JGDPA_OK;
}

struct Cache4Layout {
  size_t err, join, part_ml, part_o, total;
  int sms, grid;  // grid: CTAs at most
};
bool cache4_layout(int32_t head_dim, Cache4Layout* L) {
  const int sms = jg::host_sm_count();
  if (sms <= 0) return false;
  L->sms = sms;
  L->grid = sms * std::max(jg::cache4_ctas(head_dim, 1), jg::cache4_ctas(head_dim, 2));
  const size_t parts = 2 * static_cast<size_t>(L->grid) * jg::kCache4Rows;
  size_t off = kAlign;  // the status word
  L->err = off;
  off += up(L->grid * sizeof(int));
  L->join = off;
  off += up(L->grid * sizeof(jg::CacheJoin));
  L->part_ml = off;
  off += up(parts * sizeof(float2));
  L->part_o = off;
  off += up(parts * head_dim * sizeof(float));
  L->total = off;
  return true;
}

}  // namespace

extern "C" {

size_t jgdpa_norm_rotate_workspace_bytes(int32_t head_dim, int32_t for_backward) {
  if (!head_dim_ok(head_dim)) return 0;
  if (!for_backward) return kAlign;
  const int sms = jg::host_sm_count();
  return sms <= 0 ? 0 : kAlign + jg::rotate_back_partial_bytes(head_dim, sms);
}

jgdpa_status jgdpa_norm_rotate(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int64_t total_q,
                               int32_t heads, const int32_t* q_offsets, const int32_t* q_positions,
                               const float* q_weight, const void* k, int64_t k_stride, void* k_out,
                               int64_t k_out_stride, int64_t total_kv, int32_t kv_heads, const int32_t* kv_offsets,
                               const int32_t* k_positions, const float* k_weight, int32_t batch, int32_t head_dim,
                               const float* inv_freq, int32_t pairs, int32_t interleaved, int32_t norm, float eps,
                               void* workspace, size_t workspace_bytes, jgdpa_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  JG_CHECK(check_rotation(inv_freq, pairs, interleaved, norm, eps, head_dim, q_weight, k_weight));
  JG_CHECK(check_segments(total_q, heads, batch, q_offsets, q_positions));
  JG_CHECK(check_segments(total_kv, kv_heads, batch, kv_offsets, k_positions));
  JG_CHECK(check_rows(q, q_stride, total_q, heads, head_dim));
  JG_CHECK(check_rows(q_out, q_out_stride, total_q, heads, head_dim));
  JG_CHECK(check_rows(k, k_stride, total_kv, kv_heads, head_dim));
  JG_CHECK(check_rows(k_out, k_out_stride, total_kv, kv_heads, head_dim));
  JG_CHECK(check_status(workspace, workspace_bytes, kAlign));
  const int sms = jg::host_sm_count();
  if (sms <= 0) return JGDPA_ERR_CUDA;
  jg::RotateParams p{};
  if (total_q > 0)
    p.job[p.jobs++] = rotate_job(q, q_stride, q_out, q_out_stride, total_q, heads, q_offsets, q_positions, batch, q_weight);
  if (total_kv > 0)
    p.job[p.jobs++] = rotate_job(k, k_stride, k_out, k_out_stride, total_kv, kv_heads, kv_offsets, k_positions, batch, k_weight);
  p.inv_freq = inv_freq;
  p.pairs = pairs;
  p.eps = eps;
  JG_CHECK(start_status(&p.status, workspace, stream));
  if (p.jobs == 0) return JGDPA_OK;
  JG_CUDA(jg::launch_rotate(p, head_dim, norm != 0, interleaved != 0, sms, stream));
  return JGDPA_OK;
}

jgdpa_status jgdpa_norm_rotate_bwd(const void* dq_out, int64_t dq_out_stride, const void* q, int64_t q_stride, void* dq,
                                   int64_t dq_stride, int64_t total_q, int32_t heads, const int32_t* q_offsets,
                                   const int32_t* q_positions, const float* q_weight, float* dq_weight,
                                   const void* dk_out, int64_t dk_out_stride, const void* k, int64_t k_stride, void* dk,
                                   int64_t dk_stride, int64_t total_kv, int32_t kv_heads, const int32_t* kv_offsets,
                                   const int32_t* k_positions, const float* k_weight, float* dk_weight, int32_t batch,
                                   int32_t head_dim, const float* inv_freq, int32_t pairs, int32_t interleaved,
                                   int32_t norm, float eps, void* workspace, size_t workspace_bytes,
                                   jgdpa_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  JG_CHECK(check_rotation(inv_freq, pairs, interleaved, norm, eps, head_dim, q_weight, k_weight));
  JG_CHECK(check_segments(total_q, heads, batch, q_offsets, q_positions));
  JG_CHECK(check_segments(total_kv, kv_heads, batch, kv_offsets, k_positions));
  JG_CHECK(check_rows(dq_out, dq_out_stride, total_q, heads, head_dim));
  JG_CHECK(check_rows(dq, dq_stride, total_q, heads, head_dim));
  JG_CHECK(check_rows(dk_out, dk_out_stride, total_kv, kv_heads, head_dim));
  JG_CHECK(check_rows(dk, dk_stride, total_kv, kv_heads, head_dim));
  if (norm) {
    JG_CHECK(check_rows(q, q_stride, total_q, heads, head_dim));
    JG_CHECK(check_rows(k, k_stride, total_kv, kv_heads, head_dim));
  }
  const bool weights = dq_weight != nullptr || dk_weight != nullptr;
  if (weights && !norm) return JGDPA_ERR_INVALID_ARGUMENT;
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return JGDPA_ERR_MISALIGNED;
  const int sms = jg::host_sm_count();
  if (sms <= 0) return JGDPA_ERR_CUDA;
  if (weights && workspace == nullptr) return JGDPA_ERR_WORKSPACE_TOO_SMALL;
  JG_CHECK(check_status(workspace, workspace_bytes, weights ? kAlign + jg::rotate_back_partial_bytes(head_dim, sms) : kAlign));
  jg::RotateParams p{};
  if (total_q > 0) {
    jg::RotateJob& j = p.job[p.jobs];
    j = rotate_job(q, q_stride, dq, dq_stride, total_q, heads, q_offsets, q_positions, batch, q_weight);
    j.dy = static_cast<const __nv_bfloat16*>(dq_out);
    j.dy_stride = dq_out_stride;
    p.dweight[p.jobs++] = dq_weight;
  } else if (dq_weight != nullptr) {
    JG_CUDA(cudaMemsetAsync(dq_weight, 0, head_dim * sizeof(float), stream));
  }
  if (total_kv > 0) {
    jg::RotateJob& j = p.job[p.jobs];
    j = rotate_job(k, k_stride, dk, dk_stride, total_kv, kv_heads, kv_offsets, k_positions, batch, k_weight);
    j.dy = static_cast<const __nv_bfloat16*>(dk_out);
    j.dy_stride = dk_out_stride;
    p.dweight[p.jobs++] = dk_weight;
  } else if (dk_weight != nullptr) {
    JG_CUDA(cudaMemsetAsync(dk_weight, 0, head_dim * sizeof(float), stream));
  }
  p.inv_freq = inv_freq;
  p.pairs = pairs;
  p.eps = eps;
  JG_CHECK(start_status(&p.status, workspace, stream));
  if (p.jobs == 0) return JGDPA_OK;
  if (weights) p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kAlign);
  JG_CUDA(jg::launch_rotate_back(p, head_dim, norm != 0, interleaved != 0, sms, stream));
  return JGDPA_OK;
}

jgdpa_status jgdpa_cache_append_rotated(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                                        int32_t heads, const void* k_new, const void* v_new, int64_t k_stride,
                                        int64_t v_stride, const int32_t* slots, int32_t total_new, void* k_cache,
                                        void* v_cache, int64_t k_page_stride, int64_t v_page_stride, int32_t num_pages,
                                        int32_t page_size, int32_t kv_heads, int32_t head_dim,
                                        const int32_t* q_offsets, const int32_t* kv_lens, const int32_t* depths,
                                        int32_t batch, const float* q_weight, const float* k_weight,
                                        const float* inv_freq, int32_t pairs, int32_t interleaved, int32_t norm,
                                        float eps, void* workspace, size_t workspace_bytes, jgdpa_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (total_new < 0 || batch < 0 || heads < 0) return JGDPA_ERR_INVALID_ARGUMENT;
  JG_CHECK(jg::check_cache(k_cache, v_cache, k_page_stride, v_page_stride, num_pages, page_size, kv_heads, head_dim));
  JG_CHECK(check_rotation(inv_freq, pairs, interleaved, norm, eps, head_dim, q_weight, k_weight));
  JG_CHECK(check_status(workspace, workspace_bytes, kAlign));
  if (heads > 0) {
    JG_CHECK(check_rows(q, q_stride, total_new, heads, head_dim));
    JG_CHECK(check_rows(q_out, q_out_stride, total_new, heads, head_dim));
  }
  JG_CHECK(check_rows(k_new, k_stride, total_new, kv_heads, head_dim));
  JG_CHECK(check_rows(v_new, v_stride, total_new, kv_heads, head_dim));
  if (static_cast<int64_t>(total_new) * std::max(heads, kv_heads) > INT32_MAX || batch > kMaxBatch) return JGDPA_ERR_UNSUPPORTED;
  if (total_new > 0 && (slots == nullptr || q_offsets == nullptr || (batch > 0 && kv_lens == nullptr)))
    return JGDPA_ERR_INVALID_ARGUMENT;
  if (!aligned(slots, 4) || !aligned(q_offsets, 4) || !aligned(kv_lens, 4) || !aligned(depths, 4))
    return JGDPA_ERR_MISALIGNED;
  const int sms = jg::host_sm_count();
  if (sms <= 0) return JGDPA_ERR_CUDA;
  jg::RotateParams p{};
  JG_CHECK(start_status(&p.status, workspace, stream));
  if (total_new == 0) return JGDPA_OK;
  if (heads > 0)
    p.job[p.jobs++] = rotate_job(q, q_stride, q_out, q_out_stride, total_new, heads, q_offsets, nullptr, batch, q_weight);
  p.job[p.jobs] = rotate_job(k_new, k_stride, k_cache, 0, total_new, kv_heads, q_offsets, nullptr, batch, k_weight);
  p.job[p.jobs].slots = slots;
  p.job[p.jobs++].page_stride = k_page_stride;
  p.job[p.jobs] = rotate_job(v_new, v_stride, v_cache, 0, total_new, kv_heads, q_offsets, nullptr, batch, nullptr);
  p.job[p.jobs].slots = slots;
  p.job[p.jobs].copy = 1;
  p.job[p.jobs++].page_stride = v_page_stride;
  p.inv_freq = inv_freq;
  p.pairs = pairs;
  p.eps = eps;
  p.kv_lens = kv_lens;
  p.depths = depths;
  p.page_shift = jg::page_shift_of(page_size);
  p.slot_end = num_pages * page_size;
  JG_CUDA(jg::launch_rotate(p, head_dim, norm != 0, interleaved != 0, sms, stream));
  return JGDPA_OK;
}

size_t jgdpa_verify_workspace_bytes(void) { return kAlign; }

jgdpa_status jgdpa_verify(const void* target, int64_t target_stride, int32_t target_bf16, const void* draft,
                          int64_t draft_stride, int32_t draft_bf16, const int32_t* tokens, const int32_t* parents,
                          const float* uniforms, const int32_t* q_offsets, int32_t batch, int32_t total_q,
                          int32_t vocab, const int32_t* kv_lens, const int32_t* slots, int32_t* accepted,
                          int32_t* next_tokens, int32_t* places, int32_t* keep_lens, int32_t* keep_slots,
                          void* workspace, size_t workspace_bytes, jgdpa_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (batch < 0 || total_q < 0 || vocab < 1 || (target_bf16 != 0 && target_bf16 != 1) || (draft_bf16 != 0 && draft_bf16 != 1))
    return JGDPA_ERR_INVALID_ARGUMENT;
  if (draft != nullptr && parents != nullptr) return JGDPA_ERR_INVALID_ARGUMENT;
  if (batch > jg::kCacheMaxBatch || vocab > (1 << 30)) return JGDPA_ERR_UNSUPPORTED;
  if (target_stride < vocab || (draft != nullptr && draft_stride < vocab)) return JGDPA_ERR_INVALID_ARGUMENT;
  if (target_stride >= kMaxStride || (draft != nullptr && draft_stride >= kMaxStride)) return JGDPA_ERR_UNSUPPORTED;
  if (batch > 0 && (q_offsets == nullptr || accepted == nullptr || next_tokens == nullptr)) return JGDPA_ERR_INVALID_ARGUMENT;
  if (total_q > 0 && (target == nullptr || tokens == nullptr || uniforms == nullptr || places == nullptr))
    return JGDPA_ERR_INVALID_ARGUMENT;
  if ((keep_lens != nullptr && batch > 0 && kv_lens == nullptr) || (keep_slots != nullptr && total_q > 0 && slots == nullptr))
    return JGDPA_ERR_INVALID_ARGUMENT;
  if (!aligned(target, target_bf16 ? 2 : 4) || !aligned(draft, draft_bf16 ? 2 : 4)) return JGDPA_ERR_MISALIGNED;
  for (const void* a : std::initializer_list<const void*>{tokens, parents, uniforms, q_offsets, kv_lens, slots, accepted,
                                                          next_tokens, places, keep_lens, keep_slots})
    if (!aligned(a, 4)) return JGDPA_ERR_MISALIGNED;
  JG_CHECK(check_status(workspace, workspace_bytes, kAlign));
  const int sms = jg::host_sm_count();
  if (sms <= 0) return JGDPA_ERR_CUDA;
  jg::VerifyParams p{};
  JG_CHECK(start_status(&p.status, workspace, stream));
  if (batch == 0) {
    if (total_q > 0) {  // (-1 in every byte)
      JG_CUDA(cudaMemsetAsync(places, 0xFF, static_cast<size_t>(total_q) * sizeof(int32_t), stream));
      if (keep_slots != nullptr) JG_CUDA(cudaMemsetAsync(keep_slots, 0xFF, static_cast<size_t>(total_q) * sizeof(int32_t), stream));
    }
    return JGDPA_OK;
  }
  p.target = target;
  p.draft = draft;
  p.target_stride = target_stride;
  p.draft_stride = draft_stride;
  p.tokens = tokens;
  p.parents = parents;
  p.uniforms = uniforms;
  p.q_off = q_offsets;
  p.kv_lens = kv_lens;
  p.slots = slots;
  p.total = total_q;
  p.batch = batch;
  p.vocab = vocab;
  p.accepted = accepted;
  p.next = next_tokens;
  p.places = places;
  p.keep_lens = keep_lens;
  p.keep_slots = keep_slots;
  JG_CUDA(jg::launch_verify(p, target_bf16 != 0, draft != nullptr ? draft_bf16 != 0 : target_bf16 != 0, sms, stream));
  return JGDPA_OK;
}

jgdpa_status jgdpa_cache4_append(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                                 const int32_t* slots, int32_t total_new, void* k_codes, void* k_scales, void* v_codes,
                                 void* v_scales, int64_t k_code_stride, int64_t k_scale_stride, int64_t v_code_stride,
                                 int64_t v_scale_stride, int32_t num_pages, int32_t page_size, int32_t kv_heads,
                                 int32_t head_dim, jgdpa_stream_t stream) {
  return cache4_rows(true, k_new, v_new, nullptr, nullptr, k_stride, v_stride, slots, total_new,
                     cache4(k_codes, k_scales, k_code_stride, k_scale_stride),
                     cache4(v_codes, v_scales, v_code_stride, v_scale_stride), num_pages, page_size, kv_heads, head_dim,
                     reinterpret_cast<cudaStream_t>(stream));
}

jgdpa_status jgdpa_cache4_read(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                               int64_t k_code_stride, int64_t k_scale_stride, int64_t v_code_stride,
                               int64_t v_scale_stride, int32_t num_pages, int32_t page_size, int32_t kv_heads,
                               int32_t head_dim, const int32_t* slots, int32_t rows, void* k_out, void* v_out,
                               int64_t k_stride, int64_t v_stride, jgdpa_stream_t stream) {
  return cache4_rows(false, nullptr, nullptr, k_out, v_out, k_stride, v_stride, slots, rows,
                     cache4(k_codes, k_scales, k_code_stride, k_scale_stride),
                     cache4(v_codes, v_scales, v_code_stride, v_scale_stride), num_pages, page_size, kv_heads, head_dim,
                     reinterpret_cast<cudaStream_t>(stream));
}

size_t jgdpa_cache4_fwd_workspace_bytes(int32_t head_dim) {
  Cache4Layout L;
  return head_dim_ok(head_dim) && cache4_layout(head_dim, &L) ? L.total : 0;
}

jgdpa_status jgdpa_cache4_fwd(const void* q, int64_t q_stride, const void* k_codes, const void* k_scales,
                              const void* v_codes, const void* v_scales, int64_t k_code_stride, int64_t k_scale_stride,
                              int64_t v_code_stride, int64_t v_scale_stride, int32_t num_pages, int32_t page_size,
                              const int32_t* block_table, int32_t table_width, const int32_t* q_offsets,
                              const int32_t* kv_lens, int32_t batch, int64_t total_q, int32_t max_q, int32_t heads,
                              int32_t kv_heads, int32_t head_dim, jgdpa_act act, float scale, const float* bias_table,
                              int32_t bias_len, int32_t window, const int32_t* tree_mask, int32_t mask_words,
                              const int32_t* depths, void* out, float* lse, void* workspace, size_t workspace_bytes,
                              jgdpa_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (batch < 0 || total_q < 0 || max_q < 0 || heads < 1 || table_width < 0 || window < 0 || mask_words < 0)
    return JGDPA_ERR_INVALID_ARGUMENT;
  JG_CHECK(check_cache4(k_codes, k_scales, k_code_stride, k_scale_stride, num_pages, page_size, kv_heads, head_dim));
  JG_CHECK(check_cache4(v_codes, v_scales, v_code_stride, v_scale_stride, num_pages, page_size, kv_heads, head_dim));
  if (heads % kv_heads) return JGDPA_ERR_INVALID_ARGUMENT;
  if (heads > 65535) return JGDPA_ERR_UNSUPPORTED;
  if (act < JGDPA_ACT_GELU || act > JGDPA_ACT_SOFTMAX || !std::isfinite(scale)) return JGDPA_ERR_INVALID_ARGUMENT;
  if (bias_len < 0 || (bias_len > 0) != (bias_table != nullptr) || (bias_len > 0 && bias_len % 2 == 0))
    return JGDPA_ERR_INVALID_ARGUMENT;
  if (bias_len > jg::kMaxBiasLen) return JGDPA_ERR_UNSUPPORTED;
  if (total_q > 0 && (mask_words > 0) != (tree_mask != nullptr)) return JGDPA_ERR_INVALID_ARGUMENT;
  if (act != JGDPA_ACT_SOFTMAX && lse != nullptr) return JGDPA_ERR_INVALID_ARGUMENT;
  const int64_t max_rows = static_cast<int64_t>(max_q) * (heads / kv_heads);
  if (total_q > INT32_MAX || batch > jg::kCacheMaxBatch || max_rows > INT32_MAX / 2 ||
      static_cast<int64_t>(table_width) * page_size > jg::kMaxTokens || static_cast<int64_t>(mask_words) * 32 > INT32_MAX)
    return JGDPA_ERR_UNSUPPORTED;
  if (batch > 0 && (q_offsets == nullptr || kv_lens == nullptr || (table_width > 0 && block_table == nullptr)))
    return JGDPA_ERR_INVALID_ARGUMENT;
  if (total_q > 0) {
    JG_CHECK(check_rows(q, q_stride, total_q, heads, head_dim));
    if (out == nullptr) return JGDPA_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(bias_table, 4) || !aligned(q_offsets, 4) || !aligned(kv_lens, 4) ||
      !aligned(block_table, 4) || !aligned(tree_mask, 4) || !aligned(depths, 4))
    return JGDPA_ERR_MISALIGNED;
  Cache4Layout L;
  if (!cache4_layout(head_dim, &L)) return JGDPA_ERR_CUDA;
  if (workspace == nullptr || workspace_bytes < L.total) return JGDPA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, kAlign)) return JGDPA_ERR_MISALIGNED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (batch == 0) {
    JG_CUDA(cudaMemsetAsync(ws, 0, sizeof(int), stream));
    return JGDPA_OK;
  }
  int grid = L.sms * jg::cache4_ctas(head_dim, jg::cache4_columns(max_rows));
  if (total_q == 0 || max_q == 0) {  // no row is allowed: one CTA sees that the offsets hold none
    max_q = 0;
    grid = 1;
  }
  jg::Cache4FwdParams pp{};
  pp.k = cache4(k_codes, k_scales, k_code_stride, k_scale_stride);
  pp.v = cache4(v_codes, v_scales, v_code_stride, v_scale_stride);
  jg::CacheFwdParams& p = pp.f;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.table = block_table;
  p.q_off = q_offsets;
  p.kv_lens = kv_lens;
  p.bias = bias_table;
  p.mask = tree_mask;
  p.depth = depths;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.part_o = reinterpret_cast<float*>(ws + L.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  p.join = reinterpret_cast<jg::CacheJoin*>(ws + L.join);
  p.err = reinterpret_cast<int*>(ws + L.err);
  p.status = reinterpret_cast<int*>(ws);
  p.total_q = total_q;
  p.batch = batch;
  p.max_q = max_q;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.group = heads / kv_heads;
  p.page_shift = jg::page_shift_of(page_size);
  p.width = table_width;
  p.num_pages = num_pages;
  p.mask_words = mask_words;
  p.bias_len = bias_len;
  p.window = window;
  p.rows_per_tile = jg::kCache4Rows;
  p.heads_per_item = 1;
  // what an item's start and end take, in tiles of 64 keys, measured (half or
  // twice as many: up to 10% more on ragged lengths)
  p.item_cost = head_dim == 32 ? 16 : 8;
  p.min_part = 1;
  p.scale = act == JGDPA_ACT_SOFTMAX ? scale * jg::kLog2e : scale;
  p.wait_limit_ns = jg::host_wait_limit_ns();
  // no more CTAs than the longest line that these sizes allow has ranges
  const double tiles = std::ceil(static_cast<double>(table_width) * page_size / 64);
  const double row_tiles = std::ceil(static_cast<double>(max_rows) / jg::kCache4Rows);
  const double ranges = std::ceil(static_cast<double>(batch) * kv_heads * row_tiles * (p.item_cost + tiles) / jg::kCache4MinRange);
  if (ranges < grid) grid = std::max(1, static_cast<int>(ranges));
  const int tile_rows = static_cast<int>(std::clamp<int64_t>(max_rows, 1, jg::kCache4Rows));  // that may live
  auto launch = [&](auto dim) -> cudaError_t {
    constexpr int D = decltype(dim)::value;
    const cudaError_t e = jg::launch_cache4_fwd_d<D>(pp, act, grid, stream);
    return e != cudaSuccess ? e : jg::launch_cache_join_d<D>(p, act, grid, tile_rows, stream);
  };
  JG_CUDA(head_dim == 128  ? launch(std::integral_constant<int, 128>{})
          : head_dim == 64 ? launch(std::integral_constant<int, 64>{})
                           : launch(std::integral_constant<int, 32>{}));
  return JGDPA_OK;
}

}  // extern "C"
