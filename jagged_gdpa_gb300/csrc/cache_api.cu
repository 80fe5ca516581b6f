// Entry points of the paged key/value cache: argument checks, tensor maps,
// workspace layout and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/jgdpa.h"
#include "act.cuh"
#include "cache.cuh"
#include "host.h"

namespace jg {
template <int D>
cudaError_t launch_cache_fwd_d(const CacheFwdParams& p, int act, int grid, cudaStream_t stream);
template <int D>
cudaError_t launch_cache_fwd_wide_d(const CacheFwdParams& p, int act, bool pairs, int grid, cudaStream_t stream);
template <int D>
cudaError_t launch_cache_join_d(const CacheFwdParams& p, int act, int n_ctas, int tile_rows, cudaStream_t stream);
cudaError_t launch_cache_plan(const CachePlanParams& p, int sms, cudaStream_t stream);
cudaError_t launch_cache_append(const CacheAppendParams& p, cudaStream_t stream);

int page_shift_of(int32_t page_size) {
  for (int s = 4; s <= 10; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

jgdpa_status check_cache(const void* k_cache, const void* v_cache, int64_t k_page_stride, int64_t v_page_stride,
                         int32_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim) {
  if (num_pages < 1 || page_size < 1 || kv_heads < 1) return JGDPA_ERR_INVALID_ARGUMENT;
  if (head_dim != 32 && head_dim != 64 && head_dim != 128) return JGDPA_ERR_UNSUPPORTED;
  if (page_shift_of(page_size) < 0 || kv_heads > 65535) return JGDPA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_pages) * page_size > kMaxTokens) return JGDPA_ERR_UNSUPPORTED;
  if (k_cache == nullptr || v_cache == nullptr) return JGDPA_ERR_INVALID_ARGUMENT;
  const int64_t page = static_cast<int64_t>(page_size) * kv_heads * head_dim;
  if (k_page_stride < page || v_page_stride < page) return JGDPA_ERR_INVALID_ARGUMENT;
  if (k_page_stride >= (int64_t{1} << 39) || v_page_stride >= (int64_t{1} << 39)) return JGDPA_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(k_cache) % 16 || reinterpret_cast<uintptr_t>(v_cache) % 16 || k_page_stride % 8 ||
      v_page_stride % 8)
    return JGDPA_ERR_MISALIGNED;
  return JGDPA_OK;
}
}  // namespace jg

namespace {

constexpr size_t kAlign = 256;
using jg::check_cache;
using jg::kMaxTokens;
using jg::page_shift_of;
size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct CacheLayout {
  size_t err, join, part_ml, part_o, total;
  int rows, grid;  // query rows of one item per key/value head, CTAs
  int heads;       // key/value heads of one item
  int heads_together, grid_together;  // the same with small heads side by side
  int tokens;      // of a 128-row tile
  bool wide;       // 128-row tiles through tensor memory
  bool pairs;      // of them, two at a time
};
bool cache_layout(int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t max_q, CacheLayout* L) {
  const int sms = jg::host_sm_count();
  if (sms <= 0) return false;
  const int group = heads / kv_heads;
  const int64_t max_rows = static_cast<int64_t>(max_q) * group;
  // (a tile of the wide kernel holds whole tokens, so at most 128 heads share a key/value head there)
  L->wide = max_rows > jg::cache_narrow_rows(head_dim) && group <= jg::kTile;
  if (L->wide) {
    L->tokens = std::min(jg::kTile / group, max_q);
    L->pairs = max_q > L->tokens;
    L->rows = group * L->tokens * (L->pairs ? 2 : 1);
    L->grid = sms;
    L->heads = 1;
    L->heads_together = 1;
  } else {
    L->heads_together = kv_heads % (128 / head_dim) == 0 ? 128 / head_dim : 1;
    L->heads = 1;
    L->rows = max_rows <= 16 ? 16 : jg::cache_narrow_rows(head_dim);
    L->pairs = false;
    L->tokens = 0;
    L->grid = sms * jg::cache_ctas(head_dim, L->rows / 16);
  }
  L->grid_together = L->heads_together > 1 ? sms * jg::cache_ctas(128, L->rows / 16) : L->grid;
  // (room for either)
  const size_t most = std::max(L->grid, L->grid_together);
  const size_t parts = 2 * static_cast<size_t>(std::max(L->grid * L->heads, L->grid_together * L->heads_together)) * L->rows;
  size_t off = kAlign;  // the status word
  L->err = off;
  off += up(most * sizeof(int));
  L->join = off;
  off += up(most * sizeof(jg::CacheJoin));
  L->part_ml = off;
  off += up(parts * sizeof(float2));
  L->part_o = off;
  off += up(parts * head_dim * sizeof(float));
  L->total = off;
  return true;
}

// Small heads side by side (cache_fwd.cu) read whole 256-byte pieces and start
// and end fewer items, but each with more steps to its first and last result.
// From about 12 tiles per CTA on, as far as the host can tell (the table's width
// is its bound of the lengths), that pays: d = 32, 16 heads, 64 requests of 4,100
// tokens 96 us against 190, of 30 to 300 tokens (8 tiles) 28 against 22; d = 64, 8
// heads, 92 against 117, and 15 against 12.5 for 4 requests of 191 to 553 (where a
// table much wider than they need takes the slower way; the window, which bounds an
// item's tiles too, is not looked at).
void put_together(CacheLayout* L, int32_t batch, int32_t kv_heads, int64_t max_rows, int64_t table_tokens) {
  if (L->heads_together == 1) return;
  const int64_t items = static_cast<int64_t>(batch) * kv_heads * ((max_rows + L->rows - 1) / L->rows);
  if (static_cast<double>(items) * static_cast<double>((table_tokens + 63) / 64) <= 12.0 * L->grid) return;
  L->heads = L->heads_together;
  L->grid = L->grid_together;
}

// The cache as one tensor map: (column of a 64-column half, token of the page,
// half, head, page).  A box is one head of up to box_tokens tokens of a page,
// both halves or one.
bool cache_map(CUtensorMap* m, const void* ptr, int64_t page_stride, int32_t num_pages, int32_t page_size,
               int32_t kv_heads, int32_t head_dim, int32_t box_tokens, bool both_halves) {
  std::memset(m, 0, sizeof(*m));
  const jg::EncodeFn enc = jg::host_encode_fn();
  if (!enc) return false;
  const cuuint64_t cols = std::min(head_dim, 64), halves = head_dim / cols;
  cuuint64_t dims[5] = {cols, static_cast<cuuint64_t>(page_size), halves, static_cast<cuuint64_t>(kv_heads),
                        static_cast<cuuint64_t>(num_pages)};
  cuuint64_t strides[4] = {static_cast<cuuint64_t>(kv_heads) * head_dim * 2, cols * 2,
                           static_cast<cuuint64_t>(head_dim) * 2, static_cast<cuuint64_t>(page_stride) * 2};
  cuuint32_t box[5] = {static_cast<cuuint32_t>(cols), static_cast<cuuint32_t>(std::min(page_size, box_tokens)),
                       static_cast<cuuint32_t>(both_halves ? halves : 1), 1, 1};
  cuuint32_t es[5] = {1, 1, 1, 1, 1};
  // what L2 fetches at a time: no more than a head's piece of a token, as its
  // neighbours are other heads', read at another time
  const CUtensorMapL2promotion promotion = head_dim >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                           : head_dim == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                            : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries: (column, token, head), a box one 64-column half of a tile's
// tokens, head by head.
bool query_map(CUtensorMap* m, const void* ptr, int64_t q_stride, int64_t total_q, int32_t heads, int32_t head_dim,
               int32_t group, int32_t tokens) {
  std::memset(m, 0, sizeof(*m));
  const jg::EncodeFn enc = jg::host_encode_fn();
  if (!enc) return false;
  const cuuint32_t cols = std::min(head_dim, 64);
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(total_q),
                        static_cast<cuuint64_t>(heads)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(q_stride) * 2, static_cast<cuuint64_t>(head_dim) * 2};
  cuuint32_t box[3] = {cols, static_cast<cuuint32_t>(tokens), static_cast<cuuint32_t>(group)};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

#define JG_CUDA(x)                              \
  do {                                          \
    if ((x) != cudaSuccess) return JGDPA_ERR_CUDA; \
  } while (0)

}  // namespace

extern "C" {

size_t jgdpa_cache_plan_workspace_bytes(void) { return kAlign; }

jgdpa_status jgdpa_cache_plan(const int32_t* ctx_lens, const int32_t* new_lens, const int32_t* held_pages,
                              int32_t batch, int32_t page_size, int32_t* block_table, int32_t table_width,
                              int32_t* free_pages, int32_t num_pages, const int32_t* free_count, int32_t total_new,
                              int32_t* held_out, int32_t* free_count_out, int32_t* q_offsets, int32_t* kv_lens,
                              int32_t* slots, void* workspace, size_t workspace_bytes, jgdpa_stream_t stream_) {
  if (batch < 0 || table_width < 0 || num_pages < 0 || total_new < 0 || page_size < 1)
    return JGDPA_ERR_INVALID_ARGUMENT;
  const int shift = page_shift_of(page_size);
  if (shift < 0 || batch > jg::kCacheMaxBatch) return JGDPA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_pages) * page_size > kMaxTokens ||
      static_cast<int64_t>(table_width) * page_size > kMaxTokens)
    return JGDPA_ERR_UNSUPPORTED;
  if (free_count == nullptr || free_count_out == nullptr || q_offsets == nullptr) return JGDPA_ERR_INVALID_ARGUMENT;
  if (batch > 0 && (ctx_lens == nullptr || new_lens == nullptr || held_pages == nullptr || held_out == nullptr ||
                    kv_lens == nullptr || (table_width > 0 && block_table == nullptr)))
    return JGDPA_ERR_INVALID_ARGUMENT;
  if ((num_pages > 0 && free_pages == nullptr) || (total_new > 0 && slots == nullptr)) return JGDPA_ERR_INVALID_ARGUMENT;
  // results are written while other parts of the call still read their inputs
  if ((batch > 0 && (held_out == held_pages || kv_lens == ctx_lens || kv_lens == held_pages || held_out == ctx_lens ||
                     held_out == new_lens || kv_lens == new_lens)) || free_count_out == free_count)
    return JGDPA_ERR_INVALID_ARGUMENT;
  for (const void* a : {static_cast<const void*>(ctx_lens), static_cast<const void*>(new_lens),
                        static_cast<const void*>(held_pages), static_cast<const void*>(block_table),
                        static_cast<const void*>(free_pages), static_cast<const void*>(free_count),
                        static_cast<const void*>(held_out), static_cast<const void*>(free_count_out),
                        static_cast<const void*>(q_offsets), static_cast<const void*>(kv_lens),
                        static_cast<const void*>(slots)})
    if (!aligned(a, 4)) return JGDPA_ERR_MISALIGNED;
  if (workspace != nullptr && workspace_bytes < kAlign) return JGDPA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, kAlign)) return JGDPA_ERR_MISALIGNED;
  const int sms = jg::host_sm_count();
  if (sms <= 0) return JGDPA_ERR_CUDA;
  jg::CachePlanParams p{};
  p.ctx = ctx_lens;
  p.add = new_lens;
  p.held = held_pages;
  p.batch = batch;
  p.page_shift = shift;
  p.width = table_width;
  p.pool = num_pages;
  p.total = total_new;
  p.table = block_table;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.held_out = held_out;
  p.free_count_out = free_count_out;
  p.q_off = q_offsets;
  p.kv_lens = kv_lens;
  p.slots = slots;
  p.status = static_cast<int*>(workspace);
  JG_CUDA(jg::launch_cache_plan(p, sms, reinterpret_cast<cudaStream_t>(stream_)));
  return JGDPA_OK;
}

jgdpa_status jgdpa_cache_append(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                                const int32_t* slots, int32_t total_new, void* k_cache, void* v_cache,
                                int64_t k_page_stride, int64_t v_page_stride, int32_t num_pages, int32_t page_size,
                                int32_t kv_heads, int32_t head_dim, jgdpa_stream_t stream_) {
  if (total_new < 0) return JGDPA_ERR_INVALID_ARGUMENT;
  jgdpa_status st = check_cache(k_cache, v_cache, k_page_stride, v_page_stride, num_pages, page_size, kv_heads, head_dim);
  if (st != JGDPA_OK) return st;
  if (total_new == 0) return JGDPA_OK;
  if (k_new == nullptr || v_new == nullptr || slots == nullptr) return JGDPA_ERR_INVALID_ARGUMENT;
  const int64_t row = static_cast<int64_t>(kv_heads) * head_dim;
  if (k_stride < row || v_stride < row) return JGDPA_ERR_INVALID_ARGUMENT;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(slots, 4) || k_stride % 8 || v_stride % 8)
    return JGDPA_ERR_MISALIGNED;
  jg::CacheAppendParams p{};
  p.k = static_cast<const __nv_bfloat16*>(k_new);
  p.v = static_cast<const __nv_bfloat16*>(v_new);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = slots;
  p.rows = total_new;
  p.chunks = static_cast<int32_t>(row / 8);
  p.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  p.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  p.k_page_stride = k_page_stride;
  p.v_page_stride = v_page_stride;
  p.page_shift = page_shift_of(page_size);
  p.slot_end = num_pages * page_size;
  JG_CUDA(jg::launch_cache_append(p, reinterpret_cast<cudaStream_t>(stream_)));
  return JGDPA_OK;
}

size_t jgdpa_cache_fwd_workspace_bytes(int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t max_q) {
  if (heads < 1 || kv_heads < 1 || heads % kv_heads || max_q < 0) return 0;
  if (head_dim != 32 && head_dim != 64 && head_dim != 128) return 0;
  CacheLayout L;
  return cache_layout(heads, kv_heads, head_dim, max_q, &L) ? L.total : 0;
}

jgdpa_status jgdpa_cache_fwd(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                             int64_t k_page_stride, int64_t v_page_stride, int32_t num_pages, int32_t page_size,
                             const int32_t* block_table, int32_t table_width, const int32_t* q_offsets,
                             const int32_t* kv_lens, int32_t batch, int64_t total_q, int32_t max_q, int32_t heads,
                             int32_t kv_heads, int32_t head_dim, jgdpa_act act, float scale, const float* bias_table,
                             int32_t bias_len, int32_t window, const int32_t* tree_mask, int32_t mask_words,
                             const int32_t* depths, void* out, float* lse, void* workspace, size_t workspace_bytes,
                             jgdpa_stream_t stream_) {
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (batch < 0 || total_q < 0 || max_q < 0 || heads < 1 || table_width < 0 || window < 0 || mask_words < 0)
    return JGDPA_ERR_INVALID_ARGUMENT;
  jgdpa_status st = check_cache(k_cache, v_cache, k_page_stride, v_page_stride, num_pages, page_size, kv_heads, head_dim);
  if (st != JGDPA_OK) return st;
  if (heads % kv_heads || heads > 65535) return heads % kv_heads ? JGDPA_ERR_INVALID_ARGUMENT : JGDPA_ERR_UNSUPPORTED;
  if (act < JGDPA_ACT_GELU || act > JGDPA_ACT_SOFTMAX || !std::isfinite(scale)) return JGDPA_ERR_INVALID_ARGUMENT;
  if (bias_len < 0 || (bias_len > 0) != (bias_table != nullptr) || (bias_len > 0 && bias_len % 2 == 0))
    return JGDPA_ERR_INVALID_ARGUMENT;
  if (bias_len > jg::kMaxBiasLen) return JGDPA_ERR_UNSUPPORTED;
  if (total_q > 0 && (mask_words > 0) != (tree_mask != nullptr)) return JGDPA_ERR_INVALID_ARGUMENT;
  if (act != JGDPA_ACT_SOFTMAX && lse != nullptr) return JGDPA_ERR_INVALID_ARGUMENT;
  const int64_t max_rows = static_cast<int64_t>(max_q) * (heads / kv_heads);
  if (total_q > INT32_MAX || batch > jg::kCacheMaxBatch || max_rows > INT32_MAX / 2 ||
      static_cast<int64_t>(table_width) * page_size > kMaxTokens || static_cast<int64_t>(mask_words) * 32 > INT32_MAX)
    return JGDPA_ERR_UNSUPPORTED;
  if (batch > 0 && (q_offsets == nullptr || kv_lens == nullptr || (table_width > 0 && block_table == nullptr)))
    return JGDPA_ERR_INVALID_ARGUMENT;
  if (total_q > 0 && (q == nullptr || out == nullptr)) return JGDPA_ERR_INVALID_ARGUMENT;
  if (q_stride < static_cast<int64_t>(heads) * head_dim) return JGDPA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || q_stride % 8 || !aligned(out, 16) || !aligned(lse, 4) || !aligned(bias_table, 4) ||
      !aligned(q_offsets, 4) || !aligned(kv_lens, 4) || !aligned(block_table, 4) || !aligned(tree_mask, 4) ||
      !aligned(depths, 4))
    return JGDPA_ERR_MISALIGNED;
  if (q_stride >= (int64_t{1} << 39)) return JGDPA_ERR_UNSUPPORTED;
  CacheLayout L;
  if (!cache_layout(heads, kv_heads, head_dim, max_q, &L)) return JGDPA_ERR_CUDA;
  if (workspace == nullptr || workspace_bytes < L.total) return JGDPA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, kAlign)) return JGDPA_ERR_MISALIGNED;
  put_together(&L, batch, kv_heads, max_rows, static_cast<int64_t>(table_width) * page_size);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (batch == 0) {
    JG_CUDA(cudaMemsetAsync(ws, 0, sizeof(int), stream));
    return JGDPA_OK;
  }
  if (total_q == 0 || max_q == 0) {  // no row is allowed: one CTA sees that the offsets hold none
    max_q = 0;
    L.wide = L.pairs = false;
    L.rows = 16;
    L.heads = L.grid = 1;
    L.tokens = 0;
  }
  jg::CacheFwdParams p{};
  const int32_t box = L.wide ? jg::kTile : 64;
  const int32_t map_heads = kv_heads / L.heads, map_dim = head_dim * L.heads;  // heads that go together as one
  if (!cache_map(&p.tm_k, k_cache, k_page_stride, num_pages, page_size, map_heads, map_dim, box, !L.wide) ||
      !cache_map(&p.tm_v, v_cache, v_page_stride, num_pages, page_size, map_heads, map_dim, box, !L.wide) ||
      (L.wide && !query_map(&p.tm_q, q, q_stride, total_q, heads, head_dim, heads / kv_heads, L.tokens)))
    return JGDPA_ERR_CUDA;
  p.k_cache = static_cast<const __nv_bfloat16*>(k_cache);
  p.v_cache = static_cast<const __nv_bfloat16*>(v_cache);
  p.k_page_stride = k_page_stride;
  p.v_page_stride = v_page_stride;
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
  p.page_shift = page_shift_of(page_size);
  p.width = table_width;
  p.num_pages = num_pages;
  p.mask_words = mask_words;
  p.bias_len = bias_len;
  p.window = window;
  p.rows_per_tile = L.rows;
  p.tile_tokens = L.tokens;
  p.heads_per_item = L.heads;
  // what an item's start and end take, measured: about 4 tiles of 64 keys, or in
  // the 128-row kernel 14 half tiles of 128 keys, 24 with a bias table, whose
  // tiles near the new tokens take longer (8 lengths off cost 5 to 10% on ragged
  // lengths)
  p.item_cost = L.wide ? (bias_len ? 24 : 14) : 4;
  p.min_part = L.wide ? 2 : 1;
  p.scale = act == JGDPA_ACT_SOFTMAX ? scale * jg::kLog2e : scale;
  p.wait_limit_ns = jg::host_wait_limit_ns();
  const int tile_rows = L.wide ? L.rows : static_cast<int>(std::clamp<int64_t>(max_rows, 1, L.rows));  // that may live
  auto launch = [&](auto dim) -> cudaError_t {
    constexpr int D = decltype(dim)::value;
    cudaError_t e = L.wide ? jg::launch_cache_fwd_wide_d<D>(p, act, L.pairs, L.grid, stream)
                           : jg::launch_cache_fwd_d<D>(p, act, L.grid, stream);
    return e != cudaSuccess ? e : jg::launch_cache_join_d<D>(p, act, L.grid, tile_rows, stream);
  };
  JG_CUDA(head_dim == 128  ? launch(std::integral_constant<int, 128>{})
          : head_dim == 64 ? launch(std::integral_constant<int, 64>{})
                           : launch(std::integral_constant<int, 32>{}));
  return JGDPA_OK;
}

}  // extern "C"
