// Pages and slots of a paged key/value cache, and the writes into them.
#include <algorithm>

#include "cache.cuh"

namespace jg {

// ------------------------------------------------------------------- plan
// With P tokens per page, want_b = ceil((ctx_b + add_b) / P), request b gives
// back max(0, held_b - want_b) pages and takes max(0, want_b - held_b).  Laid
// on the free stack F[0, n) in (request, page) order the returned pages make a
// stack S of N entries; the i-th page handed out is S[N - 1 - i].
//
// The work is a few integers per request and one slot per token, so the call is
// bound by its latency: 3.3 us for 8 requests of one token, 5.2 for 256 of up to
// 64, 5.3 for 64 prompts of 262,000 tokens in all.  Every CTA forms all prefix sums for itself in shared
// memory (one pass, one block-wide scan) instead of waiting for another CTA or
// another launch, then writes its share.  Nothing that a CTA reads is written:
// table entries are read in [0, held) and written in [held, want), the stack is
// read below n and written from n on, and the new page counts go to arrays of
// their own.
constexpr int kPlanThreads = 256;

struct PlanPrefix {
  int32_t *row, *take, *back;  // exclusive sums, [batch + 1]
};

// The request whose share of the prefix holds x (x below the total).
__device__ __forceinline__ int plan_find(const int32_t* prefix, int batch, int x) {
  int lo = 0, hi = batch;  // prefix[lo] <= x < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct PlanReq {
  int ctx, add, held, want;
  bool ok;
};
__device__ __forceinline__ PlanReq plan_req(const CachePlanParams& p, int b) {
  PlanReq r;
  r.ctx = __ldg(p.ctx + b);
  r.add = __ldg(p.add + b);
  r.held = __ldg(p.held + b);
  const int64_t tokens = static_cast<int64_t>(r.ctx) + r.add;
  r.ok = r.ctx >= 0 && r.add >= 0 && r.held >= 0 && r.held <= p.width &&
         tokens <= static_cast<int64_t>(p.width) << p.page_shift;
  r.want = r.ok ? static_cast<int>((tokens + (1 << p.page_shift) - 1) >> p.page_shift) : 0;
  return r;
}

// Entry j (0 <= j < N) of the stack with the returned pages on it.
__device__ __forceinline__ int plan_stack(const CachePlanParams& p, const PlanPrefix& pre, int n, int j) {
  if (j < n) return __ldg(p.free_pages + j);
  const int b = plan_find(pre.back, p.batch, j - n);
  const PlanReq r = plan_req(p, b);
  return p.table[static_cast<int64_t>(b) * p.width + r.want + (j - n - pre.back[b])];
}

__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const CachePlanParams p) {
  extern __shared__ int32_t plan_smem[];
  __shared__ int64_t warp_sum[3][kPlanThreads / 32];
  const PlanPrefix pre{plan_smem, plan_smem + p.batch + 1, plan_smem + 2 * (p.batch + 1)};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (p.batch + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * each, p.batch), b1 = min(b0 + each, p.batch);
  const int n = __ldg(p.free_count);
  bool ok = n >= 0 && n <= p.pool;
  int64_t sum[3] = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const PlanReq r = plan_req(p, b);
    ok = ok && r.ok;
    sum[0] += r.add;
    sum[1] += max(0, r.want - r.held);
    sum[2] += max(0, r.held - r.want);
  }
  int64_t incl[3] = {sum[0], sum[1], sum[2]};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += v;
    }
    if (lane == 31) warp_sum[k][warp] = incl[k];
  }
  ok = __syncthreads_and(ok) != 0;
  int64_t total[3] = {0, 0, 0};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int64_t base = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      const int64_t v = warp_sum[k][w];
      if (w < warp) base += v;
      total[k] += v;
    }
    incl[k] += base - sum[k];  // exclusive
  }
  int status = kOk;
  if (!ok || total[0] > p.total || n + total[2] > p.pool) status = kErrBadOffsets;
  else if (total[1] > n + total[2]) status = kErrOutOfPages;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
  if (at == 0 && p.status != nullptr) *p.status = status;
  if (status != kOk) {  // nothing is handed out: no new tokens, no slots, the pages as they were
    for (int64_t b = at; b < p.batch; b += step) {
      p.held_out[b] = __ldg(p.held + b);
      p.kv_lens[b] = __ldg(p.ctx + b);
    }
    for (int64_t b = at; b <= p.batch; b += step) p.q_off[b] = 0;
    for (int64_t r = at; r < p.total; r += step) p.slots[r] = -1;
    if (at == 0) *p.free_count_out = n;
    return;
  }
  for (int b = b0; b < b1; ++b) {
    const PlanReq r = plan_req(p, b);
    pre.row[b] = static_cast<int32_t>(incl[0]);
    pre.take[b] = static_cast<int32_t>(incl[1]);
    pre.back[b] = static_cast<int32_t>(incl[2]);
    incl[0] += r.add;
    incl[1] += max(0, r.want - r.held);
    incl[2] += max(0, r.held - r.want);
  }
  if (tid == 0) {
    pre.row[p.batch] = static_cast<int32_t>(total[0]);
    pre.take[p.batch] = static_cast<int32_t>(total[1]);
    pre.back[p.batch] = static_cast<int32_t>(total[2]);
  }
  __syncthreads();
  const int rows = static_cast<int>(total[0]), taken = static_cast<int>(total[1]), given = static_cast<int>(total[2]);
  const int top = n + given;
  for (int64_t b = at; b < p.batch; b += step) {
    const PlanReq r = plan_req(p, static_cast<int>(b));
    p.held_out[b] = r.want;
    p.kv_lens[b] = r.ctx + r.add;
    p.q_off[b] = pre.row[b];
  }
  if (at == 0) {
    p.q_off[p.batch] = rows;
    *p.free_count_out = top - taken;
  }
  for (int64_t i = at; i < taken; i += step) {
    const int b = plan_find(pre.take, p.batch, static_cast<int>(i));
    p.table[static_cast<int64_t>(b) * p.width + __ldg(p.held + b) + (i - pre.take[b])] =
        plan_stack(p, pre, n, top - 1 - static_cast<int>(i));
  }
  for (int64_t j = n + at; j < top - taken; j += step) p.free_pages[j] = plan_stack(p, pre, n, static_cast<int>(j));
  const int mask = (1 << p.page_shift) - 1;
  for (int64_t r = at; r < p.total; r += step) {
    int slot = -1;
    if (r < rows) {
      const int b = plan_find(pre.row, p.batch, static_cast<int>(r));
      const PlanReq q = plan_req(p, b);
      const int pos = q.ctx + static_cast<int>(r) - pre.row[b], pg = pos >> p.page_shift;
      const int page = pg < q.held ? p.table[static_cast<int64_t>(b) * p.width + pg]
                                   : plan_stack(p, pre, n, top - 1 - (pre.take[b] + pg - q.held));
      if (static_cast<uint32_t>(page) < static_cast<uint32_t>(p.pool)) slot = (page << p.page_shift) | (pos & mask);
    }
    p.slots[r] = slot;
  }
}

cudaError_t launch_cache_plan(const CachePlanParams& p, int sms, cudaStream_t stream) {
  const int smem = 3 * (p.batch + 1) * static_cast<int>(sizeof(int32_t));
  static DeviceFlags attr_set = {};
  cudaError_t e = smem_attr_once(cache_plan_kernel, 3 * (kCacheMaxBatch + 1) * static_cast<int>(sizeof(int32_t)), attr_set);
  if (e != cudaSuccess) return e;
  // One token per thread as far as four CTAs per SM go: a token is a chain of
  // loads (its request, its page), and four in a row took twice the time.  How
  // many pages come back only the device knows; one CTA per SM where the table
  // has entries for them took 6.1 us against 14.1 with threads for the tokens
  // alone (256 requests, 62,000 pages back; 1,024 requests, 271,000 pages back:
  // 10.8 against 17.2), and nothing more where none come back (1,024 requests:
  // 6.2).  Four CTAs per SM for them: 9.3, but 7.8 where none come back.
  const int64_t tokens = (static_cast<int64_t>(std::max(p.total, p.batch)) + kPlanThreads - 1) / kPlanThreads;
  const int64_t pages = (std::min<int64_t>(static_cast<int64_t>(p.batch) * p.width, p.pool) + kPlanThreads - 1) / kPlanThreads;
  const int64_t ctas = std::max<int64_t>({1, std::min<int64_t>(tokens, 4 * sms), std::min<int64_t>(pages, sms)});
  cache_plan_kernel<<<static_cast<unsigned>(ctas), kPlanThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

// ----------------------------------------------------------------- append
// Copies row r of the new keys and values to slot r of the cache.  Bound by
// HBM; a row is a contiguous piece of both sides, so 2^lg lanes take one row's
// 16-byte pieces side by side, four loads of K and four of V in flight each.
// 32,768 rows of 8 heads of 128: 41.7 us, 0.95 of the measured copy bandwidth;
// 32 rows: 2.5 us, the launch's latency.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const CacheAppendParams p, int lg) {
  const int width = 1 << lg;  // lanes per row
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x) >> lg;
  if (row >= p.rows) return;
  const int slot = __ldg(p.slots + row);
  if (static_cast<uint32_t>(slot) >= static_cast<uint32_t>(p.slot_end)) return;
  const int64_t page = slot >> p.page_shift, place = slot & ((1 << p.page_shift) - 1);
  const uint4* ks = reinterpret_cast<const uint4*>(p.k + row * p.k_stride);
  const uint4* vs = reinterpret_cast<const uint4*>(p.v + row * p.v_stride);
  uint4* kd = reinterpret_cast<uint4*>(p.k_cache + page * p.k_page_stride) + place * p.chunks;
  uint4* vd = reinterpret_cast<uint4*>(p.v_cache + page * p.v_page_stride) + place * p.chunks;
  // blockIdx.y: a stretch of 4 width pieces
  const int c0 = blockIdx.y * 4 * width + (threadIdx.x & (width - 1));
  uint4 a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c0 + i * width < p.chunks) {
      a[i] = ld_stream(ks + c0 + i * width);
      b[i] = ld_stream(vs + c0 + i * width);
    }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c0 + i * width < p.chunks) {
      kd[c0 + i * width] = a[i];
      vd[c0 + i * width] = b[i];
    }
}

cudaError_t launch_cache_append(const CacheAppendParams& p, cudaStream_t stream) {
  int lg = 0;
  while (lg < 5 && (4 << lg) < p.chunks) ++lg;
  const int64_t threads = static_cast<int64_t>(p.rows) << lg;
  const dim3 grid(static_cast<unsigned>((threads + kAppendThreads - 1) / kAppendThreads),
                  static_cast<unsigned>((p.chunks + (4 << lg) - 1) / (4 << lg)), 1);
  cache_append_kernel<<<grid, kAppendThreads, 0, stream>>>(p, lg);
  return cudaGetLastError();
}

}  // namespace jg
