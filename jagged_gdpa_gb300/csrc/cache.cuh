// Parameters, work division and small helpers of the paged key/value cache
// kernels (cache_plan.cu, cache_fwd.cu, cache_fwd_wide.cu, cache_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "act.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace jg {

// Status codes of the cache calls (same values as jgdpa_status).
enum : int { kErrOutOfPages = 8, kErrBadPage = 9 };

constexpr int kCacheMaxBatch = 16384;  // requests per call (the plan's prefix sums live in shared memory)

// Query rows per key/value head up to which the kernel for few rows
// (cache_fwd.cu) runs, and the 128-row one (cache_fwd_wide.cu) from there on.
// At 24 rows, softmax, 64 requests of 4,100 tokens, 32-row tiles of the former took
// 264 us against 183 at d = 128 (8 key/value heads), but 140 against 114 at d = 64
// (8) and 169 against 192 at d = 32 (16); on 256 requests of 100 to 800 tokens 100
// against 177 at d = 64 and 124 against 321 at d = 32; on one of 100,000 tokens 62
// against 55 and 72 against 80.  (Lengths are not known to the host; at d = 64 the
// short ones have more to lose.)
__host__ __device__ constexpr int cache_narrow_rows(int d) { return d < 128 ? 32 : 16; }

// CTAs per SM of the attention kernel for up to 16 mt rows and w columns of K
// and V per item (cache_fwd.cu).
__host__ __device__ constexpr int cache_ctas(int w, int mt) {
  return mt == 1 ? (w == 128 ? 2 : w == 64 ? 3 : 4) : (w == 128 ? 1 : 2);
}

struct CachePlanParams {
  const int32_t* ctx;
  const int32_t* add;
  const int32_t* held;
  int32_t batch, page_shift, width, pool, total;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* held_out;
  int32_t* free_count_out;
  int32_t* q_off;
  int32_t* kv_lens;
  int32_t* slots;
  int* status;  // or nullptr
};

struct CacheAppendParams {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t k_stride, v_stride;  // elements from one new row to the next
  const int32_t* slots;
  int32_t rows, chunks;        // chunks: 16-byte pieces of a row
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  int64_t k_page_stride, v_page_stride;  // elements from one page to the next
  int32_t page_shift;
  int32_t slot_end;            // num_pages * page_size
};

// The item that a range starts inside of, written for the joining kernel: valid
// only from the second of the ranges that share it.
struct CacheJoin {
  int32_t valid, h, rt;
  int32_t c0, c1;  // its ranges
  int32_t q0, T;   // its request's first query row, its tokens
  int32_t pad;
};

struct CacheFwdParams {
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  CUtensorMap tm_q;          // (column, head, token), boxes of one 128-row tile (128-row kernel)
  const __nv_bfloat16* q;
  int64_t q_stride;          // elements from one query row to the next
  const __nv_bfloat16* k_cache;
  const __nv_bfloat16* v_cache;
  int64_t k_page_stride, v_page_stride;  // elements from one page to the next
  const int32_t* table;      // [batch][width]
  const int32_t* q_off;
  const int32_t* kv_lens;
  const float* bias;         // [heads][bias_len] or nullptr
  const int32_t* mask;       // [total_q][mask_words] or nullptr
  const int32_t* depth;      // [total_q] or nullptr
  __nv_bfloat16* out;        // [total_q][heads][D]
  float* lse;                // [heads][total_q] or nullptr
  // parts of items that several ranges share, two per range: the end (or the
  // middle) of an item that its range starts with, and the start of its last
  float* part_o;             // [2 ranges][heads per item][rows per tile][D]
  float2* part_ml;           // [2 ranges][heads per item][rows per tile]: maximum (log2 units) and sum
  CacheJoin* join;           // [ranges]
  int* err;                  // [grid]: one status word per CTA, joined into `status`
  int* status;
  int64_t total_q;
  int32_t batch, max_q, heads, kv_heads, group;
  int32_t page_shift, width, num_pages;
  int32_t mask_words, bias_len, window;
  int32_t rows_per_tile;     // query rows (token, head of the group) of one item
  int32_t tile_tokens;       // tokens of a 128-row tile (128-row kernel; 0 otherwise)
  int32_t heads_per_item;    // key/value heads of one item
  int32_t item_cost;         // what an item's start and end are worth, in lengths of the work division
  int32_t min_part;          // tiles below which a part of an item is not worth a cut
  float scale;               // s (GELU / SiLU) or s log2(e) (softmax)
  unsigned long long wait_limit_ns;
};

// One request: its tokens, cached context and the key tiles its items visit.
struct CacheReq {
  int q0, T, L, C;
  int kt0, n;  // first key tile and tiles of every item
  int rt;      // row tiles
  int u;       // length of a key tile on the line
};

template <int KT>
__device__ __forceinline__ CacheReq cache_req(const CacheFwdParams& p, int b) {
  CacheReq r;
  r.q0 = __ldg(p.q_off + b);
  r.T = __ldg(p.q_off + b + 1) - r.q0;
  r.L = __ldg(p.kv_lens + b);
  r.C = r.L - r.T;
  // new tokens sit at positions >= C, so no cached key at or below C - window is seen
  r.kt0 = p.window > 0 ? static_cast<uint32_t>(max(0, r.C - p.window + 1)) / KT : 0;
  r.n = static_cast<int>((static_cast<uint32_t>(r.L) + KT - 1) / KT) - r.kt0;
  // (T group <= 2^30 by the checks; before them the value is not used)
  r.rt = static_cast<int>((static_cast<uint32_t>(r.T) * p.group + p.rows_per_tile - 1) / static_cast<uint32_t>(p.rows_per_tile));
  // (128-row kernel: two tiles of rows take about 1.4 times as long as one)
  r.u = p.tile_tokens == 0 ? 1 : (r.T > p.tile_tokens ? 3 : 2);
  return r;
}
// The length of one of its items on the line.
__device__ __forceinline__ int cache_len(const CacheFwdParams& p, const CacheReq& r) { return p.item_cost + r.n * r.u; }
__device__ __forceinline__ int64_t cache_cost(const CacheFwdParams& p, const CacheReq& r) {
  return r.T <= 0 ? 0 : static_cast<int64_t>(p.kv_heads / p.heads_per_item) * r.rt *
                             cache_len(p, r);
}
__device__ __forceinline__ bool cache_req_ok(const CacheFwdParams& p, const CacheReq& r) {
  return r.T >= 0 && r.T <= p.max_q && r.L >= r.T &&
         static_cast<int64_t>(r.L) <= static_cast<int64_t>(p.width) << p.page_shift &&
         (p.mask == nullptr || r.T <= 32 * p.mask_words);
}

// Work division.  The items are (request, kv head, row tile), each a lead of
// item_cost, what its start and end take, and n key tiles of length u.  Laid end
// to end (request by request, row tiles of a head next to each other) they form
// one line that is cut into ranges of equal length, one per CTA.
// (Without the lead, ranges that fall on many short requests took half as long
// again as the others.)  A border inside an item cuts it, and the joining kernel
// puts the parts together; a border that would leave a part of fewer than
// min_part tiles moves to the item's start or end.
//
// n counts the request's key tiles from the first on that any of its new tokens
// sees under the window.  What one row tile of many does not see of them is not
// taken off: in a causal prompt the early row tiles skip the later keys (`tiles`
// below), so that ranges over them end sooner (one prompt of 8,192 tokens: the
// busiest CTA visits 1.9 times the mean), and under a window the late ones visit
// tiles that their own window has left behind.
//
// A CTA that gets several row tiles of one head reads its keys from HBM for
// each.  Laying the row tiles of 512-row requests out in two passes over the
// batch, so that two CTAs read them at once, left the time as it was: those
// items are bound by their products.
struct CacheRange {
  int64_t per, begin, end;
  int b;        // request that `begin` lies in (or at the end of)
  int64_t rem;  // begin minus the request's start
  bool ok;
};
struct CacheRangeShared {
  int64_t warp_sum[16];
  int64_t border[2], rem;
  int b;
};

// a / b for a >= 0: the 64-bit division, some 100 instructions, only where it is
// needed, and out of the way.
static __device__ __noinline__ int64_t cache_div64(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t cache_div(int64_t a, int b) {
  return a <= 0xFFFFFFFFll ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : cache_div64(a, b);
}

// The key tile of an item that a border `from` after the item's start cuts
// before, or 0 if it goes to the item's start, or n to its end.  (The borders
// keep their order.)
__device__ __forceinline__ int cache_cut(const CacheFwdParams& p, int64_t from, const CacheReq& r) {
  const int t = static_cast<int>(from < p.item_cost ? 0 : cache_div(from - p.item_cost, r.u));
  if (t >= p.min_part && t <= r.n - p.min_part) return t;
  const bool to_start = r.n >= 2 * p.min_part ? t < p.min_part : 2 * from < cache_len(p, r);
  return to_start ? 0 : r.n;
}

// This CTA's range.  Run by every thread of the CTA (a whole number of warps, at
// most 512); ends in a barrier.
template <int KT>
__device__ CacheRange cache_range(const CacheFwdParams& p, CacheRangeShared* sh, int min_range) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
  const int each = (p.batch + nt - 1) / nt;
  const int b0 = min(tid * each, p.batch), b1 = min(b0 + each, p.batch);
  int64_t sum = 0;
  bool ok = true;
  if (tid == 0) ok = __ldg(p.q_off) == 0 && static_cast<int64_t>(__ldg(p.q_off + p.batch)) <= p.total_q;
  for (int b = b0; b < b1; ++b) {
    const CacheReq r = cache_req<KT>(p, b);
    ok = ok && cache_req_ok(p, r);
    sum += cache_cost(p, r);
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sh->warp_sum[warp] = incl;
  const bool all_ok = __syncthreads_and(ok) != 0;
  int64_t base = 0, total = 0;
  for (int w = 0; w < nw; ++w) {
    const int64_t v = sh->warp_sum[w];
    if (w < warp) base += v;
    total += v;
  }
  CacheRange R;
  R.ok = all_ok;
  const int g = gridDim.x;
  R.per = max(cache_div(total + g - 1, g), static_cast<int64_t>(min_range));
  R.begin = min(R.per * blockIdx.x, total);
  R.end = min(R.begin + R.per, total);
  // the thread whose requests hold a border moves it, if need be
  const int64_t mine = base + incl - sum;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const int64_t x = side == 0 ? R.begin : R.end;
    if (!all_ok || x >= total || x < mine || x >= mine + sum) continue;
    int64_t at = mine;
    for (int b = b0;; ++b) {
      const CacheReq r = cache_req<KT>(p, b);
      const int64_t c = cache_cost(p, r);
      if (x >= at + c) {
        at += c;
        continue;
      }
      const int len = cache_len(p, r);
      const int64_t from_req = x - at, item0 = cache_div(from_req, len) * len;
      const int cut = cache_cut(p, from_req - item0, r);
      const int64_t moved = item0 + (cut == 0 ? 0 : p.item_cost + cut * r.u);
      sh->border[side] = at + moved;
      if (side == 0) {
        sh->b = b;
        sh->rem = moved;
      }
      break;
    }
  }
  __syncthreads();
  if (R.begin < total) {
    R.begin = sh->border[0];
    R.b = sh->b;
    R.rem = sh->rem;
  }
  if (R.end < total) R.end = sh->border[1];
  return R;
}

// Walks the parts of items in a CTA's range, in order; every role of the CTA
// walks the same parts.
struct CacheWalk {
  int64_t left;  // length left in the range
  int64_t rem;   // place in the request's length
  int b;
  // the current part
  CacheReq r;
  int h, row_tile, tile0, count;  // count tiles from the item's tile0
  int step;                       // its length
  bool whole;                     // the part is the whole item

  __device__ __forceinline__ void init(const CacheRange& R) {
    left = R.ok ? R.end - R.begin : 0;
    rem = R.rem;
    b = R.b;
  }
  template <int KT>
  __device__ __forceinline__ bool next(const CacheFwdParams& p) {
    if (left <= 0) return false;
    int64_t cost;
    for (;; ++b, rem = 0) {
      r = cache_req<KT>(p, b);
      cost = cache_cost(p, r);
      if (rem < cost) break;
    }
    const int len = cache_len(p, r);
    const int64_t item = cache_div(rem, len);
    const int from = static_cast<int>(rem - item * len);
    step = static_cast<int>(min(static_cast<int64_t>(len - from), left));
    // (a border lies between two tiles or items, never in the lead)
    tile0 = static_cast<uint32_t>(max(0, from - p.item_cost)) / static_cast<uint32_t>(r.u);
    count = static_cast<uint32_t>(from + step - p.item_cost) / static_cast<uint32_t>(r.u) - tile0;
    h = static_cast<int>(cache_div(item, r.rt));
    row_tile = static_cast<int>(item - static_cast<int64_t>(h) * r.rt);
    whole = count == r.n;
    return true;
  }
  __device__ __forceinline__ void advance() {
    rem += step;
    left -= step;
  }
  // The range's place for a part that is not a whole item.
  __device__ __forceinline__ int slot() const { return tile0 > 0 ? 0 : 1; }
  // The tiles [lo, hi) (of the request's) of this part that are visited: without
  // a mask, rows of tokens up to t see keys up to C + t, so later tiles are neither
  // loaded nor computed.  (The window trims the request's first tile only, kt0.)
  template <int KT>
  __device__ __forceinline__ void tiles(const CacheFwdParams& p, int& lo, int& hi) const {
    lo = r.kt0 + tile0;
    hi = lo + count;
    if (p.mask == nullptr) {
      const int last_row = min(r.T * p.group, (row_tile + 1) * p.rows_per_tile) - 1;
      const int64_t keys = static_cast<int64_t>(r.C) + static_cast<uint32_t>(last_row) / static_cast<uint32_t>(p.group) + 1;
      hi = max(lo, static_cast<int>(min(static_cast<int64_t>(hi), (keys + KT - 1) / KT)));
    }
  }
};

// The attention and joining kernels are launched so that a kernel's blocks may
// be set up while the kernel before it on the stream still runs (programmatic
// dependent launch).  Each block waits for that kernel's end before it touches
// global memory, and none ends without having waited.
__device__ __forceinline__ void cache_wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void cache_let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... Params, typename... Args>
inline cudaError_t cache_launch(void (*kern)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
                                const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Writes a range's join record (one thread).
template <int KT>
__device__ __forceinline__ void cache_open(const CacheFwdParams& p, const CacheRange& R) {
  const int c = blockIdx.x;
  if (!R.ok) p.err[c] = kErrBadOffsets;
  CacheJoin j{};
  if (R.ok && R.begin < R.end) {
    const CacheReq r = cache_req<KT>(p, R.b);
    const int len = cache_len(p, r);
    const int64_t item = cache_div(R.rem, len), from = R.rem - item * len;  // (at a request's end: from is 0)
    if (from > 0) {  // the range starts at a border that cuts the item; is it the first?
      const int64_t at = from + R.per * c - R.begin;  // the border before it was moved
      const int64_t before = at - R.per;
      const int cut = before <= 0 ? 0 : cache_cut(p, before, r);
      j.valid = cut == 0;
      j.q0 = r.q0;
      j.T = r.T;
      j.h = static_cast<int>(cache_div(item, r.rt));
      j.rt = static_cast<int>(item - static_cast<int64_t>(j.h) * r.rt);
      j.c0 = c - 1;
      j.c1 = c;
      // the last border that cuts it
      const int64_t last = p.item_cost + static_cast<int64_t>(r.n - p.min_part + 1) * r.u - 1;
      if (last > at) j.c1 = c + static_cast<int>(cache_div(last - at, static_cast<int>(min(R.per, static_cast<int64_t>(INT32_MAX)))));
    }
  }
  p.join[c] = j;
}

// What the kernels keep of a query row.
struct CcRow {
  int t;            // token, or -1: no row
  int pos;          // C + depth
  int head;
  float far_bias;   // bias of keys at least R behind every new token
};

// GELU(x) or SiLU(x) of two scores from hx = x / 2, each right to bf16's last
// place relative to itself.  (The packed kernels' hx + hx tanh(u) is a difference
// of nearly equal numbers below zero, whose error of some 1e-3 is as large as the
// weight itself from about -3 on: a long context whose bias pushes most scores
// there would add up noise.)
//   GELU(x) = max(x, 0) - a Phi(-a), a = |x|, with log2 Phi(-a) as a polynomial
//     on [0, 13] (csrc/fit_constants.py; beyond it a Phi(-a) is below 2^-122): of degree 6, Phi within
//     1.9e-3 (degree 7, within 5.2e-4, took 2% more time in the 128-row kernel), or 8, within 1.5e-4
//   SiLU(x) = x / (1 + 2^(-x log2 e))
// NaN stays NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float rcp_sfu(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int ACT, int DEG = 6>
__device__ __forceinline__ float2 cc_act2(float2 hx) {
  if constexpr (ACT == 0) {
    constexpr float c6[7] = {-1.00261784f,  -1.1279366f,     -0.492554843f, -0.0349358097f,
                             0.0033006093f, -0.000168592655f, 3.53243581e-06f};
    constexpr float c8[9] = {-1.00016737f,    -1.14921916f,    -0.462455243f,    -0.0510253534f, 0.00749332923f,
                             -0.00075733976f, 4.89184131e-05f, -1.80116172e-06f, 2.86048483e-08f};
    static_assert(DEG == 6 || DEG == 8, "degrees with constants");
    // n = -a / 2: 2 Phi(-a) = 2^(1 + c0 - 2 c1 n + 4 c2 n^2 ..), and hx + |hx| = max(x, 0)
    const float2 n = make_float2(max_nan(-fabsf(hx.x), -6.5f), max_nan(-fabsf(hx.y), -6.5f));
    float2 w = f2(0.f);
#pragma unroll
    for (int k = DEG; k >= 0; --k) {
      const float ck = (k % 2 ? -1.f : 1.f) * static_cast<float>(1 << k) * (DEG == 6 ? c6[k % 7] : c8[k]) + (k == 0 ? 1.f : 0.f);
      w = k == DEG ? f2(ck) : __ffma2_rn(w, n, f2(ck));
    }
    return __ffma2_rn(n, make_float2(ex2_sfu(w.x), ex2_sfu(w.y)), make_float2(hx.x + fabsf(hx.x), hx.y + fabsf(hx.y)));
  } else {
    const float2 w = __fmul2_rn(hx, f2(-2.f * kLog2e));
    const float2 a = __ffma2_rn(make_float2(ex2_sfu(w.x), ex2_sfu(w.y)), f2(0.5f), f2(0.5f));
    return __fmul2_rn(hx, make_float2(rcp_sfu(a.x), rcp_sfu(a.y)));
  }
}
// act(x) of the few weights that are formed one by one.
template <int ACT>
__device__ __forceinline__ float cc_act(float x) { return cc_act2<ACT>(f2(0.5f * x)).x; }

// A bias table's entry in the units of the scores, log2 units for softmax.
template <int ACT>
__device__ __forceinline__ float cc_bias_unit() { return ACT == 2 ? kLog2e : 1.0f; }
// Of a softmax bias, -inf hides its key as a mask would (an infinity or NaN there
// as well), and a finite entry that would leave fp32 in log2 units (the type's
// lowest value as a mask) counts as the largest that does not: where nothing else
// is seen, such keys weigh the same.  Both are rare: the kernels look for entries
// beyond kHugeBias and put things right afterwards, if there are any.
constexpr float kHugeBias = 2.358e38f, kHugeScore = kHugeBias * kLog2e;
__device__ __forceinline__ float cc_huge(float b) {  // in log2 units
  return fabsf(b) > kHugeBias ? copysignf(kHugeScore, b) : b * kLog2e;
}
// The LSE of a row from its maximum (log2 units) and sum.
__device__ __forceinline__ float cc_lse(float m, float l) {
  if (l == 0.f) return -INFINITY;
  return fabsf(m) == kHugeScore ? copysignf(3.402823466e38f, m) : (m + log2f(l)) * kLn2;
}

// The halves of a packed bf16 pair that are infinite or NaN, as a mask.
__device__ __forceinline__ uint32_t cc_nonfinite(uint32_t v) {
  return ((v & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((v & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}

// The position of new token u: C + depth, a negative depth taken as 0 and a
// position beyond 2^31 - 1 as that, which keeps what follows from positions (keys
// behind the window or the bias table's reach, in 32 bits) true of any input.
__device__ __forceinline__ int cc_new_pos(const CacheFwdParams& p, const CacheReq& r, int u) {
  if (p.depth == nullptr) return r.C + u;
  const int depth = max(__ldg(p.depth + r.q0 + u), 0);
  return static_cast<int>(min(static_cast<uint32_t>(r.C) + static_cast<uint32_t>(depth), 0x7FFFFFFFu));
}
// The same for the token of a query row; depths out of range are reported.
__device__ __forceinline__ int cc_row_pos(const CacheFwdParams& p, const CacheReq& r, int t, int* status) {
  if (p.depth != nullptr) {
    const int depth = __ldg(p.depth + r.q0 + t);
    if (depth < 0 || depth > INT32_MAX - r.C) atomicCAS(status, kOk, kErrBadOffsets);
  }
  return cc_new_pos(p, r, t);
}
// The position of key j (C for places behind the last token).
__device__ __forceinline__ int cc_pos(const CacheFwdParams& p, const CacheReq& r, int j) {
  return j < r.C ? j : (j < r.L ? cc_new_pos(p, r, j - r.C) : r.C);
}

__device__ __forceinline__ uint32_t cc_ones(int n) { return n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u); }

// Which of the keys key0 .. key0 + 31 a row sees by length and mask (bit c:
// key0 + c), whatever the window.
static __device__ __noinline__ uint32_t cc_vis32(const CacheFwdParams& p, CacheReq r, CcRow q, int key0) {
  if (q.t < 0) return 0u;
  if (p.mask == nullptr) return cc_ones(min(r.L, r.C + q.t + 1) - key0);
  const int u0 = key0 - r.C;
  uint32_t bits = 0xFFFFFFFFu;
  if (u0 > -32) {  // words i and i + 1 of the row's mask, the context's ones before the first
    const int32_t* words = p.mask + static_cast<int64_t>(r.q0 + q.t) * p.mask_words;
    const int i = u0 >> 5;
    const uint32_t lo = i < 0 ? 0xFFFFFFFFu : (i < p.mask_words ? static_cast<uint32_t>(__ldg(words + i)) : 0u);
    const uint32_t hi = i + 1 < p.mask_words ? static_cast<uint32_t>(__ldg(words + i + 1)) : 0u;
    bits = __funnelshift_r(lo, hi, u0 & 31);
  }
  return bits & cc_ones(r.L - key0);
}
// Whether the window joins a row and a key, by their positions.
__device__ __forceinline__ bool cc_near(const CacheFwdParams& p, int pos, int key_pos) {
  const int apart = pos - key_pos;
  return p.window <= 0 || (apart < p.window && apart > -p.window);
}
// Whether the keys key0 .. key0 + 31 are at the positions of their numbers (the
// context's are, and the new tokens' without depths), and which of them the
// window then joins with a row: those in (pos - w, pos + w).
__device__ __forceinline__ bool cc_in_order(const CacheFwdParams& p, const CacheReq& r, int key0) {
  return p.depth == nullptr || key0 + 31 < r.C;
}
__device__ __forceinline__ uint32_t cc_near32(const CacheFwdParams& p, int pos, int key0) {
  const int64_t at = static_cast<int64_t>(pos) - key0;
  const int lo = static_cast<int>(min(max(at - p.window + 1, int64_t{0}), int64_t{32}));
  const int hi = static_cast<int>(min(max(at + p.window, int64_t{0}), int64_t{32}));
  return cc_ones(hi) & ~cc_ones(lo);
}
// The bias table's entry of a row for a key position (any position: the index is clamped).
__device__ __forceinline__ float cc_bias(const CacheFwdParams& p, const CcRow& q, int reach, int key_pos) {
  const int at = min(max(q.pos - key_pos, -reach), reach) + reach;
  return __ldg(p.bias + static_cast<int64_t>(q.head) * p.bias_len + at);
}

// x innermost: columns, rows of the page, column halves, heads, pages
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int u, int w) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(w)
      : "memory");
}

}  // namespace jg
