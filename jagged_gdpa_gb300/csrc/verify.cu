// Verification of drafted tokens.  Row 0 of a request is the token it ended
// with, every other row a drafted token that continues an earlier row, its parent.
// From the root on, a row's children are tried in order, child c with token x:
//
//   drafts with probabilities (chains):  u_c q_c(x) < p_parent(x)
//   drafts without (chains and trees):   u_c (1 - sum of p_parent over the tokens
//                                        refused before) < p_parent(x)
//
// and the first that passes is the next row.  Where none passes, the next token
// is drawn from what is left of the last row's distribution: max(p - q, 0), each
// difference rounded to fp32, or p without the refused tokens: the first i whose
// prefix sum exceeds u times the sum.
//
// What takes time is one row of the vocabulary per request (two with the draft's):
// a cluster of 1 to 8 CTAs reads it once, each warp a contiguous piece; the pieces' sums
// meet through distributed shared memory, and the CTA that holds the piece the number falls
// into reads that again (from L2).  With V borders between tokens, an error of e
// in the prefix sums draws another token with probability V e: in fp32 (2^-24)
// one row in some hundred, so the sums are held as unevaluated pairs of fp32
// (some 2^-46; FP64 runs at a sixtieth of the rate here).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "cache.cuh"
#include "common.cuh"
#include "verify.cuh"

namespace jg {

namespace cg = cooperative_groups;

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerMaxCluster = 8;

// hi + lo, |lo| at most half a last place of hi
struct Sum2 {
  float hi, lo;
};
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}
__device__ __forceinline__ Sum2 add(Sum2 a, float v) {
  float s, e;
  two_sum(a.hi, v, s, e);
  return {s, __fadd_rn(a.lo, e)};
}
__device__ __forceinline__ Sum2 add(Sum2 a, Sum2 b) {
  float s, e;
  two_sum(a.hi, b.hi, s, e);
  e = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
  const float hi = __fadd_rn(s, e);
  return {hi, __fsub_rn(e, __fsub_rn(hi, s))};
}
__device__ __forceinline__ Sum2 times(Sum2 a, float u) {
  const float p = __fmul_rn(a.hi, u);
  const float e = __fmaf_rn(a.lo, u, __fmaf_rn(a.hi, u, -p));
  const float hi = __fadd_rn(p, e);
  return {hi, __fsub_rn(e, __fsub_rn(hi, p))};
}
__device__ __forceinline__ bool above(Sum2 a, Sum2 b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ Sum2 shfl_up(Sum2 a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
}
// Sums of lanes 0 .. lane.
__device__ __forceinline__ Sum2 warp_prefix(Sum2 a) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum2 b = shfl_up(a, o);
    if ((threadIdx.x & 31) >= o) a = add(b, a);
  }
  return a;
}

__device__ __forceinline__ float prob(const float* p) { return *p; }
__device__ __forceinline__ float prob(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// What is left of a row's distribution at token i.
template <typename TP, typename TQ>
struct Rest {
  const TP* p;
  const TQ* q;          // subtracted, or nullptr
  const int* refused;   // tokens that count nothing
  int n_refused;
  __device__ __forceinline__ float operator()(int i) const {
    float r = prob(p + i);
    if (q != nullptr) r = __fsub_rn(r, prob(q + i));
    for (int k = 0; k < n_refused; ++k)
      if (refused[k] == i) return 0.f;
    return r > 0.f && r <= 3.402823466e38f ? r : 0.f;  // (a NaN or an infinity counts nothing)
  }
};

struct VerShared {
  int token[kVerifyMaxTokens], parent[kVerifyMaxTokens];
  float p[kVerifyMaxTokens];      // the parent's probability of the row's token
  int child[kVerifyMaxTokens];    // the row's first accepted child; then its place
  unsigned char first[kVerifyMaxTokens], ok[kVerifyMaxTokens];
  int kept, last, n_refused;
  Sum2 piece[kVerWarps];          // sums of the CTA's pieces, read by the whole cluster
  Sum2 warp_sum[kVerWarps];
  Sum2 before, target;
  int win, winner, last_one;
};

// Which rows stay; every CTA of the cluster comes to the same.
template <typename TP, typename TQ>
__device__ void verify_walk(const VerifyParams& p, VerShared* sh, int q0, int T) {
  const int tid = threadIdx.x;
  const TP* target = static_cast<const TP*>(p.target);
  const TQ* draft = static_cast<const TQ*>(p.draft);
  for (int t = tid; t < T; t += kVerThreads) {
    const int x = p.tokens[q0 + t], up = t == 0 ? -1 : p.parents != nullptr ? p.parents[q0 + t] : t - 1;
    const bool valid = t > 0 && up >= 0 && up < t && x >= 0 && x < p.vocab;
    if (t > 0 && !valid && p.status != nullptr) atomicCAS(p.status, kOk, kErrBadOffsets);
    sh->token[t] = x;
    sh->parent[t] = valid ? up : -1;
    sh->child[t] = INT32_MAX;
    sh->first[t] = valid;
    const float pt = valid ? prob(target + (q0 + up) * p.target_stride + x) : 0.f;
    sh->p[t] = pt;
    if (draft != nullptr && valid)
      sh->ok[t] = static_cast<double>(p.uniforms[q0 + t]) * prob(draft + (q0 + t) * p.draft_stride + x) < pt;
    else
      sh->ok[t] = 0;
  }
  __syncthreads();
  if (draft == nullptr) {
    if (p.parents != nullptr) {  // (a chain has no siblings) of equal tokens the first counts
      for (int t = tid; t < T; t += kVerThreads)
        for (int s = 1; s < t; ++s)
          if (sh->parent[s] == sh->parent[t] && sh->token[s] == sh->token[t]) sh->first[t] = 0;
      __syncthreads();
    }
    for (int t = tid; t < T; t += kVerThreads) {
      if (!sh->first[t]) continue;
      double gone = 0.0;
      if (p.parents != nullptr)
        for (int s = 1; s < t; ++s)
          if (sh->first[s] && sh->parent[s] == sh->parent[t]) gone += sh->p[s];
      sh->ok[t] = p.uniforms[q0 + t] * (1.0 - gone) < sh->p[t];
    }
    __syncthreads();
  }
  for (int t = tid; t < T; t += kVerThreads)
    if (sh->ok[t]) atomicMin(&sh->child[sh->parent[t]], t);
  __syncthreads();
  if (tid == 0) {
    int at = 0, n = 0;
    for (;;) {
      const int to = sh->child[at];
      sh->child[at] = -1 - n++;  // its place, -1 - n, which no child is
      if (to == INT32_MAX) break;
      at = to;
    }
    sh->kept = n;
    sh->last = at;
    sh->n_refused = 0;
  }
  __syncthreads();
}

template <typename TP, typename TQ>
__global__ void __launch_bounds__(kVerThreads, 2) verify_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ VerShared sh;
  cache_let_next();
  cache_wait_before();
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_cta = cluster.num_blocks(), rank = cluster.block_rank(), b = blockIdx.x / n_cta;
  const int q0 = p.q_off[b], q1 = p.q_off[b + 1];
  const bool valid = q0 >= 0 && q1 >= q0 && q1 <= p.total && (b > 0 || q0 == 0);
  const int T = valid && q1 - q0 <= kVerifyMaxTokens ? q1 - q0 : 0;
  if (T != q1 - q0 && tid == 0 && p.status != nullptr) atomicCAS(p.status, kOk, kErrBadOffsets);
  // rows behind the last request
  const int last_row = p.q_off[p.batch];
  if (last_row >= 0 && last_row < p.total)
    for (int64_t r = last_row + static_cast<int64_t>(blockIdx.x) * kVerThreads + tid; r < p.total;
         r += static_cast<int64_t>(gridDim.x) * kVerThreads) {
      p.places[r] = -1;
      if (p.keep_slots != nullptr) p.keep_slots[r] = -1;
    }
  if (T == 0) {  // (the whole cluster)
    if (rank != 0) return;
    if (tid == 0) {
      p.accepted[b] = 0;
      p.next[b] = -1;
      if (p.keep_lens != nullptr) p.keep_lens[b] = p.kv_lens[b];
    }
    for (int r = q0 + tid; valid && r < q1; r += kVerThreads) {
      p.places[r] = -1;
      if (p.keep_slots != nullptr) p.keep_slots[r] = -1;
    }
    return;
  }
  verify_walk<TP, TQ>(p, &sh, q0, T);
  const int kept = sh.kept, last = sh.last;
  if (rank == 0) {
    if (tid == 0) {
      p.accepted[b] = kept;
      if (p.keep_lens != nullptr) p.keep_lens[b] = p.kv_lens[b] - T + kept;
    }
    for (int t = tid; t < T; t += kVerThreads) {
      const int place = sh.child[t] < 0 ? -1 - sh.child[t] : -1;
      p.places[q0 + t] = place;
      if (p.keep_slots != nullptr) p.keep_slots[q0 + t] = place >= 0 && place != t ? p.slots[q0 + place] : -1;
    }
  }
  Rest<TP, TQ> rest{static_cast<const TP*>(p.target) + (q0 + last) * p.target_stride, nullptr, sh.token, 0};
  if (p.draft != nullptr) {
    if (last + 1 < T) rest.q = static_cast<const TQ*>(p.draft) + (q0 + last + 1) * p.draft_stride;
  } else {
    // the refused children's tokens, to the front of the list of tokens, which is of no further use
    __syncthreads();
    int mine[kVerifyMaxTokens / kVerThreads];
#pragma unroll
    for (int i = 0; i < kVerifyMaxTokens / kVerThreads; ++i) {
      const int t = tid + i * kVerThreads;
      mine[i] = t < T && sh.parent[t] == last && sh.first[t] ? sh.token[t] : -1;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kVerifyMaxTokens / kVerThreads; ++i)
      if (mine[i] >= 0) sh.token[atomicAdd(&sh.n_refused, 1)] = mine[i];
    __syncthreads();
    rest.n_refused = sh.n_refused;
  }
  // pieces of the vocabulary: warp w of CTA c takes piece 16 c + w
  const int pieces = n_cta * kVerWarps;
  const int piece = (p.vocab + pieces - 1) / pieces;
  const int64_t from = static_cast<int64_t>(rank * kVerWarps + warp) * piece;
  const int lo = static_cast<int>(min(from, static_cast<int64_t>(p.vocab)));
  const int hi = static_cast<int>(min(from + piece, static_cast<int64_t>(p.vocab)));
  int next = -1;
#pragma unroll 1
  for (int attempt = 0; attempt < 2; ++attempt) {
    Rest<TP, TQ> here = rest;
    if (rest.n_refused > 0) {
      bool any = false;
      for (int k = 0; k < rest.n_refused; ++k) any = any || (sh.token[k] >= lo && sh.token[k] < hi);
      if (!any) here.n_refused = 0;
    }
    constexpr int kWays = 8;
    Sum2 part[kWays];
#pragma unroll
    for (int i = 0; i < kWays; ++i) part[i] = {0.f, 0.f};
    int at = lo + lane;
    if (here.n_refused == 0)
      for (; at + (kWays - 1) * 32 < hi; at += kWays * 32) {
        float v[kWays];
#pragma unroll
        for (int i = 0; i < kWays; ++i) v[i] = here(at + 32 * i);
#pragma unroll
        for (int i = 0; i < kWays; ++i) part[i] = add(part[i], v[i]);
      }
    for (; at < hi; at += 32) part[0] = add(part[0], here(at));
    Sum2 sum = part[0];
#pragma unroll
    for (int i = 1; i < kWays; ++i) sum = add(sum, part[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1)
      sum = add(sum, Sum2{__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)});
    if (lane == 0) sh.piece[warp] = sum;
    cluster.sync();
    if (warp == 0) {  // the piece that the number falls into
      constexpr int kEach = kVerMaxCluster * kVerWarps / 32;
      Sum2 own[kEach], run[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int k = lane * kEach + i;
        own[i] = {0.f, 0.f};
        if (k < pieces) own[i] = *cluster.map_shared_rank(&sh.piece[k % kVerWarps], k / kVerWarps);
        run[i] = i == 0 ? own[0] : add(run[i - 1], own[i]);
      }
      const Sum2 prefix = warp_prefix(run[kEach - 1]);
      const Sum2 total = {__shfl_sync(0xffffffffu, prefix.hi, 31), __shfl_sync(0xffffffffu, prefix.lo, 31)};
      Sum2 before = shfl_up(prefix, 1);
      if (lane == 0) before = {0.f, 0.f};
      const Sum2 goal = times(total, p.uniforms[q0]);
      int win = INT32_MAX, some = -1;
      Sum2 win_before = {0.f, 0.f}, some_before = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (own[i].hi > 0.f) {
          const Sum2 start = i == 0 ? before : add(before, run[i - 1]);
          some = lane * kEach + i;
          some_before = start;
          if (win == INT32_MAX && above(add(before, run[i]), goal)) {
            win = some;
            win_before = start;
          }
        }
      }
      // (the number at the very end of the sum, by rounding or because it is no number below 1: the last piece with any)
      const int best = __reduce_min_sync(0xffffffffu, win), rest_of = __reduce_max_sync(0xffffffffu, some);
      if (best == INT32_MAX) {
        win = some;
        win_before = some_before;
      }
      const int pick = best == INT32_MAX ? rest_of : best;
      if (lane == 0 && pick < 0) sh.win = -1;
      if (pick >= 0 && win == pick) {
        sh.win = pick;
        sh.before = win_before;
        sh.target = goal;
      }
    }
    if (tid == 0) {
      sh.winner = INT32_MAX;
      sh.last_one = -1;
    }
    cluster.sync();  // the sums have been read by all
    if (sh.win >= 0) break;
    // nothing left to draw from: the row itself
    rest.q = nullptr;
    rest.n_refused = 0;
  }
  if (sh.win < 0) {
    if (rank == 0 && tid == 0) p.next[b] = -1;
    return;
  }
  if (sh.win / kVerWarps != rank) return;
  // this CTA's: each thread some tokens in a row
  const int w0 = sh.win * piece, w1 = min(w0 + piece, p.vocab);
  const int each = (piece + kVerThreads - 1) / kVerThreads;
  const int i0 = min(w0 + tid * each, w1), i1 = min(i0 + each, w1);
  Sum2 sum = {0.f, 0.f};
  for (int i = i0; i < i1; ++i) sum = add(sum, rest(i));
  const Sum2 prefix = warp_prefix(add(sum, Sum2{0.f, 0.f}));
  if (lane == 31) sh.warp_sum[warp] = prefix;
  __syncthreads();
  Sum2 before = sh.before;
  for (int w = 0; w < warp; ++w) before = add(before, sh.warp_sum[w]);
  const Sum2 to_here = add(before, prefix);
  Sum2 start = shfl_up(prefix, 1);
  start = lane == 0 ? before : add(before, start);
  if (sum.hi > 0.f) {
    atomicMax(&sh.last_one, tid);
    if (above(to_here, sh.target)) atomicMin(&sh.winner, tid);
  }
  __syncthreads();
  const int winner = sh.winner == INT32_MAX ? sh.last_one : sh.winner;
  if (tid == winner) {
    Sum2 run = start;
    for (int i = i0; i < i1; ++i) {
      const float r = rest(i);
      if (r > 0.f) {
        next = i;
        run = add(run, Sum2{r, 0.f});
        if (above(run, sh.target)) break;
      }
    }
    p.next[b] = next;
  }
}

template <typename TP, typename TQ>
static cudaError_t launch_verify_t(const VerifyParams& p, int cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * cluster);
  cfg.blockDim = dim3(kVerThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<TP, TQ>, p);
}

cudaError_t launch_verify(const VerifyParams& p, bool target_half, bool draft_half, int sms, cudaStream_t stream) {
  // a row is split as long as that fills SMs and leaves a warp 128 tokens
  int cluster = 1;
  while (cluster < kVerMaxCluster && static_cast<int64_t>(p.batch) * cluster < sms && p.vocab / (2 * cluster) >= 128 * kVerWarps)
    cluster *= 2;
  if (target_half)
    return draft_half ? launch_verify_t<__nv_bfloat16, __nv_bfloat16>(p, cluster, stream)
                      : launch_verify_t<__nv_bfloat16, float>(p, cluster, stream);
  return draft_half ? launch_verify_t<float, __nv_bfloat16>(p, cluster, stream)
                    : launch_verify_t<float, float>(p, cluster, stream);
}

}  // namespace jg
