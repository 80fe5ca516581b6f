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
//
// Chains of 2 to 6 with drafts' probabilities, fp32, 128,000 tokens: 64 requests 19 us
// (the two rows 9.7 at the copy bandwidth), 256 requests 48 us, 0.80 of it.  What few
// requests take is latency: gathers along the chain, two meetings of the cluster
// and the second reading of a piece, some 8 to 9 us.  With one value at a time
// instead of 16 bytes in paired sums: 28 and 79 us.  That (with 8 loads at once) is still the way of rows of
// target and draft that lie otherwise in their 16 bytes, which contiguous rows do unless the vocabulary is a
// multiple of 4 (fp32) or 8 (bf16), and of types that differ: 23 and 55 us at 128,001 tokens in fp32; in bf16 20
// and 48 us, where 128,000 tokens take 16 and 34.  8 trees of 8 to 33 over 50,001
// tokens: 11 us (14 with a thread per row that went through the rows before it in FP64).
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

__device__ __forceinline__ Sum2 warp_sum(Sum2 a) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    a = add(a, Sum2{__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)});
  return a;
}

__device__ __forceinline__ float prob(const float* p) { return *p; }
__device__ __forceinline__ float prob(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// (An entry that is negative, infinite or NaN counts nothing.)
__device__ __forceinline__ float counted(float r) { return r > 0.f && r <= 3.402823466e38f ? r : 0.f; }

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
    return counted(r);
  }
};

// Two sums side by side.
struct Sums2 {
  float2 hi, lo;
};
__device__ __forceinline__ float2 minus(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.f, -1.f), a); }
__device__ __forceinline__ void add(Sums2& a, float2 v) {
  const float2 s = __fadd2_rn(a.hi, v), t = minus(s, a.hi);
  a.lo = __fadd2_rn(a.lo, __fadd2_rn(minus(a.hi, minus(s, t)), minus(v, t)));
  a.hi = s;
}
// 16 bytes of a row as fp32 pairs.
template <typename T>
struct Piece {
  static constexpr int kValues = 16 / sizeof(T);
  float2 v[kValues / 2];
  __device__ __forceinline__ explicit Piece(const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < kValues / 2; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
      else v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
  }
};

// The sum of what is left at tokens [lo, hi), the warp's, in 16-byte pieces from the first
// that starts one (lo, but for a row's head) on.  r0 and r1 count nothing.  Infinities are not looked for:
// the sum is no number then.
template <typename T>
__device__ __forceinline__ Sum2 verify_sum_pieces(const T* p, const T* q, int lo, int hi, int r0, int r1) {
  constexpr int kV = Piece<T>::kValues, kWays = 4;
  const int lane = threadIdx.x & 31;
  Sums2 part[kWays];
#pragma unroll
  for (int i = 0; i < kWays; ++i) part[i].hi = part[i].lo = make_float2(0.f, 0.f);
  auto take = [&](Sums2& to, const uint4& a, const uint4& b, int at) {
    Piece<T> x(a);
    if (q != nullptr) {
      const Piece<T> y(b);
#pragma unroll
      for (int i = 0; i < kV / 2; ++i) x.v[i] = minus(x.v[i], y.v[i]);
    }
    const uint32_t o0 = static_cast<uint32_t>(r0 - at), o1 = static_cast<uint32_t>(r1 - at);
    if (o0 < kV || o1 < kV) {
#pragma unroll
      for (int i = 0; i < kV / 2; ++i) {
        if (o0 == 2 * i || o1 == 2 * i) x.v[i].x = 0.f;
        if (o0 == 2 * i + 1 || o1 == 2 * i + 1) x.v[i].y = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kV / 2; ++i) add(to, make_float2(fmaxf(x.v[i].x, 0.f), fmaxf(x.v[i].y, 0.f)));
  };
  const int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p + lo) & 15)) & 15) / static_cast<int>(sizeof(T));
  const int first = min(lo + head, hi), end = first + (hi - first) / kV * kV;
  // the row's head and tail, a lane each (fewer than 8)
  const int rest = lane < 8 ? lo + lane : end + lane - 8;
  float edge = 0.f;
  if (lane < 16 && (lane < 8 ? rest < first : rest < hi) && rest != r0 && rest != r1) {
    edge = prob(p + rest);
    if (q != nullptr) edge = __fsub_rn(edge, prob(q + rest));
  }
  int at = first + lane * kV;
  const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll 1
  for (; at + (kWays - 1) * 32 * kV < end; at += kWays * 32 * kV) {
    uint4 a[kWays], b[kWays];
#pragma unroll
    for (int i = 0; i < kWays; ++i) {
      a[i] = *reinterpret_cast<const uint4*>(p + at + i * 32 * kV);
      b[i] = q != nullptr ? *reinterpret_cast<const uint4*>(q + at + i * 32 * kV) : none;
    }
#pragma unroll
    for (int i = 0; i < kWays; ++i) take(part[i], a[i], b[i], at + i * 32 * kV);
  }
  {
    uint4 a[kWays - 1], b[kWays - 1];
#pragma unroll
    for (int i = 0; i < kWays - 1; ++i) {
      const bool in = at + i * 32 * kV < end;
      a[i] = in ? *reinterpret_cast<const uint4*>(p + at + i * 32 * kV) : none;
      b[i] = in && q != nullptr ? *reinterpret_cast<const uint4*>(q + at + i * 32 * kV) : none;
    }
#pragma unroll
    for (int i = 0; i < kWays - 1; ++i) take(part[i], a[i], b[i], at + i * 32 * kV);
  }
  Sum2 sum{fmaxf(edge, 0.f), 0.f};
#pragma unroll
  for (int i = 0; i < kWays; ++i) {
    sum = add(sum, Sum2{part[i].hi.x, part[i].lo.x});
    sum = add(sum, Sum2{part[i].hi.y, part[i].lo.y});
  }
  return sum;
}

struct VerShared {
  int token[kVerifyMaxTokens], parent[kVerifyMaxTokens];
  float p[kVerifyMaxTokens];      // the parent's probability of the row's token
  float u[kVerifyMaxTokens];
  int child[kVerifyMaxTokens];    // the row's first accepted child; then its place
  Sum2 gone[kVerifyMaxTokens];    // the probabilities of its earlier siblings
  unsigned char first[kVerifyMaxTokens], ok[kVerifyMaxTokens];
  int kept, last, n_refused;
  Sum2 piece[kVerWarps];          // sums of the CTA's pieces, read by the whole cluster
  Sum2 warp_sum[kVerWarps];
  Sum2 before, target;
  int win, winner, last_one, n_here;
  int here[kVerifyMaxTokens];     // refused tokens of the piece that is searched
};

// Which rows stay; every CTA of the cluster comes to the same.
template <typename TP, typename TQ>
__device__ void verify_walk(const VerifyParams& p, VerShared* sh, int q0, int T) {
  const int tid = threadIdx.x;
  const TP* target = static_cast<const TP*>(p.target);
  const TQ* draft = static_cast<const TQ*>(p.draft);
  for (int t = tid; t < T; t += kVerThreads) {
    const int x = p.tokens[q0 + t], up = t == 0 ? -1 : p.parents != nullptr ? p.parents[q0 + t] : t - 1;
    const float u = p.uniforms[q0 + t];
    const bool valid = t > 0 && up >= 0 && up < t && x >= 0 && x < p.vocab;
    if (t > 0 && !valid && p.status != nullptr) atomicCAS(p.status, kOk, kErrBadOffsets);
    const float pt = valid ? counted(prob(target + (q0 + up) * p.target_stride + x)) : 0.f;
    const float qt = valid && draft != nullptr ? prob(draft + (q0 + t) * p.draft_stride + x) : 0.f;
    sh->token[t] = x;
    sh->parent[t] = valid ? up : -1;
    sh->child[t] = INT32_MAX;
    sh->first[t] = valid;
    sh->p[t] = pt;
    sh->u[t] = u;
    sh->ok[t] = draft != nullptr && pt > 0.f && static_cast<double>(u) * qt < pt;
  }
  __syncthreads();
  if (draft == nullptr) {
    if (p.parents != nullptr) {  // (a chain has no siblings)
      // a warp per row, its lanes over the earlier ones: of equal siblings the first counts
      const int lane = tid & 31, warp = tid >> 5;
      for (int t = 1 + warp; t < T; t += kVerWarps) {
        const int up = sh->parent[t], x = sh->token[t];
        bool twin = false;
        for (int s = 1 + lane; s < t; s += 32) twin = twin || (sh->parent[s] == up && sh->token[s] == x);
        if (__any_sync(0xffffffffu, twin) && lane == 0) sh->first[t] = 0;
      }
      __syncthreads();
      for (int t = 1 + warp; t < T; t += kVerWarps) {
        if (!sh->first[t]) continue;
        const int up = sh->parent[t];
        Sum2 sum{0.f, 0.f};
        bool some = false;
        for (int s = 1 + lane; s < t; s += 32)
          if (sh->parent[s] == up && sh->first[s]) {
            sum = add(sum, sh->p[s]);
            some = true;
          }
        if (__any_sync(0xffffffffu, some)) sum = warp_sum(sum);
        if (lane == 0) sh->gone[t] = sum;
      }
      __syncthreads();
    }
    for (int t = tid; t < T; t += kVerThreads) {
      if (!sh->first[t]) continue;
      double left = 1.0;
      if (p.parents != nullptr && sh->gone[t].hi != 0.f) left -= static_cast<double>(sh->gone[t].hi) + sh->gone[t].lo;
      sh->ok[t] = sh->u[t] * left < sh->p[t];
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

// The rows that stay, written out.
__device__ __forceinline__ void verify_kept(const VerifyParams& p, const VerShared* sh, int b, int q0, int T) {
  if (threadIdx.x == 0) {
    p.accepted[b] = sh->kept;
    if (p.keep_lens != nullptr) p.keep_lens[b] = p.kv_lens[b] - T + sh->kept;
  }
  for (int t = threadIdx.x; t < T; t += kVerThreads) {
    const int place = sh->child[t] < 0 ? -1 - sh->child[t] : -1;
    p.places[q0 + t] = place;
    if (p.keep_slots != nullptr) p.keep_slots[q0 + t] = place >= 0 && place != t ? p.slots[q0 + place] : -1;
  }
}

// Rows behind the last request.  (Offsets that are out of order lead from row 0 to here in steps of which
// the forward ones are some request's rows and the rest these, so that every row is written.)
__device__ __forceinline__ void verify_padding(const VerifyParams& p) {
  const int last = max(p.q_off[p.batch], 0);
  if (last >= p.total) return;
  for (int64_t r = last + static_cast<int64_t>(blockIdx.x) * kVerThreads + threadIdx.x; r < p.total;
       r += static_cast<int64_t>(gridDim.x) * kVerThreads) {
    p.places[r] = -1;
    if (p.keep_slots != nullptr) p.keep_slots[r] = -1;
  }
}

// The token the number falls into, of [w0, w1), by one CTA: each thread some tokens in a row.
template <typename TP, typename TQ>
__device__ __forceinline__ void verify_next(const VerifyParams& p, VerShared* sh, Rest<TP, TQ> rest, int b, int w0, int w1) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (rest.n_refused > 0) {
    for (int k = tid; k < rest.n_refused; k += kVerThreads) {
      const int x = rest.refused[k];
      if (x >= w0 && x < w1) sh->here[atomicAdd(&sh->n_here, 1)] = x;
    }
    __syncthreads();
    rest.refused = sh->here;
    rest.n_refused = sh->n_here;
  }
  const int each = (w1 - w0 + kVerThreads - 1) / kVerThreads;
  const int i0 = min(w0 + tid * each, w1), i1 = min(i0 + each, w1);
  Sum2 sum = {0.f, 0.f};
  for (int i = i0; i < i1; ++i) sum = add(sum, rest(i));
  const Sum2 prefix = warp_prefix(add(sum, Sum2{0.f, 0.f}));
  if (lane == 31) sh->warp_sum[warp] = prefix;
  __syncthreads();
  Sum2 before = sh->before;
  for (int w = 0; w < warp; ++w) before = add(before, sh->warp_sum[w]);
  const Sum2 to_here = add(before, prefix);
  Sum2 start = shfl_up(prefix, 1);
  start = lane == 0 ? before : add(before, start);
  if (sum.hi > 0.f) {
    atomicMax(&sh->last_one, tid);
    if (above(to_here, sh->target)) atomicMin(&sh->winner, tid);
  }
  __syncthreads();
  // the winner's tokens, a lane of its warp each
  const int winner = sh->winner == INT32_MAX ? sh->last_one : sh->winner;
  if (winner >> 5 != warp) return;
  Sum2 run = {__shfl_sync(0xffffffffu, start.hi, winner & 31), __shfl_sync(0xffffffffu, start.lo, winner & 31)};
  const int j0 = __shfl_sync(0xffffffffu, i0, winner & 31), j1 = __shfl_sync(0xffffffffu, i1, winner & 31);
  int next = -1;
  for (int j = j0; j < j1; j += 32) {
    const float r = j + lane < j1 ? rest(j + lane) : 0.f;
    const Sum2 sums = warp_prefix(Sum2{r, 0.f});
    const unsigned some = __ballot_sync(0xffffffffu, r > 0.f);
    const unsigned over = __ballot_sync(0xffffffffu, r > 0.f && above(add(run, sums), sh->target));
    if (over != 0) {
      next = j + __ffs(over) - 1;
      break;
    }
    if (some != 0) next = j + 31 - __clz(some);
    run = add(run, Sum2{__shfl_sync(0xffffffffu, sums.hi, 31), __shfl_sync(0xffffffffu, sums.lo, 31)});
  }
  if (lane == 0) p.next[b] = next;
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
  if ((!valid || T != q1 - q0) && tid == 0 && p.status != nullptr) atomicCAS(p.status, kOk, kErrBadOffsets);
  if (T == 0) {  // (the whole cluster)
    if (rank == 0) {
      if (tid == 0) {
        p.accepted[b] = 0;
        p.next[b] = -1;
        if (p.keep_lens != nullptr) p.keep_lens[b] = p.kv_lens[b];
      }
      const int64_t begin = b == 0 ? 0 : max(q0, 0), end = min(q1, p.total);  // (64 bits: offsets of 2^31 - 1)
      for (int64_t r = begin + tid; r < end; r += kVerThreads) {
        p.places[r] = -1;
        if (p.keep_slots != nullptr) p.keep_slots[r] = -1;
      }
    }
    verify_padding(p);
    return;
  }
  verify_walk<TP, TQ>(p, &sh, q0, T);
  const int last = sh.last;
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
  // Pieces of the vocabulary: warp w of CTA c takes piece 16 c + w.  They are cut at whole
  // 16 bytes of the row in memory, which `shift` entries in front of it start.
  constexpr int kV = Piece<TP>::kValues;
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(rest.p) & 15) / static_cast<int>(sizeof(TP));
  const int pieces = n_cta * kVerWarps;
  const int piece = ((p.vocab + shift + pieces - 1) / pieces + kV - 1) / kV * kV;
  auto piece_lo = [&](int k) { return static_cast<int>(min(max(static_cast<int64_t>(k) * piece - shift, int64_t{0}), static_cast<int64_t>(p.vocab))); };
  const int lo = piece_lo(rank * kVerWarps + warp), hi = piece_lo(rank * kVerWarps + warp + 1);
#pragma unroll 1
  for (int attempt = 0; attempt < 2; ++attempt) {
    int r0 = -1, r1 = -1, n_here = 0;  // the piece's refused tokens
    for (int k0 = 0; k0 < rest.n_refused; k0 += 32) {
      const int x = k0 + lane < rest.n_refused ? rest.refused[k0 + lane] : -1;
      unsigned in = __ballot_sync(0xffffffffu, x >= lo && x < hi);
      n_here += __popc(in);
      for (; in != 0; in &= in - 1) {
        r1 = r0;
        r0 = __shfl_sync(0xffffffffu, x, __ffs(in) - 1);
      }
    }
    Sum2 sum{0.f, 0.f};
    bool good = false;
    if constexpr (sizeof(TP) == sizeof(TQ)) {
      // (rows of a draft that lie otherwise in their 16 bytes: one by one)
      if (n_here <= 2 && (rest.q == nullptr || ((reinterpret_cast<uintptr_t>(rest.p) ^ reinterpret_cast<uintptr_t>(rest.q)) & 15) == 0)) {
        sum = verify_sum_pieces<TP>(rest.p, reinterpret_cast<const TP*>(rest.q), lo, hi, r0, r1);
        good = __all_sync(0xffffffffu, sum.hi <= 3.402823466e38f);
      }
    }
    if (!good) {
      constexpr int kWays = 8;
      Rest<TP, TQ> here = rest;
      if (n_here == 0) here.n_refused = 0;
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
      sum = part[0];
#pragma unroll
      for (int i = 1; i < kWays; ++i) sum = add(sum, part[i]);
    }
    sum = warp_sum(sum);
    if (lane == 0) sh.piece[warp] = sum;
    __syncwarp();
    cluster.barrier_arrive();
    if (rank == 0 && attempt == 0) verify_kept(p, &sh, b, q0, T);  // (while the others arrive)
    __syncwarp();
    cluster.barrier_wait();
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
      sh.n_here = 0;
    }
    __syncwarp();
    cluster.barrier_arrive();  // (the sums have been read)
    __syncthreads();
    if (sh.win >= 0 || attempt == 1) break;
    cluster.barrier_wait();
    // nothing left to draw from: the row itself
    rest.q = nullptr;
    rest.n_refused = 0;
  }
  // the CTA that the number falls into looks on; the others wait until all have read their sums
  if (sh.win < 0 || sh.win / kVerWarps != rank) {
    if (sh.win < 0 && rank == 0 && tid == 0) p.next[b] = -1;
  } else {
    verify_next<TP, TQ>(p, &sh, rest, b, piece_lo(sh.win), piece_lo(sh.win + 1));
  }
  verify_padding(p);
  __syncwarp();
  cluster.barrier_wait();
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
