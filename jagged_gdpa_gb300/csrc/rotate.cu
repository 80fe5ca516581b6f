// Norms of queries and keys for each head and the rotation by position, in one
// pass: packed rows (forward and backward) and rows on their way into a paged
// cache.
//
//   h = x r w,  r = 1 / sqrt(mean x^2 + eps)          (over a head's D columns)
//   (y_a, y_b) = (h_a cos t - h_b sin t, h_b cos t + h_a sin t),  t = pos f_i
//
// and backward, with g the gradient rotated back, h0 = x r and dh = g w:
//
//   dx = r (dh - h0 mean(dh h0)),  dw = sum over rows and heads of g h0.
//
// A few operations per value: bound by HBM.  D / 16 lanes take a vector (one
// head of one row), each two 16-byte pieces that hold whole pairs, so the only
// exchange between lanes is that of the norm's sum.  Such a group of lanes walks a run of
// vectors in (row, head) order, so that a row's angles, times the norm's weights,
// are formed once for the heads of the run; a few vectors are loaded before the
// first is used.  Two values at a time (fp32 pairs).
//
// 121,249 rows of 8 + 8 heads of 128: forward 162 us, 0.91 of the copy bandwidth
// (with angles formed anew for every vector 223); backward 264 us, 0.83.  135,492 rows
// of 8 + 2 heads, interleaved, slices of a wider row: backward 206 us, 0.75.  Backward is bound
// by the latency of loads and of the two sums per vector, with 16 warps per SM, and
// by a row's sines and cosines, which fewer key/value heads share.  16,600 rows of 16 + 4 heads
// of 64 into the cache: 22 us, 0.66, of them some 4 start and end.
#include <algorithm>

#include "cache.cuh"
#include "common.cuh"
#include "ptx.cuh"
#include "rotate.cuh"

namespace jg {

constexpr int kRotThreads = 256;
constexpr int kRotWarps = kRotThreads / 32;
constexpr int kRotBatch = 4, kRotBackBatch = 2;  // vectors loaded at a time (forward 2, with 3 CTAs: 229 us for 162)
constexpr int kRotRun = 8;                       // vectors of a run in calls that fill the GPU (4 and 16 were slower)
constexpr int kRotCtas = 2, kRotBackCtas = 2;    // per SM

template <int D>
struct RotShape {
  static constexpr int kLanes = D / 16;        // of a vector
  static constexpr int kGroups = 32 / kLanes;  // vectors side by side in a warp
};

// An angle is kept as a fraction of a turn in 64-bit fixed point: the product of
// a position and a frequency's fraction, modulo 2^64, drops whole turns exactly,
// so that a far position is as exact as a near one.  f / 2 pi is formed in integers from those bits of
// 1 / (2 pi) that count (M. Payne, R. Hanek, Radian reduction for trigonometric functions, 1983), to
// 2^-64 for any f, which is 2^-33 of a turn at position 2^31.  (As a product in FP64, right to 2^-53 of f, a
// frequency of 10^6 was off by 2^-5 of a turn there; in two, small calls took 0.2 us more.)
__device__ __forceinline__ uint64_t turn_of(float f) {
  // 1 / (2 pi), from 2^-1 on
  constexpr uint32_t w0 = 0x28BE60DBu, w1 = 0x9391054Au, w2 = 0x7F09D5F4u, w3 = 0x7D4D3770u, w4 = 0x36D8A566u, w5 = 0x4F10E410u,
                     w6 = 0x7F9458EAu;
  const uint32_t u = __float_as_uint(f), e = (u >> 23) & 255;
  const uint32_t m = (u & 0x7FFFFFu) | (e != 0 ? 0x800000u : 0u);  // |f| = m 2^s
  const int s = max(static_cast<int>(e), 1) - 150;
  // 96 bits behind the point of 2^s / (2 pi), or (s < 0) of 1 / (2 pi)
  uint32_t a0 = w0, a1 = w1, a2 = w2;
  if (s > 0) {
    const int k = s >> 5;  // 0 to 3
    const uint32_t b0 = k == 0 ? w0 : k == 1 ? w1 : k == 2 ? w2 : w3, b1 = k == 0 ? w1 : k == 1 ? w2 : k == 2 ? w3 : w4,
                   b2 = k == 0 ? w2 : k == 1 ? w3 : k == 2 ? w4 : w5, b3 = k == 0 ? w3 : k == 1 ? w4 : k == 2 ? w5 : w6;
    a0 = __funnelshift_l(b1, b0, s);  // (by s % 32)
    a1 = __funnelshift_l(b2, b1, s);
    a2 = __funnelshift_l(b3, b2, s);
  }
  // times m: 32 bits before the point and 32 behind it in p0, 64 more in low
  const uint64_t p2 = static_cast<uint64_t>(m) * a2, p1 = static_cast<uint64_t>(m) * a1 + (p2 >> 32),
                 p0 = static_cast<uint64_t>(m) * a0 + (p1 >> 32);
  const uint64_t low = (p1 << 32) | static_cast<uint32_t>(p2);
  const int n = max(-s, 0);  // further on
  const uint64_t r = n < 32 ? (n == 0 ? (p0 << 32) | (low >> 32) : (p0 << (32 - n)) | (low >> (32 + n))) : n < 96 ? p0 >> (n - 32) : 0;
  return u >> 31 ? 0 - r : r;
}
__device__ __forceinline__ void sincos_turn(uint64_t f, int pos, float& s, float& c) {
  // bits 32 to 63 of the product, half a turn on, to 23 bits as a number of [1, 2)
  const uint32_t turn = static_cast<uint32_t>(pos) * static_cast<uint32_t>(f >> 32) + __umulhi(static_cast<uint32_t>(pos), static_cast<uint32_t>(f)) -
                        (pos < 0 ? static_cast<uint32_t>(f) : 0u);
  const float x = __uint_as_float(((turn + 0x80000100u) >> 9) | 0x3F800000u) - 1.5f;
  // [-pi, pi), where the hardware's sine and cosine are within 2^-20.9
  const float a = x * 6.283185307179586f;
  s = __sinf(a);
  c = __cosf(a);
}

// The segment of a row (any value where the offsets are not in order, but one
// of [0, batch)); the whole warp asks for the same row.
__device__ __forceinline__ int segment_of(const int32_t* off, int batch, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = batch;  // off[lo] <= row < off[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const unsigned below = __ballot_sync(0xffffffffu, at < hi && off[min(at, hi)] <= row);
    const int n = __ffs(~below) - 1, from = n < 0 ? 32 : n;  // steps that start at or before the row
    hi = min(lo + (from + 1) * step, hi);
    lo += from * step;
  }
  return lo;
}

// Where a lane's two pieces of a vector lie and how its 8 pairs are formed.
// Halves: piece p of the first 2n columns meets piece p + n / 8, both one
// lane's; the other pieces follow in order.  Interleaved: two pieces in order,
// their pairs side by side.
template <int D, bool PAIRS>
struct RotLane {
  int a, b;        // first columns of the two pieces
  int first;       // the first pair's frequency
  __device__ __forceinline__ RotLane(int n) {
    const int l = threadIdx.x % RotShape<D>::kLanes;
    if constexpr (PAIRS) {
      a = 16 * l;
      b = a + 8;
      first = 8 * l;
    } else {
      const bool turns = l < (n >> 3);
      a = turns ? 8 * l : 16 * l;
      b = turns ? 8 * l + n : 16 * l + 8;
      first = 8 * l;
    }
  }
};

// A lane's 8 pairs (a, b), two to a register pair: halves: a's from the first
// piece, b's from the second; interleaved: both from every word.
struct Pairs {
  float2 a[4], b[4];
};
__device__ __forceinline__ float2 rot_pair(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool PAIRS>
__device__ __forceinline__ void rot_unpack(const uint4& u, const uint4& v, Pairs& f) {
  const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (PAIRS) {
      const float2 p = rot_pair(i < 2 ? x[2 * i] : y[2 * i - 4]), q = rot_pair(i < 2 ? x[2 * i + 1] : y[2 * i - 3]);
      f.a[i] = make_float2(p.x, q.x);
      f.b[i] = make_float2(p.y, q.y);
    } else {
      f.a[i] = rot_pair(x[i]);
      f.b[i] = rot_pair(y[i]);
    }
  }
}
template <bool PAIRS>
__device__ __forceinline__ void rot_pack(const Pairs& f, uint4& u, uint4& v) {
  uint32_t x[4], y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (PAIRS) {
      (i < 2 ? x[2 * i] : y[2 * i - 4]) = pack_bf16(f.a[i].x, f.b[i].x);
      (i < 2 ? x[2 * i + 1] : y[2 * i - 3]) = pack_bf16(f.a[i].y, f.b[i].y);
    } else {
      x[i] = pack_bf16(f.a[i].x, f.a[i].y);
      y[i] = pack_bf16(f.b[i].x, f.b[i].y);
    }
  }
  u = make_uint4(x[0], x[1], x[2], x[3]);
  v = make_uint4(y[0], y[1], y[2], y[3]);
}
// (Not by the read-only path: the output may be the input itself.)
__device__ __forceinline__ uint4 rot_load(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Columns of a lane's pieces of w, in the order of its pairs.
template <bool PAIRS>
__device__ __forceinline__ void rot_weight(const float* w, int a, int b, Pairs& out) {
  float x[8], y[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    *reinterpret_cast<float4*>(x + 4 * i) = *reinterpret_cast<const float4*>(w + a + 4 * i);
    *reinterpret_cast<float4*>(y + 4 * i) = *reinterpret_cast<const float4*>(w + b + 4 * i);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (PAIRS) {
      const float* z = i < 2 ? x + 4 * i : y + 4 * i - 8;
      out.a[i] = make_float2(z[0], z[2]);
      out.b[i] = make_float2(z[1], z[3]);
    } else {
      out.a[i] = make_float2(x[2 * i], x[2 * i + 1]);
      out.b[i] = make_float2(y[2 * i], y[2 * i + 1]);
    }
  }
}

template <int LANES>
__device__ __forceinline__ float rot_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Follows the rows of one job: segment, position, angles.
template <int D, bool PAIRS>
struct RotRow {
  int row = -1, b = 0, start = 0, end = 0;
  bool live = false;  // not behind the last segment

  // At a job's first row of the warp's.
  __device__ __forceinline__ void enter(const RotateJob& j, int first_row) {
    row = -1;
    if (j.positions != nullptr || j.batch == 0) return;
    b = segment_of(j.offsets, j.batch, first_row);
    start = j.offsets[b];
    end = j.offsets[b + 1];
  }
  // Moves on to another row, one that is not before the last (an own one for
  // every group of lanes), and forms the sines and cosines of its angles.
  __device__ __forceinline__ void to(const RotateParams& p, const RotateJob& j, const RotLane<D, PAIRS>& l,
                                     const uint64_t* turn, int r, float2 (&s)[4], float2 (&c)[4]) {
    row = r;
    int64_t pos;
    if (j.positions != nullptr) {
      live = true;
      pos = j.positions[r];
    } else {
      while (r >= end && b + 1 < j.batch) {
        ++b;
        start = end;
        end = j.offsets[b + 1];
      }
      live = r >= start && r < end;
      pos = r - start;
      if (p.kv_lens != nullptr && live) {
        const int64_t ctx = static_cast<int64_t>(p.kv_lens[b]) - (end - start);
        if (p.depths != nullptr) {
          pos = p.depths[r];
          if (p.status != nullptr && pos < 0) atomicCAS(p.status, kOk, kErrBadOffsets);
        }
        pos += ctx;
        if (p.status != nullptr && (ctx < 0 || pos > INT32_MAX)) atomicCAS(p.status, kOk, kErrBadOffsets);
      }
    }
    if (j.copy) return;
    // (columns that do not rotate have frequencies of 0: sine 0, cosine 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(turn + l.first + 2 * i);
      sincos_turn(f.x, static_cast<int>(pos), s[i].x, c[i].x);
      sincos_turn(f.y, static_cast<int>(pos), s[i].y, c[i].y);
    }
  }
};

// The call's frequencies and weights, in shared memory.
template <int D>
struct RotShared {
  alignas(16) uint64_t turn[D / 2];
  alignas(16) float weight[2][D];
};
template <int D>
__device__ __forceinline__ void rot_setup(const RotateParams& p, RotShared<D>* sh) {
  const int tid = threadIdx.x;
  if (tid < D / 2) sh->turn[tid] = tid < p.pairs ? turn_of(p.inv_freq[tid]) : 0;
  for (int i = tid; i < 2 * D; i += kRotThreads) {
    const float* w = p.job[i / D].weight;
    sh->weight[i / D][i % D] = w != nullptr ? w[i % D] : 1.f;
  }
  __syncthreads();
}
// One CTA looks whether the offsets are in order.  (Rows are found in [0, rows)
// whatever the offsets hold.)
__device__ __forceinline__ void rot_check(const RotateParams& p) {
  bool ok = true;
  for (int k = 0; k < p.jobs; ++k) {
    const RotateJob& j = p.job[k];
    if (j.positions != nullptr) continue;
    if (k > 0) {  // (the same offsets of as many rows have been looked at)
      const RotateJob& i = p.job[k - 1];
      if (i.positions == nullptr && i.offsets == j.offsets && i.rows == j.rows) continue;
    }
    for (int i = threadIdx.x; i <= j.batch; i += kRotThreads) {
      const int v = j.offsets[i];
      ok = ok && (i == 0 ? v == 0 : v >= j.offsets[i - 1]) && v <= j.rows;
    }
  }
  if (!__syncthreads_and(ok) && threadIdx.x == 0) atomicCAS(p.status, kOk, kErrBadOffsets);
}

// A warp's units: an equal, contiguous share of the call's.
struct RotShare {
  int64_t at, end;
  __device__ __forceinline__ RotShare(int64_t units) {
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kRotWarps;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kRotWarps + (threadIdx.x >> 5);
    const int64_t each = units / warps, more = units - each * warps;
    at = w * each + min(w, more);
    end = at + each + (w < more ? 1 : 0);
  }
};

// A place among the vectors of a job.
struct RotAt {
  uint32_t row, head;
  __device__ __forceinline__ void next(uint32_t heads) {
    if (++head == heads) {
      head = 0;
      ++row;
    }
  }
};

__device__ __forceinline__ float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }

template <int D, bool NORM, bool PAIRS>
__global__ void __launch_bounds__(kRotThreads, kRotCtas) rotate_kernel(const __grid_constant__ RotateParams p) {
  using S = RotShape<D>;
  __shared__ RotShared<D> sh;
  cache_let_next();
  cache_wait_before();
  rot_setup<D>(p, &sh);
  if (blockIdx.x == 0 && p.status != nullptr) rot_check(p);
  const int group = (threadIdx.x & 31) / S::kLanes;
  const RotLane<D, PAIRS> lane(p.pairs);
  RotRow<D, PAIRS> at;
  // y_a = r (x_a ca - x_b sb), y_b = r (x_b cb + x_a sa): cosines and sines times
  // the weights of their columns (without a norm: cosines and sines)
  float2 ca[4] = {}, sa[4] = {}, cb[NORM ? 4 : 1] = {}, sb[NORM ? 4 : 1] = {};
  int k = -1;
#pragma unroll 1
  for (RotShare share(p.units); share.at < share.end; ++share.at) {
    bool enter = k < 0;
    if (enter) k = 0;
    while (k + 1 < p.jobs && share.at >= p.job[k + 1].unit0) {
      ++k;
      enter = true;
    }
    const RotateJob& j = p.job[k];
    const uint32_t heads = j.heads, vecs = static_cast<uint32_t>(j.rows) * heads;
    const uint32_t vec = (static_cast<uint32_t>(share.at - j.unit0) * S::kGroups + group) * p.run;
    const int n = static_cast<int>(min(vecs - min(vec, vecs), static_cast<uint32_t>(p.run)));
    RotAt here{vec / heads, 0};
    here.head = vec - here.row * heads;
    if (enter) at.enter(j, __shfl_sync(0xffffffffu, here.row, 0));
#pragma unroll 1
    for (int i0 = 0; i0 < p.run; i0 += kRotBatch) {
      uint4 u[kRotBatch], v[kRotBatch];
      RotAt load = here;
#pragma unroll
      for (int i = 0; i < kRotBatch; ++i) {
        u[i] = v[i] = make_uint4(0, 0, 0, 0);
        if (i0 + i < n) {
          const __nv_bfloat16* src = j.x + load.row * j.x_stride + load.head * D;
          u[i] = rot_load(src + lane.a);
          v[i] = rot_load(src + lane.b);
        }
        load.next(heads);
      }
#pragma unroll
      for (int i = 0; i < kRotBatch; ++i) {
        if (i0 + i >= p.run) break;
        if (i0 + i < n && static_cast<int>(here.row) != at.row) {
          float2 s[4], c[4];
          at.to(p, j, lane, sh.turn, here.row, s, c);
          if constexpr (NORM) {
            if (!j.copy) {
              Pairs w;
              rot_weight<PAIRS>(sh.weight[k], lane.a, lane.b, w);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                ca[e] = __fmul2_rn(c[e], w.a[e]);
                sa[e] = __fmul2_rn(s[e], w.a[e]);
                cb[e] = __fmul2_rn(c[e], w.b[e]);
                sb[e] = neg2(__fmul2_rn(s[e], w.b[e]));
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              ca[e] = c[e];
              sa[e] = s[e];
            }
          }
        }
        if (!j.copy) {
          Pairs f;
          rot_unpack<PAIRS>(u[i], v[i], f);
          float2 r = make_float2(1.f, 1.f);
          if constexpr (NORM) {
            float2 sq = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) sq = __ffma2_rn(f.b[e], f.b[e], __ffma2_rn(f.a[e], f.a[e], sq));
            r.x = r.y = rsqrtf(rot_sum<S::kLanes>(sq.x + sq.y) * (1.f / D) + p.eps);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 a = f.a[e], b = f.b[e];
            f.a[e] = __ffma2_rn(b, NORM ? sb[NORM ? e : 0] : neg2(sa[e]), __fmul2_rn(a, ca[e]));
            f.b[e] = __ffma2_rn(a, sa[e], __fmul2_rn(b, NORM ? cb[NORM ? e : 0] : ca[e]));
            if constexpr (NORM) {
              f.a[e] = __fmul2_rn(f.a[e], r);
              f.b[e] = __fmul2_rn(f.b[e], r);
            }
          }
          rot_pack<PAIRS>(f, u[i], v[i]);
        }
        if (i0 + i < n && at.live) {
          __nv_bfloat16* dst = j.y + here.row * j.y_stride;
          bool write = true;
          if (j.slots != nullptr) {
            const int slot = j.slots[here.row];
            write = static_cast<uint32_t>(slot) < static_cast<uint32_t>(p.slot_end);
            dst = j.y + (slot >> p.page_shift) * j.page_stride + static_cast<int64_t>(slot & ((1 << p.page_shift) - 1)) * (j.heads * D);
          }
          if (write) {
            dst += here.head * D;
            *reinterpret_cast<uint4*>(dst + lane.a) = u[i];
            *reinterpret_cast<uint4*>(dst + lane.b) = v[i];
          }
        }
        here.next(heads);
      }
    }
  }
}

// Backward of N vectors of a row, side by side (what lanes exchange and what is
// looked up costs the latency of one):
//   dx = r dh - x r^3 mean(dh x),  dw += (g x) r
// u, v: x; du, dv: dy, then dx.
template <int D, bool NORM, bool PAIRS, int N>
__device__ __forceinline__ void rot_back(const RotLane<D, PAIRS>& lane, const float* weight, float eps, const float2 (&s)[4],
                                         const float2 (&c)[4], const uint4* u, const uint4* v, uint4* du, uint4* dv, bool live,
                                         Pairs& acc) {
  Pairs g[N], x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    rot_unpack<PAIRS>(du[i], dv[i], g[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // the other way round
      const float2 a = g[i].a[e], b = g[i].b[e];
      g[i].a[e] = __ffma2_rn(b, s[e], __fmul2_rn(a, c[e]));
      g[i].b[e] = __ffma2_rn(a, neg2(s[e]), __fmul2_rn(b, c[e]));
    }
  }
  if constexpr (NORM) {
    Pairs w;
    rot_weight<PAIRS>(weight, lane.a, lane.b, w);
    float sq[N], dot[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      rot_unpack<PAIRS>(u[i], v[i], x[i]);
      float2 sq2 = make_float2(0.f, 0.f), dot2 = sq2;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sq2 = __ffma2_rn(x[i].b[e], x[i].b[e], __ffma2_rn(x[i].a[e], x[i].a[e], sq2));
        dot2 = __ffma2_rn(__fmul2_rn(g[i].a[e], x[i].a[e]), w.a[e], dot2);
        dot2 = __ffma2_rn(__fmul2_rn(g[i].b[e], x[i].b[e]), w.b[e], dot2);
      }
      sq[i] = sq2.x + sq2.y;
      dot[i] = dot2.x + dot2.y;
    }
#pragma unroll
    for (int o = RotShape<D>::kLanes / 2; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], o);
        dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], o);
      }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float r1 = rsqrtf(sq[i] * (1.f / D) + eps), m1 = (r1 * r1) * (r1 * dot[i]) * (-1.f / D);
      const float2 r = make_float2(r1, r1), m = make_float2(m1, m1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (live) {
          acc.a[e] = __ffma2_rn(__fmul2_rn(g[i].a[e], x[i].a[e]), r, acc.a[e]);
          acc.b[e] = __ffma2_rn(__fmul2_rn(g[i].b[e], x[i].b[e]), r, acc.b[e]);
        }
        g[i].a[e] = __ffma2_rn(x[i].a[e], m, __fmul2_rn(__fmul2_rn(g[i].a[e], w.a[e]), r));
        g[i].b[e] = __ffma2_rn(x[i].b[e], m, __fmul2_rn(__fmul2_rn(g[i].b[e], w.b[e]), r));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) rot_pack<PAIRS>(g[i], du[i], dv[i]);
}

// Backward.  The weights' gradients are sums over every row and head: a lane
// keeps its 16 columns' in registers over its warp's units of a job, the warps of
// a CTA meet in shared memory, the CTAs in `partial`, each in a fixed order (the
// same bits on every run).  Two vectors of a row are worked on side by side, so that
// one's sums hide the other's (one at a time: 267 and 215 us).  Inputs copied ahead into
// shared memory instead of registers took 240 to 290 and 252 to 307 us.
template <int D, bool NORM, bool PAIRS>
__global__ void __launch_bounds__(kRotThreads, kRotBackCtas) rotate_back_kernel(const __grid_constant__ RotateParams p) {
  using S = RotShape<D>;
  __shared__ RotShared<D> sh;
  __shared__ float sums[NORM ? kRotWarps : 1][2][D];
  cache_let_next();
  cache_wait_before();
  rot_setup<D>(p, &sh);
  if (blockIdx.x == 0 && p.status != nullptr) rot_check(p);
  const int lane32 = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane32 / S::kLanes;
  const RotLane<D, PAIRS> lane(p.pairs);
  Pairs acc;
  const float2 zero = make_float2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 4; ++e) acc.a[e] = acc.b[e] = zero;
  if constexpr (NORM) {
    for (int i = lane32; i < 2 * D; i += 32) sums[warp][i / D][i % D] = 0.f;
    __syncwarp();
  }
  auto flush = [&](int k) {  // (a warp comes through a job once)
    if constexpr (NORM) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float2& two = e < 8 ? acc.a[e >> 1] : acc.b[(e >> 1) - 4];
        float v = e & 1 ? two.y : two.x;
#pragma unroll
        for (int o = S::kLanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        // pair e % 8, a's or b's
        const int column = PAIRS ? (e % 8 < 4 ? lane.a + 2 * (e % 8) : lane.b + 2 * (e % 8) - 8) + (e >> 3) : (e < 8 ? lane.a : lane.b) + e % 8;
        if (group == 0) sums[warp][k][column] = v;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc.a[e] = acc.b[e] = zero;
    }
  };
  RotRow<D, PAIRS> at;
  float2 s[4], c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] = c[e] = zero;
  int k = -1;
#pragma unroll 1
  for (RotShare share(p.units); share.at < share.end; ++share.at) {
    bool enter = k < 0;
    if (enter) k = 0;
    while (k + 1 < p.jobs && share.at >= p.job[k + 1].unit0) {
      if (!enter) flush(k);
      ++k;
      enter = true;
    }
    const RotateJob& j = p.job[k];
    const uint32_t heads = j.heads, vecs = static_cast<uint32_t>(j.rows) * heads;
    const uint32_t vec = (static_cast<uint32_t>(share.at - j.unit0) * S::kGroups + group) * p.run;
    const int n = static_cast<int>(min(vecs - min(vec, vecs), static_cast<uint32_t>(p.run)));
    RotAt here{vec / heads, 0};
    here.head = vec - here.row * heads;
    if (enter) at.enter(j, __shfl_sync(0xffffffffu, here.row, 0));
#pragma unroll 1
    for (int i0 = 0; i0 < p.run; i0 += kRotBackBatch) {
      uint4 u[kRotBackBatch], v[kRotBackBatch], du[kRotBackBatch], dv[kRotBackBatch];
      RotAt load = here;
#pragma unroll
      for (int i = 0; i < kRotBackBatch; ++i) {
        u[i] = v[i] = du[i] = dv[i] = make_uint4(0, 0, 0, 0);
        if (i0 + i < n) {
          const __nv_bfloat16* dy = j.dy + load.row * j.dy_stride + load.head * D;
          du[i] = rot_load(dy + lane.a);
          dv[i] = rot_load(dy + lane.b);
          if constexpr (NORM) {
            const __nv_bfloat16* x = j.x + load.row * j.x_stride + load.head * D;
            u[i] = rot_load(x + lane.a);
            v[i] = rot_load(x + lane.b);
          }
        }
        load.next(heads);
      }
      // both of one row, in every group of the warp: side by side
      static_assert(kRotBackBatch == 2, "pairs");
      const bool both = i0 + 1 < n && here.head + 1 < heads;
      if (__all_sync(0xffffffffu, both)) {
        if (static_cast<int>(here.row) != at.row) at.to(p, j, lane, sh.turn, here.row, s, c);
        rot_back<D, NORM, PAIRS, 2>(lane, sh.weight[k], p.eps, s, c, u, v, du, dv, at.live, acc);
        if (at.live) {
          __nv_bfloat16* dst = j.y + here.row * j.y_stride + here.head * D;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<uint4*>(dst + i * D + lane.a) = du[i];
            *reinterpret_cast<uint4*>(dst + i * D + lane.b) = dv[i];
          }
        }
        here.next(heads);
        here.next(heads);
        continue;
      }
#pragma unroll
      for (int i = 0; i < kRotBackBatch; ++i) {
        if (i0 + i >= p.run) break;
        if (i0 + i < n && static_cast<int>(here.row) != at.row) at.to(p, j, lane, sh.turn, here.row, s, c);
        const bool live = i0 + i < n && at.live;
        rot_back<D, NORM, PAIRS, 1>(lane, sh.weight[k], p.eps, s, c, u + i, v + i, du + i, dv + i, live, acc);
        if (live) {
          __nv_bfloat16* dst = j.y + here.row * j.y_stride + here.head * D;
          *reinterpret_cast<uint4*>(dst + lane.a) = du[i];
          *reinterpret_cast<uint4*>(dst + lane.b) = dv[i];
        }
        here.next(heads);
      }
    }
  }
  if constexpr (NORM) {
    if (p.partial == nullptr) return;
    if (k >= 0) flush(k);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kRotThreads) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kRotWarps; ++w) t += sums[w][i / D][i % D];
      p.partial[static_cast<int64_t>(blockIdx.x) * (2 * D) + i] = t;
    }
  }
}

// Sums the CTAs' parts of the weights' gradients: a block takes 32 columns, a warp
// every 32nd part, then the warps' sums in order.
template <int D>
__global__ void __launch_bounds__(1024) rotate_weights_kernel(const __grid_constant__ RotateParams p, int parts) {
  __shared__ float sums[32][33];
  cache_let_next();
  cache_wait_before();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int column = blockIdx.x * 32 + lane;
  float t = 0.f;
#pragma unroll 4
  for (int c = warp; c < parts; c += 32) t += p.partial[static_cast<int64_t>(c) * (2 * D) + column];
  sums[warp][lane] = t;
  __syncthreads();
  if (warp != 0) return;
  t = 0.f;
#pragma unroll
  for (int w = 0; w < 32; ++w) t += sums[w][lane];
  float* dw = p.dweight[column / D];
  if (dw != nullptr) dw[column % D] = t;
}

// ------------------------------------------------------------------ launch
// The units of the call's jobs (a run of every group of a warp), and the CTAs for
// them.  The run gets shorter as long as warps would have none (64 single tokens of
// 48 vectors of 128: 96 CTAs with runs of one, 12 with runs of 8).
template <int D>
static int rotate_units(RotateParams& p, int ctas) {
  int64_t vecs = 0;
  for (int k = 0; k < p.jobs; ++k) vecs += static_cast<int64_t>(p.job[k].rows) * p.job[k].heads;
  p.run = kRotRun;
  while (p.run > 1 && vecs < static_cast<int64_t>(ctas) * kRotWarps * p.run * RotShape<D>::kGroups) p.run /= 2;
  const int64_t each = static_cast<int64_t>(p.run) * RotShape<D>::kGroups;
  p.units = 0;
  for (int k = 0; k < p.jobs; ++k) {
    p.job[k].unit0 = p.units;
    p.units += (static_cast<int64_t>(p.job[k].rows) * p.job[k].heads + each - 1) / each;
  }
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((p.units + kRotWarps - 1) / kRotWarps, ctas)));
}

template <int D>
static cudaError_t launch_rotate_d(RotateParams p, bool norm, bool pairs, int sms, cudaStream_t stream) {
  const int grid = rotate_units<D>(p, sms * kRotCtas);
  return cache_launch(norm ? (pairs ? rotate_kernel<D, true, true> : rotate_kernel<D, true, false>)
                           : (pairs ? rotate_kernel<D, false, true> : rotate_kernel<D, false, false>),
                      dim3(grid), kRotThreads, 0, stream, p);
}
cudaError_t launch_rotate(const RotateParams& p, int head_dim, bool norm, bool pairs, int sms, cudaStream_t stream) {
  return head_dim == 128  ? launch_rotate_d<128>(p, norm, pairs, sms, stream)
         : head_dim == 64 ? launch_rotate_d<64>(p, norm, pairs, sms, stream)
                          : launch_rotate_d<32>(p, norm, pairs, sms, stream);
}

template <int D>
static cudaError_t launch_rotate_back_d(RotateParams p, bool norm, bool pairs, int sms, cudaStream_t stream) {
  const int grid = rotate_units<D>(p, sms * kRotBackCtas);
  const cudaError_t e =
      cache_launch(norm ? (pairs ? rotate_back_kernel<D, true, true> : rotate_back_kernel<D, true, false>)
                        : (pairs ? rotate_back_kernel<D, false, true> : rotate_back_kernel<D, false, false>),
                   dim3(grid), kRotThreads, 0, stream, p);
  if (e != cudaSuccess || p.partial == nullptr) return e;
  return cache_launch(rotate_weights_kernel<D>, dim3(2 * D / 32), 1024, 0, stream, p, grid);
}
cudaError_t launch_rotate_back(const RotateParams& p, int head_dim, bool norm, bool pairs, int sms, cudaStream_t stream) {
  return head_dim == 128  ? launch_rotate_back_d<128>(p, norm, pairs, sms, stream)
         : head_dim == 64 ? launch_rotate_back_d<64>(p, norm, pairs, sms, stream)
                          : launch_rotate_back_d<32>(p, norm, pairs, sms, stream);
}
size_t rotate_back_partial_bytes(int head_dim, int sms) {
  return static_cast<size_t>(sms) * kRotBackCtas * 2 * head_dim * sizeof(float);
}

}  // namespace jg
