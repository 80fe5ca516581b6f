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
// exchange between lanes is that of the norm's sum.  A warp's unit is some
// vectors side by side, in (row, head) order whatever the number of heads, up to
// four (backward two) after one another, which it loads before it uses the first.
#include <algorithm>

#include "cache.cuh"
#include "common.cuh"
#include "ptx.cuh"
#include "rotate.cuh"

namespace jg {

constexpr int kRotThreads = 256;
constexpr int kRotWarps = kRotThreads / 32;
constexpr int kRotSteps = 4, kRotBackSteps = 2;  // vectors after one another, at most
constexpr int kRotCtas = 3, kRotBackCtas = 2;    // per SM

template <int D>
struct RotShape {
  static constexpr int kLanes = D / 16;        // of a vector
  static constexpr int kGroups = 32 / kLanes;  // vectors side by side in a warp
};

// An angle is kept as a fraction of a turn in 64-bit fixed point: the product of
// a position and a frequency's fraction, modulo 2^64, drops whole turns exactly,
// so that a far position is as exact as a near one (f / 2 pi is right to 2^-53,
// which at position 2^31 is 2^-24 of a turn for f = 1).
__device__ __forceinline__ uint64_t turn_of(float f) {
  const double turns = static_cast<double>(f) * 0.15915494309189533577;  // 1 / (2 pi)
  return static_cast<uint64_t>(__double2ll_rn((turns - rint(turns)) * 18446744073709551616.0));
}
__device__ __forceinline__ void sincos_turn(uint64_t turn, float& s, float& c) {
  // [-pi, pi), where the hardware's sine and cosine are within 2^-20.9
  const float a = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 1.46291807926715968e-9f;  // pi 2^-31
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
  bool turns;      // some of the lane's columns rotate
  __device__ __forceinline__ RotLane(int n) {
    const int l = threadIdx.x % RotShape<D>::kLanes;
    if constexpr (PAIRS) {
      a = 16 * l;
      b = a + 8;
      first = 8 * l;
      turns = first < n;
    } else {
      const int m = n >> 3;
      turns = l < m;
      a = turns ? 8 * l : 16 * l;
      b = turns ? 8 * l + n : 16 * l + 8;
      first = 8 * l;
    }
  }
};

__device__ __forceinline__ void rot_unpack(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 rot_pack(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
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

__device__ __forceinline__ void rot_weight(const float* w, int a, int b, float (&out)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4*>(out + 4 * i) = *reinterpret_cast<const float4*>(w + (i < 2 ? a + 4 * i : b + 4 * i - 8));
}

// Rotates a lane's 16 columns (8 of each piece) by its 8 angles; BACK: the other way.
template <bool PAIRS, bool BACK>
__device__ __forceinline__ void rot_turn(float (&f)[16], const float (&s)[8], const float (&c)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& x = f[PAIRS ? 2 * i : i];
    float& y = f[PAIRS ? 2 * i + 1 : i + 8];
    const float sn = BACK ? -s[i] : s[i];
    const float u = x * c[i] - y * sn;
    y = y * c[i] + x * sn;
    x = u;
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
  float s[8], c[8];

  // At a job's first row of the warp's.
  __device__ __forceinline__ void enter(const RotateJob& j, int first_row) {
    row = -1;
    if (j.positions != nullptr || j.batch == 0) return;
    b = segment_of(j.offsets, j.batch, first_row);
    start = j.offsets[b];
    end = j.offsets[b + 1];
  }
  // Moves on to a row that is not before the last one (an own one for every group of lanes).
  __device__ __forceinline__ void to(const RotateParams& p, const RotateJob& j, const RotLane<D, PAIRS>& l,
                                     const uint64_t* turn, int r, bool want_angles) {
    if (r == row) return;
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
    if (!want_angles) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = l.first + i;
      s[i] = 0.f;
      c[i] = 1.f;
      if (l.turns && at < p.pairs) sincos_turn(turn[at] * static_cast<uint64_t>(pos), s[i], c[i]);
    }
  }
};

// The call's frequencies and weights, in shared memory.
template <int D>
struct RotShared {
  uint64_t turn[D / 2];
  alignas(16) float weight[2][D];
};
template <int D>
__device__ __forceinline__ void rot_setup(const RotateParams& p, RotShared<D>* sh) {
  const int tid = threadIdx.x;
  if (tid < p.pairs) sh->turn[tid] = turn_of(p.inv_freq[tid]);
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
    if (j.positions != nullptr || (k > 0 && j.offsets == p.job[k - 1].offsets)) continue;
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

// Vector of a job -> row and head.
struct RotVec {
  uint32_t row, head;
  bool here;
  __device__ __forceinline__ RotVec(const RotateJob& j, uint32_t vec) {
    const uint32_t heads = j.heads;
    here = vec < static_cast<uint32_t>(j.rows) * heads;
    row = vec / heads;
    head = vec - row * heads;
  }
};

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
    const uint32_t vec0 = static_cast<uint32_t>(share.at - j.unit0) * (p.steps * S::kGroups) + group;
    uint4 v[kRotSteps][2];
#pragma unroll
    for (int i = 0; i < kRotSteps; ++i) {
      const RotVec vec(j, vec0 + i * S::kGroups);
      v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
      if (i < p.steps && vec.here) {
        const __nv_bfloat16* src = j.x + vec.row * j.x_stride + vec.head * D;
        v[i][0] = rot_load(src + lane.a);
        v[i][1] = rot_load(src + lane.b);
      }
    }
    if (enter) at.enter(j, __shfl_sync(0xffffffffu, RotVec(j, vec0).row, 0));
#pragma unroll
    for (int i = 0; i < kRotSteps; ++i) {
      if (i >= p.steps) break;
      const RotVec vec(j, vec0 + i * S::kGroups);
      if (vec.here) at.to(p, j, lane, sh.turn, vec.row, !j.copy);
      if (!j.copy) {
        float f[16];
        rot_unpack(v[i][0], f);
        rot_unpack(v[i][1], f + 8);
        if constexpr (NORM) {
          float sq = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) sq = __fmaf_rn(f[e], f[e], sq);
          const float r = rsqrtf(rot_sum<S::kLanes>(sq) * (1.f / D) + p.eps);
          float w[16];
          rot_weight(sh.weight[k], lane.a, lane.b, w);
#pragma unroll
          for (int e = 0; e < 16; ++e) f[e] = f[e] * r * w[e];
        }
        rot_turn<PAIRS, false>(f, at.s, at.c);
        v[i][0] = rot_pack(f);
        v[i][1] = rot_pack(f + 8);
      }
      if (!vec.here || !at.live) continue;
      __nv_bfloat16* dst = j.y + vec.row * j.y_stride;
      if (j.slots != nullptr) {
        const int slot = j.slots[vec.row];
        if (static_cast<uint32_t>(slot) >= static_cast<uint32_t>(p.slot_end)) continue;
        dst = j.y + (slot >> p.page_shift) * j.page_stride + static_cast<int64_t>(slot & ((1 << p.page_shift) - 1)) * (j.heads * D);
      }
      dst += vec.head * D;
      *reinterpret_cast<uint4*>(dst + lane.a) = v[i][0];
      *reinterpret_cast<uint4*>(dst + lane.b) = v[i][1];
    }
  }
}

// Backward.  The weights' gradients are sums over every row and head: a lane
// keeps its 16 columns' in registers over its warp's units of a job, the warps of
// a CTA meet in shared memory, the CTAs in `partial`, each in a fixed order (the
// same bits on every run).
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
  float acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  if constexpr (NORM) {
    for (int i = lane32; i < 2 * D; i += 32) sums[warp][i / D][i % D] = 0.f;
    __syncwarp();
  }
  auto flush = [&](int k) {  // (a warp comes through a job once)
    if constexpr (NORM) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
#pragma unroll
        for (int o = S::kLanes; o < 32; o <<= 1) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
        if (group == 0) sums[warp][k][(e < 8 ? lane.a : lane.b - 8) + e] = acc[e];
        acc[e] = 0.f;
      }
    }
  };
  RotRow<D, PAIRS> at;
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
    const uint32_t vec0 = static_cast<uint32_t>(share.at - j.unit0) * (p.steps * S::kGroups) + group;
    uint4 v[kRotBackSteps][2], d[kRotBackSteps][2];
#pragma unroll
    for (int i = 0; i < kRotBackSteps; ++i) {
      const RotVec vec(j, vec0 + i * S::kGroups);
      v[i][0] = v[i][1] = d[i][0] = d[i][1] = make_uint4(0, 0, 0, 0);
      if (i < p.steps && vec.here) {
        const __nv_bfloat16* dy = j.dy + vec.row * j.dy_stride + vec.head * D;
        d[i][0] = rot_load(dy + lane.a);
        d[i][1] = rot_load(dy + lane.b);
        if constexpr (NORM) {
          const __nv_bfloat16* x = j.x + vec.row * j.x_stride + vec.head * D;
          v[i][0] = rot_load(x + lane.a);
          v[i][1] = rot_load(x + lane.b);
        }
      }
    }
    if (enter) at.enter(j, __shfl_sync(0xffffffffu, RotVec(j, vec0).row, 0));
#pragma unroll
    for (int i = 0; i < kRotBackSteps; ++i) {
      if (i >= p.steps) break;
      const RotVec vec(j, vec0 + i * S::kGroups);
      if (vec.here) at.to(p, j, lane, sh.turn, vec.row, true);
      const bool live = vec.here && at.live;
      float g[16];
      rot_unpack(d[i][0], g);
      rot_unpack(d[i][1], g + 8);
      rot_turn<PAIRS, true>(g, at.s, at.c);
      if constexpr (NORM) {
        float h[16], w[16];
        rot_unpack(v[i][0], h);
        rot_unpack(v[i][1], h + 8);
        float sq = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) sq = __fmaf_rn(h[e], h[e], sq);
        const float r = rsqrtf(rot_sum<S::kLanes>(sq) * (1.f / D) + p.eps);
        rot_weight(sh.weight[k], lane.a, lane.b, w);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          h[e] *= r;
          if (live) acc[e] = __fmaf_rn(g[e], h[e], acc[e]);
          g[e] *= w[e];
          dot = __fmaf_rn(g[e], h[e], dot);
        }
        dot = rot_sum<S::kLanes>(dot) * (1.f / D);
#pragma unroll
        for (int e = 0; e < 16; ++e) g[e] = r * __fmaf_rn(-h[e], dot, g[e]);
      }
      if (!live) continue;
      __nv_bfloat16* dst = j.y + vec.row * j.y_stride + vec.head * D;
      *reinterpret_cast<uint4*>(dst + lane.a) = rot_pack(g);
      *reinterpret_cast<uint4*>(dst + lane.b) = rot_pack(g + 8);
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
// The units of the call's jobs, and the CTAs for them.  Calls that would leave
// SMs idle with full units take one vector at a time (64 single tokens of 48
// vectors of 128: 96 CTAs instead of 24).
template <int D>
static int rotate_units(RotateParams& p, int most, int ctas) {
  p.steps = most;
  int64_t vecs = 0;
  for (int k = 0; k < p.jobs; ++k) vecs += static_cast<int64_t>(p.job[k].rows) * p.job[k].heads;
  if (vecs < static_cast<int64_t>(ctas) * kRotWarps * most * RotShape<D>::kGroups) p.steps = 1;
  const int64_t each = p.steps * RotShape<D>::kGroups;
  p.units = 0;
  for (int k = 0; k < p.jobs; ++k) {
    p.job[k].unit0 = p.units;
    p.units += (static_cast<int64_t>(p.job[k].rows) * p.job[k].heads + each - 1) / each;
  }
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((p.units + kRotWarps - 1) / kRotWarps, ctas)));
}

template <int D>
static cudaError_t launch_rotate_d(RotateParams p, bool norm, bool pairs, int sms, cudaStream_t stream) {
  const int grid = rotate_units<D>(p, kRotSteps, sms * kRotCtas);
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
  const int grid = rotate_units<D>(p, kRotBackSteps, sms * kRotBackCtas);
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
