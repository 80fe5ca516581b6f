// Writes rows of keys and values into a cache held in 4 bits, and reads them back.
//
// Of a token's head, with lo and hi its least and largest value:
//
//   s = bf16((hi - lo) / 15),  z = bf16(lo + 8 s),
//   c = clamp(rint((x - z) / s), -8, 7) + 8       (s = 0: 8)
//
// in fp32, each operation rounded once (halves to even), so that the codes are
// the same wherever they are formed.  A few operations per value: bound by HBM (2.5
// bytes a value each way and 4 a head).  D / 16 lanes take a head, 16 columns each.
// The quotient is q = d y, y = 1 / s rounded, corrected by its remainder, q + (d -
// q s) y (after P. Markstein, Computation of elementary functions on the IBM RISC
// System/6000 processor, 1990): the remainder is exact, as s has 8 bits, so that a quotient that is a half is met
// exactly, which values of 8 bits often are; any other differs from a half by
// more than the correction leaves (d - (k + 1/2) s is a multiple of d's last place, which
// is more than s 2^-24 of the quotient's power of two), so that the code is that of the divided
// quotient.  (With 16 divisions per lane the write of 32,768 rows x 8 x 128 took 84 us.)
//
// 32,768 rows of 8 x 128, written and read back: 64.6 us, 0.78 of the copy bandwidth.  The
// write is bound by its instructions (issue slots 66% in use); the read by HBM.
#include <algorithm>
#include <type_traits>

#include "cache4.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace jg {

constexpr int kRows4Threads = 256;
constexpr int kRows4Steps = 4;  // heads after one another

__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint4 ld_rows4(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// A place among the heads of the rows, and where it lies in the cache.
struct Rows4At {
  uint32_t row, head;
  int slot = -1;         // of the row, or -1
  int64_t page = 0;
  int place = 0;         // of the row in its page
  __device__ __forceinline__ Rows4At(const Cache4RowsParams& p, uint32_t vec) {
    row = vec / static_cast<uint32_t>(p.heads);
    head = vec - row * p.heads;
    find(p);
  }
  __device__ __forceinline__ void find(const Cache4RowsParams& p) {
    slot = row < static_cast<uint32_t>(p.rows) ? p.slots[row] : -1;
    if (static_cast<uint32_t>(slot) >= static_cast<uint32_t>(p.slot_end)) slot = -1;
    page = slot >> p.page_shift;
    place = slot & ((1 << p.page_shift) - 1);
  }
  __device__ __forceinline__ void next(const Cache4RowsParams& p) {
    if (++head == static_cast<uint32_t>(p.heads)) {
      head = 0;
      ++row;
      find(p);
    }
  }
  __device__ __forceinline__ int64_t in_page(const Cache4RowsParams& p) const { return (static_cast<int64_t>(head) << p.page_shift) + place; }
};

// blockIdx.y: K or V.
template <int D>
__global__ void __launch_bounds__(kRows4Threads) cache4_append_kernel(const __grid_constant__ Cache4RowsParams p, int steps) {
  constexpr int L = D / 16, G = 32 / L;
  cache_let_next();
  cache_wait_before();
  const int half = blockIdx.y, l = threadIdx.x % L;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kRows4Threads / 32) + (threadIdx.x >> 5);
  Rows4At at(p, (static_cast<uint32_t>(warp) * G + (threadIdx.x & 31) / L) * steps);
  uint4 v[kRows4Steps][2];
  {
    uint32_t row = at.row, head = at.head;
#pragma unroll
    for (int i = 0; i < kRows4Steps; ++i) {
      v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
      if (i >= steps) continue;
      if (row < static_cast<uint32_t>(p.rows)) {
        const __nv_bfloat16* src = p.in[half] + row * p.stride[half] + head * D + 16 * l;
        v[i][0] = ld_rows4(src);
        v[i][1] = ld_rows4(src + 8);
      }
      if (++head == static_cast<uint32_t>(p.heads)) {
        head = 0;
        ++row;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows4Steps; ++i) {
    if (i >= steps) break;
    const uint32_t w[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
    uint32_t least = w[0], most = w[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      least = min_nan2(least, w[e]);
      most = max_nan2(most, w[e]);
    }
    // the least value and the largest's negative side by side
    most ^= 0x80008000u;
    uint32_t both = min_nan2(__byte_perm(least, most, 0x5410), __byte_perm(least, most, 0x7632));
#pragma unroll
    for (int o = L / 2; o; o >>= 1) both = min_nan2(both, __shfl_xor_sync(0xffffffffu, both, o));
    const float lo = __uint_as_float(both << 16), hi = -__uint_as_float(both & 0xFFFF0000u);
    const __nv_bfloat16 step = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
    const float s = __bfloat162float(step);
    const __nv_bfloat16 middle = __float2bfloat16_rn(__fadd_rn(lo, 8.f * s));
    const float z = __bfloat162float(middle);
    // rounded by the addition of 1.5 2^23, with c + 8 in the last bits of the sum
    constexpr float kRound = 12582912.f + 8.f;
    constexpr uint32_t kBits = 0x4B400000u, kRest = kBits * 0x111u;  // 16^3 kBits and on leave 32 bits
    const float inv = __frcp_rn(s);
    const bool usual = s >= 0x1p-100f && s <= 0x1p100f;  // (1 / s and the remainders are normal numbers)
    uint32_t code[2] = {0, 0};
    auto form = [&](auto clamp) {
#pragma unroll
      for (int e = 7; e >= 0; --e) {
        const float2 x = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
        const float2 d = __fadd2_rn(x, make_float2(-z, -z)), y = make_float2(inv, inv);
        float2 q = __fmul2_rn(d, y);
        q = __ffma2_rn(__ffma2_rn(q, make_float2(-s, -s), d), y, q);
        if (decltype(clamp)::value) q = make_float2(fminf(fmaxf(q.x, -8.f), 7.f), fminf(fmaxf(q.y, -8.f), 7.f));
        const float2 t = __fadd2_rn(q, make_float2(kRound, kRound));
        uint32_t& c = code[e >> 2];
        c = (c * 16 + __float_as_uint(t.y)) * 16 + __float_as_uint(t.x);
      }
      code[0] -= kRest;
      code[1] -= kRest;
    };
    // (the roundings of s and z take q beyond -8 - 1/2 or 7 + 1/2 only if the middle is far from zero)
    if (__all_sync(0xffffffffu, usual && fabsf(z) < 64.f * s)) form(std::false_type{});
    else form(std::true_type{});
    if (!usual) {
      code[0] = code[1] = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float x = __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
        const float q = s > 0.f ? __fdiv_rn(__fsub_rn(x, z), s) : 0.f;
        code[e >> 3] |= static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(q), -8.f), 7.f)) + 8) << (4 * (e & 7));
      }
    }
    if (at.slot >= 0) {
      const Cache4& c = p.cache[half];
      const int64_t place = at.in_page(p);
      *reinterpret_cast<uint2*>(c.codes + at.page * c.code_stride + place * (D / 2) + 8 * l) = make_uint2(code[0], code[1]);
      if (l == 0) {
        __nv_bfloat162 pair;
        pair.x = step;
        pair.y = middle;
        *reinterpret_cast<__nv_bfloat162*>(c.scales + at.page * c.scale_stride + place * 2) = pair;
      }
    }
    at.next(p);
  }
}

template <int D>
__global__ void __launch_bounds__(kRows4Threads) cache4_read_kernel(const __grid_constant__ Cache4RowsParams p, int steps) {
  constexpr int L = D / 16, G = 32 / L;
  cache_let_next();
  cache_wait_before();
  const int half = blockIdx.y, l = threadIdx.x % L;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kRows4Threads / 32) + (threadIdx.x >> 5);
  Rows4At at(p, (static_cast<uint32_t>(warp) * G + (threadIdx.x & 31) / L) * steps);
  const Cache4& c = p.cache[half];
  uint32_t row = at.row, head = at.head;
  uint2 code[kRows4Steps];
  uint32_t scale[kRows4Steps];
#pragma unroll
  for (int i = 0; i < kRows4Steps; ++i) {
    code[i] = make_uint2(0, 0);
    scale[i] = 0;
    if (i >= steps) continue;
    if (at.slot >= 0) {
      const int64_t place = at.in_page(p);
      code[i] = *reinterpret_cast<const uint2*>(c.codes + at.page * c.code_stride + place * (D / 2) + 8 * l);
      scale[i] = *reinterpret_cast<const uint32_t*>(c.scales + at.page * c.scale_stride + place * 2);
    }
    at.next(p);
  }
#pragma unroll
  for (int i = 0; i < kRows4Steps; ++i) {
    if (i >= steps || row >= static_cast<uint32_t>(p.rows)) break;
    const float s = __uint_as_float(scale[i] << 16), z = __uint_as_float(scale[i] & 0xFFFF0000u);
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t two = (e < 4 ? code[i].x : code[i].y) >> (8 * (e & 3));
      const float a = static_cast<float>(static_cast<int>(two & 15) - 8), b = static_cast<float>(static_cast<int>((two >> 4) & 15) - 8);
      // (the product has 12 bits: the sum is rounded to fp32, then to bf16)
      w[e] = pack_bf16(__fmaf_rn(s, a, z), __fmaf_rn(s, b, z));
    }
    __nv_bfloat16* dst = p.out[half] + row * p.stride[half] + head * D + 16 * l;
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    if (++head == static_cast<uint32_t>(p.heads)) {
      head = 0;
      ++row;
    }
  }
}

template <int D>
static cudaError_t launch_rows4(const Cache4RowsParams& p, bool append, int sms, cudaStream_t stream) {
  constexpr int G = 512 / D;  // heads side by side in a warp
  const int64_t vecs = static_cast<int64_t>(p.rows) * p.heads;
  const int steps = vecs >= static_cast<int64_t>(sms) * 8 * G * kRows4Steps ? kRows4Steps : 1;  // (K and V: two CTAs per SM)
  const int64_t per_cta = static_cast<int64_t>(kRows4Threads / 32) * G * steps;
  return cache_launch(append ? cache4_append_kernel<D> : cache4_read_kernel<D>,
                      dim3(static_cast<unsigned>((vecs + per_cta - 1) / per_cta), 2, 1), kRows4Threads, 0, stream, p, steps);
}
cudaError_t launch_cache4_rows(const Cache4RowsParams& p, int head_dim, bool append, int sms, cudaStream_t stream) {
  return head_dim == 128  ? launch_rows4<128>(p, append, sms, stream)
         : head_dim == 64 ? launch_rows4<64>(p, append, sms, stream)
                          : launch_rows4<32>(p, append, sms, stream);
}

}  // namespace jg
