// Attention over a paged cache held in 4 bits (cache4.cuh), few query rows per
// key/value head.
//
// An item is (request, key/value head, tile of 16 query rows), a row (new token,
// query head of the group); items are divided among the CTAs and their parts
// joined as in the bf16 kernel (cache.cuh, cache_fwd.cu).  With a key's step s,
// middle z and codes c,
//
//   x = scale (s <q, c - 8> + z sum q),   O = sum_j (P_j s_j) (c_j - 8) + sum_j P_j z_j
//
// so that the products take the codes themselves, small whole numbers that bf16
// holds exactly, and steps and middles enter in fp32: no value of the cache is
// rounded again, and what a masked place holds (its codes are always finite)
// never meets a row that does not see it.
//
// Bytes per key and head are D + 8 instead of the bf16 cache's 4 D, and what a
// byte costs in instructions counts: 5 per 2 codes (a shift, a mask, a
// subtraction, their share of the products).  Every warp works by itself, on blocks of 32 keys
// that it copies (cp.async) into a ring of its own, a few blocks ahead: no
// barrier but an item's end.  The order of columns within a product and of keys within
// a block is free, so both are chosen such that a lane's codes come in one load
// per key and turn into operands by shifts and masks:
//   K: key n of a product of 8 is key (n / 2) + 4 (n % 2), and lane t of a key's
//      four takes columns D / 4 t and on; nibbles i and i + 4 of a word side by side
//   V: lane g of a key's eight takes columns D / 8 g and on; two keys' words are
//      put together by halves, nibble i of both side by side.
#include "act.cuh"
#include "cache4.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace jg {

constexpr int kC4Keys = 64;    // tokens per tile of the work division
constexpr int kC4Block = 32;   // keys of a warp's step
constexpr int kC4Warps = 4;
constexpr int kC4Rows = kCache4Rows;
constexpr int kC4MinRange = 5;  // the least length of a range

template <int D>
struct C4Cfg {
  static constexpr int kRow = D / 2;  // bytes of a key's codes
  static constexpr int kCodes = kC4Block * kRow;
  static constexpr int kStage = 2 * kCodes + 2 * kC4Block * 4;  // codes of K and V, scales of K and V
  static constexpr int kStages = D == 128 ? 4 : D == 64 ? 5 : 6;
  static constexpr int kRing = kStage * kStages > kC4Rows * D * 4 ? kStage * kStages : kC4Rows * D * 4;  // (O meets there)
  static constexpr int kSmem = kC4Warps * kRing;
  static_assert(kSmem <= 233472 / cache4_ctas(D) - 2048, "shared memory per CTA");
};

template <int D>
struct C4Shared {
  CacheRangeShared range;
  float2 ml[kC4Warps][kC4Rows];
};

__device__ __forceinline__ void c4_copy(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;  // (0: zeros, nothing is read)
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void c4_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void c4_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void c4_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Nibble 0 of both halves of w as a bf16 pair, less 8: 128 + c is the bits of
// 128 with c in its last four.
__device__ __forceinline__ uint32_t c4_pair(uint32_t w) {
  const uint32_t v = (w & 0x000F000Fu) | 0x43004300u;
  uint32_t y;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(v), "r"(0x43084308u));
  return y;
}
template <int N>
__device__ __forceinline__ void c4_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 4) ld_shared_v4(addr, w[0], w[1], w[2], w[3]);
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
  else asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
}
__device__ __forceinline__ float2 c4_scale(uint32_t addr) {  // step, middle
  uint32_t w;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(addr) : "memory");
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// Where four columns of O's row lie in a warp's part of shared memory (no bank
// conflicts, neither as the fragments are written nor as the rows are read).
template <int D>
__device__ __forceinline__ int c4_place(int row, int q4) {
  const int x = D == 128 ? (q4 >> 3) | ((row & 1) << 2) : D == 64 ? ((q4 >> 3) & 1) | ((row & 1) << 1) : row & 1;
  return row * (D / 4) + (q4 ^ x);
}

template <int D, int ACT>
__global__ void __launch_bounds__(kC4Warps * 32, cache4_ctas(D)) cache4_fwd_kernel(const __grid_constant__ Cache4FwdParams pp) {
  using C = C4Cfg<D>;
  constexpr int WK = D / 32;      // words of K's codes of a lane and key
  constexpr int KS = D / 16;      // k steps of S
  constexpr int NT = D / 8;       // n tiles of O
  constexpr int kTiles = kC4Block / 8;
  const CacheFwdParams& p = pp.f;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ C4Shared<D> sh;
  cache_let_next();
  cache_wait_before();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tig = lane & 3;
  int* status = p.err + blockIdx.x;
  if (tid == 0) *status = kOk;
  const CacheRange R = cache_range<kC4Keys>(p, &sh.range, kC4MinRange);
  if (tid == 0) cache_open<kC4Keys>(p, R);
  const uint32_t ring = smem_u32(smem) + warp * C::kRing;
  const int reach = (p.bias_len - 1) / 2;
  // scores in log2 units, or halved as cc_act2 takes them
  constexpr float kUnit = ACT == 2 ? kLog2e : 0.5f;
  const float scale = ACT == 2 ? p.scale : 0.5f * p.scale;

  CacheWalk w;
  w.init(R);
#pragma unroll 1
  for (; w.template next<kC4Keys>(p); w.advance()) {
    const CacheReq& r = w.r;
    int lo, hi;
    w.template tiles<kC4Keys>(p, lo, hi);
    const int32_t* table = p.table + static_cast<int64_t>(w.b) * p.width;
    const int blocks_end = min(hi * (kC4Keys / kC4Block), static_cast<int>((static_cast<uint32_t>(r.L) + kC4Block - 1) / kC4Block));
    int kb = lo * (kC4Keys / kC4Block) + warp;
    // lane i: the page of key 16 (i % 2) of a block, or -1
    auto page_of = [&](int block) {
      int id = -1;
      const int key = block * kC4Block + 16 * (lane & 1);
      if (block < blocks_end && key < r.L) {
        id = table[key >> p.page_shift];
        if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(p.num_pages)) {
          atomicCAS(status, kOk, kErrBadPage);
          id = -1;
        }
      }
      return id;
    };
    auto copy = [&](int block, int id, int stage) {  // (the whole warp)
      const int id0 = __shfl_sync(0xffffffffu, id, 0), id1 = __shfl_sync(0xffffffffu, id, 1);
      if (block < blocks_end) {
        const int mask = (1 << p.page_shift) - 1, first = block * kC4Block;
        const uint32_t to = ring + stage * C::kStage;
        auto where = [&](int key, int& page) {  // place in the head's part of a page
          page = key < 16 ? id0 : id1;
          return (static_cast<int64_t>(w.h) << p.page_shift) + ((first + key) & mask);
        };
        constexpr int kPieces = C::kRow / 16;  // of a key
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int key = (i * 32 + lane) / kPieces, c = lane % kPieces;
          int page;
          const int64_t at = where(key, page) * C::kRow + 16 * c;
          const bool live = page >= 0;
          const int64_t pg = live ? page : 0;
          // K's keys in the order of their products, V's pieces turned by key
          const int n = (key & ~7) | ((key & 3) << 1) | ((key >> 2) & 1);
          c4_copy(to + n * C::kRow + 16 * c, pp.k.codes + pg * pp.k.code_stride + at, live);
          const int cv = D == 128 ? c ^ (key & 2) : c;
          c4_copy(to + C::kCodes + key * C::kRow + 16 * cv, pp.v.codes + pg * pp.v.code_stride + at, live);
        }
        if (lane < 16) {  // four keys' scales each
          const int key = (lane & 7) * 4;
          const Cache4& c = lane < 8 ? pp.k : pp.v;
          int page;
          const int64_t at = where(key, page) * 2;
          const bool live = page >= 0;
          c4_copy(to + 2 * C::kCodes + lane * 16, c.scales + (live ? page : 0) * c.scale_stride + at, live);
        }
      }
      c4_commit();
    };
    // the first blocks are on their way before anything else of the item
    int ids = page_of(kb);
#pragma unroll
    for (int i = 0; i < C::kStages; ++i) {
      const int next_ids = page_of(kb + (i + 1) * kC4Warps);
      copy(kb + i * kC4Warps, ids, i);
      ids = next_ids;
    }

    const int n_rows = min(kC4Rows, r.T * p.group - w.row_tile * kC4Rows);
    CcRow rows[2];  // g and g + 8
    const __nv_bfloat16* qrow[2];
    float far_bias[2];
    int pos_min = INT32_MAX;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int lr = g + 8 * i, flat = w.row_tile * kC4Rows + lr;
      CcRow& q = rows[i];
      const int t = static_cast<uint32_t>(flat) / static_cast<uint32_t>(p.group);
      q.t = lr < n_rows ? t : -1;
      q.head = w.h * p.group + (lr < n_rows ? flat - t * p.group : 0);
      q.pos = r.C;
      q.far_bias = 0.f;
      qrow[i] = nullptr;
      if (q.t >= 0) {
        q.pos = cc_row_pos(p, r, q.t, status);
        qrow[i] = p.q + static_cast<int64_t>(r.q0 + q.t) * p.q_stride + static_cast<int64_t>(q.head) * D;
        pos_min = min(pos_min, q.pos);
      }
      far_bias[i] = 0.f;
      if (q.t >= 0 && p.bias_len)
        far_bias[i] = __ldg(p.bias + static_cast<int64_t>(q.head) * p.bias_len + 2 * reach) * kUnit;
    }
    // some row's bias hides all far keys, or is beyond what log2 units hold
    const bool hides = ACT == 2 && __any_sync(0xffffffffu, fabsf(far_bias[0]) > kHugeScore || fabsf(far_bias[1]) > kHugeScore);
    pos_min = __reduce_min_sync(0xffffffffu, pos_min);
    const int pos_max = __reduce_max_sync(0xffffffffu, max(rows[0].t >= 0 ? rows[0].pos : 0, rows[1].t >= 0 ? rows[1].pos : 0));
    // Q's fragments in the order of K's nibbles, and its sums
    uint32_t qa[KS][4];
    float q_sum[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < WK; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (qrow[i] != nullptr) v = *reinterpret_cast<const uint4*>(qrow[i] + (D / 4) * tig + 8 * j);
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};  // columns 2 e, 2 e + 1
#pragma unroll
        for (int e = 0; e < 4; ++e) q_sum[i] += __uint_as_float(x[e] << 16) + __uint_as_float(x[e] & 0xFFFF0000u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // columns 2 h and 2 h + 4, 2 h + 1 and 2 h + 5
          qa[2 * j + h][i] = __byte_perm(x[h], x[h + 2], 0x5410);
          qa[2 * j + h][2 + i] = __byte_perm(x[h], x[h + 2], 0x7632);
        }
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      q_sum[i] += __shfl_xor_sync(0xffffffffu, q_sum[i], 1);
      q_sum[i] += __shfl_xor_sync(0xffffffffu, q_sum[i], 2);
    }
    float o[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, pz[2] = {0.f, 0.f};  // pz: sum P z

    int stage = 0;
#pragma unroll 1
    for (; kb < blocks_end; kb += kC4Warps) {
      c4_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t kt = ring + stage * C::kStage, vt = kt + C::kCodes, ks = vt + C::kCodes, vs = ks + kC4Block * 4;
      const int key0 = kb * kC4Block;
      const bool far = p.bias_len == 0 || (!hides && key0 + kC4Block - 1 < r.C && pos_min - (key0 + kC4Block - 1) >= reach);
      bool plain = key0 + kC4Block - 1 < r.C && (p.window <= 0 || pos_max - key0 < p.window);
      // lane's columns: keys key0 + col(tile, e)
      auto col = [&](int nt, int e) { return 8 * nt + tig + 4 * e; };
      uint32_t see[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
      if (!plain) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t bits = cc_vis32(p, r, rows[h], key0);
          if (p.window > 0) {
            uint32_t near = 0;
            if (cc_in_order(p, r, key0)) {
              near = cc_near32(p, rows[h].pos, key0);
            } else {
#pragma unroll 1
              for (int c = 0; c < 2 * kTiles; ++c) {
                const int at = col(c >> 1, c & 1);
                near |= (cc_near(p, rows[h].pos, cc_pos(p, r, key0 + at)) ? 1u : 0u) << at;
              }
            }
            bits &= near;  // (only this lane's columns are kept)
          }
          see[h] = bits;
        }
      }
      float s[kTiles][4];
#pragma unroll
      for (int nt = 0; nt < kTiles; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
        uint32_t word[WK];
        c4_words<WK>(kt + (8 * nt + g) * C::kRow + tig * (4 * WK), word);
#pragma unroll
        for (int j = 0; j < WK; ++j) {
          c4_mma(s[nt], qa[2 * j], c4_pair(word[j]), c4_pair(word[j] >> 4));
          c4_mma(s[nt], qa[2 * j + 1], c4_pair(word[j] >> 8), c4_pair(word[j] >> 12));
        }
      }
#pragma unroll
      for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float2 k = c4_scale(ks + 4 * col(nt, c));
          const float step = k.x * scale, middle = k.y * scale;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            s[nt][2 * h + c] = __fmaf_rn(s[nt][2 * h + c], step, __fmaf_rn(middle, q_sum[h], far ? far_bias[h] : 0.f));
        }
      if (!far) {
        float top = 0.f;
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int key_pos = cc_pos(p, r, key0 + col(nt, c));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float bias = cc_bias(p, rows[h], reach, key_pos);
              s[nt][2 * h + c] = __fmaf_rn(bias, kUnit, s[nt][2 * h + c]);
              if constexpr (ACT == 2) top = fmaxf(top, fabsf(bias));
            }
          }
        if (ACT == 2 && __any_sync(0xffffffffu, top > kHugeBias)) {
          plain = false;
#pragma unroll
          for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int h = e >> 1, at = col(nt, e & 1);
              const float bias = cc_bias(p, rows[h], reach, cc_pos(p, r, key0 + at));
              if (bias == -INFINITY) see[h] &= ~(1u << at);
              else if (fabsf(bias) > kHugeBias && s[nt][e] == s[nt][e]) s[nt][e] = cc_huge(bias);
            }
        }
      }
      if (!plain) {
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((see[e >> 1] >> col(nt, e & 1)) & 1)) s[nt][e] = ACT == 2 ? -INFINITY : 0.f;  // act(0) = 0
      }
      if constexpr (ACT == 2) {
        // m: within 8 (log2 units) of the maximum or above, as in the bf16 kernel
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) mx[i] = fmaxf(mx[i], fmaxf(s[nt][2 * i], s[nt][2 * i + 1]));
        if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            const float mn = fmaxf(m[i], fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2)));
            const float f = mn == -INFINITY ? 1.f : ex2_sfu(m[i] - mn);
            m[i] = mn;
            l[i] *= f;
            pz[i] *= f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              o[nt][2 * i] *= f;
              o[nt][2 * i + 1] *= f;
            }
          }
        }
        const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[nt][e] = ex2_sfu(s[nt][e] - ref[e >> 1]);
            l[e >> 1] += s[nt][e];
          }
      } else {
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 y = cc_act2<ACT>(make_float2(s[nt][e], s[nt][e + 1]));
            s[nt][e] = y.x;
            s[nt][e + 1] = y.y;
          }
      }
#pragma unroll
      for (int kk = 0; kk < kTiles / 2; ++kk) {  // 16 keys
        // P s rounds to bf16 as the A operand (half a step, 2^-8 of each at most)
        uint32_t pa[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int nt = 2 * kk + i;
          float2 v[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) v[c] = c4_scale(vs + 4 * col(nt, c));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float y[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float weight = s[nt][2 * h + c];
              // (a place that the row does not see may hold any step and middle)
              const bool sees = plain || ((see[h] >> col(nt, c)) & 1);
              y[c] = sees ? weight * v[c].x : 0.f;
              if (sees) pz[h] = __fmaf_rn(weight, v[c].y, pz[h]);
            }
            pa[2 * i + h] = pack_bf16(y[0], y[1]);
          }
        }
        // V's codes of four keys: columns NT g and on of keys tig, tig + 4, + 8, + 12
        constexpr int WV = NT >= 8 ? NT / 8 : 1;
        uint32_t word[4][WV];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = 16 * kk + tig + 4 * i;
          const uint32_t at = vt + key * C::kRow;
          if constexpr (D == 128) c4_words<2>(at + (((g >> 1) ^ (key & 2)) << 4) + ((g & 1) << 3), word[i]);
          else if constexpr (D == 64) c4_words<1>(at + 4 * g, word[i]);
          else {
            unsigned short x;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at + 2 * g) : "memory");
            word[i][0] = x;
          }
        }
#pragma unroll
        for (int j = 0; j < WV; ++j)
#pragma unroll
          for (int u = 0; u < (NT >= 8 ? 2 : 1); ++u) {
            const uint32_t sel = u == 0 ? 0x5410 : 0x7632;
            const uint32_t a = __byte_perm(word[0][j], word[1][j], sel), b = __byte_perm(word[2][j], word[3][j], sel);
#pragma unroll
            for (int i = 0; i < 4; ++i) c4_mma(o[8 * j + 4 * u + i], pa, c4_pair(a >> (4 * i)), c4_pair(b >> (4 * i)));
          }
      }
      __syncwarp();  // the block has been read
      const int next_ids = page_of(kb + (C::kStages + 1) * kC4Warps);
      copy(kb + C::kStages * kC4Warps, ids, stage);
      ids = next_ids;
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
    }
    c4_wait<0>();
    __syncwarp();

    // the item's end: the warps' O, maxima and sums meet in shared memory
    float* mine = reinterpret_cast<float*>(smem + warp * C::kRing);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      pz[i] += __shfl_xor_sync(0xffffffffu, pz[i], 1);
      pz[i] += __shfl_xor_sync(0xffffffffu, pz[i], 2);
      if constexpr (ACT == 2) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if (tig == 0) sh.ml[warp][g + 8 * i] = make_float2(m[i], l[i]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int c = 0; c < NT / 4; ++c)
          *reinterpret_cast<float4*>(mine + 4 * c4_place<D>(g + 8 * i, (NT / 4) * (2 * tig + e) + c)) =
              make_float4(o[4 * c][2 * i + e] + pz[i], o[4 * c + 1][2 * i + e] + pz[i], o[4 * c + 2][2 * i + e] + pz[i],
                          o[4 * c + 3][2 * i + e] + pz[i]);
    }
    __syncthreads();
#pragma unroll 1
    for (int at = tid; at < n_rows * (D / 4); at += kC4Warps * 32) {
      const int lr = at / (D / 4), q4 = at % (D / 4);
      const int flat = w.row_tile * kC4Rows + lr, t = static_cast<uint32_t>(flat) / static_cast<uint32_t>(p.group);
      const int64_t token = r.q0 + t, prow = (2 * static_cast<int64_t>(blockIdx.x) + w.slot()) * kC4Rows + lr;
      const int head = w.h * p.group + flat - t * p.group;
      float inv = 1.f, f[kC4Warps];
#pragma unroll
      for (int i = 0; i < kC4Warps; ++i) f[i] = 1.f;
      if constexpr (ACT == 2) {
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int i = 0; i < kC4Warps; ++i) M = fmaxf(M, sh.ml[i][lr].x);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int i = 0; i < kC4Warps; ++i) {
          f[i] = ex2_sfu(sh.ml[i][lr].x - ref);
          L = __fmaf_rn(sh.ml[i][lr].y, f[i], L);
        }
        if (w.whole) inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // no key seen: 0 (a NaN sum stays NaN)
        if (q4 == 0) {
          if (!w.whole) p.part_ml[prow] = make_float2(M, L);
          else if (p.lse != nullptr) p.lse[static_cast<int64_t>(head) * p.total_q + token] = cc_lse(M, L);
        }
      }
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kC4Warps; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(smem + i * C::kRing + 16 * c4_place<D>(lr, q4));
        a.x = __fmaf_rn(v.x, f[i], a.x);
        a.y = __fmaf_rn(v.y, f[i], a.y);
        a.z = __fmaf_rn(v.z, f[i], a.z);
        a.w = __fmaf_rn(v.w, f[i], a.w);
      }
      if (w.whole)
        *reinterpret_cast<uint2*>(p.out + (token * p.heads + head) * D + 4 * q4) =
            make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
      else *reinterpret_cast<float4*>(p.part_o + prow * D + 4 * q4) = a;
    }
    __syncthreads();  // the rings are free again
  }
}

// ------------------------------------------------------------------ launch
#ifndef JGDPA_HEAD_DIM
#error "compile cache4_fwd.cu with -DJGDPA_HEAD_DIM=32, 64 or 128"
#endif

template <int D, int ACT>
static cudaError_t launch_c4(const Cache4FwdParams& p, int grid, cudaStream_t stream) {
  auto kern = cache4_fwd_kernel<D, ACT>;
  static DeviceFlags attr_set = {};
  cudaError_t e = smem_attr_once(kern, C4Cfg<D>::kSmem, attr_set);
  if (e != cudaSuccess) return e;
  return cache_launch(kern, dim3(grid), kC4Warps * 32, C4Cfg<D>::kSmem, stream, p);
}
template <int D>
cudaError_t launch_cache4_fwd_d(const Cache4FwdParams& p, int act, int grid, cudaStream_t stream) {
  if (act == 0) return launch_c4<D, 0>(p, grid, stream);
  if (act == 1) return launch_c4<D, 1>(p, grid, stream);
  return launch_c4<D, 2>(p, grid, stream);
}
template cudaError_t launch_cache4_fwd_d<JGDPA_HEAD_DIM>(const Cache4FwdParams&, int, int, cudaStream_t);

}  // namespace jg
