// Attention over a paged cache held in 4 bits (cache4.cuh), few query rows per
// key/value head.
//
// An item is (request, key/value head, tile of 16 query rows), a row (new token,
// query head of the group); items are divided among the CTAs and their parts
// joined as in the bf16 kernel (cache.cuh, cache_fwd.cu).  With a key's step s,
// middle z and codes c,
//
//   x = scale (s <q, c> + (z - 8 s) sum q),   O = sum_j (P_j s_j) (c_j - 8) + sum_j P_j z_j
//
// so that the products take the codes themselves, small whole numbers that 16-bit
// types hold exactly, and steps and middles enter in fp32: no value of the cache is
// rounded again, and what a masked place holds (its codes are always finite)
// never meets a row that does not see it.
//
// Bytes per key and head are D + 8 instead of the bf16 cache's 4 D, so what a
// byte costs in instructions counts.
//   S^T = K Q^T and O^T += V^T P^T: the cache is the operand of 16 rows, the
//     query rows the one of 8 columns, one set of them (up to 8 rows) or two; with the rows on the
//     side of 16, as in the bf16 kernel, a single token's 4 heads took twice the
//     products and twice the work on scores.
//   K is fp16: a nibble in the last four bits, or the next four, of a half is
//     2^-24 c or 2^-20 c, a subnormal that takes no instruction but a mask.  Q follows: a row
//     times the power of two that brings its largest value to 2^14 (what falls
//     below fp16 then is 2^-38 of that), the columns of high nibbles times 2^-4 more.
//   V is bf16, as P has its range: 128 + c is 128's bits with c in its last four, less 136.
//   P s goes in two bf16 operands, its rounding and what that leaves: in one (2^-8 of each term) errors
//      average out over many keys that count alike, but where few carry the weight (a peaked softmax of
//      any length, a prompt's first rows) results had up to 1.25 times the error of one rounding, and
//      by the number of keys such rows cannot be told.  With both 1.00 times; 85 us for 81, 35 for 32 on trees of
//      up to 32 rows (d = 64, GELU), 224 for 199 on trees of 64 rows (d = 128).
//   GELU's Phi is right to 1.5e-4 (1.9e-3, as in the bf16 kernels, is as much as the result's own rounding:
//      1.45 to 1.65 times its error at scores near -2 and -4.5; trees 34.6 us for 35.3).
// Every warp works by itself, on blocks of 32 keys
// that it copies (cp.async) into a ring of its own, a few blocks ahead: no
// barrier but an item's end.
//   K: lane t of a key's four takes columns D / 4 t and on, in one load; the order of columns within a
//      product is free, so nibbles i and i + 4 of a word go side by side, masked where they stand.
//   V: a transposing matrix load gives a lane the same four columns of two keys side by side; what is
//      left is a shift and a mask per nibble (with loads key by key and a
//      permutation of bytes: 82 us for 79, 95 for 88 at D = 32).
//
// 64 single tokens over up to 8,192 tokens each (8 x 4 heads, D = 128, softmax): 85 us, 0.45
// of the copy bandwidth (the bf16 cache's bytes alone would take 145).  Bound by latency at few warps: 12 per
// SM by registers, 0.83 of them ready per scheduler and cycle, each taking one block after the other.  Of the 5.3
// cycles per instruction 1.5 are fixed latencies, 0.6 another warp's turn, 0.5 each the integer unit and copies
// and tables; nothing is full (issue slots 52%, integer unit 49%, DRAM 42%, matrix unit 27%).  Some 740 instructions
// per block and warp; copies alone take 52 us.  Measured slower
// (before the second operand): four chains of K's products for two (84 for 82),
// a fifth CTA per SM at the price of spills (127), V's shifts by multiplication
// (86 for 83), blocks of 64 keys (before the last two steps: 77 for 82 here, but 74 for 64 on short
// contexts and 115 for 104 at D = 32).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "act.cuh"
#include "cache4.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace jg {

constexpr int kC4Keys = 64;    // tokens per tile of the work division
constexpr int kC4Block = 32;   // keys of a warp's step
constexpr int kC4Warps = 4;
constexpr int kC4Rows = kCache4Rows;

template <int D, int NQ>
struct C4Cfg {
  static constexpr int kRow = D / 2;  // bytes of a key's codes
  static constexpr int kCodes = kC4Block * kRow;
  static constexpr int kStage = 2 * kCodes + 2 * kC4Block * 4;  // codes of K and V, scales of K and V
  static constexpr int kStages = D == 128 ? (NQ == 1 ? 3 : 4) : D == 64 ? (NQ == 1 ? 4 : 5) : 6;
  static constexpr int kRing = kStage * kStages > kC4Rows * D * 4 ? kStage * kStages : kC4Rows * D * 4;  // (O meets there)
  static constexpr int kQ = NQ * D / 32 * 32 * 16;  // Q's fragments, a copy for every warp
  static constexpr int kQOff = kC4Warps * kRing;
  static constexpr int kSmem = kQOff + kC4Warps * kQ;
  static_assert(kSmem <= 233472 / cache4_ctas(D, NQ) - 2048, "shared memory per CTA");
};

struct C4Shared {
  CacheRangeShared range;
  float2 ml[kC4Warps][kC4Rows];
  CcRow row[kC4Warps][kC4Rows];  // of the item, a copy for every warp
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
__device__ __forceinline__ void c4_mma_k(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void c4_mma_v(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The warp's 8 x 8 matrix of 16-bit values, rows to columns.
__device__ __forceinline__ uint32_t c4_transpose(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Nibble 0 of both halves of w as a bf16 pair, less 8.
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
__device__ __forceinline__ uint32_t c4_word(uint32_t addr) {
  uint32_t w;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(addr) : "memory");
  return w;
}
__device__ __forceinline__ float2 c4_scale(uint32_t w) {  // step, middle
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t c4_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Where four columns of O's row lie in a warp's part of shared memory: no bank
// conflicts, neither as the fragments are written (8 lanes: 4 rows 2 apart, 2
// places side by side) nor as rows are read.
template <int D>
__device__ __forceinline__ int c4_place(int row, int q4) {
  return row * (D / 4) + (q4 ^ (row & 6));
}
// Four 8 x 8 matrices of 16-bit values: a lane's two of each are column lane / 4 of rows
// 2 (lane % 4) and the next; lanes 8 i to 8 i + 7 name matrix i's rows.
__device__ __forceinline__ void c4_matrices(uint32_t addr, uint32_t (&x)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(addr)
               : "memory");
}

// NQ: columns of query rows, by 8.
template <int D, int ACT, int NQ>
__global__ void __launch_bounds__(kC4Warps * 32, cache4_ctas(D, NQ)) cache4_fwd_kernel(const __grid_constant__ Cache4FwdParams pp) {
  using C = C4Cfg<D, NQ>;
  constexpr int WK = D / 32;      // words of K's codes of a lane and key
  constexpr int MT = D / 16;      // tiles of 16 columns of O
  constexpr int R2 = 2 * NQ;      // a lane's query rows: 2 tig + (i % 2) + 8 (i / 2)
  const CacheFwdParams& p = pp.f;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ C4Shared sh;
  cache_let_next();
  cache_wait_before();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tig = lane & 3;
  int* status = p.err + blockIdx.x;
  if (tid == 0) *status = kOk;
  const CacheRange R = cache_range<kC4Keys>(p, &sh.range, kCache4MinRange);
  if (tid == 0) cache_open<kC4Keys>(p, R);
  const uint32_t ring = smem_u32(smem) + warp * C::kRing, q_at = smem_u32(smem) + C::kQOff + warp * C::kQ + lane * 16;
  const int reach = (p.bias_len - 1) / 2;
  // scores in log2 units, or halved as cc_act2 takes them
  constexpr float kUnit = ACT == 2 ? kLog2e : 0.5f;
  const float scale = ACT == 2 ? p.scale : 0.5f * p.scale;
  const int page_mask = (1 << p.page_shift) - 1;

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
    // the pages of a block's keys 0 and 16 on, or -1
    auto pages_of = [&](int block) {
      int2 id = make_int2(-1, -1);
      const int key = block * kC4Block;
      if (block < blocks_end) {
        id.x = table[key >> p.page_shift];
        id.y = key + 16 < r.L ? (p.page_shift == 4 ? table[(key >> 4) + 1] : id.x) : -1;
        const bool bad_x = static_cast<uint32_t>(id.x) >= static_cast<uint32_t>(p.num_pages);
        const bool bad_y = key + 16 < r.L && static_cast<uint32_t>(id.y) >= static_cast<uint32_t>(p.num_pages);
        if (bad_x || bad_y) {
          atomicCAS(status, kOk, kErrBadPage);
          if (bad_x) id.x = -1;
          if (bad_y) id.y = -1;
        }
      }
      return id;
    };
    // A block's copies: a half of 16 keys lies in one page, side by side.
    auto v_turn = [](int key) { return D == 128 ? (key >> 1) & 3 : D == 64 ? (key >> 2) & 1 : 0; };
    constexpr int kPieces = C::kRow / 16;                   // of a key
    constexpr int kHalf = 16 * kPieces;                     // of 16 keys' codes
    constexpr int kEach = kHalf >= 32 ? kHalf / 32 : 1;     // of them a lane's
    // A lane's place in a half's codes (with kHalf = 16 lanes 16 and on take the second half): key and piece,
    // and where they go: V's pieces turned by key, so that one piece of 8 keys is read without bank conflicts.
    const int c_key = lane / kPieces, c_piece = lane % kPieces;
    const int k_to = c_key * C::kRow + 16 * c_piece;
    const int v_to = C::kCodes + c_key * C::kRow + 16 * (c_piece ^ v_turn(c_key));
    // a lane's places in the head's part of page 0: codes, and (lanes 0 to 7 K's, 8 to 15 V's) scales of four keys
    const int64_t head_at = static_cast<int64_t>(w.h) << p.page_shift;
    const uint8_t* const k_lane = pp.k.codes + head_at * C::kRow + 16 * (kHalf >= 32 ? lane : lane & 15);
    const uint8_t* const v_lane = pp.v.codes + head_at * C::kRow + 16 * (kHalf >= 32 ? lane : lane & 15);
    const Cache4& s_half = lane < 8 ? pp.k : pp.v;
    const __nv_bfloat16* const s_lane = s_half.scales + head_at * 2;
    const int64_t s_stride = s_half.scale_stride;
    auto copy = [&](int block, int2 id, int stage) {  // (the whole warp)
      if (block < blocks_end) {
        const uint32_t to = ring + stage * C::kStage;
        const int first = block * kC4Block;
#pragma unroll
        for (int half = 0; half < (kHalf >= 32 ? 2 : 1); ++half) {
          const int h = kHalf >= 32 ? half : lane >> 4;
          const int page = h ? id.y : id.x;
          const bool live = page >= 0;
          const int pg = max(page, 0), at = ((first + 16 * h) & page_mask) * C::kRow;
          const uint8_t* ks = k_lane + pg * pp.k.code_stride + at;
          const uint8_t* vs = v_lane + pg * pp.v.code_stride + at;
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            const int from = ((kHalf >= 32 ? 16 * half : 0) + i * (32 / kPieces)) * C::kRow;  // (8 keys or more, in order)
            c4_copy(to + k_to + from, ks + 512 * i, live);
            c4_copy(to + v_to + from, vs + 512 * i, live);
          }
        }
        if (lane < 16) {
          const int key = (lane & 7) * 4, page = key & 16 ? id.y : id.x;
          c4_copy(to + 2 * C::kCodes + lane * 16, s_lane + max(page, 0) * s_stride + ((first + key) & page_mask) * 2, page >= 0);
        }
      }
      c4_commit();
    };
    // the first blocks are on their way before anything else of the item
    int2 ids = pages_of(kb);
#pragma unroll
    for (int i = 0; i < C::kStages; ++i) {
      const int2 next_ids = pages_of(kb + (i + 1) * kC4Warps);
      copy(kb + i * kC4Warps, ids, i);
      ids = next_ids;
    }

    const int n_rows = min(kC4Rows, r.T * p.group - w.row_tile * kC4Rows);
    // the rows, lanes 0 to 15 one each; by the loop they are only asked for where a block is not plain
    int pos_min = INT32_MAX, pos_max = 0;
    bool hides = false;  // some row's bias hides all far keys, or is beyond what log2 units hold
    if (lane < kC4Rows) {
      const int flat = w.row_tile * kC4Rows + lane, t = static_cast<uint32_t>(flat) / static_cast<uint32_t>(p.group);
      CcRow q{-1, r.C, w.h * p.group, 0.f};
      if (lane < n_rows) {
        q.t = t;
        q.head += flat - t * p.group;
        q.pos = cc_row_pos(p, r, t, status);
        pos_min = pos_max = q.pos;
        if (p.bias_len) q.far_bias = __ldg(p.bias + static_cast<int64_t>(q.head) * p.bias_len + 2 * reach) * kUnit;
        hides = ACT == 2 && fabsf(q.far_bias) > kHugeScore;
      }
      sh.row[warp][lane] = q;
    }
    hides = __any_sync(0xffffffffu, hides);
    pos_min = __reduce_min_sync(0xffffffffu, pos_min);
    pos_max = __reduce_max_sync(0xffffffffu, pos_max);
    __syncwarp();
    auto row_of = [&](int i) -> const CcRow& { return sh.row[warp][2 * tig + (i & 1) + 8 * (i >> 1)]; };
    // Q's fragments (query row g + 8 n) in the order of K's nibbles, and what a lane's rows (2 tig ..) need of it
    float q_sum[R2], q_unit[R2];  // sum q, and what brings <q, c> back
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int lr = g + 8 * n, flat = w.row_tile * kC4Rows + lr, t = static_cast<uint32_t>(flat) / static_cast<uint32_t>(p.group);
      const __nv_bfloat16* src = p.q + static_cast<int64_t>(r.q0 + t) * p.q_stride +
                                 static_cast<int64_t>(w.h * p.group + flat - t * p.group) * D + (D / 4) * tig;
      uint4 v[WK];
      float sum = 0.f, top = 0.f;
#pragma unroll
      for (int j = 0; j < WK; ++j) {
        v[j] = make_uint4(0, 0, 0, 0);
        if (lr < n_rows) v[j] = *reinterpret_cast<const uint4*>(src + 8 * j);
        const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = __uint_as_float(x[e] << 16), b = __uint_as_float(x[e] & 0xFFFF0000u);
          sum += a + b;
          top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      // 2^e <= top < 2^(e + 1): the row times 2^(14 - e), in two factors that fp32 holds
      const int e = top > 0.f ? max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -124) : 0;
      const int up = min(14 - e, 123);
      const float f0 = __uint_as_float(static_cast<uint32_t>(up + 127) << 23), f1 = __uint_as_float(static_cast<uint32_t>(14 - e - up + 127) << 23);
#pragma unroll
      for (int j = 0; j < WK; ++j) {
        const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};  // columns 2 e, 2 e + 1
        float y[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          y[2 * c] = __uint_as_float(x[c] << 16) * f0 * f1;
          y[2 * c + 1] = __uint_as_float(x[c] & 0xFFFF0000u) * f0 * f1 * 0.0625f;
        }
        // columns 2 h and 2 h + 4, 2 h + 1 and 2 h + 5
        st_shared_v4(q_at + (n * WK + j) * 512, c4_half2(y[0], y[4]), c4_half2(y[1], y[5]), c4_half2(y[2], y[6]), c4_half2(y[3], y[7]));
      }
      // 2^24 of the codes (half of it with the step) and 2^(e - 14) of the row; lane 4 (2 tig + i) has row 2 tig + i
      const float back = __uint_as_float(static_cast<uint32_t>(12 + e - 14 + 127) << 23);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        q_sum[2 * n + i] = __shfl_sync(0xffffffffu, sum, 4 * (2 * tig + i));
        q_unit[2 * n + i] = __shfl_sync(0xffffffffu, back, 4 * (2 * tig + i));
      }
    }
    float o[NQ][MT][4];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][mt][e] = 0.f;
    float m[R2], l[R2], pz[R2];  // pz: sum P z
#pragma unroll
    for (int i = 0; i < R2; ++i) {
      m[i] = -INFINITY;
      l[i] = pz[i] = 0.f;
    }

    int stage = 0;
    const int v_key = (lane & 7) + 8 * (lane / 8 / kPieces);
    const int v_lane_at = v_key * C::kRow + 16 * ((lane / 8) % kPieces ^ v_turn(v_key));
#pragma unroll 1
    for (; kb < blocks_end; kb += kC4Warps) {
      c4_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t kt = ring + stage * C::kStage, vt = kt + C::kCodes, ks = vt + C::kCodes, vs = ks + kC4Block * 4;
      // everything of the block that is read, at once: what follows is cut by branches, across which loads do not move
      auto key_of = [&](int kk, int e) { return 16 * kk + 8 * e + g; };  // a lane's keys
      uint32_t k_word[4][WK], k_scale[4], v_scale[4], v_word[kPieces][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c4_words<WK>(kt + (8 * e + g) * C::kRow + tig * (4 * WK), k_word[e]);
        k_scale[e] = c4_word(ks + 4 * key_of(e >> 1, e & 1));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v_scale[e] = c4_word(vs + 4 * key_of(e >> 1, e & 1));
      // matrix i of a read: piece i % kPieces of the 8 keys 8 (i / kPieces) and on
#pragma unroll
      for (int i = 0; i < kPieces; ++i) c4_matrices(vt + v_lane_at + i * (4 / kPieces) * 8 * C::kRow, v_word[i]);
      const int key0 = kb * kC4Block;
      const bool far = p.bias_len == 0 || (!hides && key0 + kC4Block - 1 < r.C && pos_min - (key0 + kC4Block - 1) >= reach);
      bool plain = key0 + kC4Block - 1 < r.C && (p.window <= 0 || pos_max - key0 < p.window);
      float far_bias[R2];
#pragma unroll
      for (int i = 0; i < R2; ++i) far_bias[i] = 0.f;
      if (p.bias_len != 0 && far) {
#pragma unroll
        for (int i = 0; i < R2; ++i) far_bias[i] = row_of(i).far_bias;
      }
      uint32_t see[R2];
#pragma unroll
      for (int i = 0; i < R2; ++i) see[i] = 0xFFFFFFFFu;
      if (!plain) {
#pragma unroll
        for (int i = 0; i < R2; ++i) {
          uint32_t bits = cc_vis32(p, r, row_of(i), key0);
          if (p.window > 0) {
            uint32_t near = 0;
            if (cc_in_order(p, r, key0)) {
              near = cc_near32(p, row_of(i).pos, key0);
            } else {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                const int at = key_of(c >> 1, c & 1);
                near |= (cc_near(p, row_of(i).pos, cc_pos(p, r, key0 + at)) ? 1u : 0u) << at;
              }
            }
            bits &= near;  // (only this lane's keys are kept)
          }
          see[i] = bits;
        }
      }
      // S^T: s[n][kk][2 e + i] is key_of(kk, e) with row 2 n + i
      float s[NQ][2][4];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[n][e >> 2][e & 3] = 0.f;
      {
#pragma unroll
        for (int j = 0; j < WK; ++j)
        {
          uint32_t qb[NQ][4];
#pragma unroll
          for (int n = 0; n < NQ; ++n) ld_shared_v4(q_at + (n * WK + j) * 512, qb[n][0], qb[n][1], qb[n][2], qb[n][3]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              const uint32_t x = k_word[2 * kk][j] >> (8 * h), y = k_word[2 * kk + 1][j] >> (8 * h);
              const uint32_t a[4] = {x & 0x000F000Fu, y & 0x000F000Fu, x & 0x00F000F0u, y & 0x00F000F0u};
#pragma unroll
              for (int n = 0; n < NQ; ++n) c4_mma_k(s[n][kk], a, qb[n][2 * h], qb[n][2 * h + 1]);
            }
        }
      }
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 k = c4_scale(k_scale[2 * kk + e]);
          const float step = k.x * (4096.f * scale), middle = __fmaf_rn(-8.f, k.x, k.y) * scale;
          const float2 step2 = make_float2(step, step), middle2 = make_float2(middle, middle);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            float* x = &s[n][kk][2 * e];
            const float2 y = __ffma2_rn(__fmul2_rn(make_float2(x[0], x[1]), make_float2(q_unit[2 * n], q_unit[2 * n + 1])), step2,
                                        __ffma2_rn(middle2, make_float2(q_sum[2 * n], q_sum[2 * n + 1]),
                                                   make_float2(far_bias[2 * n], far_bias[2 * n + 1])));
            x[0] = y.x;
            x[1] = y.y;
          }
        }
      if (!far) {
        float top = 0.f;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key_pos = cc_pos(p, r, key0 + key_of(kk, e));
#pragma unroll
            for (int i = 0; i < R2; ++i) {
              const float bias = cc_bias(p, row_of(i), reach, key_pos);
              float& x = s[i >> 1][kk][2 * e + (i & 1)];
              x = __fmaf_rn(bias, kUnit, x);
              if constexpr (ACT == 2) top = fmaxf(top, fabsf(bias));
            }
          }
        if (ACT == 2 && __any_sync(0xffffffffu, top > kHugeBias)) {
          plain = false;
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int i = 0; i < R2; ++i) {
                const int at = key_of(kk, e);
                const float bias = cc_bias(p, row_of(i), reach, cc_pos(p, r, key0 + at));
                float& x = s[i >> 1][kk][2 * e + (i & 1)];
                if (bias == -INFINITY) see[i] &= ~(1u << at);
                else if (fabsf(bias) > kHugeBias && x == x) x = cc_huge(bias);
              }
        }
      }
      if (!plain) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < R2; ++i)
              if (!((see[i] >> key_of(kk, e)) & 1)) s[i >> 1][kk][2 * e + (i & 1)] = ACT == 2 ? -INFINITY : 0.f;  // act(0) = 0
      }
      if constexpr (ACT == 2) {
        // m: within 8 (log2 units) of the maximum or above, as in the bf16 kernel
        float mx[R2];
        bool over = false;
#pragma unroll
        for (int i = 0; i < R2; ++i) {
          const int n = i >> 1, c = i & 1;
          mx[i] = fmaxf(fmaxf(s[n][0][c], s[n][0][2 + c]), fmaxf(s[n][1][c], s[n][1][2 + c]));
          over = over || mx[i] > m[i] + 8.f;
        }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int i = 0; i < R2; ++i) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], x));
            const float mn = fmaxf(m[i], mx[i]);
            const float f = mn == -INFINITY ? 1.f : ex2_sfu(m[i] - mn);
            m[i] = mn;
            l[i] *= f;
            pz[i] *= f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              o[i >> 1][mt][i & 1] *= f;
              o[i >> 1][mt][2 + (i & 1)] *= f;
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const float2 ref = make_float2(m[2 * n] == -INFINITY ? 0.f : -m[2 * n], m[2 * n + 1] == -INFINITY ? 0.f : -m[2 * n + 1]);
          float2 sum = make_float2(l[2 * n], l[2 * n + 1]);
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float* x = &s[n][kk][2 * e];
              const float2 y = __fadd2_rn(make_float2(x[0], x[1]), ref);
              x[0] = ex2_sfu(y.x);
              x[1] = ex2_sfu(y.y);
              sum = __fadd2_rn(sum, make_float2(x[0], x[1]));
            }
          l[2 * n] = sum.x;
          l[2 * n + 1] = sum.y;
        }
      } else {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const float2 y = cc_act2<ACT, 8>(make_float2(s[n][kk][e], s[n][kk][e + 1]));
              s[n][kk][e] = y.x;
              s[n][kk][e + 1] = y.y;
            }
      }
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {  // 16 keys
        // P s as two bf16 operands, its rounding and what that leaves (2^-16 of it at most)
        uint32_t pb[NQ][2], pl[NQ][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 v = c4_scale(v_scale[2 * kk + e]);
          float2 y[NQ];
          if (plain) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              const float2 weight = make_float2(s[n][kk][2 * e], s[n][kk][2 * e + 1]);
              y[n] = __fmul2_rn(weight, make_float2(v.x, v.x));
              const float2 b = __ffma2_rn(weight, make_float2(v.y, v.y), make_float2(pz[2 * n], pz[2 * n + 1]));
              pz[2 * n] = b.x;
              pz[2 * n + 1] = b.y;
            }
          } else {  // (a place that the row does not see may hold any step and middle)
#pragma unroll
            for (int i = 0; i < R2; ++i) {
              const float weight = s[i >> 1][kk][2 * e + (i & 1)];
              const bool sees = (see[i] >> key_of(kk, e)) & 1;
              (i & 1 ? y[i >> 1].y : y[i >> 1].x) = sees ? weight * v.x : 0.f;
              if (sees) pz[i] = __fmaf_rn(weight, v.y, pz[i]);
            }
          }
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            const uint32_t top = pack_bf16(y[n].x, y[n].y);
            const float2 rest = __ffma2_rn(c4_scale(top), make_float2(-1.f, -1.f), y[n]);  // (of an infinity: NaN)
            pb[n][e] = c4_transpose(top);
            pl[n][e] = c4_transpose(pack_bf16(rest.x, rest.y));
          }
        }
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {  // 32 columns
          // (8 keys' piece c is number kPieces (2 kk) + c of the matrices read)
          constexpr int kP = kPieces;
          const uint32_t x = v_word[(kP * 2 * kk + c) / 4][(kP * 2 * kk + c) % 4], y = v_word[(kP * (2 * kk + 1) + c) / 4][(kP * (2 * kk + 1) + c) % 4];
          uint32_t a[2][4];  // nibbles 2 i and 2 i + 1: columns 32 c + 4 g + 2 i and + 1
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            a[i][0] = c4_pair(x >> (8 * i)), a[i][1] = c4_pair(x >> (8 * i + 4));
            a[i][2] = c4_pair(y >> (8 * i)), a[i][3] = c4_pair(y >> (8 * i + 4));
#pragma unroll
            for (int n = 0; n < NQ; ++n) c4_mma_v(o[n][2 * c + i], a[i], pb[n][0], pb[n][1]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < NQ; ++n) c4_mma_v(o[n][2 * c + i], a[i], pl[n][0], pl[n][1]);
        }
      }
      __syncwarp();  // the block has been read
      const int2 next_ids = pages_of(kb + (C::kStages + 1) * kC4Warps);
      copy(kb + C::kStages * kC4Warps, ids, stage);
      ids = next_ids;
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
    }
    c4_wait<0>();
    __syncwarp();

    // the item's end: the warps' O, maxima and sums meet in shared memory
    float* mine = reinterpret_cast<float*>(smem + warp * C::kRing);
#pragma unroll
    for (int i = 0; i < R2; ++i) {
      const int row = 2 * tig + (i & 1) + 8 * (i >> 1);
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        pz[i] += __shfl_xor_sync(0xffffffffu, pz[i], x);
        if constexpr (ACT == 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
      }
      if (ACT == 2 && g == 0) sh.ml[warp][row] = make_float2(m[i], l[i]);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const float(&a)[4] = o[i >> 1][2 * c], (&b)[4] = o[i >> 1][2 * c + 1];
        *reinterpret_cast<float4*>(mine + 4 * c4_place<D>(row, 8 * c + g)) =
            make_float4(a[i & 1] + pz[i], a[2 + (i & 1)] + pz[i], b[i & 1] + pz[i], b[2 + (i & 1)] + pz[i]);
      }
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

template <int D, int ACT, int NQ>
static cudaError_t launch_c4(const Cache4FwdParams& p, int grid, cudaStream_t stream) {
  auto kern = cache4_fwd_kernel<D, ACT, NQ>;
  static DeviceFlags attr_set = {};
  cudaError_t e = smem_attr_once(kern, C4Cfg<D, NQ>::kSmem, attr_set);
  if (e != cudaSuccess) return e;
  return cache_launch(kern, dim3(grid), kC4Warps * 32, C4Cfg<D, NQ>::kSmem, stream, p);
}
template <int D, int ACT>
static cudaError_t launch_c4_rows(const Cache4FwdParams& p, int grid, cudaStream_t stream) {
  return cache4_columns(static_cast<int64_t>(p.f.max_q) * p.f.group) == 1 ? launch_c4<D, ACT, 1>(p, grid, stream)
                                                                           : launch_c4<D, ACT, 2>(p, grid, stream);
}
template <int D>
cudaError_t launch_cache4_fwd_d(const Cache4FwdParams& p, int act, int grid, cudaStream_t stream) {
  if (act == 0) return launch_c4_rows<D, 0>(p, grid, stream);
  if (act == 1) return launch_c4_rows<D, 1>(p, grid, stream);
  return launch_c4_rows<D, 2>(p, grid, stream);
}
template cudaError_t launch_cache4_fwd_d<JGDPA_HEAD_DIM>(const Cache4FwdParams&, int, int, cudaStream_t);

}  // namespace jg
