// Attention over a paged key/value cache, few query rows per key/value head.
//
// One item is (request, key/value head, tile of 16 or 32 query rows); a row is
// (new token, query head of the group), so the heads that share a key/value
// head share its loads.  Of small heads (d < 128) an item takes 128 / d side by
// side where their number allows and the work is large enough: their columns are
// one contiguous 256-byte piece per token, and an item's start and end are paid
// once for all of them (d = 32, 16 heads, 64 requests of 4,100 tokens: 98 us
// against 190 one by one).  Its keys stream through shared memory once, in tiles
// of 64 tokens gathered from the pages by TMA.
//
//   S = Q K^T, P = act(S) or exp2(S - m), O += P V
//
// With R rows each K/V byte feeds R multiply-adds, so for R <= 16 the kernel is
// bound by HBM.  Rows of 16 are the m of mma.sync m16n8k16, whose fragments
// keep S, P and O in registers: no tensor-memory round trip and no block-wide
// step per tile.  (The 128-row tensor-memory form is cache_fwd_wide.cu.)  Four
// warps share a tile: a head's keys are divided among them, or, of heads side by
// side, each takes one head (d = 32) or half the keys of one (d = 64), each with
// its own running maximum, sum and O; those of a head meet once per item.  (With
// every warp at all four heads of a quarter of the keys the d = 32 case above
// took 120 us: a step with few independent instructions per head,
// four times.)  With 32-row tiles (d < 128) a second group of four warps takes
// the second 16 rows of the same keys.
//
// A TMA producer runs up to 96 KB ahead, across items, and several CTAs share
// an SM, so that neither an item's end (the warps' exchange) nor its start
// stops the loads.
//
// Measured, d = 128: 64 requests of 118 to 8,000 tokens, 8 key/value heads, 4
// rows each: 171 to 175 us from GPU to GPU, 0.93 to 0.91 of the copy bandwidth; one
// of 131,072 tokens: 94 us with the joining, 0.84.  d = 32, 128 requests, SiLU,
// window 1,024: 59 us, 0.64: items of 17 tiles, of which two or three are masked.
#include "act.cuh"
#include "cache.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace jg {

constexpr int kCKeys = 64;        // tokens per tile
constexpr int kCGroupWarps = 4;   // warps that share a tile's keys
constexpr int kCMinRange = 5;     // the least length of a range
constexpr int kCChunk = 32;       // columns of O that meet at a time at an item's end

// W: columns of K and V that an item streams, the head dimension times the
// heads that it takes together.
template <int W, int MT, int HP>
struct CcCfg {
  static constexpr int kWarps = kCGroupWarps * MT;  // consumer warps
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kTileBytes = kCKeys * W * 2;  // K or V of one tile
  // CTAs per SM and stages of K and V: 130 to 190 KB of loads in flight on an
  // SM (at d = 128, 64 KB reached 0.67 of the copy bandwidth on one long
  // request, 128 KB 0.82)
  static constexpr int kCtas = cache_ctas(W, MT);
  static constexpr int kStages = MT == 1 ? (W == 128 ? 3 : W == 64 ? 4 : 5) : (W == 128 ? 6 : W == 64 ? 5 : 10);
  static constexpr int kSlotBytes = 16 * kCChunk * 4;  // one warp's chunk of O
  static constexpr int kOOff = kStages * 2 * kTileBytes;
  static constexpr int kBarOff = kOOff + kWarps * kSlotBytes;
  static constexpr int kSmemBytes = kBarOff + 768 + kWarps * 16 * 8 + 1024;
  // A group's warps: a head each, or a head's keys shared by several
  static constexpr int kKeyGroups = kCGroupWarps / HP;
  static_assert(kSmemBytes <= 233472 / kCtas - 1024, "shared memory per CTA");
};

template <int MT>
struct CcShared {
  uint64_t full[16], empty[16];
  CacheRangeShared range;
  int abort;
  float2 ml[MT * kCGroupWarps][16];  // a warp's maxima and sums
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte piece c of key n in a K or V tile: the tile is a row
// of TMA boxes of `pr` = min(page size, 64) tokens, each [halves][pr][row],
// its pieces swizzled over the bytes of a row by the row's place in 8.
template <int W>
__device__ __forceinline__ uint32_t cc_offset(int n, int c, int pr) {
  const int r = n & (pr - 1);
  if constexpr (W >= 64) return (n - r) * (W * 2) + (c >> 3) * (pr * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  else return (n - r) * (W * 2) + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// ------------------------------------------------------------- producer
template <int W, int MT, int HP>
__device__ void cc_producer(const CacheFwdParams& p, uint8_t* smem, CcShared<MT>* sh, const CacheRange& R, Fail fail) {
  using C = CcCfg<W, MT, HP>;
  const int lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem);
  const int pr = min(1 << p.page_shift, kCKeys), pieces = kCKeys / pr;  // pieces: 1, 2 or 4
  uint32_t it = 0;
  bool ok = true;
  CacheWalk w;
  w.init(R);
  for (; ok && w.template next<kCKeys>(p); w.advance()) {
    int lo, hi;
    w.template tiles<kCKeys>(p, lo, hi);
    const int32_t* row = p.table + static_cast<int64_t>(w.b) * p.width;
    for (int t = lo; t < hi && ok; ++t) {
      // lane i: piece i / 2 of K (even) or V (odd)
      const int key = t * kCKeys + (lane >> 1) * pr;
      const bool mine = (lane >> 1) < pieces && key < w.r.L;
      int page = p.num_pages;
      if (mine) {
        page = __ldg(row + (key >> p.page_shift));
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) {
          atomicCAS(fail.status, kOk, kErrBadPage);
          page = p.num_pages;  // outside the map: the copy writes zeros and reads nothing
        }
      }
      const int n = min(pieces, (w.r.L - t * kCKeys + pr - 1) / pr);
      const int st = it % C::kStages;
      if (!(ok = mbar_wait_warp(&sh->empty[st], ((it / C::kStages) & 1) ^ 1, fail))) break;
      if (lane == 0) mbar_arrive_tx(&sh->full[st], 2 * n * pr * W * 2);
      __syncwarp();
      if (mine) {
        const uint32_t dst = base + st * 2 * C::kTileBytes + (lane & 1) * C::kTileBytes + (lane >> 1) * pr * W * 2;
        tma_load_5d(dst, (lane & 1) ? &p.tm_v : &p.tm_k, &sh->full[st], 0, key & ((1 << p.page_shift) - 1), 0, w.h,
                    page);
      }
      ++it;
    }
  }
  // the copies issued land before the CTA exits, also when the consumers gave up
  for (uint32_t i = it > C::kStages ? it - C::kStages : 0; i < it; ++i)
    mbar_wait_drain(&sh->full[i % C::kStages], (i / C::kStages) & 1);
}

// ------------------------------------------------------------- consumers
template <int D, int ACT, int MT, int HP>
__device__ void cc_consumer(const CacheFwdParams& p, uint8_t* smem, CcShared<MT>* sh, const CacheRange& R, Fail fail) {
  constexpr int W = D * HP;
  using C = CcCfg<W, MT, HP>;
  constexpr int KS = D / 16;  // k steps of S = Q K^T
  constexpr int NT = D / 8;   // n tiles of O
  constexpr int kRows = 16 * MT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int KG = C::kKeyGroups, KB = HP;  // warps that share a head's keys, blocks of 16 keys of a warp
  static_assert(KB * KG * 16 == kCKeys, "keys of a tile");
  const int grp = warp / kCGroupWarps, hw = warp % kCGroupWarps / KG, kg = warp % KG;  // which rows, head, keys
  const int pr = min(1 << p.page_shift, kCKeys);
  const uint32_t base = smem_u32(smem);
  // this warp's keys: piece addresses for ldmatrix (the four 8x8 blocks of a
  // load are keys 0-7 / 8-15 by 16-byte piece for K, and transposed for V); the
  // lane's part of an address is fixed, a piece comes in by exclusive or, a
  // block of 16 keys by addition
  const int half = W >= 64 ? pr * 128 : 0;  // bytes of a box's column half
  auto head_at = [&](uint32_t at) {         // the warp's head's first piece
    return W >= 64 ? (at ^ ((hw * (D / 8) & 7) << 4)) + (hw * D >= 64 ? half : 0) : at;
  };
  const int first = 16 * KB * kg;
  const uint32_t kl = head_at(cc_offset<W>(first + (lane & 7) + ((lane & 16) ? 8 : 0), (lane >> 3) & 1, pr));
  const uint32_t vl = head_at(cc_offset<W>(first + (lane & 7) + ((lane & 8) ? 8 : 0), lane >> 4, pr));
  auto piece = [&](uint32_t at, int c) {  // of the head's even piece c
    return (at ^ ((c & (W >= 64 ? 6 : 2)) << 4)) + (W >= 64 && c >= 8 ? half : 0);
  };
  const uint32_t row_bytes = W >= 64 ? 128 : 64;
  const uint32_t step1 = 16 * (pr >= 32 ? row_bytes : 2 * W), step2 = 32 * (pr >= 64 ? row_bytes : 2 * W);
  auto block = [&](int kb) { return (kb & 1) * step1 + (kb >> 1) * step2; };
  const int reach = (p.bias_len - 1) / 2;
  // scores in log2 units, or halved as cc_act2 takes them
  constexpr float kUnit = ACT == 2 ? kLog2e : 0.5f;
  const float scale = ACT == 2 ? p.scale : 0.5f * p.scale;
  uint32_t it = 0;
  bool dead = false;
  CacheWalk w;
  w.init(R);
  for (; w.template next<kCKeys>(p); w.advance()) {
    const CacheReq& r = w.r;
    int lo, hi;
    w.template tiles<kCKeys>(p, lo, hi);
    const int n_rows = min(kRows, r.T * p.group - w.row_tile * kRows);
    CcRow rows[2];  // lane / 4 and lane / 4 + 8 of the warp's 16
    const __nv_bfloat16* qrow[2];
    float far_bias[2];
    int pos_min = INT32_MAX;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int lr = 16 * grp + (lane >> 2) + 8 * i;
      const int flat = w.row_tile * kRows + lr;
      CcRow& q = rows[i];
      const int t = static_cast<uint32_t>(flat) / static_cast<uint32_t>(p.group);
      q.t = lr < n_rows ? t : -1;
      q.head = (w.h * HP + hw) * p.group + (lr < n_rows ? flat - t * p.group : 0);
      q.pos = r.C;
      q.far_bias = 0.f;
      qrow[i] = nullptr;
      if (q.t >= 0) {
        q.pos = cc_row_pos(p, r, q.t, fail.status);
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
    // Q fragments: rows lane / 4 (+ 8), columns 16 ks + 2 (lane % 4) (+ 8).  By
    // ordinary loads: Q may be what the call before wrote while this block was
    // being set up, and so is not constant over the kernel's life.
    uint32_t qa[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat16* src = qrow[e & 1];
        qa[ks][e] = src != nullptr ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * (lane & 3) + ((e & 2) ? 8 : 0)) : 0u;
      }
    float o[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int t = lo; t < hi; ++t, ++it) {
      const int st = it % C::kStages;
      if (!dead && !mbar_wait(&sh->full[st], (it / C::kStages) & 1, fail)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      const int key0 = t * kCKeys + first;  // this warp's first key
      if (!dead && key0 < r.L) {
        const uint32_t kt = base + st * 2 * C::kTileBytes, vt = kt + C::kTileBytes;
        // plain: every key of the warp's is seen by every row; far: R or more behind
        const int last = key0 + 16 * KB - 1;
        const bool far = p.bias_len == 0 || (!hides && last < r.C && pos_min - last >= reach);
        bool plain = last < r.C && (p.window <= 0 || pos_max - key0 < p.window);
        uint32_t see[(KB + 1) / 2][2];  // by 32 keys
        if (!plain) {
#pragma unroll
          for (int j = 0; j < (KB + 1) / 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t bits = cc_vis32(p, r, rows[h], key0 + 32 * j);
              if (p.window > 0) {
                uint32_t near = 0;
                if (cc_in_order(p, r, key0 + 32 * j)) {
                  near = cc_near32(p, rows[h].pos, key0 + 32 * j);
                } else {
#pragma unroll 1
                  for (int c = 0; c < (KB > 1 ? 8 : 4); ++c) {
                    const int col = 8 * (c >> 1) + 2 * (lane & 3) + (c & 1);
                    near |= (cc_near(p, rows[h].pos, cc_pos(p, r, key0 + 32 * j + col)) ? 1u : 0u) << col;
                  }
                }
                bits &= near;  // (only this lane's columns are kept)
              }
              see[j][h] = bits;
            }
        }
        float s[KB][2][4];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[kb][i][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            uint32_t b[4];
            ldsm4(piece(kt + block(kb) + kl, 2 * ks), b);
            mma16816(s[kb][0], qa[ks], b[0], b[1]);
            mma16816(s[kb][1], qa[ks], b[2], b[3]);
          }
        if (far) {
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[kb][i][e] = __fmaf_rn(s[kb][i][e], scale, far_bias[e >> 1]);
        } else {
          float top = 0.f;
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int key_pos = cc_pos(p, r, key0 + 16 * kb + 8 * i + 2 * (lane & 3) + c);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float bias = cc_bias(p, rows[h], reach, key_pos);
                  s[kb][i][2 * h + c] = __fmaf_rn(s[kb][i][2 * h + c], scale, bias * kUnit);
                  if constexpr (ACT == 2) top = fmaxf(top, fabsf(bias));
                }
              }
          if (ACT == 2 && __any_sync(0xffffffffu, top > kHugeBias)) {
            if (plain) {
#pragma unroll
              for (int j = 0; j < (KB + 1) / 2; ++j) see[j][0] = see[j][1] = 0xFFFFFFFFu;
              plain = false;
            }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int i = e >> 2, h = (e >> 1) & 1, col = 16 * (kb & 1) + 8 * i + 2 * (lane & 3) + (e & 1);
                const float bias = cc_bias(p, rows[h], reach, cc_pos(p, r, key0 + 32 * (kb >> 1) + col));
                float& x = s[kb][i][e & 3];
                if (bias == -INFINITY) see[kb >> 1][h] &= ~(1u << col);
                else if (fabsf(bias) > kHugeBias && x == x) x = cc_huge(bias);
              }
          }
        }
        bool odd = false;
        if (!plain) {
          // Some rows do not see some of these keys, and 0 * NaN = NaN: rows of
          // V past the request's end (whatever the page held) count as zeros,
          // and where others hold an infinity or NaN (`odd`) those are left out
          // of the product and added to the rows that see them.
          const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
          __nv_bfloat162 sum = zero;  // of 0 * v
#pragma unroll 1
          for (int k = lane & 15; k < 16 * KB && key0 + k < r.L; k += 16)
#pragma unroll 1
            for (int c = lane >> 4; c < D / 8; c += 2) {
              uint32_t x[4];
              ld_shared_v4(vt + cc_offset<W>(first + k, hw * (D / 8) + c, pr), x[0], x[1], x[2], x[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) sum = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&x[e]), zero, sum);
            }
          odd = __any_sync(0xffffffffu, !(__low2float(sum) == 0.f && __high2float(sum) == 0.f));
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (!((see[kb >> 1][e >> 1] >> (16 * (kb & 1) + 8 * i + 2 * (lane & 3) + (e & 1))) & 1))
                  s[kb][i][e] = ACT == 2 ? -INFINITY : 0.f;  // act(0) = 0
        }
        float(&pv)[KB][2][4] = s;  // in place
        if constexpr (ACT == 2) {
          // m need not be the maximum, only within 8 (in log2 units) of it or
          // above: weights up to 2^8, and a step, with the exchange between the
          // lanes of a row, that most tiles skip (5% at d = 32)
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              mx[i] = fmaxf(mx[i], fmaxf(fmaxf(s[kb][0][2 * i], s[kb][0][2 * i + 1]), fmaxf(s[kb][1][2 * i], s[kb][1][2 * i + 1])));
          if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
              const float mn = fmaxf(m[i], fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2)));
              const float f = mn == -INFINITY ? 1.f : ex2_sfu(m[i] - mn);
              m[i] = mn;
              l[i] *= f;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                o[nt][2 * i] *= f;
                o[nt][2 * i + 1] *= f;
              }
            }
          }
          const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                pv[kb][i][e] = ex2_sfu(s[kb][i][e] - ref[e >> 1]);
                l[e >> 1] += pv[kb][i][e];
              }
        } else {
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const float2 y = cc_act2<ACT>(make_float2(s[kb][i][e], s[kb][i][e + 1]));
                pv[kb][i][e] = y.x;
                pv[kb][i][e + 1] = y.y;
              }
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          // P rounds to bf16 as the A operand (half a step, 2^-8 of each weight at most)
          uint32_t pa[4], keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
#pragma unroll
          for (int i = 0; i < 4; ++i) pa[i] = pack_bf16(pv[kb][i >> 1][2 * (i & 1)], pv[kb][i >> 1][2 * (i & 1) + 1]);
          if (!plain) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int j = key0 + 16 * kb + 8 * i + 2 * (lane & 3);
              keep[i] = j + 1 < r.L ? 0xFFFFFFFFu : (j < r.L ? 0xFFFFu : 0u);
            }
          }
#pragma unroll
          for (int n2 = 0; n2 < NT / 2; ++n2) {
            uint32_t b[4];
            ldsm4_t(piece(vt + block(kb) + vl, 2 * n2), b);
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] &= keep[e & 1];
            if (odd) {
#pragma unroll
              for (int e = 0; e < 4; ++e) b[e] &= ~cc_nonfinite(b[e]);
            }
            mma16816(o[2 * n2], pa, b[0], b[1]);
            mma16816(o[2 * n2 + 1], pa, b[2], b[3]);
          }
          if (odd) {
#pragma unroll 1
            for (int kk = 0; kk < 16 && key0 + 16 * kb + kk < r.L; ++kk) {
              // the lane with this key's weights for the same rows, and what the rows see
              const int from = (lane & ~3) | ((kk & 7) >> 1), bit = 16 * (kb & 1) + kk;
              const uint32_t see0 = __shfl_sync(0xffffffffu, see[kb >> 1][0], from) >> bit;
              const uint32_t see1 = __shfl_sync(0xffffffffu, see[kb >> 1][1], from) >> bit;
              const float w0 = __shfl_sync(0xffffffffu, kk < 8 ? ((kk & 1) ? pv[kb][0][1] : pv[kb][0][0])
                                                               : ((kk & 1) ? pv[kb][1][1] : pv[kb][1][0]), from);
              const float w1 = __shfl_sync(0xffffffffu, kk < 8 ? ((kk & 1) ? pv[kb][0][3] : pv[kb][0][2])
                                                               : ((kk & 1) ? pv[kb][1][3] : pv[kb][1][2]), from);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                uint32_t v;
                asm volatile("ld.shared.b32 %0, [%1];"
                             : "=r"(v)
                             : "r"(vt + cc_offset<W>(first + 16 * kb + kk, hw * (D / 8) + nt, pr) + 4 * (lane & 3))
                             : "memory");
                v &= cc_nonfinite(v);
                if (v == 0) continue;
                const float x = __uint_as_float(v << 16), y = __uint_as_float(v & 0xFFFF0000u);
                if (see0 & 1) {
                  if (x != 0.f) o[nt][0] += w0 * x;
                  if (y != 0.f) o[nt][1] += w0 * y;
                }
                if (see1 & 1) {
                  if (x != 0.f) o[nt][2] += w1 * x;
                  if (y != 0.f) o[nt][3] += w1 * y;
                }
              }
            }
          }
        }
      }
      // (a warp that gave up releases nothing: what it did not wait for may
      // still be on its way)
      if (!dead) mbar_arrive_warp(&sh->empty[st]);
    }

    // the item's end: the warps' O, maxima and sums meet in shared memory
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (ACT != 2) continue;
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if ((lane & 3) == 0) sh->ml[warp][(lane >> 2) + 8 * i] = make_float2(m[i], l[i]);
    }
    // O by chunks of 32 columns of every head: a warp's slot holds its 16 rows,
    // row g's column pair c at pair c ^ 4 (g % 4) (no bank conflicts); a thread
    // sums 4 columns of a row over the slots of each head in turn
    constexpr int kPerRow = kCChunk / 4;  // threads per row
    const int lr = tid / kPerRow, cc = (tid % kPerRow) * 4;
    const int g = lr & 15, w0 = (lr >> 4) * kCGroupWarps;
    const bool live = lr < n_rows;
    const int flat = w.row_tile * kRows + lr;
    const int t_out = static_cast<uint32_t>(flat) / static_cast<uint32_t>(p.group);
    const int64_t token = r.q0 + (live ? t_out : 0);
    const int head0 = w.h * HP * p.group + (live ? flat - t_out * p.group : 0);
    const int64_t part0 = (2 * static_cast<int64_t>(blockIdx.x) + w.slot()) * (HP * kRows) + lr;
    float* slot = reinterpret_cast<float*>(smem + C::kOOff + warp * C::kSlotBytes);
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += kCChunk) {
#pragma unroll
      for (int nt = 0; nt < kCChunk / 8; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int gr = (lane >> 2) + 8 * i, c2 = (4 * nt + (lane & 3)) ^ ((gr & 3) << 2);
          *reinterpret_cast<float2*>(slot + gr * kCChunk + 2 * c2) = make_float2(o[c0 / 8 + nt][2 * i], o[c0 / 8 + nt][2 * i + 1]);
        }
      named_bar(1, C::kWarps * 32);
#pragma unroll
      for (int hh = 0; hh < HP; ++hh) {
        if (!live) break;
        const int head = head0 + hh * p.group, from = w0 + hh * KG;
        const int64_t prow = part0 + hh * kRows;
        float inv = 1.f, f[KG];
#pragma unroll
        for (int i = 0; i < KG; ++i) f[i] = 1.f;
        if constexpr (ACT == 2) {
          float M = -INFINITY, L = 0.f;
#pragma unroll
          for (int i = 0; i < KG; ++i) M = fmaxf(M, sh->ml[from + i][g].x);
          const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
          for (int i = 0; i < KG; ++i) {
            f[i] = ex2_sfu(sh->ml[from + i][g].x - ref);
            L = __fmaf_rn(sh->ml[from + i][g].y, f[i], L);
          }
          if (w.whole) inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // no key seen: 0 (a NaN sum stays NaN)
          if (c0 == 0 && cc == 0) {
            if (!w.whole) p.part_ml[prow] = make_float2(M, L);
            else if (p.lse != nullptr)
              p.lse[static_cast<int64_t>(head) * p.total_q + token] = cc_lse(M, L);
          }
        }
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < KG; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(smem + C::kOOff + (from + i) * C::kSlotBytes +
                                                            (g * kCChunk + (cc ^ ((g & 3) << 3))) * 4);
          a.x = __fmaf_rn(v.x, f[i], a.x);
          a.y = __fmaf_rn(v.y, f[i], a.y);
          a.z = __fmaf_rn(v.z, f[i], a.z);
          a.w = __fmaf_rn(v.w, f[i], a.w);
        }
        if (w.whole)
          *reinterpret_cast<uint2*>(p.out + (token * p.heads + head) * D + c0 + cc) =
              make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
        else
          *reinterpret_cast<float4*>(p.part_o + prow * D + c0 + cc) = a;
      }
      named_bar(1, C::kWarps * 32);  // the slots are free again
    }
  }
}

template <int D, int ACT, int MT, int HP>
__global__ void __launch_bounds__((CcCfg<D * HP, MT, HP>::kThreads), (CcCfg<D * HP, MT, HP>::kCtas))
    cache_fwd_kernel(const __grid_constant__ CacheFwdParams p) {
  using C = CcCfg<D * HP, MT, HP>;
  static_assert(sizeof(CcShared<MT>) <= C::kSmemBytes - 1024 - C::kBarOff, "shared block");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  CcShared<MT>* sh = reinterpret_cast<CcShared<MT>*>(smem + C::kBarOff);
  cache_let_next();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], C::kWarps);
    }
    sh->abort = 0;
    fence_mbar_init();
  }
  cache_wait_before();
  if (threadIdx.x == 0) p.err[blockIdx.x] = kOk;
  const CacheRange R = cache_range<kCKeys>(p, &sh->range, kCMinRange);
  if (threadIdx.x == (C::kWarps - 1) * 32) cache_open<kCKeys>(p, R);
  Fail fail{&sh->abort, p.err + blockIdx.x, p.wait_limit_ns};
  if (threadIdx.x >= C::kWarps * 32) cc_producer<D * HP, MT, HP>(p, smem, sh, R, fail);
  else cc_consumer<D, ACT, MT, HP>(p, smem, sh, R, fail);
}

// ------------------------------------------------------------------ joining
// Joins the parts of the items that range borders cut, and the CTAs' status
// words.  Block (i, y): border i + 1, and of its item the rows (of which a head
// has at most tile_rows that live) 8 / SPLIT y and on.  SPLIT warps share a row's
// parts, every SPLIT-th each, then their sums in order: the same bits on every
// run.  Few rows meet with many parts (16-row tiles on a long request: SPLIT 4),
// many rows with few (128-row tiles: SPLIT 1).  Bound by latency:
// with cold caches 7 to 10 us after 16-row items, 9 to 13 after 128-row ones.
constexpr int kJoinWarps = 8;

template <int D, bool SOFTMAX, int SPLIT>
__global__ void __launch_bounds__(kJoinWarps * 32) cache_join_kernel(const __grid_constant__ CacheFwdParams p, int n_ctas,
                                                                     int tile_rows) {
  constexpr int V = D / 32, kRows = kJoinWarps / SPLIT;
  __shared__ int worst[kJoinWarps];
  __shared__ float sums[SPLIT > 1 ? kRows : 1][SPLIT][D];
  __shared__ float2 ml[kRows][SPLIT];
  cache_let_next();
  cache_wait_before();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    int e = kOk;
    for (int c = threadIdx.x; c < n_ctas; c += kJoinWarps * 32) e = max(e, p.err[c]);
    e = __reduce_max_sync(0xffffffffu, e);
    if (lane == 0) worst[warp] = e;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < kJoinWarps; ++i) e = max(e, worst[i]);
      *p.status = e;
    }
  }
  const int border = blockIdx.x + 1;
  if (border >= n_ctas) return;
  const CacheJoin j = p.join[border];
  if (!j.valid) return;
  const int R = p.rows_per_tile, part = warp % SPLIT;
  const int row = kRows * blockIdx.y + warp / SPLIT;
  const int hh = row / tile_rows, lr = row - hh * tile_rows;  // head of the item's, row of its tile
  int token_at, g;  // of the request, of the group
  if (p.tile_tokens) {  // 128-row tiles: head by head
    const int tile = p.tile_tokens * p.group, s = lr / tile, r = lr - s * tile;
    g = r / p.tile_tokens;
    token_at = j.rt * (R / p.group) + s * p.tile_tokens + r - g * p.tile_tokens;
  } else {  // token by token
    const int flat = j.rt * R + lr;
    token_at = flat / p.group;
    g = flat - token_at * p.group;
  }
  const bool live = hh < p.heads_per_item && token_at < j.T;
  auto row_of = [&](int c) {
    return (2 * static_cast<int64_t>(c) + (c == j.c0 ? 1 : 0)) * (p.heads_per_item * R) + hh * R + lr;
  };
  float M = -INFINITY, L = 0.f;
  float acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  if (live) {
    if constexpr (SOFTMAX) {
      for (int c = j.c0 + lane; c <= j.c1; c += 32) M = fmaxf(M, p.part_ml[row_of(c)].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    }
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
    for (int c = j.c0 + part; c <= j.c1; c += SPLIT) {
      const int64_t at = row_of(c);
      float f = 1.f;
      if constexpr (SOFTMAX) {
        const float2 x = p.part_ml[at];
        f = ex2_sfu(x.x - ref);
        L = __fmaf_rn(x.y, f, L);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = __fmaf_rn(p.part_o[at * D + lane * V + e], f, acc[e]);
    }
  }
  if constexpr (SPLIT > 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) sums[warp / SPLIT][part][lane * V + e] = acc[e];
    if (lane == 0) ml[warp / SPLIT][part] = make_float2(M, L);
    __syncthreads();
  }
  if (!live || part != 0) return;
#pragma unroll
  for (int i = 1; i < SPLIT; ++i) {
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] += sums[warp / SPLIT][i][lane * V + e];
    L += ml[warp / SPLIT][i].y;
  }
  const int64_t token = j.q0 + token_at;
  const int head = (j.h * p.heads_per_item + hh) * p.group + g;
  if constexpr (SOFTMAX) {
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= inv;
    if (lane == 0 && p.lse != nullptr)
      p.lse[static_cast<int64_t>(head) * p.total_q + token] = cc_lse(M, L);
  }
  __nv_bfloat16* dst = p.out + (token * p.heads + head) * D + lane * V;
  if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]));
  else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(dst) = pack_bf16(acc[0], acc[1]);
  else *dst = __float2bfloat16_rn(acc[0]);
}

// ------------------------------------------------------------------ launch
#ifndef JGDPA_HEAD_DIM
#error "compile cache_fwd.cu with -DJGDPA_HEAD_DIM=32, 64 or 128"
#endif

template <int D, int ACT, int MT, int HP>
static cudaError_t launch_cc(const CacheFwdParams& p, int grid, cudaStream_t stream) {
  using C = CcCfg<D * HP, MT, HP>;
  auto kern = cache_fwd_kernel<D, ACT, MT, HP>;
  static DeviceFlags attr_set = {};
  cudaError_t e = smem_attr_once(kern, C::kSmemBytes, attr_set);
  if (e != cudaSuccess) return e;
  return cache_launch(kern, dim3(grid), C::kThreads, C::kSmemBytes, stream, p);
}

template <int D, int ACT, int HP>
static cudaError_t launch_cc_rows(const CacheFwdParams& p, int grid, cudaStream_t stream) {
  if constexpr (cache_narrow_rows(D) > 16)
    if (p.rows_per_tile > 16) return launch_cc<D, ACT, 2, HP>(p, grid, stream);
  return launch_cc<D, ACT, 1, HP>(p, grid, stream);
}

template <int D, int ACT>
static cudaError_t launch_cc_act(const CacheFwdParams& p, int grid, cudaStream_t stream) {
  if constexpr (D < 128)
    if (p.heads_per_item > 1) return launch_cc_rows<D, ACT, 128 / D>(p, grid, stream);
  return launch_cc_rows<D, ACT, 1>(p, grid, stream);
}

template <int D>
cudaError_t launch_cache_fwd_d(const CacheFwdParams& p, int act, int grid, cudaStream_t stream) {
  if (act == 0) return launch_cc_act<D, 0>(p, grid, stream);
  if (act == 1) return launch_cc_act<D, 1>(p, grid, stream);
  return launch_cc_act<D, 2>(p, grid, stream);
}

template <int D, bool SOFTMAX>
static cudaError_t launch_join(const CacheFwdParams& p, int n_ctas, int tile_rows, cudaStream_t stream) {
  const int split = p.rows_per_tile <= 32 ? 4 : 1, rows = kJoinWarps / split;
  const dim3 grid(n_ctas > 1 ? n_ctas - 1 : 1, (p.heads_per_item * tile_rows + rows - 1) / rows, 1);
  return cache_launch(split == 4 ? cache_join_kernel<D, SOFTMAX, 4> : cache_join_kernel<D, SOFTMAX, 1>, grid,
                      kJoinWarps * 32, 0, stream, p, n_ctas, tile_rows);
}
template <int D>
cudaError_t launch_cache_join_d(const CacheFwdParams& p, int act, int n_ctas, int tile_rows, cudaStream_t stream) {
  return act == 2 ? launch_join<D, true>(p, n_ctas, tile_rows, stream) : launch_join<D, false>(p, n_ctas, tile_rows, stream);
}

template cudaError_t launch_cache_fwd_d<JGDPA_HEAD_DIM>(const CacheFwdParams&, int, int, cudaStream_t);
template cudaError_t launch_cache_join_d<JGDPA_HEAD_DIM>(const CacheFwdParams&, int, int, int, cudaStream_t);

}  // namespace jg
