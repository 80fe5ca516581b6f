// Attention over a paged key/value cache, few query rows per key/value head.
//
// One item is (request, key/value head, tile of 16 or 32 query rows); a row is
// (new token, query head of the group), so the heads that share a key/value
// head share its loads.  Its keys stream through shared memory once, in tiles
// of 64 tokens gathered from the pages by TMA.
//
//   S = Q K^T, P = act(S) or exp2(S - m), O += P V
//
// With R rows each K/V byte feeds R multiply-adds, so for R <= 32 the kernel is
// bound by HBM.  Rows of 16 are the m of mma.sync m16n8k16, whose fragments
// keep S, P and O in registers: no tensor-memory round trip and no block-wide
// step per tile.  (The 128-row tensor-memory form is cache_fwd_wide.cu.)  Each
// of four warps takes 16 of a tile's keys with its own running maximum, sum and
// O; they meet once per item.  With 32-row tiles a second group of four warps
// takes the second 16 rows of the same keys.
//
// A TMA producer runs up to 96 KB ahead, across items, and several CTAs share
// an SM, so that neither an item's end (the warps' exchange) nor its start
// stops the loads.
#include "act.cuh"
#include "cache.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace jg {

constexpr int kCKeys = 64;        // tokens per tile
constexpr int kCGroupWarps = 4;   // warps that share a tile's keys
constexpr int kCMinRange = 6;     // a range below this many tiles is not worth its own CTA
constexpr int kCChunk = 32;       // columns of O that meet at a time at an item's end

template <int D, int MT>
struct CcCfg {
  static constexpr int kWarps = kCGroupWarps * MT;  // consumer warps
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kBlockCols = D < 64 ? D : 64;
  static constexpr int kRowBytes = kBlockCols * 2;
  static constexpr int kTileBytes = kCKeys * D * 2;  // K or V of one tile
  // CTAs per SM and stages of K and V: 130 to 190 KB of loads in flight on an
  // SM (at d = 128, 64 KB reached 0.67 of the copy bandwidth on one long
  // request, 128 KB 0.82)
  static constexpr int kCtas = MT == 1 ? cache_ctas_narrow(D) : (D == 128 ? 1 : 2);
  static constexpr int kStages = MT == 1 ? (D == 128 ? 3 : D == 64 ? 4 : 5) : (D == 128 ? 6 : D == 64 ? 5 : 10);
  static constexpr int kSlotBytes = 16 * kCChunk * 4;  // one warp's chunk of O
  static constexpr int kOOff = kStages * 2 * kTileBytes;
  static constexpr int kBarOff = kOOff + kWarps * kSlotBytes;
  static constexpr int kSmemBytes = kBarOff + 2048 + 1024;
  static_assert(kSmemBytes <= 233472 / kCtas - 1024, "shared memory per CTA");
};

struct CcShared {
  uint64_t full[16], empty[16];
  float ml[2 * kCGroupWarps][16][2];
  CacheRangeShared range;
  int abort;
};
static_assert(sizeof(CcShared) <= 2048, "shared block");

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
template <int D>
__device__ __forceinline__ uint32_t cc_offset(int n, int c, int pr) {
  using C = CcCfg<D, 1>;
  const int r = n & (pr - 1);
  uint32_t off = (n - r) * (D * 2) + r * C::kRowBytes;
  if constexpr (C::kRowBytes == 128) {
    off += (c >> 3) * (pr * 128) + (((c & 7) ^ (r & 7)) << 4);
  } else {
    off += (c ^ ((r >> 1) & 3)) << 4;
  }
  return off;
}

// ------------------------------------------------------------- producer
template <int D, int MT>
__device__ void cc_producer(const CacheFwdParams& p, uint8_t* smem, CcShared* sh, const CacheRange& R, Fail fail) {
  using C = CcCfg<D, MT>;
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
      if (lane == 0) mbar_arrive_tx(&sh->full[st], 2 * n * pr * D * 2);
      __syncwarp();
      if (mine) {
        const uint32_t dst = base + st * 2 * C::kTileBytes + (lane & 1) * C::kTileBytes + (lane >> 1) * pr * D * 2;
        tma_load_5d(dst, (lane & 1) ? &p.tm_v : &p.tm_k, &sh->full[st], 0, key & ((1 << p.page_shift) - 1), 0, w.h,
                    page);
      }
      ++it;
    }
  }
  if (!ok) {  // let the copies already issued land before the CTA exits
    for (uint32_t i = it > C::kStages ? it - C::kStages : 0; i < it; ++i)
      mbar_wait_drain(&sh->full[i % C::kStages], (i / C::kStages) & 1);
  }
}

// ------------------------------------------------------------- consumers
template <int D, int ACT, int MT>
__device__ void cc_consumer(const CacheFwdParams& p, uint8_t* smem, CcShared* sh, const CacheRange& R, Fail fail) {
  using C = CcCfg<D, MT>;
  constexpr int KS = D / 16;  // k steps of S = Q K^T
  constexpr int NT = D / 8;   // n tiles of O
  constexpr int kRows = 16 * MT;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = warp / kCGroupWarps, kw = warp % kCGroupWarps;
  const int row0 = 16 * grp;
  const int pr = min(1 << p.page_shift, kCKeys);
  const uint32_t base = smem_u32(smem);
  // this warp's 16 keys: piece addresses for ldmatrix (the four 8x8 blocks of
  // a load are keys 0-7 / 8-15 by 16-byte piece for K, and transposed for V)
  const int kn = 16 * kw + (lane & 7) + ((lane & 16) ? 8 : 0), kc = (lane >> 3) & 1;
  const int vn = 16 * kw + (lane & 7) + ((lane & 8) ? 8 : 0), vc = lane >> 4;
  const int bias_reach = (p.bias_len - 1) / 2;
  uint32_t it = 0;
  bool dead = false;
  CacheWalk w;
  w.init(R);
  for (; w.template next<kCKeys>(p); w.advance()) {
    const CacheReq& r = w.r;
    int lo, hi;
    w.template tiles<kCKeys>(p, lo, hi);
    const int n_rows = min(static_cast<int64_t>(kRows), static_cast<int64_t>(r.T) * p.group -
                                                            static_cast<int64_t>(w.row_tile) * kRows);
    CcRow rows[2];
    const __nv_bfloat16* qrow[2];
    int pos_min = INT32_MAX;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int lr = row0 + (lane >> 2) + 8 * i;
      const int flat = w.row_tile * kRows + lr;
      CcRow& q = rows[i];
      q.t = lr < n_rows ? flat / p.group : -1;
      q.head = w.h * p.group + (lr < n_rows ? flat % p.group : 0);
      q.pos = r.C;
      q.far_bias = 0.f;
      qrow[i] = nullptr;
      if (q.t >= 0) {
        q.pos = r.C + (p.depth != nullptr ? __ldg(p.depth + r.q0 + q.t) : q.t);
        if (p.bias_len) q.far_bias = __ldg(p.bias + static_cast<int64_t>(q.head) * p.bias_len + 2 * bias_reach) * cc_bias_unit<ACT>();
        qrow[i] = p.q + static_cast<int64_t>(r.q0 + q.t) * p.q_stride + static_cast<int64_t>(q.head) * D;
        pos_min = min(pos_min, q.pos);
      }
    }
    pos_min = __reduce_min_sync(0xffffffffu, pos_min);
    const int pos_max = __reduce_max_sync(0xffffffffu, max(rows[0].t >= 0 ? rows[0].pos : 0, rows[1].t >= 0 ? rows[1].pos : 0));
    // Q fragments: rows lane / 4 (+ 8), columns 16 ks + 2 (lane % 4) (+ 8)
    uint32_t qa[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat16* src = qrow[e & 1];
        qa[ks][e] = src != nullptr
                        ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * (lane & 3) + ((e & 2) ? 8 : 0)))
                        : 0u;
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
      const int key0 = t * kCKeys + 16 * kw;  // this warp's first key
      if (!dead && key0 < r.L) {
        const uint32_t kb = base + st * 2 * C::kTileBytes, vb = kb + C::kTileBytes;
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t b[4];
          ldsm4(kb + cc_offset<D>(kn, 2 * ks + kc, pr), b);
          mma16816(s[0], qa[ks], b[0], b[1]);
          mma16816(s[1], qa[ks], b[2], b[3]);
        }
        // every key of these 16 is seen by every row, and R or more behind
        const int last = key0 + 15;
        const bool plain = last < r.C && (p.window <= 0 || pos_max - key0 < p.window);
        const bool far = p.bias_len == 0 || (last < r.C && pos_min - last >= bias_reach);
        float pv[2][4];
        uint32_t vis = 0;  // bit 4 i + e: that element's row sees its key (not kept on the plain path)
        if (plain && far) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][e] = __fmaf_rn(s[i][e], p.scale, rows[e >> 1].far_bias);
        } else {
          // (written without branches, so that the loads run side by side)
          const uint32_t see[2] = {cc_vis32(p, r, rows[0], key0), cc_vis32(p, r, rows[1], key0)};
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int col = 8 * i + 2 * (lane & 3) + c;
              const int key_pos = cc_pos(p, r, key0 + col);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const CcRow& q = rows[h];
                const bool sees = ((see[h] >> col) & 1) && cc_near(p, q.pos, key_pos);
                float bias = q.far_bias;
                if (!far) bias = cc_bias(p, q, bias_reach, key_pos) * cc_bias_unit<ACT>();
                const float x = __fmaf_rn(s[i][2 * h + c], p.scale, bias);
                s[i][2 * h + c] = sees ? x : (ACT == 2 ? -INFINITY : 0.f);  // act(0) = 0
                vis |= (sees ? 1u : 0u) << (4 * i + 2 * h + c);
              }
            }
        }
        if constexpr (ACT == 2) {
          float mx[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
          }
          if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float mn = fmaxf(m[i], mx[i]);
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
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              pv[i][e] = ex2_sfu(s[i][e] - ref[e >> 1]);
              l[e >> 1] += pv[i][e];
            }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) pv[i][e] = cc_act<ACT>(s[i][e]);
        }
        // P rounds to bf16 as the A operand (half a step, 2^-9 of each weight)
        uint32_t pa[4] = {pack_bf16(pv[0][0], pv[0][1]), pack_bf16(pv[0][2], pv[0][3]), pack_bf16(pv[1][0], pv[1][1]),
                          pack_bf16(pv[1][2], pv[1][3])};
        if (plain) {
#pragma unroll
          for (int n2 = 0; n2 < NT / 2; ++n2) {
            uint32_t b[4];
            ldsm4_t(vb + cc_offset<D>(vn, 2 * n2 + vc, pr), b);
            mma16816(o[2 * n2], pa, b[0], b[1]);
            mma16816(o[2 * n2 + 1], pa, b[2], b[3]);
          }
        } else {
          // Some rows do not see some of these keys, and 0 * NaN = NaN: rows
          // of V past the request's end (whatever the page held) count as
          // zeros, and infinities or NaN of the others are left out of the
          // product and added below to the rows that see them.
          uint32_t keep[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int j = key0 + 8 * i + 2 * (lane & 3);
            keep[i] = j + 1 < r.L ? 0xFFFFFFFFu : (j < r.L ? 0xFFFFu : 0u);
          }
          bool odd = false;
#pragma unroll
          for (int n2 = 0; n2 < NT / 2; ++n2) {
            uint32_t b[4];
            ldsm4_t(vb + cc_offset<D>(vn, 2 * n2 + vc, pr), b);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              b[e] &= keep[e & 1];
              const uint32_t bad = cc_nonfinite(b[e]);
              odd = odd || bad != 0;
              b[e] &= ~bad;
            }
            mma16816(o[2 * n2], pa, b[0], b[1]);
            mma16816(o[2 * n2 + 1], pa, b[2], b[3]);
          }
          if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
            for (int kk = 0; kk < 16 && key0 + kk < r.L; ++kk) {
              const int from = (lane & ~3) | ((kk & 7) >> 1);  // the lane with this key's weights for the same rows
              const uint32_t see = __shfl_sync(0xffffffffu, vis, from) >> (4 * (kk >> 3) + (kk & 1));
              const float w0 = __shfl_sync(0xffffffffu, kk < 8 ? ((kk & 1) ? pv[0][1] : pv[0][0])
                                                               : ((kk & 1) ? pv[1][1] : pv[1][0]), from);
              const float w1 = __shfl_sync(0xffffffffu, kk < 8 ? ((kk & 1) ? pv[0][3] : pv[0][2])
                                                               : ((kk & 1) ? pv[1][3] : pv[1][2]), from);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                uint32_t v;
                asm volatile("ld.shared.b32 %0, [%1];"
                             : "=r"(v)
                             : "r"(vb + cc_offset<D>(16 * kw + kk, nt, pr) + 4 * (lane & 3))
                             : "memory");
                v &= cc_nonfinite(v);
                if (v == 0) continue;
                const float x = __uint_as_float(v << 16), y = __uint_as_float(v & 0xFFFF0000u);
                if (see & 1) {
                  if (x != 0.f) o[nt][0] += w0 * x;
                  if (y != 0.f) o[nt][1] += w0 * y;
                }
                if (see & 4) {
                  if (x != 0.f) o[nt][2] += w1 * x;
                  if (y != 0.f) o[nt][3] += w1 * y;
                }
              }
            }
          }
        }
      }
      mbar_arrive_warp(&sh->empty[st]);
    }

    // the item's end: the warps' O, maxima and sums meet in shared memory
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (ACT == 2 && (lane & 3) == 0) {
        sh->ml[warp][(lane >> 2) + 8 * i][0] = m[i];
        sh->ml[warp][(lane >> 2) + 8 * i][1] = l[i];
      }
    }
    // O by chunks of 32 columns: a warp's slot holds its 16 rows, row g's
    // column pair c at pair c ^ 4 (g % 4) (no bank conflicts); a thread sums 4
    // columns of a row over the group's four slots
    constexpr int kPerRow = kCChunk / 4;  // threads per row
    const int lr = tid / kPerRow, cc = (tid % kPerRow) * 4;
    const int g = lr & 15, w0 = (lr >> 4) * kCGroupWarps;
    const bool live = lr < n_rows;
    const int flat = w.row_tile * kRows + lr;
    const int64_t token = r.q0 + (live ? flat / p.group : 0);
    const int head = w.h * p.group + (live ? flat % p.group : 0);
    const int64_t prow = (2 * static_cast<int64_t>(blockIdx.x) + (w.first ? 0 : 1)) * kRows + lr;
    float M = -INFINITY, L = 0.f, inv = 1.f, f[kCGroupWarps] = {1.f, 1.f, 1.f, 1.f};
    float* slot = reinterpret_cast<float*>(smem + C::kOOff + warp * C::kSlotBytes);
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += kCChunk) {
#pragma unroll
      for (int nt = 0; nt < kCChunk / 8; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int gr = (lane >> 2) + 8 * i, c2 = (4 * nt + (lane & 3)) ^ ((gr & 3) << 2);
          *reinterpret_cast<float2*>(slot + gr * kCChunk + 2 * c2) =
              make_float2(o[c0 / 8 + nt][2 * i], o[c0 / 8 + nt][2 * i + 1]);
        }
      named_bar(1, C::kWarps * 32);
      if (live) {
        if (ACT == 2 && c0 == 0) {
#pragma unroll
          for (int i = 0; i < kCGroupWarps; ++i) M = fmaxf(M, sh->ml[w0 + i][g][0]);
          const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
          for (int i = 0; i < kCGroupWarps; ++i) {
            f[i] = ex2_sfu(sh->ml[w0 + i][g][0] - ref);
            L = __fmaf_rn(sh->ml[w0 + i][g][1], f[i], L);
          }
          if (w.whole) inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // no key seen: 0 (a NaN sum stays NaN)
        }
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kCGroupWarps; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(smem + C::kOOff + (w0 + i) * C::kSlotBytes +
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
    if (ACT == 2 && live && cc == 0) {
      if (!w.whole) p.part_ml[prow] = make_float2(M, L);
      else if (p.lse != nullptr)
        p.lse[static_cast<int64_t>(head) * p.total_q + token] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
  }
}

template <int D, int ACT, int MT>
__global__ void __launch_bounds__((CcCfg<D, MT>::kThreads), (CcCfg<D, MT>::kCtas))
    cache_fwd_kernel(const __grid_constant__ CacheFwdParams p) {
  using C = CcCfg<D, MT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  CcShared* sh = reinterpret_cast<CcShared*>(smem + C::kBarOff);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], C::kWarps);
    }
    sh->abort = 0;
    p.err[blockIdx.x] = kOk;
    fence_mbar_init();
  }
  const CacheRange R = cache_range<kCKeys>(p, &sh->range, kCMinRange);  // (ends in a barrier)
  if (threadIdx.x == (C::kWarps - 1) * 32) cache_open<kCKeys>(p, R);
  Fail fail{&sh->abort, p.err + blockIdx.x, p.wait_limit_ns};
  if (threadIdx.x >= C::kWarps * 32) cc_producer<D, MT>(p, smem, sh, R, fail);
  else cc_consumer<D, ACT, MT>(p, smem, sh, R, fail);
}

// ------------------------------------------------------------------ joining
// Joins the parts of the items that range borders cut, in the order of the
// ranges (the same bits on every run), and the CTAs' status words.  Block
// (i, y): border i + 1, rows 4 y ..; one warp per row.
template <int D, bool SOFTMAX>
__global__ void __launch_bounds__(128) cache_join_kernel(const __grid_constant__ CacheFwdParams p, int n_ctas) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // every block waits: none may end before the attention has
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    int e = kOk;
    for (int c = threadIdx.x; c < n_ctas; c += 128) e = max(e, p.err[c]);
    __shared__ int worst[4];
    e = __reduce_max_sync(0xffffffffu, e);
    if (lane == 0) worst[warp] = e;
    __syncthreads();
    if (threadIdx.x == 0) *p.status = max(max(worst[0], worst[1]), max(worst[2], worst[3]));
  }
  const int border = blockIdx.x + 1;
  if (border >= n_ctas) return;
  const CacheJoin j = p.join[border];
  if (!j.valid) return;
  const int q0 = __ldg(p.q_off + j.b), T = __ldg(p.q_off + j.b + 1) - q0;
  const int R = p.rows_per_tile;
  const int64_t flat = static_cast<int64_t>(j.rt) * R + 4 * blockIdx.y + warp;
  if (4 * static_cast<int>(blockIdx.y) + warp >= R || flat >= static_cast<int64_t>(T) * p.group) return;
  const int lr = 4 * blockIdx.y + warp;
  // (the first range that holds one of its tiles, the last)
  const int c0 = static_cast<int>((j.t0 + p.item_cost) / j.per), c1 = static_cast<int>((j.t1 - 1) / j.per);
  // CTA c's part lies in its first slot when its range starts inside the item (or at its start)
  auto row_of = [&](int c) { return (2 * static_cast<int64_t>(c) + (c * j.per < j.t0 ? 1 : 0)) * R + lr; };
  float M = -INFINITY, L = 0.f;
  if constexpr (SOFTMAX) {
    for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, p.part_ml[row_of(c)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  }
  const float ref = M == -INFINITY ? 0.f : M;
  constexpr int V = D / 32;
  float acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const int64_t pr = row_of(c);
    float f = 1.f;
    if constexpr (SOFTMAX) {
      const float2 x = p.part_ml[pr];
      f = ex2_sfu(x.x - ref);
      L = __fmaf_rn(x.y, f, L);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = __fmaf_rn(p.part_o[pr * D + lane * V + e], f, acc[e]);
  }
  const int64_t token = q0 + flat / p.group;
  const int head = j.h * p.group + static_cast<int>(flat % p.group);
  if constexpr (SOFTMAX) {
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= inv;
    if (lane == 0 && p.lse != nullptr)
      p.lse[static_cast<int64_t>(head) * p.total_q + token] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
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

template <int D, int ACT, int MT>
static cudaError_t launch_cc(const CacheFwdParams& p, int grid, cudaStream_t stream) {
  auto kern = cache_fwd_kernel<D, ACT, MT>;
  constexpr int kSmem = CcCfg<D, MT>::kSmemBytes;
  static DeviceFlags attr_set = {};
  cudaError_t e = smem_attr_once(kern, kSmem, attr_set);
  if (e != cudaSuccess) return e;
  kern<<<grid, CcCfg<D, MT>::kThreads, kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_cache_fwd_d(const CacheFwdParams& p, int act, int grid, cudaStream_t stream) {
  if (p.rows_per_tile == 16) {
    if (act == 0) return launch_cc<D, 0, 1>(p, grid, stream);
    if (act == 1) return launch_cc<D, 1, 1>(p, grid, stream);
    return launch_cc<D, 2, 1>(p, grid, stream);
  }
  if (act == 0) return launch_cc<D, 0, 2>(p, grid, stream);
  if (act == 1) return launch_cc<D, 1, 2>(p, grid, stream);
  return launch_cc<D, 2, 2>(p, grid, stream);
}

// Launched so that its blocks may be set up while the attention still runs
// (programmatic dependent launch); they wait for its end before they read.
template <int D>
cudaError_t launch_cache_join_d(const CacheFwdParams& p, int act, int n_ctas, int max_rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_ctas > 1 ? n_ctas - 1 : 1, (max_rows + 3) / 4, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return act == 2 ? cudaLaunchKernelEx(&cfg, cache_join_kernel<D, true>, p, n_ctas)
                  : cudaLaunchKernelEx(&cfg, cache_join_kernel<D, false>, p, n_ctas);
}

template cudaError_t launch_cache_fwd_d<JGDPA_HEAD_DIM>(const CacheFwdParams&, int, int, cudaStream_t);
template cudaError_t launch_cache_join_d<JGDPA_HEAD_DIM>(const CacheFwdParams&, int, int, int, cudaStream_t);

}  // namespace jg
