// Attention over a paged key/value cache, many query rows per key/value head.
//
// One item is (request, key/value head, block of query rows); a row is (new
// token, query head of the group).  Tiles of 128 rows and 128 keys run on the
// tensor cores through tensor memory:
//
//   S = Q K^T (128 x 128), P = act(S) or exp2(S - m) as bf16 over S's columns,
//   O += P V (128 x d)
//
// The register form (cache_fwd.cu) would read the keys once for every 16 or 32
// rows and be bound by its matrix and special-function work; here a tile's two
// products take about 1,500 cycles at d = 128 (110 per 128 x 128 x 16 with both
// operands in shared memory, 80 with P in tensor memory) against the 2,700 in
// which HBM delivers its K and V, so up to 128 rows the kernel is bound by HBM
// and above by the products.
//
// Two streams, each with its S, O and a warpgroup of activation threads, keep
// the tensor core fed: while one stream's S is turned into P, the other's
// products run.  A part with more than 128 rows gives each stream its own rows
// and uses every K and V tile twice (half the shared-memory fills and L2 reads
// per product); a part with fewer gives both streams the same rows and every
// other key tile, and joins their O, maxima and sums at its end.
//
// Warps: 0 TMA producer, 1 MMA issuer (owns tensor memory), 2-3 the masked
// tiles' V, 4-7 and 8-11 the streams' activation and epilogue (one row per
// thread).
// TMEM: S_s at 128 s, O_s at 256 + 128 s.
//
// Measured, d = 128: 64 requests of 4,100 tokens, 8 key/value heads, 64 rows: 187
// us, 0.87 of the copy bandwidth; 32 trees of 8 to 33 tokens, 32 to 132 rows, over
// 177 to 13,900 tokens: 74 to 77 us, 0.60 (the items' starts and ends); 64 trees of
// 64 tokens, 512 rows, GELU with a bias over 134 to 8,066 tokens: 322 us, 0.46 of
// the products at cuBLAS's burst rate (284 with the packed kernels' GELU, which is
// not right far below zero, see cc_act2).  At d = 64 the same 64 requests take 112
// to 115 us (softmax; GELU 141, SiLU 149), at d = 32 (16 heads) 185 to 194 (258,
// 271) where the bytes take 80: the way of a tile's 128 x 128 weights from S to P no
// longer hides behind half or a quarter of the bytes.
#include "act.cuh"
#include "cache.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace jg {

constexpr int kWideMinRange = 12;  // the least length of a range
constexpr int kWideThreads = 384;

// PAIR: items of more than 128 rows.
template <int D, bool PAIR>
struct CwCfg {
  static constexpr int kBlockCols = D < 64 ? D : 64;
  static constexpr int kRowBytes = kBlockCols * 2;
  static constexpr int kBlockBytes = kTile * kRowBytes;  // 128 rows of one column block
  static constexpr int kBlocks = D / kBlockCols;
  static constexpr int kTileBytes = kTile * D * 2;
  // K and V go through one ring of `kStages` tiles in the order K0 K1 V0 K2 V1
  // ..: a V is not needed before its P, more than a tile's time after its K, and
  // would only hold its stage meanwhile
  static constexpr int kSlots = PAIR ? 2 : 1;  // Q tiles
  static constexpr int kStages = D == 128 ? 7 - kSlots : (D == 64 ? 14 - kSlots : 16);
  static constexpr uint32_t kSwizzle = kRowBytes == 128 ? 2u : 4u;
  static constexpr int kSBO = 8 * kRowBytes;
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = kQOff + kSlots * kTileBytes;
  static constexpr int kBarOff = kRingOff + kStages * kTileBytes;
  static constexpr int kSmemBytes = kBarOff + 2048 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  // Ring entries of the CTA's tile `it`.  (The K entry before the very last V
  // is skipped; the ring does not come round to it.)
  static __device__ __forceinline__ uint32_t entry_k(uint32_t it) { return it == 0 ? 0 : 2 * it - 1; }
  static __device__ __forceinline__ uint32_t entry_v(uint32_t it) { return 2 * it + 2; }
  static __device__ __forceinline__ int stage(uint32_t entry) { return entry % kStages; }
  static __device__ __forceinline__ uint32_t parity(uint32_t entry) { return (entry / kStages) & 1; }
};

struct CwShared {
  uint64_t q_full[2], q_empty[2];
  uint64_t full[16], empty[16];
  // The CTA's n-th masked tile, at n % 2: asked for when its S is issued, its V
  // safe.  (Each stream has at most one tile whose S is issued and P V is not.)
  uint64_t fix_ask[2], fixed[2];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t o_empty, drain;
  CacheRangeShared range;
  uint32_t tmem_base;
  int abort;
  int hides;         // softmax with a bias table: 1, or 2 where an entry of -inf hides all far keys of some head
  int odd[16];       // number of the last part (mod 16) whose masked tiles hold a V that is not finite
  float2 ml[kTile];  // the streams' maxima and sums at the end of a part that they share
};
static_assert(sizeof(CwShared) <= 2048, "shared block");

// What every role works out about a part.
struct CwPart {
  int lo, n;        // key tiles [lo, lo + n)
  int first_token;  // of the part's rows
  int tokens;       // of them
  bool pair;        // two tiles of rows; otherwise one
  int plain_lo, plain_hi;  // tiles in which every row sees every key, whatever the bias table's entries
  int far_hi;              // tiles below it are plain in the bias: R or more behind every row

  __device__ __forceinline__ CwPart() {}
  // (whole warp)
  __device__ __forceinline__ CwPart(const CacheFwdParams& p, const CacheWalk& w, int hides) {
    int hi;
    w.tiles<kTile>(p, lo, hi);
    n = hi - lo;
    const int most = p.rows_per_tile / p.group;
    first_token = w.row_tile * most;
    tokens = min(most, w.r.T - first_token);
    pair = tokens > p.tile_tokens;
    const int C = w.r.C, last_token = first_token + tokens - 1;
    plain_lo = 0;
    plain_hi = (p.window <= 0 && p.mask == nullptr ? min(w.r.L, C + first_token + 1) : C) / kTile;
    if (p.window > 0) {
      int depth = last_token;  // the rows' largest
      if (p.depth != nullptr) {
        depth = 0;
        for (int t = first_token + (threadIdx.x & 31); t <= last_token; t += 32) depth = max(depth, __ldg(p.depth + w.r.q0 + t));
        depth = __reduce_max_sync(0xffffffffu, depth);
      }
      const int64_t behind = static_cast<int64_t>(C) + depth - p.window;  // keys up to here are out of some row's window
      if (behind >= 0) plain_lo = static_cast<int>(min(behind / kTile + 1, static_cast<int64_t>(INT32_MAX)));
    }
    const int reach = max((p.bias_len - 1) / 2, 1);
    far_hi = p.bias_len == 0 ? INT32_MAX : (C >= reach ? (C - reach + 1) / kTile : 0);
    // (a softmax bias may hide near keys: only the table's entries say which)
    if (hides > 0) plain_hi = hides > 1 ? 0 : min(plain_hi, far_hi);
  }
  __device__ __forceinline__ bool plain(int tile) const { return tile >= plain_lo && tile < plain_hi; }
  // The tiles of stream s, and the one it takes as its i-th.
  __device__ __forceinline__ int count(int s) const { return pair ? n : (n + 1 - s) / 2; }
  __device__ __forceinline__ int at(int s, int i) const { return pair ? i : 2 * i + s; }
};

// ------------------------------------------------------------- producer
template <int D, bool PAIR>
struct CwProducer {
  using C = CwCfg<D, PAIR>;
  const CacheFwdParams& p;
  uint8_t* smem;
  CwShared* sh;
  Fail fail;
  uint32_t q_n = 0;          // Q loads issued
  uint32_t it = 0;           // tiles taken
  uint32_t entries = 0;      // ring entries issued, or one more (the skipped one)
  // the last tile, whose V is to come
  struct {
    int h, y, page;
    uint32_t bytes;
    bool mine;
  } held;

  // Rows of the tile from `token` on into the next Q slot (whole warp).
  __device__ __forceinline__ bool query(const CacheWalk& w, int token) {
    const int slot = q_n % C::kSlots;
    if (!mbar_wait_warp(&sh->q_empty[slot], ((q_n / C::kSlots) & 1) ^ 1, fail)) return false;
    if ((threadIdx.x & 31) == 0) {
      mbar_arrive_tx(&sh->q_full[slot], p.tile_tokens * p.group * D * 2);
#pragma unroll
      for (int b = 0; b < C::kBlocks; ++b)
        tma_load_3d(smem + C::kQOff + slot * C::kTileBytes + b * C::kBlockBytes, &p.tm_q, &sh->q_full[slot],
                    b * C::kBlockCols, w.r.q0 + token, w.h * p.group);
    }
    __syncwarp();
    ++q_n;
    return true;
  }
  // Lane: piece lane % 8 (min(page size, 128) tokens) of column block lane / 8.
  __device__ __forceinline__ bool load(uint32_t entry, const CUtensorMap* map, bool mine, uint32_t bytes, int y, int h,
                                       int page) {
    const int lane = threadIdx.x & 31, piece = lane & 7, cb = lane >> 3, st = C::stage(entry);
    if (!mbar_wait_warp(&sh->empty[st], C::parity(entry) ^ 1, fail)) return false;
    if (lane == 0) mbar_arrive_tx(&sh->full[st], bytes);
    __syncwarp();
    if (mine)
      tma_load_5d(smem_u32(smem) + C::kRingOff + st * C::kTileBytes + cb * C::kBlockBytes +
                      piece * min(1 << p.page_shift, kTile) * C::kRowBytes,
                  map, &sh->full[st], 0, y, cb, h, page);
    entries = entry + 1;
    return true;
  }
  // K of the next tile, then V of the tile before.
  __device__ __forceinline__ bool tile(const CacheWalk& w, int t) {
    const int lane = threadIdx.x & 31, piece = lane & 7;
    const int pr = min(1 << p.page_shift, kTile), pieces = kTile / pr;  // pieces: 1, 2, 4 or 8
    const int key = t * kTile + piece * pr, y = key & ((1 << p.page_shift) - 1);
    const bool mine = (lane >> 3) < C::kBlocks && piece < pieces && key < w.r.L;
    int page = p.num_pages;
    if (mine) {
      page = __ldg(p.table + static_cast<int64_t>(w.b) * p.width + (key >> p.page_shift));
      if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) {
        atomicCAS(fail.status, kOk, kErrBadPage);
        page = p.num_pages;  // outside the map: the copy writes zeros and reads nothing
      }
    }
    const uint32_t bytes = min(pieces, (w.r.L - t * kTile + pr - 1) / pr) * pr * D * 2;
    if (!load(C::entry_k(it), &p.tm_k, mine, bytes, y, w.h, page) || !value()) return false;
    held = {w.h, y, page, bytes, mine};
    ++it;
    return true;
  }
  // V of the last tile taken, if any.
  __device__ __forceinline__ bool value() {
    return it == 0 || load(C::entry_v(it - 1), &p.tm_v, held.mine, held.bytes, held.y, held.h, held.page);
  }
  // The copies issued land before the CTA exits, also when the others gave up.
  __device__ void drain() {
    for (uint32_t i = q_n > C::kSlots ? q_n - C::kSlots : 0; i < q_n; ++i)
      mbar_wait_drain(&sh->q_full[i % C::kSlots], (i / C::kSlots) & 1);
    for (uint32_t e = entries > C::kStages ? entries - C::kStages : 0; e < entries; ++e)
      if (e != C::entry_k(it) || entries <= e + 1)  // (the skipped one has the last V behind it)
        mbar_wait_drain(&sh->full[C::stage(e)], C::parity(e));
  }
};

template <int D, bool PAIR>
__device__ void cw_producer(const CacheFwdParams& p, uint8_t* smem, CwShared* sh, const CacheRange& R, Fail fail) {
  CwProducer<D, PAIR> load{p, smem, sh, fail};
  bool ok = true;
  CacheWalk w;
  w.init(R);
  for (; ok && w.next<kTile>(p); w.advance()) {
    const CwPart part(p, w, sh->hides);
    if (part.n == 0) continue;
    ok = load.query(w, part.first_token);
    if (PAIR && part.pair && ok) ok = load.query(w, part.first_token + p.tile_tokens);
    for (int t = part.lo; t < part.lo + part.n && ok; ++t) ok = load.tile(w, t);
  }
  if (ok) load.value();
  load.drain();
}

// ------------------------------------------------------------- MMA issuer
template <int D>
__device__ __forceinline__ void cw_issue_qk(uint32_t t_s, uint32_t q_addr, uint32_t k_addr, bool leader) {
  using C = CwCfg<D, false>;  // (the layouts are the same)
  constexpr uint32_t idesc = idesc_bf16(kTile, kTile, 0, 0);
  const uint64_t a0 = sdesc(q_addr, 16, C::kSBO, C::kSwizzle), b0 = sdesc(k_addr, 16, C::kSBO, C::kSwizzle);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t off = static_cast<uint64_t>((kk * 16 / C::kBlockCols) * C::kBlockBytes + (kk * 16 % C::kBlockCols) * 2) >> 4;
    if (leader) mma_ss(t_s, a0 + off, b0 + off, idesc, kk > 0 ? 1u : 0u);
  }
}
template <int D>
__device__ __forceinline__ void cw_issue_pv(uint32_t t_o, uint32_t t_p, uint32_t v_addr, bool accumulate, bool leader) {
  using C = CwCfg<D, false>;
  constexpr uint32_t idesc = idesc_bf16(kTile, D, 0, 1);  // V is MN-major
  const uint64_t b0 = sdesc(v_addr, C::kBlockBytes, C::kSBO, C::kSwizzle);
#pragma unroll
  for (int kk = 0; kk < kTile / 16; ++kk) {
    const uint64_t off = static_cast<uint64_t>(kk * 16 * C::kRowBytes) >> 4;
    if (leader) mma_ts(t_o, t_p + kk * 8, b0 + off, idesc, (accumulate || kk > 0) ? 1u : 0u);
  }
}

// Per pair of tiles: O_0 += P_0 V, S_0 of the stream's next tile, O_1 += P_1 V,
// S_1 of its next.  A stream's S overwrites the columns of its P; it is issued
// after the product that reads them, and MMAs execute in issue order.  For the
// same reason a stream's S being complete says that its O is, too.
template <int D, bool PAIR>
struct CwIssuer {
  using C = CwCfg<D, PAIR>;
  CwShared* sh;
  uint32_t tmem, q_base, ring;
  bool leader;
  Fail fail;
  uint32_t p_n[2] = {0, 0};
  uint32_t asked = 0, fixed = 0;  // masked tiles

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) { return mbar_wait_warp(bar, parity, fail); }
  __device__ __forceinline__ void commit(uint64_t* bar) {
    if (leader) mma_commit(bar);
  }
  // S of stream s from a Q slot and the K of tile `it`; `masked`: has its V made safe meanwhile.
  __device__ __forceinline__ bool issue_s(int s, int slot, uint32_t it, bool masked) {
    const uint32_t e = C::entry_k(it);
    if (!wait(&sh->full[C::stage(e)], C::parity(e))) return false;
    tc_fence_after();
    cw_issue_qk<D>(tmem + 128 * s, q_base + slot * C::kTileBytes, ring + C::stage(e) * C::kTileBytes, leader);
    commit(&sh->s_full[s]);
    if (masked) {
      if (leader) mbar_arrive(&sh->fix_ask[asked & 1]);
      ++asked;
    }
    return true;
  }
  // O of stream s from its P and the V of tile `it`.
  __device__ __forceinline__ bool issue_o(int s, uint32_t it, bool first, bool masked) {
    const uint32_t e = C::entry_v(it);
    if (!wait(&sh->full[C::stage(e)], C::parity(e)) || !wait(&sh->p_full[s], p_n[s] & 1)) return false;
    ++p_n[s];
    if (masked) {
      if (!wait(&sh->fixed[fixed & 1], (fixed >> 1) & 1)) return false;
      ++fixed;
    }
    tc_fence_after();
    cw_issue_pv<D>(tmem + 256 + 128 * s, tmem + 128 * s, ring + C::stage(e) * C::kTileBytes, !first, leader);
    return true;
  }
  __device__ __forceinline__ void free_k(uint32_t it) { commit(&sh->empty[C::stage(C::entry_k(it))]); }
  __device__ __forceinline__ void free_v(uint32_t it) { commit(&sh->empty[C::stage(C::entry_v(it))]); }
};

template <int D, bool PAIR>
__device__ void cw_mma(const CacheFwdParams& p, uint8_t* smem, CwShared* sh, uint32_t tmem, const CacheRange& R,
                       Fail fail) {
  using C = CwCfg<D, PAIR>;
  CwIssuer<D, PAIR> mma{sh, tmem, smem_u32(smem + C::kQOff), smem_u32(smem + C::kRingOff), elect_one(), fail};
  bool ok = true;
  uint32_t q_n = 0, it0 = 0, o_n = 0;
  CacheWalk w;
  w.init(R);
  for (; ok && w.next<kTile>(p); w.advance()) {
    const CwPart part(p, w, sh->hides);
    if (part.n == 0) continue;
    const bool pair = PAIR && part.pair;
    const int slot[2] = {static_cast<int>(q_n % C::kSlots), static_cast<int>(pair ? (q_n + 1) % C::kSlots : q_n % C::kSlots)};
    for (int s = 0; s < (pair ? 2 : 1) && ok; ++s, ++q_n)
      ok = mma.wait(&sh->q_full[q_n % C::kSlots], (q_n / C::kSlots) & 1);
    // (a pair has a masked V made safe once)
    auto masked = [&](int s, int t) { return (!pair || s == 0) && !part.plain(part.lo + t); };
    // S of stream s's i-th tile; frees what no later product of the part reads
    auto part_s = [&](int s, int i) -> bool {
      const int t = part.at(s, i);
      if (!mma.issue_s(s, slot[s], it0 + t, masked(s, t))) return false;
      if (!pair || s == 1) mma.free_k(it0 + t);
      if (t == part.n - 1) mma.commit(&sh->q_empty[slot[s]]);
      return true;
    };
    if (ok) ok = part_s(0, 0);
    if (ok && part.count(1) > 0) ok = part_s(1, 0);
    if (ok) ok = mma.wait(&sh->o_empty, (o_n & 1) ^ 1);  // the part before has read its O
    ++o_n;
    for (int i = 0; i < part.count(0) && ok; ++i) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (!ok || i >= part.count(s)) continue;
        const int t = part.at(s, i);
        if (!(ok = mma.issue_o(s, it0 + t, i == 0, masked(s, t)))) continue;
        if (!pair || s == 1) mma.free_v(it0 + t);
        if (i == part.count(s) - 1) mma.commit(&sh->o_full[s]);
        if (i + 1 < part.count(s)) ok = part_s(s, i + 1);
      }
    }
    it0 += part.n;
  }
  mma.commit(&sh->drain);
  mbar_wait_drain(&sh->drain, 0);
}

// ------------------------------------------------------ activation warps
// The code of a tile is kept small, in loops over 32 columns: most of it runs a
// few times per item, and instructions fetched for the first time cost more
// than the work (a fully unrolled tile took 2.1 us on its first run, 0.9 after).

// What a row needs to know of a tile's 128 keys, fetched before S is waited for:
// which of them it sees (bit c of see[k]: key0 + 32 k + c), and in lane c the
// positions of the keys key0 + 32 k + c (pos[k]; where the bias varies only).
struct CwNear {
  uint32_t see[4];
  int pos[4];
};
static __device__ __noinline__ CwNear cw_near(const CacheFwdParams& p, CacheReq r, CcRow q, bool plain, int key0) {
  CwNear t;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 4; ++k) t.pos[k] = cc_pos(p, r, key0 + 32 * k + lane);
#pragma unroll
  for (int k = 0; k < 4; ++k) t.see[k] = plain ? 0xFFFFFFFFu : cc_vis32(p, r, q, key0 + 32 * k);
  if (p.window > 0 && !plain) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t near = 0;
      if (cc_in_order(p, r, key0 + 32 * k)) {
        near = cc_near32(p, q.pos, key0 + 32 * k);
      } else {
#pragma unroll 4
        for (int c = 0; c < 32; ++c) near |= (cc_near(p, q.pos, __shfl_sync(0xffffffffu, t.pos[k], c)) ? 1u : 0u) << c;
      }
      t.see[k] &= near;
    }
  }
  return t;
}

// 32 scores of a row, formed with biases of which some are beyond kHugeBias, put
// right in place (`see`: the keys that length, mask and window let it see).
static __device__ __noinline__ void cw_huge_biases(const float* bias_row, int reach, int row_pos, int pos, uint32_t see,
                                                   uint32_t t_s) {
  uint32_t v[32];
  tmem_st_wait();
  tmem_ld32(t_s, v);
  tmem_ld_wait(v);
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    const float b = __ldg(bias_row + min(max(row_pos - __shfl_sync(0xffffffffu, pos, c), -reach), reach));
    const float x = __uint_as_float(v[c]);
    if (((see >> c) & 1) && fabsf(b) > kHugeBias && (b == -INFINITY || x == x))
      v[c] = b == -INFINITY ? 0xFF800000u : __float_as_uint(cc_huge(b));
  }
  tmem_st32(t_s, v);
}

// S -> s S + bias (in log2 units for softmax) in place, for the tiles near the
// new tokens, where the bias varies from key to key or some rows do not see
// some keys (-inf for softmax, else 0, as act(0) = 0).
template <int ACT>
__device__ __noinline__ void cw_near_tile(const CacheFwdParams& p, int C, CcRow q, CwNear t, int key0, uint32_t t_s) {
  const int reach = (p.bias_len - 1) / 2;
  const float* bias_row = p.bias + static_cast<int64_t>(q.head) * p.bias_len + reach;
  const bool huge = ACT == 2 && __any_sync(0xffffffffu, fabsf(q.far_bias) > kHugeScore);
#pragma unroll 1
  for (int c0 = 0; c0 < kTile; c0 += 32) {
    uint32_t v[32];
    tmem_ld32(t_s + c0, v);
    // keys R or more behind every new token: one bias for all
    const bool far = p.bias_len == 0 || (!huge && key0 + c0 + 31 <= C - max(reach, 1));
    float top = 0.f;
    if (far) {
      tmem_ld_wait(v);
#pragma unroll
      for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__fmaf_rn(__uint_as_float(v[c]), p.scale, q.far_bias));
    } else {
      float bias[32];
#pragma unroll
      for (int c = 0; c < 32; ++c)
        bias[c] = __ldg(bias_row + min(max(q.pos - __shfl_sync(0xffffffffu, t.pos[0], c), -reach), reach));
      tmem_ld_wait(v);
#pragma unroll
      for (int c = 0; c < 32; ++c)
        v[c] = __float_as_uint(__fmaf_rn(__uint_as_float(v[c]), p.scale, bias[c] * cc_bias_unit<ACT>()));
      if constexpr (ACT == 2) {
#pragma unroll
        for (int c = 0; c < 32; ++c) top = fmaxf(top, fabsf(bias[c]));
      }
    }
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (!((t.see[0] >> c) & 1)) v[c] = ACT == 2 ? 0xFF800000u : 0u;
    tmem_st32(t_s + c0, v);
    if (ACT == 2 && __any_sync(0xffffffffu, top > kHugeBias))
      cw_huge_biases(bias_row, reach, q.pos, t.pos[0], t.see[0], t_s + c0);
#pragma unroll
    for (int k = 0; k < 3; ++k) {  // the next chunk's words come to the front
      t.see[k] = t.see[k + 1];
      t.pos[k] = t.pos[k + 1];
    }
  }
  tmem_st_wait();
}

// P = act(s S + bias) over S's columns, two elements per packed instruction.
template <int ACT>
__device__ __forceinline__ void cw_act_tile(uint32_t t_s, float scale, float bias) {
  const float2 hs = f2(0.5f * scale), hb = f2(0.5f * bias);
#pragma unroll 1
  for (int q = 0; q < 4; q += 2) {
    uint32_t a[32], b[32];
    tmem_ld32(t_s + 32 * q, a);
    tmem_ld32(t_s + 32 * q + 32, b);
    tmem_ld_wait2(a, b);
    uint32_t pk[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const uint32_t(&v)[32] = c < 16 ? a : b;
      const float2 hx = __ffma2_rn(make_float2(__uint_as_float(v[2 * (c % 16)]), __uint_as_float(v[2 * (c % 16) + 1])), hs, hb);
      const float2 y = cc_act2<ACT>(hx);
      pk[c] = pack_bf16(y.x, y.y);
    }
    tmem_st32(t_s + 16 * q, pk);  // columns [16 q, 16 q + 32) are read already
  }
}

// P = 2^(x - m) with a running maximum that moves only when it grows by more
// than 8 (P stays below 2^8, O and l in fp32): O is rescaled then.  At d < 128,
// where HBM does not hide a second pass over S, most tiles do without a look at
// their maximum: the weights by the m so far add up to no more than 2^8, so none
// is above it (64 requests of 4,100 tokens, 64 rows: 121 -> 114 us at d = 64, 211
// -> 192 at d = 32; at d = 128 it would change nothing there, 453 -> 441 at 512
// rows, but 209 -> 217 on short trees, whose few tiles have more to fetch).
template <int D>
__device__ __forceinline__ void cw_softmax_tile(uint32_t t_s, uint32_t t_o, float scale, float bias, bool live, bool first,
                                                float& m, float& l) {
  constexpr bool kTry = D < 128;
  if (kTry && !__any_sync(0xffffffffu, live && m == -INFINITY)) {
    const float2 off = f2(bias - m);
    float2 sum = f2(0.f);
    uint32_t pk[64];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t a[32];
      tmem_ld32(t_s + 32 * q, a);
      tmem_ld_wait(a);
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float2 z = __ffma2_rn(make_float2(__uint_as_float(a[2 * c]), __uint_as_float(a[2 * c + 1])), f2(scale), off);
        const float2 e = make_float2(ex2_sfu(z.x), ex2_sfu(z.y));
        sum = __fadd2_rn(sum, e);
        pk[16 * q + c] = pack_bf16(e.x, e.y);
      }
    }
    const float total = sum.x + sum.y;
    if (!__any_sync(0xffffffffu, live && !(total <= 256.f))) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t x[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = pk[32 * q + c];
        tmem_st32(t_s + 32 * q, x);
      }
      l += total;
      return;
    }
  }
  float mx = -INFINITY;
#pragma unroll 1
  for (int q = 0; q < 4; q += 2) {
    uint32_t a[32], b[32];
    tmem_ld32(t_s + 32 * q, a);
    tmem_ld32(t_s + 32 * q + 32, b);
    tmem_ld_wait2(a, b);
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      const float2 x = __ffma2_rn(make_float2(__uint_as_float(a[c]), __uint_as_float(a[c + 1])), f2(scale), f2(bias));
      const float2 y = __ffma2_rn(make_float2(__uint_as_float(b[c]), __uint_as_float(b[c + 1])), f2(scale), f2(bias));
      mx = fmaxf(fmaxf(mx, fmaxf(x.x, x.y)), fmaxf(y.x, y.y));
    }
  }
  const bool grow = mx > m + (kTry ? 1.0f : 8.0f);  // (128 weights of up to 2 pass the test above)
  const float factor = grow ? ex2_sfu(m - mx) : 1.0f;  // 0 on the first tile
  if (grow) m = mx;
  l *= factor;
  // x - m, with m = 0 while no key was seen: then every x is -inf and P is 0
  const float2 off = f2(m == -INFINITY ? bias : bias - m);
  float2 sum = f2(0.f);
#pragma unroll 1
  for (int q = 0; q < 4; q += 2) {
    uint32_t a[32], b[32];
    tmem_ld32(t_s + 32 * q, a);
    tmem_ld32(t_s + 32 * q + 32, b);
    tmem_ld_wait2(a, b);
    uint32_t pk[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const uint32_t(&v)[32] = c < 16 ? a : b;
      const float2 z = __ffma2_rn(make_float2(__uint_as_float(v[2 * (c % 16)]), __uint_as_float(v[2 * (c % 16) + 1])), f2(scale), off);
      const float2 e = make_float2(ex2_sfu(z.x), ex2_sfu(z.y));
      sum = __fadd2_rn(sum, e);
      pk[c] = pack_bf16(e.x, e.y);
    }
    tmem_st32(t_s + 16 * q, pk);  // columns [16 q, 16 q + 32) are read already
  }
  l += sum.x + sum.y;
  if (!first && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
      uint32_t o[32];
      tmem_ld32(t_o + c0, o);
      tmem_ld_wait(o);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
      tmem_st32(t_o + c0, o);
    }
  }
}

// Adds what the product left out: infinities and NaN in V of keys in the
// part's masked tiles, for a row that sees them, to columns [c0, c0 + n) of the
// row's result (bf16 `out` or fp32 `part`), which this thread has written.
// Rare, so it works from global memory.
template <int D, int ACT>
__device__ __noinline__ void cw_add_odd(const CacheFwdParams& p, CacheWalk w, CwPart part, CcRow q, int c0,
                                        int n, __nv_bfloat16* out, float* part_o) {
  const CacheReq& r = w.r;
  const int32_t* pages = p.table + static_cast<int64_t>(w.b) * p.width;
  for (int t = part.lo; t < part.lo + part.n; ++t) {
    if (part.plain(t)) continue;
    for (int key = t * kTile; key < min(r.L, (t + 1) * kTile); ++key) {
      const int page = __ldg(pages + (key >> p.page_shift));
      if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages)) continue;
      const int key_pos = cc_pos(p, r, key);
      if (!(cc_vis32(p, r, q, key) & 1) || !cc_near(p, q.pos, key_pos)) continue;
      if (ACT == 2 && p.bias_len && cc_bias(p, q, (p.bias_len - 1) / 2, key_pos) == -INFINITY) continue;
      const int64_t place = static_cast<int64_t>(key & ((1 << p.page_shift) - 1)) * p.kv_heads * D + w.h * D;
      const __nv_bfloat16* v = p.v_cache + page * p.v_page_stride + place;
      bool any = false;
      for (int c = 0; c < n; ++c) any = any || !isfinite(__bfloat162float(v[c0 + c]));
      if (!any) continue;
      float weight = 1.f;  // softmax weights are positive
      if constexpr (ACT != 2) {
        const __nv_bfloat16* k = p.k_cache + page * p.k_page_stride + place;
        const __nv_bfloat16* qr = p.q + static_cast<int64_t>(r.q0 + q.t) * p.q_stride + static_cast<int64_t>(q.head) * D;
        float x = 0.f;
        for (int c = 0; c < D; ++c) x = __fmaf_rn(__bfloat162float(k[c]), __bfloat162float(qr[c]), x);
        x *= p.scale;
        if (p.bias_len) x += cc_bias(p, q, (p.bias_len - 1) / 2, key_pos);
        weight = cc_act<ACT>(x);
      }
      for (int c = 0; c < n; ++c) {
        const float x = __bfloat162float(v[c0 + c]);
        if (isfinite(x)) continue;
        if (out != nullptr) out[c0 + c] = __float2bfloat16_rn(__bfloat162float(out[c0 + c]) + weight * x);
        else part_o[c0 + c] += weight * x;
      }
    }
  }
}

// Two spare warps make V of the masked tiles safe for the product: 0 * NaN =
// NaN, so V rows past the request's end (the page or an earlier tile may have
// left anything there) are zeroed, and infinities and NaN of the others taken
// out; the epilogue adds those to the rows that see them.
template <int D, bool PAIR>
__device__ void cw_fixer(const CacheFwdParams& p, uint8_t* smem, CwShared* sh, const CacheRange& R, Fail fail) {
  using C = CwCfg<D, PAIR>;
  constexpr int kPieces = C::kBlockCols / 8;
  const int lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem + C::kRingOff);
  uint32_t it = 0, asked = 0;
  int number = 0;
  CacheWalk w;
  w.init(R);
  for (; w.next<kTile>(p); w.advance()) {
    const CwPart part(p, w, sh->hides);
    if (part.n == 0) continue;
    ++number;
    for (int t = part.lo; t < part.lo + part.n; ++t, ++it) {
      if (part.plain(t)) continue;
      const uint32_t e = C::entry_v(it);
      const int st = C::stage(e), key0 = t * kTile;
      // (once its S is issued, the stage's round before this V is over)
      if (!mbar_wait_warp(&sh->fix_ask[asked & 1], (asked >> 1) & 1, fail)) return;
      if (!mbar_wait_warp(&sh->full[st], C::parity(e), fail)) return;
      for (int row = threadIdx.x & 63; row < kTile; row += 64) {
        const bool past = key0 + row >= w.r.L;
        const uint32_t vr = ring + st * C::kTileBytes + row * C::kRowBytes;
        // (pieces in any order, whatever the swizzle: from the lane's on, so
        // that the lanes, a row apart, meet different banks)
        auto piece = [&](int c) {
          return vr + (c / kPieces) * C::kBlockBytes + ((c + lane * kPieces / 8) % kPieces) * 16;
        };
        if (past) {
  #pragma unroll
          for (int c = 0; c < D / 8; ++c) st_shared_v4(piece(c), 0u, 0u, 0u, 0u);
          continue;
        }
        // 0 * x summed over the row is NaN when one of its values is not finite
        const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
        __nv_bfloat162 sum = zero;
  #pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint32_t x[4];
          ld_shared_v4(piece(c), x[0], x[1], x[2], x[3]);
  #pragma unroll
          for (int e = 0; e < 4; ++e) sum = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&x[e]), zero, sum);
        }
        if (__low2float(sum) == 0.f && __high2float(sum) == 0.f) continue;
        *const_cast<volatile int*>(&sh->odd[number & 15]) = number;
  #pragma unroll 1
        for (int c = 0; c < D / 8; ++c) {
          uint32_t x[4];
          ld_shared_v4(piece(c), x[0], x[1], x[2], x[3]);
  #pragma unroll
          for (int e = 0; e < 4; ++e) x[e] &= ~cc_nonfinite(x[e]);
          st_shared_v4(piece(c), x[0], x[1], x[2], x[3]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(&sh->fixed[asked & 1]);
      ++asked;
    }
  }
}

// 16 columns of a row: bf16 to `out`, or fp32 to `part` where the item goes on elsewhere.
__device__ __forceinline__ void cw_store16(const uint32_t (&x)[16], float inv, __nv_bfloat16* out, float* part, int c0) {
  if (out != nullptr) {
    uint32_t pk[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) pk[c] = pack_bf16(__uint_as_float(x[2 * c]) * inv, __uint_as_float(x[2 * c + 1]) * inv);
    if (reinterpret_cast<uintptr_t>(out) % 32 == 0) {
      st_global_v8(out + c0, pk);
    } else {
      st_global_v4(out + c0, pk[0], pk[1], pk[2], pk[3]);
      st_global_v4(out + c0 + 8, pk[4], pk[5], pk[6], pk[7]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 16; c += 8) {
      const uint32_t w[8] = {x[c], x[c + 1], x[c + 2], x[c + 3], x[c + 4], x[c + 5], x[c + 6], x[c + 7]};
      st_global_v8(part + c0 + c, w);
    }
  }
}

template <int D, int ACT, bool PAIR>
__device__ void cw_consumer(const CacheFwdParams& p, CwShared* sh, uint32_t tmem, int stream, const CacheRange& R,
                            Fail fail) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = (warp & 3) * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t t_s = tmem + lane_off + 128 * stream, t_o = tmem + lane_off + 256;
  const int reach = (p.bias_len - 1) / 2;
  uint32_t s_n = 0, o_n[2] = {0, 0};
  int number = 0;  // of the part with tiles, from 1
  bool dead = false;
  CacheWalk w;
  w.init(R);
  for (; w.next<kTile>(p); w.advance()) {
    CwPart part(p, w, sh->hides);
    const CacheReq& r = w.r;
    if (part.n > 0) ++number;  // (the ring lets no more than 8 later parts be loaded, let alone made safe)
    __syncwarp();
    const bool pair = PAIR && part.pair;
    // a tile's rows go head by head, so that the lanes of a warp are neighbours
    // in their mask words and bias entries
    const int before = pair && stream == 1 ? p.tile_tokens : 0;  // tokens of the part
    const int g = static_cast<uint32_t>(row) / static_cast<uint32_t>(p.tile_tokens), at = row - g * p.tile_tokens;
    const bool row_ok = g < p.group && before + at < part.tokens;
    CcRow q;
    q.t = row_ok ? part.first_token + before + at : -1;
    q.head = w.h * p.group + (row_ok ? g : 0);
    q.pos = row_ok ? cc_row_pos(p, r, q.t, fail.status) : r.C;
    q.far_bias = 0.f;
    if (row_ok && p.bias_len)
      q.far_bias = __ldg(p.bias + static_cast<int64_t>(q.head) * p.bias_len + 2 * reach) * cc_bias_unit<ACT>();
    const bool warp_live = __any_sync(0xffffffffu, row_ok);
    // a far bias beside which scores are lost takes the near tiles' way, where it is added to them first
    if (ACT == 2 && __any_sync(0xffffffffu, fabsf(q.far_bias) > 1e18f)) part.far_hi = 0;
    const int count = part.count(stream);
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < count; ++i) {
      const int tile = part.lo + part.at(stream, i);
      const bool far = tile < part.far_hi, plain = part.plain(tile);
      CwNear near;
      if ((!plain || !far) && warp_live) near = cw_near(p, r, q, plain, tile * kTile);
      if (!dead && !mbar_wait(&sh->s_full[stream], s_n & 1, fail)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      ++s_n;
      if (dead) continue;
      tc_fence_after();
      if (warp_live) {
        float scale = p.scale, bias = q.far_bias;
        if (!far || !plain) {
          cw_near_tile<ACT>(p, r.C, q, near, tile * kTile, t_s);
          scale = 1.f;
          bias = 0.f;
        }
        if constexpr (ACT == 2) cw_softmax_tile<D>(t_s, t_o + 128 * stream, scale, bias, row_ok, i == 0, m, l);
        else cw_act_tile<ACT>(t_s, scale, bias);
        tmem_st_wait();
      }
      tc_fence_before();
      mbar_arrive_warp(&sh->p_full[stream]);
    }

    // the part's end
    const bool share = !pair && part.n > 0;  // both streams hold parts of the same rows
    int o_col = 0;            // first column this warpgroup writes
    float f[2] = {1.f, 1.f};  // factors of the streams' O
    bool use[2] = {stream == 0 && part.n > 0, stream == 1 && part.n > 0};
    if (share) {  // each warpgroup joins and writes half the columns
      use[0] = true;
      use[1] = part.count(1) > 0;
      o_col = stream * (D / 2);
      if constexpr (ACT == 2) {
        // the two threads of a row exchange through one place, there and back
        float2 other = make_float2(m, l);
        if (stream == 1) sh->ml[row] = other;
        named_bar(1, 256);
        if (stream == 0) {
          other = sh->ml[row];
          sh->ml[row] = make_float2(m, l);
        }
        named_bar(1, 256);
        if (stream == 1) other = sh->ml[row];
        const float top = fmaxf(m, other.x), ref = top == -INFINITY ? 0.f : top;
        f[stream] = ex2_sfu(m - ref);
        f[stream ^ 1] = ex2_sfu(other.x - ref);
        // (in stream order, so that both warpgroups get the same bits)
        const float l0 = stream == 0 ? l : other.y, l1 = stream == 0 ? other.y : l;
        l = __fmaf_rn(l0, f[0], l1 * f[1]);
        m = top;
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (use[s] && !dead && !mbar_wait(&sh->o_full[s], o_n[s] & 1, fail)) dead = true;
      if (part.n > 0 && part.count(s) > 0) ++o_n[s];
    }
    dead = __any_sync(0xffffffffu, dead);
    const bool odd = part.n > 0 && *const_cast<volatile int*>(&sh->odd[number & 15]) == number;
    const float inv = ACT != 2 || !w.whole ? 1.f : (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l));
    const int64_t token = r.q0 + (row_ok ? q.t : 0);
    const int64_t prow = (2 * static_cast<int64_t>(blockIdx.x) + w.slot()) * p.rows_per_tile + before * p.group + row;
    __nv_bfloat16* out = w.whole ? p.out + (token * p.heads + q.head) * D : nullptr;
    float* part_o = p.part_o + prow * D;
    tc_fence_after();
    // (a part without tiles leaves zeros; where the streams share it, both write them)
#pragma unroll 1
    for (int c0 = o_col; c0 < o_col + (share ? D / 2 : D); c0 += 16) {
      uint32_t x[16], y[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) x[c] = y[c] = 0u;
      if (!dead) {
        if (use[0]) tmem_ld16(t_o + c0, x);
        if (use[1]) tmem_ld16(t_o + 128 + c0, y);
        tmem_ld_wait16(x);
        tmem_ld_wait16(y);
      }
#pragma unroll
      for (int c = 0; c < 16; ++c)
        x[c] = __float_as_uint(__fmaf_rn(__uint_as_float(x[c]), f[0], __uint_as_float(y[c]) * f[1]));
      if (row_ok && !dead) cw_store16(x, inv, out, part_o, c0);
      __syncwarp();
    }
    if (part.n > 0 && !dead) {
      tc_fence_before();
      mbar_arrive_warp(&sh->o_empty);
    }
    if (!row_ok || dead) continue;
    if (odd) cw_add_odd<D, ACT>(p, w, part, q, o_col, share ? D / 2 : D, out, part_o);
    if (ACT == 2 && o_col == 0) {
      if (!w.whole) p.part_ml[prow] = make_float2(m, l);
      else if (p.lse != nullptr)
        p.lse[static_cast<int64_t>(q.head) * p.total_q + token] = cc_lse(m, l);
    }
  }
}

template <int D, int ACT, bool PAIR>
__global__ void __launch_bounds__(kWideThreads, 1) cache_fwd_wide_kernel(const __grid_constant__ CacheFwdParams p) {
  using C = CwCfg<D, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  CwShared* sh = reinterpret_cast<CwShared*>(smem + C::kBarOff);
  const int warp = threadIdx.x >> 5;
  cache_let_next();
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh->q_full[s], 1);
      mbar_init(&sh->q_empty[s], 1);
      mbar_init(&sh->s_full[s], 1);
      mbar_init(&sh->p_full[s], 4);
      mbar_init(&sh->o_full[s], 1);
      mbar_init(&sh->fix_ask[s], 1);
      mbar_init(&sh->fixed[s], 2);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
    }
    mbar_init(&sh->o_empty, 8);
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    for (int i = 0; i < 16; ++i) sh->odd[i] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  cache_wait_before();
  if (threadIdx.x == 0) p.err[blockIdx.x] = kOk;
  const CacheRange R = cache_range<kTile>(p, &sh->range, kWideMinRange);
  bool hides = false;
  if (ACT == 2 && p.bias != nullptr)
    for (int h = threadIdx.x; h < p.heads; h += kWideThreads)
      hides = hides || __ldg(p.bias + static_cast<int64_t>(h + 1) * p.bias_len - 1) == -INFINITY;
  tc_fence_before();
  hides = __syncthreads_or(hides) != 0;
  tc_fence_after();
  if (threadIdx.x == 0) sh->hides = ACT != 2 || p.bias == nullptr ? 0 : (hides ? 2 : 1);
  __syncthreads();
  if (threadIdx.x == 96) cache_open<kTile>(p, R);
  const uint32_t tmem = sh->tmem_base;
  Fail fail{&sh->abort, p.err + blockIdx.x, p.wait_limit_ns};
  if (warp == 0) cw_producer<D, PAIR>(p, smem, sh, R, fail);
  else if (warp == 1) cw_mma<D, PAIR>(p, smem, sh, tmem, R, fail);
  else if (warp < 4) cw_fixer<D, PAIR>(p, smem, sh, R, fail);
  else cw_consumer<D, ACT, PAIR>(p, sh, tmem, (warp - 4) >> 2, R, fail);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ launch
#ifndef JGDPA_HEAD_DIM
#error "compile cache_fwd_wide.cu with -DJGDPA_HEAD_DIM=32, 64 or 128"
#endif

template <int D, int ACT, bool PAIR>
static cudaError_t launch_cw(const CacheFwdParams& p, int grid, cudaStream_t stream) {
  auto kern = cache_fwd_wide_kernel<D, ACT, PAIR>;
  constexpr int kSmem = CwCfg<D, PAIR>::kSmemBytes;
  static DeviceFlags attr_set = {};
  cudaError_t e = smem_attr_once(kern, kSmem, attr_set);
  if (e != cudaSuccess) return e;
  return cache_launch(kern, dim3(grid), kWideThreads, kSmem, stream, p);
}

// pairs: items of two 128-row tiles.
template <int D>
cudaError_t launch_cache_fwd_wide_d(const CacheFwdParams& p, int act, bool pairs, int grid, cudaStream_t stream) {
  if (act == 0) return pairs ? launch_cw<D, 0, true>(p, grid, stream) : launch_cw<D, 0, false>(p, grid, stream);
  if (act == 1) return pairs ? launch_cw<D, 1, true>(p, grid, stream) : launch_cw<D, 1, false>(p, grid, stream);
  return pairs ? launch_cw<D, 2, true>(p, grid, stream) : launch_cw<D, 2, false>(p, grid, stream);
}
template cudaError_t launch_cache_fwd_wide_d<JGDPA_HEAD_DIM>(const CacheFwdParams&, int, bool, int, cudaStream_t);

}  // namespace jg
