// Attention of new tokens over a paged cache, bf16, on the tensor cores:
//
//   O = softmax(Q K^T scale) V over the visible keys,  lse = log sum exp
//
// One CTA an SM walks its range of units (PagedPlan).  Query rows of a (stream,
// key head) are the pairs (token, head of the group), so the heads that share
// keys share their tile: a tile is 128 rows.  Two tiles are in flight, a softmax
// warpgroup each.  A block with one tile (single tokens, a chunk's tail) takes
// two key tiles at once instead: both halves hold the same queries, half t every
// second tile of 64 keys, and their (m, l, O) are joined at the end, so that a
// single row keeps as many bytes in flight as 256 rows do.
//
// A half's work goes in steps of 64 keys with two S in tensor memory, so that
// S(i + 1) is there when the softmax of step i ends: S(i) = Q K^T (128 x 64,
// fp32), P(i) over it in place (bf16 pairs), O += P(i) V.  With 128 keys a step
// and one S a half each half waited for its own products (softmax 2800 clocks,
// products and signals 1500, one after the other); the halves hid too little of
// each other.  Order of a half's products:  S(0) S(1), then for each step i
// PV(i) S(i + 2);  the loader's ring of 16 KB tiles follows it.  S(i + 2)
// overwrites P(i) behind PV(i) in the pipe.
//
// Warps: 0 describes the segments and loads Q (one box a tile) and K, 2 loads V
// (boxes inside pages, one lane a box, page numbers fetched ahead), 1 and 3 issue
// the products of a half each, 4-7 and 8-11 softmax, O's rescaling (only when a row's maximum grows
// by more than 8 in log2 units: P <= 256) and the output; a thread has one row.
// Tensor memory: S_t, P_t of step i at t 128 + (i & 1) 64; O_t at 256 + t 128.
//
// Rounding: P and O to bf16 (half a step, 2^-8, each); S, m, l and O's sums are
// fp32.  Rows of V past the stream's keys are cleared in shared memory before a
// product sees them: what the pool holds there may be NaN.

#include "layer.h"
#include "paged_join.cuh"
#include "paged_mma.cuh"
#include "params.h"

namespace arl2 {

namespace {

constexpr int kThreads = 384;
constexpr int kRing = 10, kSegs = 4;
constexpr int kStepKeys = 64;
constexpr uint32_t kSlot = kStepKeys * 256;  // a step's K or V: two boxes of 64 columns
using Plan = PagedPlan<2, 128, 2>;

enum {
  B_QF = 0,              // Q tiles loaded (bytes)
  B_QE,                  // Q read by the segment's last S (commit, both issuers)
  B_SF,                  // [t][2] S_t of a step in tensor memory (commit)
  B_PF = B_SF + 4,       // [t][2] P_t of a step written (the warpgroup's 4 warps)
  B_PD = B_PF + 4,       // [t] a step's product with V done (commit)
  B_OF = B_PD + 2,       // [t] O_t final (commit)
  B_MG = B_OF + 2,       // half 1's statistics in shared memory (4 warps)
  B_MD,                  // half 1's O and statistics read by half 0 (4 warps)
  B_RF,                  // [kRing] ring slot loaded (bytes)
  B_RE = B_RF + kRing,   // [kRing] ring slot read (two commits)
  B_GF = B_RE + kRing,   // [kSegs] segment described
  B_GE = B_GF + kSegs,   // [kSegs] description read (the V loader, both issuers, 8 softmax warps)
  B_JN = B_GE + kSegs,   // [kSegs] the pieces of half 0's warps are in, Seg::last says whether as the last (4 warps)
  B_DRAIN = B_JN + kSegs,
  B_COUNT
};

// A segment as the roles need it, written by the K loader into a ring.
struct Seg {
  int more;            // 0: the CTA's range is done
  int b, hk;           // stream, key head
  int row0;            // first token row of the block in q and o
  int tok0;            // its token within the stream's new ones
  int n_new, kv;       // the stream's new tokens and cached keys
  int dual;            // two tiles of rows on the same key tiles; else one tile on alternate ones
  int n[2];            // steps of 64 keys of each half
  int rot;             // step with which both halves begin, of their n (cyclic)
  int j0;              // first step's tile of 64 keys (dual: of both; else of half 0, half 1's is the next)
  int rows[2];         // rows of each half's tile
  int slot;            // of this CTA's piece, and the pieces of the item (PagedSeg)
  int owner, pieces, owner_slot;
  int last;            // half 0 joins the pieces (said by one of its warps)
};

__device__ __forceinline__ void describe(Seg& g, const PagedSeg<Plan>& s, int rotation, const PagedAttnParams& p) {
  const int qt = p.qt;
  g.more = 1;
  g.last = 0;
  g.b = s.b, g.hk = s.hk;
  g.row0 = s.blk.row0;
  g.tok0 = s.blk.t0;
  g.n_new = s.blk.n, g.kv = s.blk.kv;
  g.dual = s.blk.tiles == 2;
  // the block's last token sees all its key tiles; with two row tiles the first may see fewer
  const int all = (visible_keys(s.blk.view(), p.mask, s.blk.t0 + s.blk.n_tok - 1) + kStepKeys - 1) / kStepKeys;
  if (g.dual) {
    const int nk = (visible_keys(s.blk.view(), p.mask, s.blk.t0 + qt - 1) + kStepKeys - 1) / kStepKeys;
    g.j0 = 2 * s.u0;
    g.n[0] = max(0, min(nk, 2 * s.u1) - g.j0);
    g.n[1] = max(0, min(all, 2 * s.u1) - g.j0);
    g.rows[0] = qt * p.group;
    g.rows[1] = (s.blk.n_tok - qt) * p.group;
  } else {
    g.j0 = 4 * s.u0;
    const int n = max(0, min(all, 4 * s.u1) - g.j0);
    g.n[0] = (n + 1) >> 1;
    g.n[1] = n >> 1;
    g.rows[0] = g.rows[1] = s.blk.n_tok * p.group;
  }
  g.rot = g.dual && g.n[0] == g.n[1] ? max(0, min(2 * rotation, g.n[1] - 1)) : 0;
  g.slot = s.slot;
  g.owner = s.owner, g.pieces = s.pieces, g.owner_slot = s.owner_slot;
}

// The segments as a role meets them.
struct SegReader {
  const Seg* ring;
  uint64_t* bars;
  uint32_t k = 0;
  __device__ const Seg* next(const WaitCtl& w) {  // a whole warp; null at the end
    if (!warp_wait(&bars[B_GF + k % kSegs], (k / kSegs) & 1, w)) return nullptr;
    const Seg* g = &ring[k % kSegs];
    return g->more ? g : nullptr;
  }
  __device__ void done() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars[B_GE + k % kSegs]);
    ++k;
  }
};

// ------------------------------------------------------------------ loads
// Two warps, one for K (which also describes the segments and loads Q) and one
// for V, so that neither's waits and page numbers hold up the other: one warp
// took 600 clocks a tile, where the products want one every 450.  K and V tiles
// lie in the ring in the order in which the products take them: the first steps'
// K (one tile a step in a dual segment, two otherwise, two steps), then V(y),
// K(y + first).  Each warp waits for its own tiles' slots alone: its last tile
// lies at most five places back, and both issuers release all tiles in order, so
// a slot it asks for is at most one fill behind.
struct Loader {
  const PagedAttnParams& p;
  uint64_t* bars;
  uint8_t* sR;
  const CUtensorMap* tm;
  const WaitCtl& w;
  uint32_t slot = 0, round = 0;
  __device__ void skip() {
    if (++slot == kRing) slot = 0, ++round;
  }
  __device__ __forceinline__ bool load(BoxRows<kStepKeys>& rows, int tile) {
    if (round > 0 && !warp_wait(&bars[B_RE + slot], (round - 1) & 1, w)) return false;
    if ((threadIdx.x & 31) == 0) mbar_expect_tx(&bars[B_RF + slot], kSlot);
    __syncwarp();
    rows.load(tile, sR + slot * kSlot, tm, &bars[B_RF + slot]);
    skip();
    return true;
  }
  // This warp's tiles of a segment, from its rotation's on and then those before.
  template <bool kRotate>
  __device__ __forceinline__ bool segment(const Seg& s, bool is_v) {
    const int n = s.dual ? s.n[1] : s.n[0] + s.n[1], first = s.dual ? 2 : 4, j0 = s.j0, rot = kRotate ? s.rot : 0, wrap = n - rot;
    BoxRows<kStepKeys> rows(p.s, s.b, s.kv, s.hk, p.kv_heads, j0 + rot, j0 + n, p.err);
    auto take = [&](int i) {
      if (kRotate && i == wrap) rows = BoxRows<kStepKeys>(p.s, s.b, s.kv, s.hk, p.kv_heads, j0, j0 + rot, p.err);
      return load(rows, !kRotate || i < wrap ? j0 + rot + i : j0 + i - wrap);
    };
    for (int i = -first; i < n; ++i) {
      if (i >= 0) {
        if (!is_v)
          skip();
        else if (!take(i))
          return false;
      }
      if (i + first < n) {
        if (is_v)
          skip();
        else if (!take(i + first))
          return false;
      }
    }
    return true;
  }
};

template <bool kRotate>
__device__ __forceinline__ void k_role(const PagedAttnParams& p, const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                                       uint64_t* bars, Seg* ring, uint8_t* sQ, uint8_t* sR, const WaitCtl& w) {
  const int lane = threadIdx.x & 31, qt = p.qt;
  PagedWalk<Plan> walk;
  walk.find(p, blockIdx.x, gridDim.x);
  Loader loader{p, bars, sR, tm_k, w};
  uint32_t q_loads = 0;
  for (uint32_t k = 0;; ++k) {
    const bool more = walk.next(p);
    if (k >= kSegs && !warp_wait(&bars[B_GE + k % kSegs], (k / kSegs - 1) & 1, w)) return;
    Seg& s = ring[k % kSegs];
    if (lane == 0) {
      if (more)
        describe(s, walk.seg, kRotate ? walk.rotation() : 0, p);
      else
        s.more = 0;
      mbar_arrive(&bars[B_GF + k % kSegs]);
    }
    __syncwarp();
    if (!more) return;
    walk.done(p);
    if (s.n[0] == 0 && s.n[1] == 0) continue;
    if (q_loads > 0 && !warp_wait(&bars[B_QE], (q_loads - 1) & 1, w)) return;
    ++q_loads;
    if (lane == 0) {
      const int tiles = s.dual ? 2 : 1;
      mbar_expect_tx(&bars[B_QF], 2u * uint32_t(tiles) * uint32_t(qt * p.group) * 128u);
      for (int t = 0; t < tiles; ++t)
        for (int h = 0; h < 2; ++h)
          tma_load_3d(sQ + t * kTile + h * kHalfTile, tm_q, &bars[B_QF], h * 64, s.hk * p.group, s.row0 + t * qt);
    }
    __syncwarp();
    if (!loader.segment<kRotate>(s, false)) return;
  }
}

template <bool kRotate>
__device__ __forceinline__ void v_role(const PagedAttnParams& p, const CUtensorMap* tm_v, SegReader segs, uint64_t* bars,
                                       uint8_t* sR, const WaitCtl& w) {
  Loader loader{p, bars, sR, tm_v, w};
  for (const Seg* s = segs.next(w); s; segs.done(), s = segs.next(w))
    if (s->n[0] + s->n[1] > 0 && !loader.segment<kRotate>(*s, true)) return;
}

// ------------------------------------------------------------------ products
// A place in the ring and the parity of its fill.
struct RingPos {
  uint32_t slot = 0, phase = 0;
  __device__ RingPos next() {  // this one; moves on
    const RingPos r = *this;
    if (++slot == kRing) slot = 0, phase ^= 1u;
    return r;
  }
};

// The products of half t: S(i) and O += P(i) V, one warp a half (see elect_one),
// so that one's waits and signals pass while the other's products run; each
// keeps its own order, in which S(i + 2) follows PV(i).  One warp for both took
// 3500 clocks a unit where its products take 2700.
struct Issuer {
  uint64_t* bars;
  uint8_t* sR;
  int t;
  uint32_t tS, tO, dk, dv, el;  // tensor memory; descriptors of ring slot 0 as K and as V
  const WaitCtl& w;
  uint32_t s_count = 0, p_count = 0;  // S and P so far: buffer count & 1, parity (count >> 1) & 1

  __device__ __forceinline__ bool loaded(const RingPos& r) const { return warp_wait(&bars[B_RF + r.slot], r.phase, w); }
  __device__ __forceinline__ void release(const RingPos& r) const { mma_commit_el(&bars[B_RE + r.slot], el); }
  // The next S: queries q, the K in slot r.
  __device__ __forceinline__ void scores(const RingPos& r, uint32_t q) {
    const uint32_t buf = s_count++ & 1u;
    mma_tile<kStepKeys>(tS + buf * 64, q, dk + r.slot * (kSlot >> 4), idesc_bf16(128, kStepKeys, 0, 0), el);
    mma_commit_el(&bars[B_SF + 2 * t + buf], el);
  }
  // O += P V: the next P, the V in slot r, of which `valid` rows count.
  __device__ __forceinline__ bool values(const RingPos& r, int valid, bool first) {
    const uint32_t buf = p_count & 1u;
    if (!warp_wait(&bars[B_PF + 2 * t + buf], (p_count >> 1) & 1u, w)) return false;
    ++p_count;
    if (uniform(valid < kStepKeys && (valid & 15))) {  // rows past the stream's keys, up to the product's 16
      uint8_t* tile = sR + r.slot * kSlot;
      for (int x = valid * 8 + int(threadIdx.x & 31); x < ((valid + 15) & ~15) * 8; x += 32) {
        *reinterpret_cast<uint4*>(tile + x * 16) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(tile + kSlot / 2 + x * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_async_smem();
      __syncwarp();
    }
    tc_fence_after();
    const uint32_t id = idesc_bf16(128, 128, 0, 1);
    const uint32_t a = tS + buf * 64, b = dv + r.slot * (kSlot >> 4);
    if (uniform(valid >= kStepKeys)) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) mma_ts_el(tO, a + kk * 8, b + kk * 128, id, kk > 0 || !first, el);
    } else {
      for (int kk = 0; uniform(kk * 16 < valid); ++kk) mma_ts_el(tO, a + kk * 8, b + kk * 128, id, kk > 0 || !first, el);
    }
    mma_commit_el(&bars[B_PD + t], el);
    return true;
  }
};

template <bool kRotate>
__device__ __forceinline__ void mma_role(SegReader segs, uint64_t* bars, uint8_t* sQ, uint8_t* sR, uint32_t tmem, int t,
                                         const WaitCtl& w) {
  Issuer x{bars, sR, t, tmem + t * 128, tmem + 256 + t * 128, desc_lo(sR, 16), desc_lo(sR, kSlot / 2), elect_one(), w};
  const uint32_t q0 = desc_lo(sQ, 16), q1 = q0 + t * (kTile >> 4);
  RingPos ring;
  uint32_t qf = 0;
  for (const Seg* s = segs.next(w); s; segs.done(), s = segs.next(w)) {
    const int n = s->n[t], both = s->n[0] + s->n[1];
    int left = s->kv - (s->j0 + (kRotate ? s->rot : 0)) * kStepKeys;  // keys from the tile on
    if (uniform(both == 0)) continue;
    if (!warp_wait(&bars[B_QF], qf, w)) return;
    qf ^= 1u;
    if (uniform(s->dual)) {
      // Both halves walk K(0) K(1) V(0) K(2) V(1) ... and release every tile; half
      // 0 may have fewer steps (its tokens are the earlier ones).
      const int all = s->n[1], wrap = kRotate ? all - s->rot : -1;
#pragma unroll 1
      for (int i = 0; uniform(i < 2 && i < all); ++i) {
        const RingPos k = ring.next();
        if (!x.loaded(k)) return;
        if (uniform(i < n)) x.scores(k, q1);
        x.release(k);
      }
#pragma unroll 1
      for (int i = 0; uniform(i < all); ++i, left -= kStepKeys) {
        if (kRotate && i == wrap) left += all * kStepKeys;
        const RingPos v = ring.next();
        if (!x.loaded(v)) return;
        if (uniform(i < n) && !x.values(v, left, i == 0)) return;
        x.release(v);
        if (uniform(i + 2 < all)) {
          const RingPos k = ring.next();
          if (!x.loaded(k)) return;
          if (uniform(i + 2 < n)) x.scores(k, q1);
          x.release(k);
        }
      }
    } else {
      // Tile y is half y & 1's: K(0) .. K(3) V(0) K(4) V(1) K(5) ...  Both halves
      // wait for and release every tile: who skipped the other's could run a
      // round of the ring ahead of it, where a parity says nothing.
#pragma unroll 1
      for (int y = 0; uniform(y < 4 && y < both); ++y) {
        const RingPos k = ring.next();
        if (!x.loaded(k)) return;
        if (uniform((y & 1) == t)) x.scores(k, q0);
        x.release(k);
      }
#pragma unroll 1
      for (int y = 0; uniform(y < both); ++y, left -= kStepKeys) {
        const bool mine = uniform((y & 1) == t);
        const RingPos v = ring.next();
        if (!x.loaded(v)) return;
        if (mine && !x.values(v, left, y < 2)) return;
        x.release(v);
        if (uniform(y + 4 < both)) {
          const RingPos k = ring.next();
          if (!x.loaded(k)) return;
          if (mine) x.scores(k, q0);
          x.release(k);
        }
      }
    }
    mma_commit_el(&bars[B_QE], x.el);
    if (uniform(n > 0)) mma_commit_el(&bars[B_OF + t], x.el);
  }
}

// ------------------------------------------------------------------ softmax and output
// P = 2^(S scale - m) for 32 columns of a row, packed to bf16 pairs; their sum.
// All on the MUFU: with 3 of 16 pairs on the FMA pipe (a polynomial of degree 4)
// a frame took 412 us instead of 393, as the products bound the loop.
__device__ __forceinline__ float exp_chunk(const uint32_t* r, const float2 sc, const float2 nm, uint32_t (&pk)[16]) {
  float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    const float2 y = __ffma2_rn(make_float2(__uint_as_float(r[2 * x]), __uint_as_float(r[2 * x + 1])), sc, nm);
    const float2 e = make_float2(fast_exp2(y.x), fast_exp2(y.y));
    s2[x & 1] = __fadd2_rn(s2[x & 1], e);
    pk[x] = pack_bf16x2(e.x, e.y);
  }
  const float2 sa = __fadd2_rn(s2[0], s2[1]);
  return sa.x + sa.y;
}

// 32 columns of an output row.
__device__ __forceinline__ void store_row32(__nv_bfloat16* dst, const uint32_t (&o)[32], bool sectors) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t v[8];
#pragma unroll
    for (int x = 0; x < 8; ++x)
      v[x] = pack_bf16x2(__uint_as_float(o[c * 16 + 2 * x]), __uint_as_float(o[c * 16 + 2 * x + 1]));
    if (sectors) {
      store_sector(dst + c * 16, v);
    } else {
      reinterpret_cast<uint4*>(dst + c * 16)[0] = make_uint4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<uint4*>(dst + c * 16)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
}

// Joins the pieces of a thread's own row (see join_rows).
__device__ __forceinline__ void join_own(const PagedAttnParams& p, const Seg& s, int row, int64_t orow, bool sectors) {
  auto first = [&](int k) { return int64_t(k == 0 ? 2 * s.owner + s.owner_slot : 2 * (s.owner + k)) * 256; };
  float M = -INFINITY, L = 0.f;
  for (int k = 0; k < s.pieces; ++k) M = fmaxf(M, __ldcg(&p.part_ml[first(k) + row].x));
  if (M == -INFINITY) M = 0.f;
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    float acc[32];
#pragma unroll
    for (int x = 0; x < 32; ++x) acc[x] = 0.f;
    L = 0.f;
#pragma unroll 1
    for (int k = 0; k < s.pieces; ++k) {
      const float2 ml = __ldcg(&p.part_ml[first(k) + row]);
      float4 v[8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4* src = reinterpret_cast<const float4*>(p.part_o + piece_at(first(k), row, q * 4 + c));
        v[2 * c] = __ldcg(src);
        v[2 * c + 1] = __ldcg(src + 1);
      }
      const float w = exp2f(ml.x - M);
      L = fmaf(ml.y, w, L);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        acc[4 * x] = fmaf(v[x].x, w, acc[4 * x]);
        acc[4 * x + 1] = fmaf(v[x].y, w, acc[4 * x + 1]);
        acc[4 * x + 2] = fmaf(v[x].z, w, acc[4 * x + 2]);
        acc[4 * x + 3] = fmaf(v[x].w, w, acc[4 * x + 3]);
      }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    uint32_t o[32];
#pragma unroll
    for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(acc[x] * inv);
    store_row32(static_cast<__nv_bfloat16*>(p.o) + orow * 128 + q * 32, o, sectors);
  }
  if (p.lse) p.lse[orow] = row_lse(M, L);
}

// Warpgroup t: tile t's rows, one a thread, 64 keys a step.
template <bool kRotate>
__device__ __forceinline__ void softmax_role(const PagedAttnParams& p, SegReader segs, uint64_t* bars, float* stats,
                                             uint32_t tmem, int t, const WaitCtl& w) {
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, row = quarter * 32 + lane;
  const uint32_t lane_off = uint32_t(quarter * 32) << 16;
  const uint32_t tS = tmem + t * 128 + lane_off, tO = tmem + 256 + t * 128 + lane_off;
  const float2 sc = make_float2(p.scale_log2, p.scale_log2);
  uint32_t g = 0, of = 0, merges = 0, asked = 0;  // g: steps so far; asked: parity of each B_JN
  for (const Seg* s = segs.next(w); s; segs.done(), s = segs.next(w)) {
    const int rows = s->rows[t], n = s->n[t], step = s->dual ? kStepKeys : 2 * kStepKeys;
    const bool live = row < rows, warp_live = quarter * 32 < rows;
    int left = s->kv;  // visible keys from the step's first on
    if (live)
      left = visible_keys(SeqView{0, s->n_new, s->kv}, p.mask, s->tok0 + (s->dual ? t * p.qt : 0) + p.per_group.div(row));
    left -= (s->j0 + (kRotate ? s->rot : 0) + (s->dual ? 0 : t)) * kStepKeys;
    const int wrap = kRotate ? n - s->rot : -1;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < n; ++i, ++g) {
      if (kRotate && i == wrap) left += n * step;
      const uint32_t buf = g & 1;
      if (!warp_wait(&bars[B_SF + 2 * t + buf], (g >> 1) & 1, w)) return;
      if (warp_live) {
        tc_fence_after();
        uint32_t r[64];
#pragma unroll
        for (int q = 0; q < 2; ++q) tmem_ld32(tS + buf * 64 + q * 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32 * q]));
        tmem_wait_ld();
        const bool masked = __any_sync(0xffffffffu, left < 64);
        if (masked) {
#pragma unroll
          for (int x = 0; x < 64; ++x)
            if (x >= left) r[x] = __float_as_uint(-INFINITY);
        }
        float m4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          m4[q] = fmax3(__uint_as_float(r[q]), __uint_as_float(r[4 + q]), __uint_as_float(r[8 + q]));
#pragma unroll
        for (int x = 12; x < 60; x += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q) m4[q] = fmax3(m4[q], __uint_as_float(r[x + q]), __uint_as_float(r[x + 4 + q]));
#pragma unroll
        for (int q = 0; q < 4; ++q) m4[q] = fmaxf(m4[q], __uint_as_float(r[60 + q]));
        const float mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]) * sc.x;
        const bool need = mx > m + 8.f;  // (also a row's first finite maximum)
        const float mg = need ? mx : m;
        const float ref = mg == -INFINITY ? 0.f : mg;  // nothing visible so far: every exponential is 0
        const float f = need ? fast_exp2(m - ref) : 1.f;
        if (i > 0 && __any_sync(0xffffffffu, need)) {
          // O *= 2^(old m - new m), 1 for rows that keep m, once the step before is in O
          if (!warp_wait(&bars[B_PD + t], (g - 1) & 1, w)) return;
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {
            uint32_t o[16];
            tmem_ld16(tO + q * 16, o);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
            tmem_st16(tO + q * 16, o);
          }
        }
        const float2 nm = make_float2(-ref, -ref);
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t pc[16];
          sum += exp_chunk(&r[32 * q], sc, nm, pc);
          tmem_st16(tS + buf * 64 + q * 16, pc);
        }
        l = fmaf(l, f, sum);
        m = mg;
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_PF + 2 * t + buf]);
      left -= step;
    }
    const bool have = n > 0;
    if (have) {
      if (!warp_wait(&bars[B_OF + t], of & 1, w)) return;
      ++of;
      tc_fence_after();
    }
    float a = 1.f, a1 = 0.f;  // O = a O_t + a1 O_1
    const bool join = !s->dual && s->n[1] > 0;
    if (!s->dual && t == 1) {  // half 0 writes the block's rows
      if (join) {
        stats[row] = m;
        stats[128 + row] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_MG]);
        if (!warp_wait(&bars[B_MD], merges & 1, w)) return;
        ++merges;
      }
      continue;
    }
    if (join) {
      if (!warp_wait(&bars[B_MG], merges & 1, w)) return;
      ++merges;
      const float m1 = stats[row], l1 = stats[128 + row], M = fmaxf(m, m1), ref = M == -INFINITY ? 0.f : M;
      a = fast_exp2(m - ref);
      a1 = fast_exp2(m1 - ref);
      l = l * a + l1 * a1;
      m = M;
    }
    const bool whole = s->pieces == 1;
    if (whole) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      a *= inv, a1 *= inv;
    }
    const int tok_row = s->row0 + (s->dual ? t * p.qt : 0), head0 = s->hk * p.group;
    auto out_row = [&](int r) { return int64_t(tok_row + p.per_group.div(r)) * p.heads + head0 + p.per_group.mod(r); };
    const int64_t orow = out_row(row);
    const int64_t piece = int64_t(2 * blockIdx.x + s->slot) * 256;
    const int64_t prow = piece + t * 128 + row;
    const bool sectors = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
    const bool team = !whole && !s->dual;
    if (warp_live) {
      // 32 columns at a time in a loop of its own: code that runs once costs its fetch
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t o[32], o1[32];
        tmem_ld32(tO + q * 32, o);
        if (join) tmem_ld32(tO + 128 + q * 32, o1);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          float v = have ? __uint_as_float(o[x]) * a : 0.f;
          if (join) v = fmaf(__uint_as_float(o1[x]), a1, v);
          o[x] = __float_as_uint(v);
        }
        if (!live) continue;
        if (whole) {
          store_row32(static_cast<__nv_bfloat16*>(p.o) + orow * 128 + q * 32, o, sectors);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            store_sector(p.part_o + piece_at(piece, t * 128 + row, q * 4 + c),
                         *reinterpret_cast<const uint32_t(*)[8]>(&o[c * 8]));
        }
      }
      if (live) {
        if (!whole)
          p.part_ml[prow] = make_float2(m, l);
        else if (p.lse)
          p.lse[orow] = row_lse(m, l);
      }
      if (!whole) {
        // The warp whose piece of these rows comes last joins them, in a dual segment;
        // else the last of all the rows' warps tells its warpgroup.
        __threadfence();
        __syncwarp();
        int last = 0;
        if (lane == 0)
          last = last_piece(p.joined + 8 * s->owner + (team ? 0 : 4 * t + quarter), s->pieces * (team ? (rows + 31) >> 5 : 1));
        if (team) {
          if (last) const_cast<Seg*>(s)->last = 1;
        } else if (__shfl_sync(0xffffffffu, last, 0) && live) {
          join_own(p, *s, t * 128 + row, orow, sectors);
        }
      }
    }
    if (team) {
      // Often few rows and many pieces: the four warps share the rows.  (A barrier
      // for each place of the ring of segments: one that all segments shared could
      // be two phases ahead of a warp.)
      const uint32_t at = segs.k % kSegs;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_JN + at]);
      if (!warp_wait(&bars[B_JN + at], (asked >> at) & 1, w)) return;
      asked ^= 1u << at;
      const int n = (rows + 3) >> 2;
      if (uniform(*const_cast<const volatile int*>(&s->last) != 0 && quarter * n < rows))
        join_rows(p, s->owner, s->owner_slot, s->pieces, quarter * n, min(n, rows - quarter * n),
                                            out_row);
    }
    if (join) {  // O_1 and its statistics are read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_MD]);
    }
  }
}

constexpr int kSmem = 232448;
constexpr int kLayout = 2 * kTile + kRing * kSlot + 256 * 4 + kSegs * int(sizeof(Seg)) + 8 * B_COUNT + 16;
static_assert(kLayout <= kSmem, "shared memory");

// ------------------------------------------------------------------ kernel
template <bool kRotate>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_bf16_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PagedAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // (the window begins on 1024 bytes; a layout that does not fit is refused)
  if (size_t(smem - smem_raw) + kLayout > size_t(kSmem)) {
    grid_dependency_wait();
    if (threadIdx.x == 0) record_error(p.err, kDevBadShape);
    return;
  }
  uint8_t* sQ = smem;
  uint8_t* sR = smem + 2 * kTile;
  float* stats = reinterpret_cast<float*>(sR + kRing * kSlot);  // half 1's m, l
  Seg* segs = reinterpret_cast<Seg*>(stats + 256);
  uint64_t* bars = reinterpret_cast<uint64_t*>(segs + kSegs);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      const int n = (i >= B_PF && i < B_PD) || i == B_MG || i == B_MD || (i >= B_JN && i < B_JN + kSegs) ? 4
                    : i >= B_GE && i < B_GE + kSegs                     ? 11
                    : i == B_QE || (i >= B_RE && i < B_RE + kRing) || i == B_DRAIN ? 2
                                                                        : 1;
      mbar_init(&bars[i], n);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc(tmem_holder, 512);
  if (warp == 0 && lane == 0) {
    tma_prefetch(&tm_q);
    tma_prefetch(&tm_k);
    tma_prefetch(&tm_v);
  }
  grid_dependency_wait();
  allow_dependent_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitCtl w{abort_flag, p.err, p.wait_limit_ns};
  const SegReader reader{segs, bars};
  if (warp == 0) {
    k_role<kRotate>(p, &tm_q, &tm_k, bars, segs, sQ, sR, w);
  } else if (warp == 1 || warp == 3) {
    mma_role<kRotate>(reader, bars, sQ, sR, tmem, warp >> 1, w);
  } else if (warp == 2) {
    v_role<kRotate>(p, &tm_v, reader, bars, sR, w);
  } else if (warp >= 4) {
    softmax_role<kRotate>(p, reader, bars, stats, tmem, (warp >> 2) - 1, w);
  }
  // Every product has completed once a commit behind all of them has arrived:
  // only then are shared and tensor memory released.
  __syncwarp();
  if (warp == 1 || warp == 3) {
    mma_commit_el(&bars[B_DRAIN], elect_one());
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(&bars[B_DRAIN], 0) && global_timer_ns() - t0 < 10000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {  // a wait ran out: let this CTA's own copies land first
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) {
    }
  }
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// 3-D map over rows of 128 bf16, 128-byte swizzle, boxes {64, b1, b2}.
bool encode(CUtensorMap* m, const void* base, uint64_t d1, uint64_t d2, uint64_t s1, uint64_t s2, uint32_t b1,
            uint32_t b2) {
  static const auto fn = reinterpret_cast<CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                                       const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                                       const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                                       CUtensorMapL2promotion, CUtensorMapFloatOOBfill)>(
      tensor_map_encoder());
  if (!fn) return false;
  const cuuint64_t dims[3] = {128, d1, d2}, strides[2] = {s1, s2};
  const cuuint32_t box[3] = {64, b1, b2}, step[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool paged_pool_map(CUtensorMap* m, const void* pool, int64_t rows, int page_size) {
  return encode(m, pool, uint64_t(rows), 1, 256, 256 * uint64_t(rows), uint32_t(box_keys(page_size)), 1);
}
// Query rows (token, head): boxes of one key head's group by a tile's tokens.
bool paged_query_map(CUtensorMap* m, const void* q, int64_t tokens, int heads, int group, int64_t ld) {
  return encode(m, q, uint64_t(heads), uint64_t(tokens), 256, uint64_t(ld) * 2, uint32_t(group), uint32_t(128 / group));
}

cudaError_t launch_paged_attn_bf16(PagedAttnParams p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                                   bool rotate, cudaStream_t st) {
  static unsigned done[2] = {0, 0};
  const auto kernel = rotate ? paged_attn_bf16_kernel<true> : paged_attn_bf16_kernel<false>;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), kSmem, &done[rotate]);
  if (e != cudaSuccess) return e;
  CUtensorMap tq;
  if (!paged_query_map(&tq, p.q, p.s.tokens, p.heads, p.group, p.ld_q)) return cudaErrorInvalidValue;
  return launch_overlapped(kernel, dim3(unsigned(grid)), kThreads, kSmem, st, 0, tq, tk, tv, p);
}

}  // namespace arl2
