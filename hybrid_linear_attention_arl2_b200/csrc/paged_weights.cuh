// Division of the attention weights' work over CTAs, for the float32 and the bf16
// kernel.  Units are (key block, tile of rows that sees it), stream by stream, key
// head by key head, blocks in order; CTAs take equal contiguous ranges.  A block
// cut by a range's end is joined from the CTAs' pieces, in order, by the one that
// comes last.  Sums run in the order of rows: the same bits every time.
#pragma once

#include "paged.h"

namespace arl2 {

// A stream's units.  Row tile rt holds tokens [rt qt, ...); key block jt is
// seen from the first token that sees its first key on, by all tiles after that.
template <int kKeys>
struct WeightStream {
  SeqView v;
  int n_kb, n_rt;  // key blocks, row tiles; 0 where nothing is to be summed
  int full;        // blocks that every row tile sees
  __device__ WeightStream() {}
  __device__ WeightStream(const PagedWeightParams& p, int b, uint32_t* err) : v(load_seq(p.s, b, err)) {
    const bool some = v.n > 0 && v.kv > 0;
    n_kb = some ? (v.kv + kKeys - 1) / kKeys : 0;
    n_rt = some ? p.per_tile.div(v.n - 1) + 1 : 0;
    // blocks that begin below the keys which the first token sees
    const long long seen = (long long)(v.kv - v.n) + p.mask.by;
    full = p.mask.by <= 0 ? n_kb : seen <= 0 ? 0 : int(min((long long)n_kb, (seen + kKeys - 1) / kKeys));
  }
  // the first token that sees key j
  __device__ int first_token(const FastDiv& mask, int j) const {
    if (mask.by <= 0) return 0;
    const int past = j - (v.kv - v.n);
    return past < mask.by ? 0 : past - mask.mod(past);
  }
  __device__ int first_tile(const PagedWeightParams& p, int jt) const {
    return jt < full ? 0 : p.per_tile.div(first_token(p.mask, jt * kKeys));
  }
  __device__ int units(const PagedWeightParams& p) const {
    int sum = full * n_rt;
    for (int jt = full; jt < n_kb; ++jt) sum += n_rt - first_tile(p, jt);
    return sum;
  }
};

// A key block as the roles need it: its units [rt0, rt1) within this CTA's range.
struct WeightBlk {
  int more, b, hk, jt;
  int rt0, rt1;
  int q0, n, kv;
  int fresh;   // its first unit's Q tile is not the last one of the block before
  int pieces, owner, owner_slot, slot;  // as PagedSeg's
};

// The CTA's range, walked block by block, by one warp.
template <int kKeys>
struct WeightWalk {
  using Stream = WeightStream<kKeys>;
  Stream s;
  int b, hk, jt, rt, left;
  int qb, qhk, qrt;  // the Q tile before
  int each, more, at;  // units of every range (the first `more` have one more); the next unit
  bool head;

  __device__ int begin(int cta) const { return each * cta + min(cta, more); }
  __device__ int owner(int unit) const {
    const int big = (each + 1) * more;
    return unit < big ? unit / (each + 1) : more + (unit - big) / each;
  }

  __device__ void find(const PagedWeightParams& p) {
    const int lane = threadIdx.x & 31;
    left = 0, qb = -1, qhk = qrt = 0, head = true;
    // (A sum that wraps is one of rows that several streams claim, which is recorded:
    // the search still ends inside the streams, and blocks that are never whole are
    // not joined.  A check of it, three instructions, made all launches 1.5 % longer.)
    int mine = 0;
#pragma unroll 1
    for (int i = lane; i < p.s.n_seqs; i += 32)
      mine += Stream(p, i, blockIdx.x == 0 ? p.err : nullptr).units(p) * p.kv_heads;
    const int total = __reduce_add_sync(0xffffffffu, mine), ctas = min(total, int(gridDim.x)), cta = blockIdx.x;
    if (cta >= ctas) return;
    each = total / ctas, more = total - each * ctas;
    int pos = at = begin(cta);
    const int len = each + (cta < more ? 1 : 0);
    // the index in [0, n) whose cost holds `pos`, and pos within it
    auto find_in = [&](int n, auto&& cost) {
      int before = 0;
#pragma unroll 1
      for (int i0 = 0; i0 < n; i0 += 32) {
        const int c = i0 + lane < n ? cost(i0 + lane) : 0;
        int inc = c;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        const int off = pos - (before + inc - c);
        const unsigned hit = __ballot_sync(0xffffffffu, off >= 0 && off < c);
        if (hit) {
          const int src = __ffs(hit) - 1;
          pos = __shfl_sync(0xffffffffu, off, src);
          return i0 + src;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
      return -1;
    };
    b = find_in(p.s.n_seqs, [&](int i) { return Stream(p, i, nullptr).units(p) * p.kv_heads; });
    if (b < 0) return;  // (cannot happen: the range lies inside the units)
    s = Stream(p, b, nullptr);
    const int per = s.units(p);
    hk = pos / per;
    pos -= hk * per;
    if (pos < s.full * s.n_rt) {
      jt = pos / s.n_rt;
      rt = pos - jt * s.n_rt;
    } else {
      pos -= s.full * s.n_rt;
      jt = s.full + find_in(s.n_kb - s.full, [&](int i) { return s.n_rt - s.first_tile(p, s.full + i); });
      rt = s.first_tile(p, jt) + pos;
    }
    left = len;
  }
  // Describes the next block (lane 0 writes) and moves on.
  __device__ bool next(const PagedWeightParams& p, WeightBlk& out) {
    const bool writes = (threadIdx.x & 31) == 0;
    if (left <= 0) {
      if (writes) out.more = 0;
      return false;
    }
    const int r0 = s.first_tile(p, jt), rt1 = min(s.n_rt, rt + left);
    if (writes) {
      out.more = 1;
      out.b = b, out.hk = hk, out.jt = jt;
      out.rt0 = rt, out.rt1 = rt1;
      out.q0 = s.v.q0, out.n = s.v.n, out.kv = s.v.kv;
      out.fresh = !(qb == b && qhk == hk && qrt == rt);
      out.slot = head ? 0 : 1;
      out.pieces = 1, out.owner = out.owner_slot = 0;
      if (rt > r0 || rt1 < s.n_rt) {
        const int first = at - (rt - r0);
        out.owner = owner(first);
        out.pieces = owner(first + (s.n_rt - r0) - 1) - out.owner + 1;
        out.owner_slot = begin(out.owner) == first ? 0 : 1;
      }
    }
    head = false;
    qb = b, qhk = hk, qrt = rt1 - 1;
    left -= rt1 - rt;
    at += rt1 - rt;
    if (left > 0) {  // (the block is done)
      if (++jt >= s.n_kb) {
        jt = 0;
        if (++hk >= p.kv_heads) {
          hk = 0;
          do {
            if (++b >= p.s.n_seqs) {  // (cannot happen)
              left = 0;
              return true;
            }
            s = Stream(p, b, nullptr);
          } while (s.n_kb == 0);
        }
      }
      rt = s.first_tile(p, jt);
    }
    return true;
  }
};

// What no new token adds to: rows past kv_len are cleared, and the weights of
// streams without new tokens fade.  Runs of kTail weights, a warp each: `warp` of
// `warps`.  err: null where the caller's division records what breaks a bound.
constexpr int kTail = 1024;
__device__ __forceinline__ void clear_tails(const PagedWeightParams& p, int warp, int warps, uint32_t* err = nullptr) {
  const long long per_row = (p.w_ld + kTail - 1) / kTail, items = per_row * p.s.n_seqs * p.kv_heads;
  for (long long it = warp; it < items; it += warps) {
    const long long row = it / per_row, j0 = (it - row * per_row) * kTail, j1 = min((long long)p.w_ld, j0 + kTail);
    const SeqView v = load_seq(p.s, int(row / p.kv_heads), err);
    if (v.n < 0 || (j1 <= v.kv && v.n > 0)) continue;
    const int64_t base = row * p.w_ld;
    for (long long j = j0 + (threadIdx.x & 31); j < j1; j += 32) {
      if (j >= v.kv)
        p.w_out[base + j] = 0.f;
      else if (v.n == 0)
        p.w_out[base + j] = p.decay * p.w_in[base + j];
    }
  }
}

}  // namespace arl2
