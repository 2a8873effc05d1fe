// Paged KV cache: launch parameters, the device view of a batch of streams,
// and the division of an attention launch's work over its CTAs, shared by the
// kernels (paged_*.cu) and the entry points (paged_api.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "arl2.h"

namespace arl2 {

constexpr uint32_t kDevPage = 9;  // ARL2_ERR_PAGE as kernels record it
constexpr int kPagedMaxGroup = 64;
constexpr int kMaxUnits = 0x7fffffff - (1 << 14);  // of a launch's work division: sums stay in 32 bits

// Division of numbers below 2^30 by a divisor known on the host: a product and a
// shift.  With s = ceil(log2 d) - 2 and m = ceil(2^(32 + s) / d), m d - 2^(32 + s)
// < d <= 2^(s + 2), so n m / 2^(32 + s) exceeds n / d by less than 1 / d.
struct FastDiv {
  uint32_t mul;
  int32_t shift, by;
  FastDiv() = default;
  explicit FastDiv(int d) : mul(1), shift(0), by(d) {
    if (d < 2) return;
    int log = 0;
    while ((1u << log) < unsigned(d)) ++log;
    shift = 32 + log - 2;
    mul = uint32_t(((uint64_t(1) << shift) + d - 1) / d);
  }
  __host__ __device__ int div(int n) const { return int((uint64_t(uint32_t(n)) * mul) >> shift); }
  __host__ __device__ int mod(int n) const { return n - div(n) * by; }
};

// A batch as the kernels see it (arl2_paged_batch and the pool's extents).
struct PagedSeqs {
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* pages;
  int32_t n_seqs, tokens, max_q, max_kv, pages_ld;
  int32_t page_size, n_pages;
  FastDiv page;            // by page_size
  int32_t box;             // keys of a TMA box (bf16)
};

// Keys per TMA box: the boxes of a 64-key tile lie inside pages.
inline int box_keys(int page_size) {
  int a = page_size, b = 64;
  while (b) {
    const int t = a % b;
    a = b, b = t;
  }
  return a;
}

// Attention and weights: one launch's operands.
struct PagedAttnParams {
  PagedSeqs s;
  const void* q;        // [tokens, H, d], rows ld_q apart
  int64_t ld_q;
  const void* k_pool;   // [n_pages, Hk, page_size, d]
  const void* v_pool;
  void* o;              // [tokens, H, d]
  float* lse;           // [tokens, H] or null
  int32_t heads, kv_heads, group, d;
  int32_t mask_block;
  FastDiv mask, per_group, per_blk;  // by mask_block, group, a block's tokens
  float scale_log2;     // softmax scale * log2(e)
  // work division (see PagedPlan): tokens of a tile, cost of a range at least
  int32_t qt, min_cost;
  float* part_o;        // [2 * grid][rows][d] pieces of items that several CTAs share
  float2* part_ml;      // [2 * grid][rows] their running max (log2 units) and sum
  uint32_t* joined;     // [grid][8] pieces of a CTA's cut item that are in (a count for each warp's rows); zero between launches
  uint32_t* err;
  uint64_t wait_limit_ns;
};

struct PagedWeightParams {
  PagedSeqs s;
  const void* q;
  int64_t ld_q;
  const void* k_pool;
  const float* lse;
  const float* w_in;
  float* w_out;
  int64_t w_ld;
  float decay;
  int32_t heads, kv_heads, group, d;
  int32_t mask_block;
  FastDiv mask, per_group, per_tile;  // by mask_block, group, a tile's tokens
  float scale_log2;
  float* part_w;        // [2 * grid][256, f32 64] sums of key blocks that CTAs share
  uint32_t* joined;     // as PagedAttnParams'
  uint32_t* err;
  uint64_t wait_limit_ns;
};

struct PagedEvictParams {
  PagedSeqs s;
  void* k_pool;
  void* v_pool;
  const float* w_in;
  float* w_out;
  int64_t w_ld;
  int32_t* kept;
  int32_t* kv_len_out;
  const int32_t* dst_pages;
  int32_t dst_ld;
  int32_t kv_heads, row_bytes;
  int32_t budget, sink, recent;
  uint32_t* err;
};

// Norm + rotation (and append): see paged_prep.cu.
struct PrepParams {
  const void *q, *k, *v;
  int64_t ld_q, ld_k, ld_v;    // elements between token rows
  void *q_out, *k_out;         // q_out may be null (append without Q); k_out unused by append
  int64_t ld_qo, ld_ko;
  const void *w_q, *w_k;
  const int32_t* pos;
  int64_t tokens;
  int32_t heads, kv_heads, d;
  int32_t n_axes, axis_dim[3], halves, rot;  // rot = R, 0: no rotation
  int32_t norm;
  float eps, inv_d;            // inv_d = 1 / d
  uint64_t freq[64];           // 2^64 theta^(-2 i / n) / (2 pi) of each pair
  // append
  PagedSeqs s;
  void *k_pool, *v_pool;
  uint32_t* err;
};

// Launches with programmatic stream serialisation: the grid may be scheduled
// while the kernel ahead of it on the stream finishes; every kernel launched so
// waits for that kernel's completion (grid_dependency_wait) before it touches
// global memory, in every thread, so that the stream's order is kept along any
// chain of them.  cluster: CTAs of a cluster (0: none).
template <class... P, class... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster,
                              A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 0) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

cudaError_t launch_prep(const PrepParams& p, int dtype, bool append, int sms, cudaStream_t st);
// Attention: CTAs of the launch and rows of one of their pieces at most, which
// size the handle's work space; then the launches.
// (float32: two blocks to an SM)
inline int paged_attn_grid(int dtype, int sms) { return dtype == ARL2_BF16 ? sms : 2 * sms; }
inline int paged_piece_rows(int dtype) { return dtype == ARL2_BF16 ? 256 : 64; }
cudaError_t launch_paged_attn_f32(PagedAttnParams p, int grid, cudaStream_t st);
// bf16 operands travel by TMA: maps over the pools (made once) and the queries
bool paged_pool_map(CUtensorMap* m, const void* pool, int64_t rows, int page_size);
bool paged_query_map(CUtensorMap* m, const void* q, int64_t tokens, int heads, int group, int64_t ld);
// rotate: CTAs take the key tiles of their segments in an order that brings
// those on one key head together (PagedWalk::rotation)
cudaError_t launch_paged_attn_bf16(PagedAttnParams p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                                   bool rotate, cudaStream_t st);
cudaError_t launch_paged_weights_f32(const PagedWeightParams& p, int sms, cudaStream_t st);
cudaError_t launch_paged_weights_bf16(const PagedWeightParams& p, const CUtensorMap& tk, int sms, cudaStream_t st);
cudaError_t launch_paged_evict(const PagedEvictParams& p, int sms, cudaStream_t st);

#ifdef __CUDACC__
// ------------------------------------------------------------------ device side
struct SeqView {
  int q0, n, kv;  // first row, new tokens, cached keys
};

// A stream of rows [q0, q1) and kv keys, n = -1 when they break the batch's bounds
// (it is then left out by every kernel; the error is recorded).
__device__ __forceinline__ SeqView checked_seq(const PagedSeqs& s, int q0, int q1, int kv, uint32_t* err) {
  SeqView v{q0, q1 - q0, kv};
  if (q0 < 0 || q1 < q0 || q1 > s.tokens || q1 - q0 > s.max_q || kv < 0 || kv > s.max_kv ||
      kv > int64_t(s.pages_ld) * s.page_size) {
    if (err) atomicCAS(err, 0u, kDevPage);
    v = SeqView{0, -1, 0};
  }
  return v;
}

__device__ __forceinline__ SeqView load_seq(const PagedSeqs& s, int b, uint32_t* err) {
  return checked_seq(s, s.q_start[b], s.q_start[b + 1], s.kv_len[b], err);
}

// As load_seq for the calls that use a stream's cache alone.
__device__ __forceinline__ int load_kv_len(const PagedSeqs& s, int b, uint32_t* err) {
  const int kv = s.kv_len[b];
  if (kv < 0 || kv > s.max_kv || kv > int64_t(s.pages_ld) * s.page_size) {
    if (err) atomicCAS(err, 0u, kDevPage);
    return -1;
  }
  return kv;
}

// The page that holds key j of stream b, or -1 (recorded) when the table's
// entry is no page of the pool.  j < kv_len, so the entry exists.
__device__ __forceinline__ int page_of(const PagedSeqs& s, int b, int j, uint32_t* err) {
  const int pg = s.pages[int64_t(b) * s.pages_ld + s.page.div(j)];
  if (unsigned(pg) >= unsigned(s.n_pages)) {
    if (err) atomicCAS(err, 0u, kDevPage);
    return -1;
  }
  return pg;
}

// Keys that new token t of a stream sees.
__device__ __forceinline__ int visible_keys(const SeqView& v, const FastDiv& mask, int t) {
  if (mask.by <= 0) return v.kv;
  const long long lim = (long long)(v.kv - v.n) + (long long)(mask.div(t) + 1) * mask.by;
  return lim < 0 ? 0 : lim > v.kv ? v.kv : int(lim);
}

// log sum exp of a row from its maximum (log2 units) and its sum, which is 0 where
// the row sees no key, and NaN where its logits are.
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Division of an attention launch.  Query rows of one (stream, key head) are
// the pairs (token, head of the group), token-major; a tile holds `qt` tokens, a
// block kTiles tiles.  An item is a block of a stream and a key head.  Its work is
// counted in units: with two tiles one unit is one tile of kKeys keys against both; a
// block of one tile (single tokens) splits its keys between the two halves of
// the CTA, so a unit is two key tiles.  Items lie in a row, streams first, their
// blocks and key heads within them, and the CTAs take equal contiguous ranges of
// the cost, kItemCost + units an item (its start, end and output take as long as
// that many units), so that ragged batches are spread as evenly as one long
// stream.  An item cut by a range's end is finished from the CTAs' pieces by the
// one that comes last: a CTA has at most two, one at its range's begin (slot 0) and
// one at its end (slot 1).  An item has at least one unit, so that rows which see
// no key get their zeros.  A range costs min_cost at least.  Only blocks that exist
// are looked at, tokens / block + streams at most, so that neither the time nor the
// launch's limit on units (kMaxUnits) depends on how far max_q is above the streams'
// lengths.
template <int kTiles, int kKeys, int kItemCost_>
struct PagedPlan {
  static constexpr int kItemCost = kItemCost_;
  struct Block {
    int row0, t0, n_tok;  // first token row, its token in the stream, tokens
    int tiles;            // 1 or 2
    int units;            // per key head
    int n, kv;            // the stream's new tokens and cached keys
    __device__ SeqView view() const { return SeqView{0, n, kv}; }
  };

  // Blocks of a stream's rows.
  __device__ static int blocks(const PagedAttnParams& p, const SeqView& v) {
    return v.n > 0 ? p.per_blk.div(v.n - 1) + 1 : 0;
  }
  // Block k of a stream's.
  __device__ static Block block(const PagedAttnParams& p, const SeqView& v, int k) {
    Block r;
    r.t0 = k * p.qt * kTiles;
    r.row0 = v.q0 + r.t0;
    r.n = v.n, r.kv = v.kv;
    r.n_tok = min(v.n - r.t0, p.qt * kTiles);
    r.tiles = kTiles == 2 && r.n_tok > p.qt ? 2 : 1;
    const int nk = (visible_keys(v, p.mask, r.t0 + r.n_tok - 1) + kKeys - 1) / kKeys;
    r.units = max(1, kTiles == 2 && r.tiles == 1 ? (nk + 1) >> 1 : nk);
    return r;
  }
};

// The sum of the lanes' units, each below 2^31; false where it is above kMaxUnits,
// as it can only be of rows that several streams claim.
__device__ __forceinline__ bool sum_units(unsigned mine, int& total) {
  const unsigned high = __reduce_add_sync(0xffffffffu, mine >> 8), low = __reduce_add_sync(0xffffffffu, mine & 255u);
  total = int(high << 8) + int(low);
  return high <= unsigned(kMaxUnits >> 8);
}

// One segment of a CTA's walk: units [u0, u1) of the item of block `blk` of stream b and key head hk.
template <class Plan>
struct PagedSeg {
  typename Plan::Block blk;
  int b, hk, u0, u1;
  // the item's pieces when it is cut: CTAs owner, owner + 1, ...; the owner's is in slot owner_slot, the others' in 0
  int owner, pieces, owner_slot;
  int slot;  // of this CTA's piece
  __device__ bool whole() const { return pieces == 1; }
};

template <class Plan>
struct PagedWalk {
  int each, more;  // cost of every range; the first `more` have one more
  int at, end;     // cost before the current item, and where the range ends
  int used;        // units of the segments before
  bool have, fresh;
  PagedSeg<Plan> seg;

  __device__ int begin(int cta) const { return each * cta + min(cta, more); }
  __device__ int owner(int cost) const {  // the CTA whose range holds it
    const int big = (each + 1) * more;
    return cost < big ? cost / (each + 1) : more + (cost - big) / each;
  }

  // The blocks of all streams in order, up to 32 at a time, a lane each: use(blk, b,
  // cost), with cost 0 in a lane without one, until it returns true.  A lane holds
  // one of 32 streams; where none of them has more than one block, its block too.
  template <class Use>
  __device__ static void visit(const PagedAttnParams& p, uint32_t* err, const Use& use) {
    const int lane = threadIdx.x & 31;
    int q0 = 0, q1 = 0, kv = 0;  // (a lane without a stream has one without tokens)
    auto fetch = [&](int b) {
      q0 = q1 = kv = 0;
      if (b < p.s.n_seqs) q0 = p.s.q_start[b], q1 = p.s.q_start[b + 1], kv = p.s.kv_len[b];
    };
    fetch(lane);
#pragma unroll 1
    for (int s0 = 0; s0 < p.s.n_seqs; s0 += 32) {
      const SeqView v = checked_seq(p.s, q0, q1, kv, err);
      fetch(s0 + 32 + lane);
      const int nb = Plan::blocks(p, v);
      const bool shared = __any_sync(0xffffffffu, nb > 1);
      int upto = nb, all = 32;  // blocks of the lanes up to this one, and of all
      if (shared) {
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x;
        }
        all = __shfl_sync(0xffffffffu, upto, 31);
      }
#pragma unroll 1
      for (int x0 = 0; x0 < all; x0 += 32) {
        SeqView u = v;
        int k = 0, src = lane;
        bool some = nb > 0;
        if (shared) {
          const int x = x0 + lane;
          some = x < all;
          src = 0;  // the lane whose stream block x is of
#pragma unroll 1
          for (int o = 16; o > 0; o >>= 1)
            if (__shfl_sync(0xffffffffu, upto, src + o - 1) <= x) src += o;
          k = x - __shfl_sync(0xffffffffu, upto - nb, src);
          u = SeqView{__shfl_sync(0xffffffffu, v.q0, src), __shfl_sync(0xffffffffu, v.n, src),
                      __shfl_sync(0xffffffffu, v.kv, src)};
        }
        const typename Plan::Block blk = Plan::block(p, u, k);
        if (use(blk, s0 + src, some ? (blk.units + Plan::kItemCost) * p.kv_heads : 0)) return;
      }
    }
  }

  // Finds the CTA's range; called by one warp.  Two passes over the blocks: their
  // total, then the one that holds the range's begin (of 32 blocks or fewer one).
  __device__ void find(const PagedAttnParams& p, int cta, int grid) {
    const int lane = threadIdx.x & 31;
    unsigned mine = 0;
    typename Plan::Block blk;
    int b = 0, c = 0, batches = 0;
    visit(p, cta == 0 ? p.err : nullptr, [&](const typename Plan::Block& blk_, int b_, int c_) {
      blk = blk_, b = b_, c = c_, ++batches;
      mine = min(mine + unsigned(c_), 0x7fffffffu);
      return false;
    });
    at = end = used = 0;
    have = fresh = true;
    int total;
    if (!sum_units(mine, total)) {
      if (cta == 0 && lane == 0) atomicCAS(p.err, 0u, kDevPage);
      return;
    }
    const int ctas = min((total + p.min_cost - 1) / p.min_cost, grid);
    if (cta >= ctas) return;
    each = total / ctas;
    more = total - each * ctas;
    const int pos = begin(cta);
    int before = 0;
    auto search = [&](const typename Plan::Block& blk_, int b_, int c_) {
      int inc = c_;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      const int off = pos - (before + inc - c_);
      const unsigned hit = __ballot_sync(0xffffffffu, off >= 0 && off < c_);
      before += __shfl_sync(0xffffffffu, inc, 31);
      if (!hit) return false;
      const int src = __ffs(hit) - 1;
      const int in = __shfl_sync(0xffffffffu, off, src);
      typename Plan::Block found = blk_;
      int* w = reinterpret_cast<int*>(&found);
      for (int i = 0; i < int(sizeof(found) / 4); ++i) w[i] = __shfl_sync(0xffffffffu, w[i], src);
      seg.blk = found;
      seg.b = __shfl_sync(0xffffffffu, b_, src);
      seg.hk = in / (found.units + Plan::kItemCost);
      const int inner = in - seg.hk * (found.units + Plan::kItemCost);
      at = pos - inner;
      seg.u1 = max(0, inner - Plan::kItemCost);  // (the next segment begins at u1)
      end = begin(cta + 1);
      return true;
    };
    if (batches == 1)
      search(blk, b, c);
    else
      visit(p, nullptr, search);
  }

  // The next segment with units; a range may end or begin in an item's kItemCost.
  __device__ bool next(const PagedAttnParams& p) {
    while (at < end) {
      if (!have) {
        SeqView v{seg.blk.row0 - seg.blk.t0, seg.blk.n, seg.blk.kv};
        int k = p.per_blk.div(seg.blk.t0) + 1;
        while (k >= Plan::blocks(p, v)) {
          if (++seg.b >= p.s.n_seqs) return false;  // (cannot happen: the range lies inside the items)
          v = load_seq(p.s, seg.b, nullptr);
          k = 0;
        }
        seg.blk = Plan::block(p, v, k);
        seg.hk = 0;
        have = true;
      }
      seg.u0 = seg.u1;
      seg.u1 = min(seg.blk.units, end - at - Plan::kItemCost);
      if (seg.u1 <= seg.u0) return false;  // (the range ends before the item's first unit)
      seg.slot = fresh ? 0 : 1;
      seg.owner = 0, seg.pieces = 1, seg.owner_slot = 0;
      if (seg.u1 - seg.u0 < seg.blk.units) {
        seg.owner = owner(at + Plan::kItemCost);
        seg.pieces = owner(at + Plan::kItemCost + seg.blk.units - 1) - seg.owner + 1;
        seg.owner_slot = begin(seg.owner) >= at ? 0 : 1;
      }
      fresh = false;
      return true;
    }
    return false;
  }
  // Where to begin within the segment's units, cyclically: the CTAs on one key
  // head then reach a key tile at about the same time, each at the unit that is
  // its clock modulo a range's length where its segment has it.
  __device__ int rotation() const {
    int r = (used - seg.u0) % each;
    if (r < 0) r += each;
    return r < seg.u1 - seg.u0 ? r : 0;
  }
  // After a segment's use: moves on to the next item where this one ended.
  __device__ void done(const PagedAttnParams& p) {
    used += seg.u1 - seg.u0;
    if (seg.u1 < seg.blk.units) {
      at = end;
      return;
    }
    at += seg.blk.units + Plan::kItemCost;
    seg.u1 = 0;
    if (++seg.hk == p.kv_heads) have = false;
  }
};
#endif  // __CUDACC__

// Host side: blocks of `block` tokens at most in a batch's streams (one of n tokens
// has n / block + 1 at most).
inline double most_blocks(const PagedSeqs& s, int block) {
  const double by_streams = double(s.max_q / block + 1) * s.n_seqs, by_tokens = double(s.tokens / block) + s.n_seqs;
  return by_streams < by_tokens ? by_streams : by_tokens;
}

// Of the division: fills p's tile; false where the units could pass kMaxUnits.
inline bool paged_plan(PagedAttnParams& p, int tile_rows, int tiles, int keys) {
  p.qt = tile_rows / p.group;
  const int block = p.qt * tiles;
  if (most_blocks(p.s, block) * (p.s.max_kv / keys + 8) * p.kv_heads >= double(kMaxUnits)) return false;
  p.mask = FastDiv(p.mask_block);
  p.per_group = FastDiv(p.group);
  p.per_blk = FastDiv(block);
  return true;
}

}  // namespace arl2
