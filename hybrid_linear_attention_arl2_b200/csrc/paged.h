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

// A batch as the kernels see it (arl2_paged_batch and the pool's extents).
struct PagedSeqs {
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* pages;
  int32_t n_seqs, tokens, max_q, max_kv, pages_ld;
  int32_t page_size, n_pages;
};

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
  float scale_log2;     // softmax scale * log2(e)
  // work division (see PagedPlan): blocks of query rows per stream at most
  int32_t n_qblk;
  float* part_o;        // [2 * grid][rows][d] pieces of items that several CTAs share
  float2* part_ml;      // [2 * grid][rows] their running max (log2 units) and sum
  int4* rec;            // [2 * grid] (f, kv head, starts, ends) of those pieces
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
  float scale_log2;
  float* part_w;        // bf16: [2 * grid][256] sums of key blocks that CTAs share
  int4* rec;            // [2 * grid] (stream, key head, key block, starts | ends << 1) of those pieces
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
  float eps;
  uint64_t freq[64];           // 2^64 theta^(-2 i / n) / (2 pi) of each pair
  // append
  PagedSeqs s;
  void *k_pool, *v_pool;
  uint32_t* err;
};

cudaError_t launch_prep(const PrepParams& p, int dtype, bool append, int sms, cudaStream_t st);
// Attention: CTAs of the launch and rows of one of their pieces at most, which
// size the handle's work space; then the launches (attention, combine).
// (float32: two blocks to an SM with head dims up to 64)
inline int paged_attn_grid(int dtype, int sms) { return dtype == ARL2_BF16 ? sms : 2 * sms; }
inline int paged_piece_rows(int dtype) { return dtype == ARL2_BF16 ? 256 : 64; }
cudaError_t launch_paged_attn_f32(PagedAttnParams p, int grid, cudaStream_t st);
// bf16 operands travel by TMA: maps over the pools (made once) and the queries
bool paged_pool_map(CUtensorMap* m, const void* pool, int64_t rows, int page_size);
bool paged_query_map(CUtensorMap* m, const void* q, int64_t tokens, int heads, int group, int64_t ld);
cudaError_t launch_paged_attn_bf16(PagedAttnParams p, const CUtensorMap& tk, const CUtensorMap& tv, int grid,
                                   cudaStream_t st);
cudaError_t launch_paged_weights_f32(const PagedWeightParams& p, cudaStream_t st);
cudaError_t launch_paged_weights_bf16(const PagedWeightParams& p, const CUtensorMap& tk, int sms, cudaStream_t st);
cudaError_t launch_paged_evict(const PagedEvictParams& p, int sms, cudaStream_t st);

#ifdef __CUDACC__
// ------------------------------------------------------------------ device side
struct SeqView {
  int q0, n, kv;  // first row, new tokens, cached keys
};

// Stream b, or n = -1 when its rows or lengths break the batch's bounds (it is
// then left out by every kernel; the error is recorded).
__device__ __forceinline__ SeqView load_seq(const PagedSeqs& s, int b, uint32_t* err) {
  const int q0 = s.q_start[b], q1 = s.q_start[b + 1], kv = s.kv_len[b];
  SeqView v{q0, q1 - q0, kv};
  if (q0 < 0 || q1 < q0 || q1 > s.tokens || q1 - q0 > s.max_q || kv < 0 || kv > s.max_kv ||
      (kv + s.page_size - 1) / s.page_size > s.pages_ld) {
    if (err) atomicCAS(err, 0u, kDevPage);
    v = SeqView{0, -1, 0};
  }
  return v;
}

// As load_seq for the calls that use a stream's cache alone.
__device__ __forceinline__ int load_kv_len(const PagedSeqs& s, int b, uint32_t* err) {
  const int kv = s.kv_len[b];
  if (kv < 0 || kv > s.max_kv || (kv + s.page_size - 1) / s.page_size > s.pages_ld) {
    if (err) atomicCAS(err, 0u, kDevPage);
    return -1;
  }
  return kv;
}

// The page that holds key j of stream b, or -1 (recorded) when the table's
// entry is no page of the pool.  j < kv_len, so the entry exists.
__device__ __forceinline__ int page_of(const PagedSeqs& s, int b, int j, uint32_t* err) {
  const int pg = s.pages[int64_t(b) * s.pages_ld + j / s.page_size];
  if (unsigned(pg) >= unsigned(s.n_pages)) {
    if (err) atomicCAS(err, 0u, kDevPage);
    return -1;
  }
  return pg;
}

// Keys that new token t of a stream sees.
__device__ __forceinline__ int visible_keys(const SeqView& v, int mask_block, int t) {
  if (mask_block <= 0) return v.kv;
  const long long lim = (long long)(v.kv - v.n) + (long long)(t / mask_block + 1) * mask_block;
  return lim < 0 ? 0 : lim > v.kv ? v.kv : int(lim);
}

// Division of an attention launch.  Query rows of one (stream, key head) are
// the pairs (token, head of the group), token-major; a tile holds kTileRows /
// group tokens, a block kTiles tiles.  Item (f, hk): f = b * n_qblk + block.
// Its work is counted in units: with two tiles one unit is one tile of kKeys
// keys against both; a block of one tile (single tokens) splits its keys
// between the two halves of the CTA, so a unit is two key tiles.  Items lie in
// a row, f first and key heads within it, and the CTAs take equal contiguous
// ranges of the units: no CTA has more than one unit more than another,
// however ragged the batch is.  An item cut by a range's end is finished by the
// combine kernel from the CTAs' pieces: a CTA has at most two, one at its
// range's begin (slot 0) and one at its end (slot 1).  An item has at least
// one unit, so that rows which see no key get their zeros.
template <int kTiles, int kTileRows, int kKeys>
struct PagedPlan {
  struct Block {
    int q0, t0, n_tok;  // stream's first row, the block's first token, its tokens (0: no item)
    int tiles;          // 1 or 2
    int units;          // per key head
    SeqView v;
  };
  __device__ static int tile_tokens(int group) { return kTileRows / group; }
  __device__ static Block block(const PagedSeqs& s, int b, int blk, int group, int mask_block, uint32_t* err) {
    Block r;
    r.v = load_seq(s, b, err);
    const int qt = tile_tokens(group);
    r.q0 = r.v.q0;
    r.t0 = blk * qt * kTiles;
    r.n_tok = r.v.n - r.t0;
    if (r.n_tok <= 0) {
      r.n_tok = 0;
      r.tiles = 0;
      r.units = 0;
      return r;
    }
    if (r.n_tok > qt * kTiles) r.n_tok = qt * kTiles;
    r.tiles = (r.n_tok + qt - 1) / qt;
    int nk = (visible_keys(r.v, mask_block, r.t0 + r.n_tok - 1) + kKeys - 1) / kKeys;
    if (kTiles == 2 && r.tiles == 1) nk = (nk + 1) >> 1;
    r.units = nk < 1 ? 1 : nk;
    return r;
  }
};

// What a CTA walks: segments (f, hk, units [u0, u1) of the item).
struct PagedRange {
  int f, hk, u;          // where the range begins (u: unit within the item)
  int left;              // units of the range
};

// Finds the CTA's range; called by all kThreads threads of the block.  Two
// passes over the blocks of rows: their total, then the one that holds the
// range's first unit.  `sh` is 64 shared 64-bit words.
template <class Plan, int kThreads>
__device__ __forceinline__ PagedRange paged_range(const PagedSeqs& s, int n_qblk, int group, int kv_heads,
                                                  int mask_block, int cta, int grid, uint32_t* err,
                                                  long long* sh) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps + 8 <= 64, "shared words");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long F = (long long)s.n_seqs * n_qblk;
  auto cost = [&](long long f) -> long long {
    if (f >= F) return 0;
    return (long long)Plan::block(s, int(f / n_qblk), int(f % n_qblk), group, mask_block, err).units * kv_heads;
  };
  long long first = cost(tid), sum = first;
  for (long long f = tid + kThreads; f < F; f += kThreads) sum += cost(f);
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sh[warp] = sum;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < kWarps; ++w) total += sh[w];
  const int ctas = total < grid ? int(total) : grid;
  PagedRange r{0, 0, 0, 0};
  if (cta >= ctas) return r;  // uniform over the block
  const long long u0 = total * cta / ctas, u1 = total * (cta + 1) / ctas;
  r.left = int(u1 - u0);
  __syncthreads();
  long long base = 0;
  for (long long f0 = 0; f0 < F; f0 += kThreads) {
    const long long c = f0 == 0 ? first : cost(f0 + tid);
    long long inc = c;
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) sh[warp] = inc;
    __syncthreads();
    long long before = base, all = base;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh[w];
      all += sh[w];
    }
    const long long end = before + inc, beg = end - c;
    if (c > 0 && u0 >= beg && u0 < end) {
      sh[kWarps] = f0 + tid;
      sh[kWarps + 1] = u0 - beg;
      sh[kWarps + 2] = c / kv_heads;
    }
    __syncthreads();
    if (u0 < all) break;
    base = all;
  }
  r.f = int(sh[kWarps]);
  const long long off = sh[kWarps + 1], units = sh[kWarps + 2];
  r.hk = int(off / units);
  r.u = int(off % units);
  __syncthreads();
  return r;
}

// One segment of the walk.
template <class Plan>
struct PagedSeg {
  typename Plan::Block blk;
  int b, f, hk, u0, u1;  // units [u0, u1) of item (f, hk)
  bool first;            // the range's first segment
  __device__ bool starts() const { return u0 == 0; }
  __device__ bool ends() const { return u1 == blk.units; }
  __device__ bool whole() const { return starts() && ends(); }
  // the slot of a piece: the range's first segment has slot 0
  __device__ int slot() const { return first ? 0 : 1; }
};

template <class Plan>
struct PagedWalk {
  PagedRange r;
  int b, blk;
  bool fresh, have;
  PagedSeg<Plan> seg;
  PagedWalk() = default;
  __device__ explicit PagedWalk(const PagedRange& range, int n_qblk)
      : r(range), b(range.f / n_qblk), blk(range.f % n_qblk), fresh(true), have(false) {}
  __device__ bool next(const PagedSeqs& s, int n_qblk, int group, int kv_heads, int mask_block) {
    if (r.left <= 0) return false;
    if (!have) {
      while (true) {
        if (b >= s.n_seqs) return false;  // (cannot happen: the range lies inside the items)
        seg.blk = Plan::block(s, b, blk, group, mask_block, nullptr);
        if (seg.blk.units > 0) break;
        if (++blk == n_qblk) blk = 0, ++b;
      }
      have = true;
    }
    seg.b = b;
    seg.f = b * n_qblk + blk;
    seg.hk = r.hk;
    seg.u0 = r.u;
    const int rest = seg.blk.units - r.u;
    const int take = rest < r.left ? rest : r.left;
    seg.u1 = r.u + take;
    seg.first = fresh;
    fresh = false;
    r.left -= take;
    r.u = 0;
    if (take == rest && ++r.hk == kv_heads) {
      r.hk = 0;
      have = false;
      if (++blk == n_qblk) blk = 0, ++b;
    }
    return true;
  }
};

#endif  // __CUDACC__

}  // namespace arl2
