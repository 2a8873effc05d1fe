// Paged KV cache on CUDA cores (float32 tensors): attention of new tokens over
// the pages, and the weights the cached keys received.
//
//   O = softmax(Q K^T scale) V over the visible keys,  lse = log sum exp,
//   w_out[j] = decay w_in[j] + sum over rows of exp(s_j - lse)
//
// One pass over the keys with the running maximum and sum of each row (Q K^T
// in units of log2).  A CTA holds 64 query rows (token, head of the group) of
// one key head and takes tiles of 64 keys; S and O are 4 x 4 and 4 x d/16
// register tiles a thread, in packed pairs, P passes through shared memory.  The
// f32 path is bound by the FMA pipe: 4 d FMAs a (row, key) pair.
//
// Tiles come by 16-byte asynchronous copies: V while S is computed, the next K
// while O is, the page numbers of the tile after a step earlier still.  Tiles of
// one buffer each, chunks of 16 bytes swizzled in place of padding, leave room
// for two CTAs an SM with 128 columns, and one's products pass while the other
// waits.  1000 causal tokens of 4 heads of 128 columns on 5000 keys: 320 us, 29
// TFLOP/s (541 with tiles loaded between barriers, one CTA an SM); single tokens
// of 16 heads on 2 key heads over 29300 keys: 93 us (154).  Neither pipe is full:
// shared memory moves in 58 % of the clocks, without conflicts, and an instruction
// issues in 49 %; 16 warps an SM do not hide the two barriers a tile.

#include <cuda_bf16.h>

#include "paged.h"
#include "paged_join.cuh"
#include "paged_weights.cuh"
#include "params.h"
#include "sm100.cuh"

namespace arl2 {

namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 256;
using Plan = PagedPlan<1, kKeys, 1>;

// Copies 16 bytes into shared memory asynchronously; zeros where `there` is false.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Columns of a tile's rows in shared memory: whole runs of 8 chunks of 4, since
// the chunks of K rows are swizzled by row & 7, those of Q by (row >> 2) & 1.
__host__ __device__ inline int tile_pitch(int d) { return (d + 31) & ~31; }

// How a block's threads copy rows of d columns: a power of two of lanes a row.
struct Lanes {
  int shift, chunks;
  __device__ explicit Lanes(int d) : shift(0), chunks(d >> 2) {
    while ((1 << shift) < chunks) ++shift;
  }
  // f(row, chunk) for every 16 bytes of 64 rows
  template <class F>
  __device__ __forceinline__ void each(const F& f) const {
    const int c = threadIdx.x & ((1 << shift) - 1);
    if (c < chunks)
      for (int r = threadIdx.x >> shift; r < kKeys; r += kThreads >> shift) f(r, c);
  }
};

// The page entry of key j of stream b (of a key behind the last: none), and from
// it the pool row of head hk; -1 where there is none or the entry is no page (recorded).
__device__ __forceinline__ int page_entry(const PagedSeqs& s, int b, int j, int end) {
  return j < end ? s.pages[int64_t(b) * s.pages_ld + s.page.div(j)] : -1;
}
__device__ __forceinline__ int pool_row(const PagedSeqs& s, int entry, int hk, int kv_heads, int j, int end, uint32_t* err) {
  if (j >= end) return -1;
  if (unsigned(entry) >= unsigned(s.n_pages)) {
    if (err) atomicCAS(err, 0u, kDevPage);
    return -1;
  }
  return (entry * kv_heads + hk) * s.page_size + s.page.mod(j);
}

// Starts the copy of 64 pool rows into a tile; `swizzle`: K's chunks.
__device__ __forceinline__ void copy_keys(float* dst, const float* pool, const int* rows, const Lanes& lanes, int pitch,
                                          int d, bool swizzle) {
  lanes.each([&](int r, int c) {
    const int row = rows[r];
    copy16(dst + r * pitch + 4 * (swizzle ? c ^ (r & 7) : c), pool + int64_t(max(row, 0)) * d + 4 * c, row >= 0);
  });
}

__device__ __forceinline__ float4 lds4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// S = Q K^T for this thread's 4 rows (4 ty ..) x 4 keys (tx + 16 i), even and odd columns apart.
__device__ __forceinline__ void scores(const float* sQ, const float* sK, int pitch, int chunks, int ty, int tx,
                                       float (&out)[4][4]) {
  float2 acc[4][4];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[a][i] = make_float2(0.f, 0.f);
  const float* q0 = sQ + 4 * ty * pitch;
  const float* k0 = sK + tx * pitch;
  const int xq = ty & 1, xk = tx & 7;
#pragma unroll 2
  for (int c = 0; c < chunks; ++c) {
    float4 q[4], k[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) q[a] = lds4(q0 + a * pitch + 4 * (c ^ xq));
#pragma unroll
    for (int i = 0; i < 4; ++i) k[i] = lds4(k0 + 16 * i * pitch + 4 * (c ^ xk));
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[a][i] = __ffma2_rn(make_float2(q[a].x, q[a].y), make_float2(k[i].x, k[i].y), acc[a][i]);
        acc[a][i] = __ffma2_rn(make_float2(q[a].z, q[a].w), make_float2(k[i].z, k[i].w), acc[a][i]);
      }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) out[a][i] = acc[a][i].x + acc[a][i].y;
}

__host__ __device__ inline size_t attn_smem(int d) {
  return (size_t(kRows + 2 * kKeys) * tile_pitch(d) + size_t(kKeys) * kRows) * sizeof(float);
}
__host__ __device__ inline size_t weights_smem(int d) { return size_t(2 * kRows + kKeys) * tile_pitch(d) * sizeof(float); }

// Joins the pieces of an item's rows, the whole block (see paged_join.cuh): the
// rows' maxima and sums by the lanes of a warp, 32 pieces at a time; then a thread
// has four columns of a row, and where the rows are few the threads share the
// pieces too.  One token of 4 heads of 32 on 3000 keys takes 16 us, 23 with a warp a
// row; 100 on 1000 keys 24 and 30.
template <class Out>
__device__ __forceinline__ void join_block(const PagedAttnParams& p, const PagedSeg<Plan>& s, int rows, float* scratch,
                                           const Out& out) {
  constexpr int kWarps = kThreads / 32, kEach = kRows / kWarps;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, d = p.d, pieces = s.pieces;
  float *max_of = scratch, *inv_of = scratch + kRows;
  float4* sums = reinterpret_cast<float4*>(scratch + 2 * kRows);
  auto first = [&](int k) { return int64_t(k == 0 ? 2 * s.owner + s.owner_slot : 2 * (s.owner + k)) * kRows; };
  auto add = [](float& m, float& l, float m2, float l2) {
    const float M = fmaxf(m, m2), ref = M == -INFINITY ? 0.f : M;
    l = fmaf(l, exp2f(m - ref), l2 * exp2f(m2 - ref));
    m = M;
  };
  float m[kEach], l[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) m[i] = -INFINITY, l[i] = 0.f;
  for (int k = lane; k < pieces; k += 32) {
    float2 ml[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (warp + kWarps * i < rows) ml[i] = __ldcg(&p.part_ml[first(k) + warp + kWarps * i]);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) add(m[i], l[i], ml[i].x, ml[i].y);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = warp + kWarps * i;
    if (r >= rows) break;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1)
      add(m[i], l[i], __shfl_down_sync(0xffffffffu, m[i], x), __shfl_down_sync(0xffffffffu, l[i], x));
    if (lane == 0) {
      max_of[r] = m[i] == -INFINITY ? 0.f : m[i];
      inv_of[r] = l[i] > 0.f ? 1.f / l[i] : 0.f;
      if (p.lse) p.lse[out(r)] = row_lse(m[i], l[i]);
    }
  }
  __syncthreads();
  const int chunks = d >> 2, items = rows * chunks;
  int groups = 1;  // that share an item's pieces
  while (groups < 32 && items * groups * 2 <= kThreads) groups *= 2;
  for (int x = tid; x < items * groups; x += kThreads) {  // (one round where groups > 1)
    const int g = x / items, it = x - g * items, r = it / chunks, c = it - r * chunks;
    const float M = max_of[r];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = g; k0 < pieces; k0 += 8 * groups) {
      float mk[8];
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int k = k0 + u * groups;
        mk[u] = -INFINITY;
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < pieces) {
          mk[u] = __ldcg(&p.part_ml[first(k) + r].x);
          v[u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (first(k) + r) * d + 4 * c));
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float w = exp2f(mk[u] - M);
        acc = make_float4(fmaf(v[u].x, w, acc.x), fmaf(v[u].y, w, acc.y), fmaf(v[u].z, w, acc.z), fmaf(v[u].w, w, acc.w));
      }
    }
    if (groups > 1) {
      sums[x] = acc;
    } else {
      const float inv = inv_of[r];
      store4(static_cast<float*>(p.o) + out(r) * d + 4 * c, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    }
  }
  if (groups > 1) {
    __syncthreads();
    if (tid < items) {
      const int r = tid / chunks, c = tid - r * chunks;
      const float inv = inv_of[r];
      float4 acc = sums[tid];
      for (int g = 1; g < groups; ++g) {
        const float4 v = sums[g * items + tid];
        acc = make_float4(acc.x + v.x, acc.y + v.y, acc.z + v.z, acc.w + v.w);
      }
      store4(static_cast<float*>(p.o) + out(r) * d + 4 * c, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    }
  }
}

// DC: 64-column chunks of the head dimension a thread accumulates (d <= 64 DC).
template <int DC>
__global__ void __launch_bounds__(kThreads, 2)
paged_attn_f32_kernel(const PagedAttnParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  extern __shared__ float sm[];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, d = p.d, ld = tile_pitch(d);
  const Lanes lanes(d);
  float* sQ = sm;
  float* sK = sQ + kRows * ld;
  float* sV = sK + kKeys * ld;
  float* sP = sV + kKeys * ld;  // [key][row], chunks of 4 rows swizzled by key & 7
  __shared__ int pool_rows[2][kKeys];  // of this tile's and the next one's keys
  __shared__ PagedWalk<Plan> walk;
  __shared__ int join, more;
  if (tid < 32) {
    PagedWalk<Plan> mine;
    mine.find(p, blockIdx.x, gridDim.x);
    if (tid == 0) {
      walk = mine;
      more = walk.next(p);
    }
  }
  __syncthreads();
  const float* q = static_cast<const float*>(p.q);
  while (more) {
    const PagedSeg<Plan> s = walk.seg;
    const int rows = s.blk.n_tok * p.group, b = s.b;
    const float* k_pool = static_cast<const float*>(p.k_pool);
    const float* v_pool = static_cast<const float*>(p.v_pool);
    // the first keys' pages, query rows, and each of this thread's rows' visible keys
    if (tid < kKeys) {
      const int j = s.u0 * kKeys + tid;
      pool_rows[0][tid] = pool_row(p.s, page_entry(p.s, b, j, s.blk.kv), s.hk, p.kv_heads, j, s.blk.kv, p.err);
    }
    lanes.each([&](int r, int c) {
      const int tok = r < rows ? p.per_group.div(r) : 0, head = r < rows ? p.per_group.mod(r) : 0;
      copy16(sQ + r * ld + 4 * (c ^ ((r >> 2) & 1)), q + int64_t(s.blk.row0 + tok) * p.ld_q + (s.hk * p.group + head) * d + 4 * c,
             r < rows);
    });
    __syncthreads();
    copy_keys(sK, k_pool, pool_rows[0], lanes, ld, d, true);
    copy_commit();
    int lim[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = 4 * ty + a;
      lim[a] = r < rows ? visible_keys(s.blk.view(), p.mask, s.blk.t0 + p.per_group.div(r)) : 0;
    }
    float m[4], l[4];
    float2 o[4][2 * DC];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      m[a] = -INFINITY;
      l[a] = 0.f;
#pragma unroll
      for (int c = 0; c < 2 * DC; ++c) o[a][c] = make_float2(0.f, 0.f);
    }
    for (int j = s.u0; j < s.u1; ++j) {
      const int k0 = j * kKeys, at = (j - s.u0) & 1, ahead = k0 + kKeys + tid;
      copy_wait();
      __syncthreads();  // K and Q are there, V and P are read
      copy_keys(sV, v_pool, pool_rows[at], lanes, ld, d, false);
      copy_commit();
      const bool fetch = tid < kKeys && j + 1 < s.u1;
      const int entry = fetch ? page_entry(p.s, b, ahead, s.blk.kv) : -1;
      float acc[4][4];
      scores(sQ, sK, ld, d >> 2, ty, tx, acc);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[a][i] = k0 + tx + 16 * i < lim[a] ? acc[a][i] * p.scale_log2 : -INFINITY;
          mx = fmaxf(mx, acc[a][i]);
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        const float mn = fmaxf(m[a], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;  // nothing visible so far: every exponential is 0
        const float corr = exp2f(m[a] - ref);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[a][i] = exp2f(acc[a][i] - ref);
          sum += acc[a][i];
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l[a] = fmaf(l[a], corr, sum);
        m[a] = mn;
#pragma unroll
        for (int c = 0; c < 2 * DC; ++c) o[a][c] = __fmul2_rn(o[a][c], make_float2(corr, corr));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(sP + (tx + 16 * i) * kRows + 4 * (ty ^ (tx & 7))) =
            make_float4(acc[0][i], acc[1][i], acc[2][i], acc[3][i]);
      if (fetch) pool_rows[at ^ 1][tid] = pool_row(p.s, entry, s.hk, p.kv_heads, ahead, s.blk.kv, p.err);
      copy_wait();
      __syncthreads();  // V, P and the next pages are there, K is read
      if (j + 1 < s.u1) {
        copy_keys(sK, k_pool, pool_rows[at ^ 1], lanes, ld, d, true);
        copy_commit();
      }
#pragma unroll 8
      for (int k = 0; k < kKeys; ++k) {
        const float4 pk = lds4(sP + k * kRows + 4 * (ty ^ (k & 7)));
        const float pr[4] = {pk.x, pk.y, pk.z, pk.w};
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          const int col = tx * 4 + 64 * c;
          if (col < d) {
            const float4 v = lds4(sV + k * ld + col);
#pragma unroll
            for (int a = 0; a < 4; ++a) {
              o[a][2 * c] = __ffma2_rn(make_float2(pr[a], pr[a]), make_float2(v.x, v.y), o[a][2 * c]);
              o[a][2 * c + 1] = __ffma2_rn(make_float2(pr[a], pr[a]), make_float2(v.z, v.w), o[a][2 * c + 1]);
            }
          }
        }
      }
    }
    const bool whole = s.whole();
    const int piece = 2 * blockIdx.x + s.slot;
    auto out_row = [&](int r) {
      return int64_t(s.blk.row0 + p.per_group.div(r)) * p.heads + s.hk * p.group + p.per_group.mod(r);
    };
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = 4 * ty + a;
      if (r >= rows) continue;
      const int64_t orow = out_row(r);
      const float inv = !whole ? 1.f : l[a] > 0.f ? 1.f / l[a] : 0.f;
#pragma unroll
      for (int c = 0; c < DC; ++c) {
        const int col = tx * 4 + 64 * c;
        if (col >= d) continue;
        const float4 x = make_float4(o[a][2 * c].x * inv, o[a][2 * c].y * inv, o[a][2 * c + 1].x * inv,
                                     o[a][2 * c + 1].y * inv);
        if (whole)
          store4(static_cast<float*>(p.o) + orow * d + col, x);
        else
          store4(p.part_o + (int64_t(piece) * kRows + r) * d + col, x);
      }
      if (tx == 0) {
        if (!whole)
          p.part_ml[int64_t(piece) * kRows + r] = make_float2(m[a], l[a]);
        else if (p.lse)
          p.lse[orow] = row_lse(m[a], l[a]);
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) join = last_piece(p.joined + 8 * s.owner, s.pieces);
      __syncthreads();
      if (join) {
        join_block(p, s, rows, sP, out_row);
      }
    }
    __syncthreads();  // sQ is read no more, nor the segment
    if (tid == 0) {
      walk.done(p);
      more = walk.next(p);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ weights
// A CTA takes its range of key blocks (paged_weights.cuh), 64 keys each, and the
// new tokens' rows past them in tiles of 64, the next tile's copy under way; a
// thread sums its 4 rows' weights of its 4 keys.  500 tokens of 8 heads a key
// head on 500 keys and 400 on 3000, 64 columns: 111 us, 380 with a CTA a block;
// clusters that shared a block's rows took 144, but 1800 instead of 250 (166 now)
// where most streams have one token.
__global__ void __launch_bounds__(kThreads, 2)
paged_weights_f32_kernel(const PagedWeightParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  extern __shared__ float sm[];
  __shared__ float part[16][kKeys];
  __shared__ int pool_rows[kKeys];
  __shared__ WeightWalk<kKeys> walk;
  __shared__ WeightBlk blk;
  __shared__ int join;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, d = p.d, ld = tile_pitch(d);
  const Lanes lanes(d);
  float* sK = sm;
  float* sQ = sK + kKeys * ld;  // two tiles
  const float* q = static_cast<const float*>(p.q);
  const int qt = p.per_tile.by;  // tokens of a tile
  if (tid < 32) {
    WeightWalk<kKeys> mine;
    mine.find(p);
    mine.next(p, blk);
    if (tid == 0) walk = mine;
  } else {
    clear_tails(p, int(blockIdx.x) * (kThreads / 32 - 1) + (tid >> 5) - 1, int(gridDim.x) * (kThreads / 32 - 1));
  }
  __syncthreads();
  while (blk.more) {
    const int k0 = blk.jt * kKeys, hk = blk.hk, b = blk.b, rt1 = blk.rt1;
    const SeqView v{blk.q0, blk.n, blk.kv};
    if (tid < kKeys)
      pool_rows[tid] = pool_row(p.s, page_entry(p.s, b, k0 + tid, v.kv), hk, p.kv_heads, k0 + tid, v.kv, p.err);
    auto copy_rows = [&](int tile, float* dst) {
      const int rows = min(qt, v.n - tile * qt) * p.group;
      lanes.each([&](int r, int c) {
        const int tok = r < rows ? p.per_group.div(r) : 0, head = r < rows ? p.per_group.mod(r) : 0;
        copy16(dst + r * ld + 4 * (c ^ ((r >> 2) & 1)),
               q + int64_t(v.q0 + tile * qt + tok) * p.ld_q + (hk * p.group + head) * d + 4 * c, r < rows);
      });
      copy_commit();
    };
    copy_rows(blk.rt0, sQ);
    __syncthreads();
    copy_keys(sK, static_cast<const float*>(p.k_pool), pool_rows, lanes, ld, d, true);
    copy_commit();
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    int at = 0;
    for (int t = blk.rt0; t < rt1; ++t, at ^= 1) {
      const int rows = min(qt, v.n - t * qt) * p.group;
      float lse2[4];
      int lim[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int r = 4 * ty + a;
        lim[a] = 0, lse2[a] = 0.f;
        if (r < rows) {
          const int tok = t * qt + p.per_group.div(r);
          const float lse = p.lse[int64_t(v.q0 + tok) * p.heads + hk * p.group + p.per_group.mod(r)];
          if (lse != -INFINITY) lim[a] = visible_keys(v, p.mask, tok);
          lse2[a] = -1.4426950408889634f * lse;
        }
      }
      copy_wait();
      __syncthreads();  // the tile is there, the one before is read
      if (t + 1 < rt1) copy_rows(t + 1, sQ + (at ^ 1) * kRows * ld);
      float acc[4][4];
      scores(sQ + at * kRows * ld, sK, ld, d >> 2, ty, tx, acc);
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (k0 + tx + 16 * i < lim[a]) w[i] += exp2f(fmaf(acc[a][i], p.scale_log2, lse2[a]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) part[ty][tx + 16 * i] = w[i];
    __syncthreads();
    float sum = 0.f;
    if (tid < kKeys)
      for (int y = 0; y < 16; ++y) sum += part[y][tid];
    bool mine = tid < kKeys;
    if (blk.pieces > 1) {
      if (mine) {
        p.part_w[(2 * blockIdx.x + blk.slot) * kKeys + tid] = sum;
        __threadfence();
      }
      __syncthreads();
      if (tid == 0) join = last_piece(p.joined + 8 * blk.owner, blk.pieces);
      __syncthreads();
      mine = mine && join;
      if (mine) {
        sum = __ldcg(&p.part_w[(2 * blk.owner + blk.owner_slot) * kKeys + tid]);
#pragma unroll 8
        for (int x = 1; x < blk.pieces; ++x) sum += __ldcg(&p.part_w[2 * (blk.owner + x) * kKeys + tid]);
      }
    }
    if (mine && k0 + tid < v.kv) {
      const int64_t to = (int64_t(b) * p.kv_heads + hk) * p.w_ld + k0 + tid;
      p.w_out[to] = fmaf(p.decay, p.w_in[to], sum);
    }
    __syncthreads();  // the block is read
    if (tid == 0) walk.next(p, blk);
    __syncthreads();
  }
}

template <int DC>
cudaError_t launch_attn(PagedAttnParams p, int grid, cudaStream_t st) {
  static unsigned done = 0;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(paged_attn_f32_kernel<DC>),
                                   int(attn_smem(128)), &done);
  if (e != cudaSuccess) return e;
  return launch_overlapped(paged_attn_f32_kernel<DC>, dim3(unsigned(grid)), kThreads, attn_smem(p.d), st, 0, p);
}

}  // namespace

cudaError_t launch_paged_attn_f32(PagedAttnParams p, int grid, cudaStream_t st) {
  return p.d <= 64 ? launch_attn<1>(p, grid, st) : launch_attn<2>(p, grid, st);
}

cudaError_t launch_paged_weights_f32(const PagedWeightParams& p, int sms, cudaStream_t st) {
  static unsigned done = 0;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(paged_weights_f32_kernel),
                                   int(weights_smem(128)), &done);
  if (e != cudaSuccess) return e;
  return launch_overlapped(paged_weights_f32_kernel, dim3(2 * unsigned(sms)), kThreads, weights_smem(p.d), st, 0, p);
}

}  // namespace arl2
