// Attention weights that cached keys received, bf16, on the tensor cores:
//
//   w_out[j] = decay w_in[j] + sum over rows that see j of exp(q k_j scale - lse[row])
//
// Keys lie on the accumulator's lanes: S^T = K Q^T, so that a key's sum over
// rows is one thread's, with no exchange and no maximum (lse is given).  A CTA
// holds 256 keys of one (stream, key head), two tiles of K, and takes the
// stream's rows past them in tiles of 128 (token, head of the group): each tile
// of Q serves both products, 32 bytes a clock from L2 instead of 64.  Bound: the
// exponentials (2048 clocks of the MUFU a 256 x 128 unit against the products'
// 1024; a part of them on the FMA pipe changed nothing); for single tokens the
// bytes of K.
//
// Work: paged_weights.cuh.  What lies past kv_len is cleared by the summing warps
// while the range is found.
//
// Warps: 0 finds the range, describes its blocks and loads K; 2 loads Q and puts
// the rows' lse next to it; 1 and 3 issue the products, a key tile each; four
// warpgroups sum, one for each key tile and half of the columns.  What a unit
// needs beyond its block's description is a few sums: with a walk over streams,
// heads and blocks in every role a unit took 2000 clocks without any arithmetic.
// Tensor memory: S^T of tile t, buffer i at columns (2 t + i) 128.

#include "layer.h"
#include "paged_join.cuh"
#include "paged_mma.cuh"
#include "paged_weights.cuh"
#include "params.h"

namespace arl2 {

namespace {

constexpr int kThreads = 640;
constexpr int kKeys = 256;  // of a block
constexpr int kQRing = 3, kBlks = 3;

enum {
  B_KF = 0,              // [2] a block's K loaded (bytes)
  B_KE = 2,              // [2] read (two commits)
  B_QF = 4,              // [kQRing] a Q tile loaded (bytes)
  B_QE = B_QF + kQRing,  // [kQRing] read (two commits)
  B_LF = B_QE + kQRing,  // [kQRing] its rows' lse in shared memory (warp 2)
  B_LE = B_LF + kQRing,  // [kQRing] read (16 warps)
  B_SF = B_LE + kQRing,  // [t][2] S^T in tensor memory (commit)
  B_SC = B_SF + 4,       // [t][2] read (8 warps)
  B_JF = B_SC + 4,       // [t] half 1's sums in shared memory (4 warps)
  B_JE = B_JF + 2,       // [t] read (4 warps)
  B_GF = B_JE + 2,       // [kBlks] block described
  B_GE = B_GF + kBlks,   // [kBlks] description read (Q loader, issuers, 16 summing warps)
  B_DRAIN = B_GE + kBlks,
  B_COUNT
};
constexpr int kSmem = 232448, kLayout = 2 * 2 * kTile + kQRing * kTile + kQRing * 512 + 1024 + kBlks * 56 + 8 * B_COUNT + 16;
static_assert(kLayout <= kSmem, "shared memory");

using Stream = WeightStream<kKeys>;
using Blk = WeightBlk;
using Walk = WeightWalk<kKeys>;
static_assert(sizeof(Blk) == 56 && kBlks * 56 % 8 == 0, "shared memory");

// The blocks as a role meets them (a whole warp).
struct BlkReader {
  const Blk* ring;
  uint64_t* bars;
  uint32_t k = 0;
  __device__ const Blk* next(const WaitCtl& w) {
    if (!warp_wait(&bars[B_GF + k % kBlks], (k / kBlks) & 1, w)) return nullptr;
    const Blk* g = &ring[k % kBlks];
    return g->more ? g : nullptr;
  }
  __device__ void done() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars[B_GE + k % kBlks]);
    ++k;
  }
};

// A place in the Q ring.
struct QPos {
  uint32_t slot = kQRing - 1, round = 0xffffffffu;  // before the first
  __device__ void next() {
    if (++slot == kQRing) slot = 0, ++round;
  }
};

__device__ __forceinline__ void k_role(const PagedWeightParams& p, const CUtensorMap* tm_k, uint64_t* bars, Blk* ring,
                                       uint8_t* sK, const WaitCtl& w) {
  const int lane = threadIdx.x & 31;
  Walk walk;
  walk.find(p);
  int b = -1, hk = -1;
  BoxRows<128> rows;
  for (uint32_t k = 0;; ++k) {
    if (k >= kBlks && !warp_wait(&bars[B_GE + k % kBlks], (k / kBlks - 1) & 1, w)) return;
    Blk& blk = ring[k % kBlks];
    const bool more = walk.next(p, blk);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[B_GF + k % kBlks]);
    if (!more) return;
    if (blk.b != b || blk.hk != hk) {  // a (stream, key head): its key tiles lie in a row
      b = blk.b, hk = blk.hk;
      rows = BoxRows<128>(p.s, b, blk.kv, hk, p.kv_heads, 2 * blk.jt, 2 * ((blk.kv + kKeys - 1) / kKeys), p.err);
    }
    const uint32_t i = k & 1;
    if (k >= 2 && !warp_wait(&bars[B_KE + i], ((k >> 1) - 1) & 1, w)) return;
    if (lane == 0) mbar_expect_tx(&bars[B_KF + i], 2 * kTile);
    __syncwarp();
#pragma unroll
    for (int t = 0; t < 2; ++t) rows.load(2 * blk.jt + t, sK + (2 * i + t) * kTile, tm_k, &bars[B_KF + i]);
    __syncwarp();
  }
}

// Q tiles, and their rows' -lse log2(e): -inf where a row adds nothing.
__device__ __forceinline__ void q_role(const PagedWeightParams& p, const CUtensorMap* tm_q, BlkReader blks, int qt,
                                       uint64_t* bars, uint8_t* sQ, float* sL, const WaitCtl& w) {
  const int lane = threadIdx.x & 31;
  QPos q;
  for (const Blk* k = blks.next(w); k; blks.done(), k = blks.next(w)) {
    for (int rt = k->fresh ? k->rt0 : k->rt0 + 1; rt < k->rt1; ++rt) {
      q.next();
      const int tok = rt * qt, rows = min(qt, k->n - tok) * p.group;
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = lane + 32 * i, t = p.per_group.div(r);
        x[i] = -INFINITY;
        if (r < rows) x[i] = p.lse[int64_t(k->q0 + tok + t) * p.heads + k->hk * p.group + (r - t * p.group)];
      }
      if (q.round > 0 && !warp_wait(&bars[B_QE + q.slot], (q.round - 1) & 1, w)) return;
      if (lane == 0) {
        mbar_expect_tx(&bars[B_QF + q.slot], 2u * uint32_t(qt * p.group) * 128u);
        for (int h = 0; h < 2; ++h)
          tma_load_3d(sQ + q.slot * kTile + h * kHalfTile, tm_q, &bars[B_QF + q.slot], h * 64, k->hk * p.group, k->q0 + tok);
      }
      if (q.round > 0 && !warp_wait(&bars[B_LE + q.slot], (q.round - 1) & 1, w)) return;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sL[q.slot * 128 + lane + 32 * i] = x[i] == -INFINITY ? x[i] : -1.4426950408889634f * x[i];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_LF + q.slot]);
    }
  }
}

// The products of key tile t (one warp, see elect_one).
__device__ __forceinline__ void mma_role(const PagedWeightParams& p, BlkReader blks, int qt, uint64_t* bars, uint8_t* sK,
                                         uint8_t* sQ, uint32_t tmem, int t, const WaitCtl& w) {
  const uint32_t dk = desc_lo(sK + t * kTile, 16), dq = desc_lo(sQ, 16), el = elect_one();
  QPos q;
  uint32_t g = 0;
  for (const Blk* k = blks.next(w); k; blks.done(), k = blks.next(w)) {
    const uint32_t i = blks.k & 1;
    if (!warp_wait(&bars[B_KF + i], (blks.k >> 1) & 1, w)) return;
    const int rt0 = k->rt0, units = k->rt1 - rt0, fresh = k->fresh;
    int tokens = k->n - rt0 * qt;  // from the unit's first on
#pragma unroll 2
    for (int u = 0; uniform(u < units); ++u, tokens -= qt) {
      if (uniform(u > 0 || fresh)) {
        if (uniform(q.round != 0xffffffffu)) mma_commit_el(&bars[B_QE + q.slot], el);
        q.next();
        if (!warp_wait(&bars[B_QF + q.slot], q.round & 1, w)) return;
      }
      const uint32_t buf = g & 1;
      if (g >= 2 && !warp_wait(&bars[B_SC + 2 * t + buf], ((g >> 1) - 1) & 1, w)) return;
      tc_fence_after();
      const uint32_t cols = (min(tokens, qt) * p.group + 15) & ~15;
      mma_tile<128>(tmem + (2 * t + buf) * 128, dk + 2 * i * (kTile >> 4), dq + q.slot * (kTile >> 4),
                    idesc_bf16(128, 0, 0, 0) | (cols >> 3) << 17, el);
      mma_commit_el(&bars[B_SF + 2 * t + buf], el);
      ++g;
    }
    mma_commit_el(&bars[B_KE + i], el);
  }
}

// Sum of 2^(s scale + nl) over 32 columns [c0, c0 + 32); with kMask only those
// in [lo, hi).
template <bool kMask>
__device__ __forceinline__ float2 sum_chunk(const uint32_t* r, const float4* nl, const float2 sc, int c0, int lo, int hi,
                                            float2 acc) {
#pragma unroll
  for (int x = 0; x < 16; x += 2) {
    const float4 n4 = nl[x / 2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float2 e = __ffma2_rn(make_float2(__uint_as_float(r[2 * (x + y)]), __uint_as_float(r[2 * (x + y) + 1])), sc,
                            y == 0 ? make_float2(n4.x, n4.y) : make_float2(n4.z, n4.w));
      e = make_float2(fast_exp2(e.x), fast_exp2(e.y));
      if (kMask) {
        const int c = c0 + 2 * (x + y);
        e.x = c >= lo && c < hi ? e.x : 0.f;
        e.y = c + 1 >= lo && c + 1 < hi ? e.y : 0.f;
      }
      acc = __fadd2_rn(acc, e);
    }
  }
  return acc;
}

// Warpgroup (t, half): key tile t, columns [64 half, 64 half + 64) of each unit.
// Half 1 hands its sums of a block to half 0 through sJ.
__device__ __forceinline__ void sum_role(const PagedWeightParams& p, BlkReader blks, int qt, uint64_t* bars, const float* sL,
                                         float* sJ, uint32_t tmem, int t, int half, const WaitCtl& w) {
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, row = quarter * 32 + lane;
  const uint32_t tS = tmem + t * 256 + half * 64 + (uint32_t(quarter * 32) << 16);
  const float2 sc = make_float2(p.scale_log2, p.scale_log2);
  const int col0 = half * 64;
  QPos q;
  uint32_t g = 0;
  for (const Blk* k = blks.next(w); k; blks.done(), k = blks.next(w)) {
    const int key = k->jt * kKeys + t * 128 + row, units = k->rt1 - k->rt0;
    // the key is seen by the tile's columns [lo, rows)
    int from = 0;  // tokens from the unit's first on that do not see it
    if (p.mask.by > 0) {
      Stream s;
      s.v = SeqView{0, k->n, k->kv};
      from = s.first_token(p.mask, key) - k->rt0 * qt;
    }
    int tokens = k->n - k->rt0 * qt;
    float2 sum = make_float2(0.f, 0.f);
    for (int u = 0; u < units; ++u, tokens -= qt, from -= qt) {
      if (u > 0 || k->fresh) {
        if (q.round != 0xffffffffu) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_LE + q.slot]);
        }
        q.next();
        if (!warp_wait(&bars[B_LF + q.slot], q.round & 1, w)) return;
      }
      const uint32_t buf = g & 1;
      if (!warp_wait(&bars[B_SF + 2 * t + buf], (g >> 1) & 1, w)) return;
      ++g;
      tc_fence_after();
      const int rows = min(tokens, qt) * p.group, lo = from <= 0 ? 0 : min(from, qt) * p.group;
      const bool masked = rows < 128 || __any_sync(0xffffffffu, lo > 0);
      const float4* nl = reinterpret_cast<const float4*>(sL + q.slot * 128 + col0);
      // (columns from the product's width on hold an older product, and are masked)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t r[32];
        const bool some = col0 + 32 * c < rows;
        if (some) {
          tmem_ld32(tS + buf * 128 + c * 32, r);
          tmem_wait_ld();
        }
        if (c == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_SC + 2 * t + buf]);
        }
        if (!masked)
          sum = sum_chunk<false>(r, nl + 8 * c, sc, 0, 0, 0, sum);
        else if (some)
          sum = sum_chunk<true>(r, nl + 8 * c, sc, col0 + 32 * c, lo, rows, sum);
      }
    }
    float total = sum.x + sum.y;
    if (half == 1) {
      if (blks.k > 0 && !warp_wait(&bars[B_JE + t], (blks.k - 1) & 1, w)) return;
      sJ[t * 128 + row] = total;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_JF + t]);
    } else {
      if (!warp_wait(&bars[B_JF + t], blks.k & 1, w)) return;
      total += sJ[t * 128 + row];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_JE + t]);
      if (k->pieces > 1) {
        const int mine = t * 128 + row;
        p.part_w[(2 * blockIdx.x + k->slot) * kKeys + mine] = total;
        __threadfence();
        __syncwarp();
        int last = 0;
        if (lane == 0) last = last_piece(p.joined + 8 * k->owner + 4 * t + quarter, k->pieces);
        if (!__shfl_sync(0xffffffffu, last, 0)) continue;
        total = __ldcg(&p.part_w[(2 * k->owner + k->owner_slot) * kKeys + mine]);
#pragma unroll 4
        for (int i = 1; i < k->pieces; ++i) total += __ldcg(&p.part_w[2 * (k->owner + i) * kKeys + mine]);
      }
      const int64_t at = (int64_t(k->b) * p.kv_heads + k->hk) * p.w_ld + key;
      if (key < k->kv) p.w_out[at] = fmaf(p.decay, p.w_in[at], total);
    }
  }
}

// ------------------------------------------------------------------ kernel
__global__ void __launch_bounds__(kThreads, 1)
paged_weights_bf16_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const PagedWeightParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // (the window begins on 1024 bytes; a layout that does not fit is refused)
  if (size_t(smem - smem_raw) + kLayout > size_t(kSmem)) {
    grid_dependency_wait();
    if (threadIdx.x == 0) record_error(p.err, kDevBadShape);
    return;
  }
  uint8_t* sK = smem;                // [2 blocks][2 tiles]
  uint8_t* sQ = smem + 4 * kTile;    // [kQRing]
  float* sL = reinterpret_cast<float*>(sQ + kQRing * kTile);  // [kQRing][128]
  float* sJ = sL + kQRing * 128;  // [2][128]
  Blk* blks = reinterpret_cast<Blk*>(sJ + 256);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(blks) + kBlks * sizeof(Blk));
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, qt = 128 / p.group;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i)
      mbar_init(&bars[i], i == B_KE || i == B_KE + 1 || (i >= B_QE && i < B_QE + kQRing) || i == B_DRAIN ? 2
                          : i >= B_LE && i < B_LE + kQRing                                             ? 16
                          : i >= B_SC && i < B_JF                                                      ? 8
                          : i >= B_JF && i < B_GF                                                      ? 4
                          : i >= B_GE && i < B_DRAIN                                                   ? 19
                                                                                                       : 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2) tmem_alloc(tmem_holder, 512);
  if (warp == 0 && lane == 0) {
    tma_prefetch(&tm_q);
    tma_prefetch(&tm_k);
  }
  grid_dependency_wait();
  allow_dependent_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitCtl w{abort_flag, p.err, p.wait_limit_ns};
  const BlkReader reader{blks, bars};
  if (warp == 0) {
    k_role(p, &tm_k, bars, blks, sK, w);
  } else if (warp == 2) {
    q_role(p, &tm_q, reader, qt, bars, sQ, sL, w);
  } else if (warp < 4) {
    mma_role(p, reader, qt, bars, sK, sQ, tmem, warp >> 1, w);
  } else {
    clear_tails(p, blockIdx.x * 16 + warp - 4, gridDim.x * 16);
    const int wg = (warp >> 2) - 1;
    sum_role(p, reader, qt, bars, sL, sJ, tmem, wg & 1, wg >> 1, w);
  }
  // shared and tensor memory are released once a commit behind every product has arrived
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

// Where no stream has new tokens.
__global__ void __launch_bounds__(256) paged_weights_fade_kernel(const PagedWeightParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  clear_tails(p, blockIdx.x * 8 + (threadIdx.x >> 5), gridDim.x * 8, p.err);
}

}  // namespace

cudaError_t launch_paged_weights_bf16(const PagedWeightParams& p, const CUtensorMap& tk, int sms, cudaStream_t st) {
  static unsigned done = 0;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(paged_weights_bf16_kernel), kSmem, &done);
  if (e != cudaSuccess) return e;
  if (p.s.tokens < 1 || p.s.max_q < 1 || p.s.max_kv < 1)
    return launch_overlapped(paged_weights_fade_kernel, dim3(unsigned(sms)), 256, 0, st, 0, p);
  CUtensorMap tq;
  if (!paged_query_map(&tq, p.q, p.s.tokens, p.heads, p.group, p.ld_q)) return cudaErrorInvalidValue;
  return launch_overlapped(paged_weights_bf16_kernel, dim3(unsigned(sms)), kThreads, kSmem, st, 0, tq, tk, p);
}

}  // namespace arl2
