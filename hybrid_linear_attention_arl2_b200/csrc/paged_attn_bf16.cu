// Attention of new tokens over a paged cache, bf16, on the tensor cores:
//
//   O = softmax(Q K^T scale) V over the visible keys,  lse = log sum exp
//
// One CTA an SM walks its range of units (PagedPlan).  Query rows of a (stream,
// key head) are the pairs (token, head of the group), so the heads that share
// keys share their tile: a tile is 128 rows.  Two tiles are in flight, and each
// softmax warpgroup owns one: S_t = Q_t K^T (128 x 128, fp32 in tensor memory),
// P_t over S_t in place (bf16 pairs), O_t += P_t V.  While warpgroup 0 is on its
// exponentials the tensor core does warpgroup 1's products and the other way
// round.  A block with one tile (single tokens, a chunk's tail) takes two key
// tiles at once instead: both halves hold the same queries, half t the key
// tiles 2 u + t, and their (m, l, O) are joined at the end, so that a single row
// keeps as many bytes in flight as 256 rows do.
//
// Warps: 0 loads (Q by one box a tile, K and V by boxes inside pages, one lane a
// box, page numbers fetched a tile ahead), 1 issues the products, 4-7 and 8-11
// softmax, O's rescaling (only when a row's maximum grows by more than 8 in
// log2 units: P <= 256), and the output.  A softmax thread has one row.
// The issuer's order, which the loader's ring of 32 KB tiles follows, is
//   S_0(0) S_1(0), then for each unit u:  PV_0(u) S_0(u+1) PV_1(u) S_1(u+1);
// S_t(u + 1) overwrites P_t(u) behind PV_t(u) in the pipe, and its completion
// stands for PV_t(u)'s, after which O_t may be rescaled.
// Tensor memory: S_0 / P_0 [0,128), S_1 / P_1 [128,256), O_0 [256,384), O_1 [384,512).
//
// Rounding: P and O to bf16 (half a step, 2^-8, each); S, m, l and O's sums are
// fp32.  Rows of V past the stream's keys are cleared in shared memory before a
// product sees them: what the pool holds there may be NaN.

#include "layer.h"
#include "paged_combine.cuh"
#include "paged_mma.cuh"
#include "params.h"

namespace arl2 {

namespace {

constexpr int kThreads = 384;
constexpr int kRing = 5;
// registers a thread: at launch, and after the split between the control warps and the softmax
constexpr int kLaunchRegs = 168, kCtlRegs = 72, kSoftmaxRegs = 216;
static_assert(128 * kCtlRegs + 256 * kSoftmaxRegs <= kThreads * kLaunchRegs, "register split too large");
using Plan = PagedPlan<2, 128, 128>;

enum {
  B_QF = 0,            // Q tiles loaded (bytes)
  B_QE,                // Q read by the segment's last S (commit)
  B_SF,                // [2] S_t in tensor memory (commit)
  B_PF = B_SF + 2,     // [2] P_t written (the warpgroup's 4 warps)
  B_OF = B_PF + 2,     // [2] O_t final (commit)
  B_MG = B_OF + 2,     // half 1's statistics in shared memory (4 warps)
  B_MD,                // half 1's O read by warpgroup 0 (4 warps)
  B_RF,                // [kRing] ring slot loaded (bytes)
  B_RE = B_RF + kRing, // [kRing] ring slot read (commit)
  B_DRAIN = B_RE + kRing,
  B_COUNT
};

// Key tiles of a segment for each half: the units both walk.
struct Work {
  bool dual;   // two tiles of rows on the same key tiles; else one tile on alternate ones
  int n[2];    // units each half takes part in
  int j0;      // first unit
  __device__ int tile(int t, int u) const { return dual ? j0 + u : 2 * (j0 + u) + t; }
};
__device__ __forceinline__ Work work_of(const PagedSeg<Plan>& s, int group, int mask_block) {
  Work w;
  w.dual = s.blk.tiles == 2;
  w.j0 = s.u0;
  const int qt = 128 / group;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = w.dual ? min((t + 1) * qt, s.blk.n_tok) : s.blk.n_tok;  // the tile's tokens end
    const int nk = (visible_keys(s.blk.v, mask_block, s.blk.t0 + last - 1) + 127) >> 7;
    const int units = w.dual ? nk : (nk + 1 - t) >> 1;
    w.n[t] = max(0, min(units, s.u1) - s.u0);
  }
  return w;
}

// ------------------------------------------------------------------ loads
__device__ __forceinline__ void load_role(const PagedAttnParams& p, const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                                          const CUtensorMap* tm_v, const PagedRange& range, uint64_t* bars, uint8_t* sQ,
                                          uint8_t* sR, const WaitCtl& w) {
  const int lane = threadIdx.x & 31;
  const int qt = 128 / p.group;
  uint32_t ring = 0, k = 0;
  PagedWalk<Plan> walk(range, p.n_qblk);
  while (walk.next(p.s, p.n_qblk, p.group, p.kv_heads, p.mask_block)) {
    const PagedSeg<Plan>& s = walk.seg;
    const Work wk = work_of(s, p.group, p.mask_block);
    if (wk.n[0] == 0 && wk.n[1] == 0) continue;
    if (k > 0 && !warp_wait(&bars[B_QE], (k - 1) & 1, w)) return;
    if (lane == 0) {
      const uint32_t bytes = uint32_t(qt * p.group) * 128u;
      mbar_expect_tx(&bars[B_QF], 2u * uint32_t(s.blk.tiles) * bytes);
      for (int t = 0; t < s.blk.tiles; ++t)
        for (int h = 0; h < 2; ++h)
          tma_load_3d(sQ + t * kTile + h * kHalfTile, tm_q, &bars[B_QF], h * 64, s.hk * p.group,
                      s.blk.q0 + s.blk.t0 + t * qt);
    }
    // K and V tiles in the order in which the products take them: a dual
    // segment's K(u), V(u); else K(0), K(1), V(0), K(2), V(1), ... of its tiles
    const int n = wk.dual ? wk.n[1] : wk.n[0] + wk.n[1], lag = wk.dual ? 0 : 1, j0 = wk.tile(0, 0);
    BoxRows rk(p.s, s.b, s.blk.v.kv, s.hk, p.kv_heads, j0, j0 + n, p.err), rv = rk;
    auto load = [&](BoxRows& rows, int i, const CUtensorMap* tm) {
      const uint32_t slot = ring % kRing;
      if (ring >= kRing && !warp_wait(&bars[B_RE + slot], ((ring / kRing) - 1) & 1, w)) return false;
      if (lane == 0) mbar_expect_tx(&bars[B_RF + slot], kTile);
      __syncwarp();
      rows.load(j0 + i, sR + slot * kTile, tm, &bars[B_RF + slot]);
      __syncwarp();
      ++ring;
      return true;
    };
    for (int i = 0; i < n + lag; ++i) {
      if (i < n && !load(rk, i, tm_k)) return;
      if (i >= lag && !load(rv, i - lag, tm_v)) return;
    }
    ++k;
  }
}

// ------------------------------------------------------------------ products
// One warp (see elect_one).  Its order, with S_t(u + 1) right behind PV_t(u), is the loader's.
__device__ __forceinline__ void mma_role(const PagedAttnParams& p, const PagedRange& range, uint64_t* bars,
                                         uint8_t* sQ, uint8_t* sR, uint32_t tmem, const WaitCtl& w) {
  const uint32_t id_s = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, 128, 0, 1);
  const uint64_t dq = smem_desc_sw128(smem_u32(sQ), 16, 1024), dk = smem_desc_sw128(smem_u32(sR), 16, 1024);
  const uint64_t dv = smem_desc_sw128(smem_u32(sR), kHalfTile, 1024);
  const uint32_t el = elect_one();
  const int lane = threadIdx.x & 31;
  uint32_t ring = 0, k = 0, pf = 0;  // pf: a parity bit for each half
  PagedWalk<Plan> walk(range, p.n_qblk);
  while (walk.next(p.s, p.n_qblk, p.group, p.kv_heads, p.mask_block)) {
    const PagedSeg<Plan>& s = walk.seg;
    const Work wk = work_of(s, p.group, p.mask_block);
    if (wk.n[0] == 0 && wk.n[1] == 0) continue;
    if (!warp_wait(&bars[B_QF], k & 1, w)) return;
    const bool dual = uniform(wk.dual);
    const int left = uniform(s.blk.v.kv - wk.tile(0, 0) * 128);  // keys from the first tile on
    // S of half t, with the K tile in ring position pos; `last`: the tile's last use
    auto scores = [&](int t, uint32_t pos, bool last) {
      const uint32_t slot = pos % kRing;
      if (!warp_wait(&bars[B_RF + slot], (pos / kRing) & 1, w)) return false;
      mma_tile(tmem + t * 128, dq + (dual ? t * (kTile >> 4) : 0), dk + slot * (kTile >> 4), id_s, el);
      mma_commit_el(&bars[B_SF + t], el);
      if (last) mma_commit_el(&bars[B_RE + slot], el);
      return true;
    };
    // O += P V; `clear`: the tile's first use; `fin`: the half's last product
    auto values = [&](int t, int u, uint32_t pos, bool clear, bool last, bool fin) {
      const uint32_t slot = pos % kRing;
      if (!warp_wait(&bars[B_RF + slot], (pos / kRing) & 1, w)) return false;
      const int valid = min(128, left - (dual ? u : 2 * u + t) * 128);
      if (clear && (valid & 15)) {  // rows past the stream's keys
        uint8_t* tile = sR + slot * kTile;
        for (int i = valid * 8 + lane; i < ((valid + 15) & ~15) * 8; i += 32) {
          *reinterpret_cast<uint4*>(tile + i * 16) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(tile + kHalfTile + i * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        __syncwarp();
      }
      if (!warp_wait(&bars[B_PF + t], (pf >> t) & 1, w)) return false;
      pf ^= 1u << t;
      tc_fence_after();
      const uint64_t b = dv + slot * (kTile >> 4);
      const uint32_t o = tmem + 256 + t * 128, a = tmem + t * 128;
      if (valid == 128) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mma_ts_el(o, a + kk * 8, b + kk * 128, id_o, kk > 0 || u > 0, el);
      } else {
        for (int kk = 0; kk * 16 < valid; ++kk) mma_ts_el(o, a + kk * 8, b + kk * 128, id_o, kk > 0 || u > 0, el);
      }
      if (last) mma_commit_el(&bars[B_RE + slot], el);
      if (fin) mma_commit_el(&bars[B_OF + t], el);
      return true;
    };
    if (dual) {
      const int n0 = uniform(wk.n[0]), n1 = uniform(wk.n[1]);  // n0 <= n1: the first tile's tokens are the earlier ones
      if (n0 > 0 && !scores(0, ring, false)) return;
      if (!scores(1, ring, true)) return;
      for (int u = 0; u < n1; ++u) {
        const uint32_t kp = ring + 2 * u + 2, vp = ring + 2 * u + 1;
        if (u + 1 == n1) mma_commit_el(&bars[B_QE], el);  // every S of the segment has been issued
        if (u < n0 && !values(0, u, vp, true, false, u + 1 == n0)) return;
        if (u + 1 < n0 && !scores(0, kp, false)) return;
        if (!values(1, u, vp, u >= n0, true, u + 1 == n1)) return;
        if (u + 1 < n1 && !scores(1, kp, true)) return;
      }
      ring += 2 * n1;
    } else {
      const int n = uniform(wk.n[0] + wk.n[1]);  // tile i belongs to half i & 1
      if (!scores(0, ring, true)) return;
      if (n > 1 && !scores(1, ring + 1, true)) return;
      for (int i = 0; i < n; ++i) {
        if (i + 2 == n || n == 1) mma_commit_el(&bars[B_QE], el);
        // ring: K(0) K(1) V(0) K(2) V(1) K(3) ... V(n - 2) V(n - 1)
        const uint32_t vp = ring + (n == 1 ? 1 : i + 2 < n ? 2 * i + 2 : n + i);
        if (!values(i & 1, i >> 1, vp, true, true, i + 2 >= n)) return;
        if (i + 2 < n && !scores(i & 1, ring + 2 * i + 3, true)) return;
      }
      ring += 2 * n;
    }
    ++k;
  }
}

// ------------------------------------------------------------------ softmax and output
// Of the 16 pairs of a 32-column chunk this many take the FMA-pipe exponential.
constexpr int kPolyPerChunk = 3;

template <bool kPoly>
__device__ __forceinline__ float exp_chunk(const uint32_t* r, const float2 sc, const float2 nm, uint32_t (&pk)[16]) {
  float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    const float2 y = __ffma2_rn(make_float2(__uint_as_float(r[2 * x]), __uint_as_float(r[2 * x + 1])), sc, nm);
    const bool poly = kPoly && (x % 3 == 1) && (x / 3) < kPolyPerChunk;
    const float2 e = poly ? exp2_fma_pair(y) : make_float2(fast_exp2(y.x), fast_exp2(y.y));
    s2[x & 1] = __fadd2_rn(s2[x & 1], e);
    pk[x] = pack_bf16x2(e.x, e.y);
  }
  const float2 sa = __fadd2_rn(s2[0], s2[1]);
  return sa.x + sa.y;
}

// A warp's walk, in shared memory: the rows' 128 logits leave no registers for it.
struct SharedWalk {
  PagedWalk<Plan> walk;
  Work wk;
  bool more;
};

constexpr int kSmem =
    1024 + 2 * kTile + kRing * kTile + 8 * B_COUNT + 16 + 256 * 4 + 8 * int(sizeof(SharedWalk));
static_assert(kSmem <= 232448, "shared memory");

__device__ __forceinline__ void softmax_role(const PagedAttnParams& p, const PagedRange& range, uint64_t* bars,
                                             float* stats, SharedWalk* sw, uint32_t tmem, int t, const WaitCtl& w) {
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, row = quarter * 32 + lane;
  const uint32_t lane_off = uint32_t(quarter * 32) << 16;
  const uint32_t tS = tmem + t * 128 + lane_off, tO = tmem + 256 + t * 128 + lane_off;
  const float2 sc = make_float2(p.scale_log2, p.scale_log2);
  const int qt = 128 / p.group;
  uint32_t sf = 0, of = 0, merges = 0;
  if (lane == 0) sw->walk = PagedWalk<Plan>(range, p.n_qblk);
  while (true) {
    __syncwarp();  // every lane is done with the previous segment
    if (lane == 0) {
      sw->more = sw->walk.next(p.s, p.n_qblk, p.group, p.kv_heads, p.mask_block);
      if (sw->more) sw->wk = work_of(sw->walk.seg, p.group, p.mask_block);
    }
    __syncwarp();
    if (!sw->more) return;
    const PagedSeg<Plan>& s = sw->walk.seg;
    const Work& wk = sw->wk;
    const int tok0 = s.blk.t0 + (wk.dual ? t * qt : 0);
    const int rows = (wk.dual ? min(qt, s.blk.n_tok - t * qt) : s.blk.n_tok) * p.group;
    const bool live = row < rows, warp_live = quarter * 32 < rows;
    const int lim = live ? visible_keys(s.blk.v, p.mask_block, tok0 + row / p.group) : s.blk.v.kv;
    float m = -INFINITY, l = 0.f;
    const int n = wk.n[t], step = wk.dual ? 128 : 256;
    int left = lim - wk.tile(t, 0) * 128;  // visible keys from the tile's first on
    for (int u = 0; u < n; ++u, left -= step) {
      if (!warp_wait(&bars[B_SF + t], sf & 1, w)) return;
      ++sf;
      if (warp_live) {
        tc_fence_after();
        uint32_t r[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32 * c]));
        tmem_wait_ld();
        const bool masked = __any_sync(0xffffffffu, left < 128);
        if (masked) {
#pragma unroll
          for (int x = 0; x < 128; ++x)
            if (x >= left) r[x] = __float_as_uint(-INFINITY);
        }
        float m4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          m4[q] = fmax3(__uint_as_float(r[q]), __uint_as_float(r[4 + q]), __uint_as_float(r[8 + q]));
#pragma unroll
        for (int x = 12; x < 124; x += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q) m4[q] = fmax3(m4[q], __uint_as_float(r[x + q]), __uint_as_float(r[x + 4 + q]));
#pragma unroll
        for (int q = 0; q < 4; ++q) m4[q] = fmaxf(m4[q], __uint_as_float(r[124 + q]));
        const float mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]) * sc.x;
        const bool need = mx > m + 8.f;  // (also a row's first finite maximum)
        const float mg = need ? mx : m;
        const float ref = mg == -INFINITY ? 0.f : mg;  // nothing visible so far: every exponential is 0
        const float f = fast_exp2(m - ref);
        if (u > 0 && __any_sync(0xffffffffu, need)) {  // O *= 2^(old m - new m), 1 for rows that keep m
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {
            uint32_t o[16];
            tmem_ld16(tO + q * 16, o);
            tmem_wait_ld();
            const float g = need ? f : 1.f;
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * g);
            tmem_st16(tO + q * 16, o);
          }
        }
        const float2 nm = make_float2(-ref, -ref);
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pc[16];
          sum += masked ? exp_chunk<false>(&r[32 * c], sc, nm, pc) : exp_chunk<true>(&r[32 * c], sc, nm, pc);
          tmem_st16(tS + c * 16, pc);
        }
        l = need ? fmaf(l, f, sum) : l + sum;
        m = mg;
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_PF + t]);
    }
    const bool have = n > 0;
    if (have) {
      if (!warp_wait(&bars[B_OF + t], of & 1, w)) return;
      ++of;
      tc_fence_after();
    }
    float a = 1.f, a1 = 0.f;  // O = a O_t + a1 O_1
    const bool join = !wk.dual && wk.n[1] > 0;
    if (join) {
      if (t == 1) {  // warpgroup 0 writes the block's rows
        stats[row] = m;
        stats[128 + row] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_MG]);
        if (!warp_wait(&bars[B_MD], merges & 1, w)) return;
        ++merges;
        continue;
      }
      if (!warp_wait(&bars[B_MG], merges & 1, w)) return;
      ++merges;
      const float m1 = stats[row], l1 = stats[128 + row], M = fmaxf(m, m1), ref = M == -INFINITY ? 0.f : M;
      a = fast_exp2(m - ref);
      a1 = fast_exp2(m1 - ref);
      l = l * a + l1 * a1;
      m = M;
    } else if (!wk.dual && t == 1) {
      continue;
    }
    const bool whole = s.whole();
    const int piece = 2 * blockIdx.x + s.slot();
    if (whole) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      a *= inv, a1 *= inv;
    }
    const int64_t orow = int64_t(s.blk.q0 + tok0 + row / p.group) * p.heads + s.hk * p.group + row % p.group;
    const int64_t prow = int64_t(piece) * 256 + t * 128 + row;
    if (!whole && t == 0 && row == 0) p.rec[piece] = make_int4(s.f, s.hk, s.starts(), s.ends());
    if (warp_live) {
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t o[32], o1[32];
        if (have) tmem_ld32(tO + q * 32, o);
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
          char* dst = reinterpret_cast<char*>(static_cast<__nv_bfloat16*>(p.o) + orow * 128 + q * 32);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t v[8];
#pragma unroll
            for (int x = 0; x < 8; ++x)
              v[x] = pack_bf16x2(__uint_as_float(o[c * 16 + 2 * x]), __uint_as_float(o[c * 16 + 2 * x + 1]));
            if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
              store_sector(dst + c * 32, v);
            } else {
              reinterpret_cast<uint4*>(dst + c * 32)[0] = make_uint4(v[0], v[1], v[2], v[3]);
              reinterpret_cast<uint4*>(dst + c * 32)[1] = make_uint4(v[4], v[5], v[6], v[7]);
            }
          }
        } else {
          float* dst = p.part_o + prow * 128 + q * 32;
#pragma unroll
          for (int c = 0; c < 4; ++c) store_sector(dst + c * 8, *reinterpret_cast<const uint32_t(*)[8]>(&o[c * 8]));
        }
      }
    }
    if (live) {
      if (!whole)
        p.part_ml[prow] = make_float2(m, l);
      else if (p.lse)
        p.lse[orow] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
    if (join) {  // O_1 and its statistics are read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_MD]);
    }
  }
}

// ------------------------------------------------------------------ kernel
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_bf16_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PagedAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sR = smem + 2 * kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sR + kRing * kTile);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  long long* sh = reinterpret_cast<long long*>(tmem_holder + 4);
  float* stats = reinterpret_cast<float*>(sh);  // [256], in the range search's words
  SharedWalk* walks = reinterpret_cast<SharedWalk*>(stats + 256);  // of the 8 softmax warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      const bool warps = i == B_PF || i == B_PF + 1 || i == B_MG || i == B_MD;
      mbar_init(&bars[i], warps ? 4 : 1);
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
  if (threadIdx.x < 2) p.rec[2 * blockIdx.x + threadIdx.x] = make_int4(-1, 0, 0, 0);
  const PagedRange range = paged_range<Plan, kThreads>(p.s, p.n_qblk, p.group, p.kv_heads, p.mask_block, blockIdx.x,
                                                       gridDim.x, p.err, sh);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitCtl w{abort_flag, p.err, p.wait_limit_ns};
  if (warp < 4) {
    regs_dec<kCtlRegs>();
    if (warp == 0)
      load_role(p, &tm_q, &tm_k, &tm_v, range, bars, sQ, sR, w);
    else if (warp == 1)
      mma_role(p, range, bars, sQ, sR, tmem, w);
  } else {
    regs_inc<kSoftmaxRegs>();
    softmax_role(p, range, bars, stats, walks + warp - 4, tmem, (warp >> 2) - 1, w);
  }
  // Every product has completed once a commit behind all of them has arrived:
  // only then are shared and tensor memory released.
  __syncwarp();
  if (warp == 1) {
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
                                   cudaStream_t st) {
  static unsigned done = 0;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(paged_attn_bf16_kernel), kSmem, &done);
  if (e != cudaSuccess) return e;
  static int regs = -1;
  if (regs < 0) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, paged_attn_bf16_kernel)) != cudaSuccess) return e;
    regs = fa.numRegs;
  }
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;  // the register split needs this count
  const int rows = 2 * (128 / p.group);
  p.n_qblk = (p.s.max_q + rows - 1) / rows;
  if ((long long)p.n_qblk * p.s.n_seqs >= (1LL << 31)) return cudaErrorInvalidValue;
  CUtensorMap tq;
  if (!paged_query_map(&tq, p.q, p.s.tokens, p.heads, p.group, p.ld_q)) return cudaErrorInvalidValue;
  paged_attn_bf16_kernel<<<grid, kThreads, kSmem, st>>>(tq, tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_combine<__nv_bfloat16, 2, 128, 128>(p, grid, st);
}

}  // namespace arl2
