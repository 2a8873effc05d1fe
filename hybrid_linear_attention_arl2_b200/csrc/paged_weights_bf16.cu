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
// 1024), of which a part goes to the FMA pipe; for single tokens the bytes of K.
//
// Work: units (key block, tile of rows that sees it), stream by stream, key head
// by key head, blocks in order; CTAs take equal contiguous ranges.  A block cut
// by a range's end is joined from the CTAs' pieces by the finish kernel, which
// also clears what lies past kv_len.  Sums run in the order of rows: the same
// bits every time.
//
// Warps: 0 loads, 1 issues the products, 2 puts the rows' lse next to their
// tile; four warpgroups sum, one for each key tile and half of the columns.  Tensor memory: S^T of tile t,
// buffer i at columns (2 t + i) 128.

#include "layer.h"
#include "paged_mma.cuh"
#include "params.h"

namespace arl2 {

namespace {

constexpr int kThreads = 640;
constexpr int kKeys = 256;  // of a block
constexpr int kQRing = 3;

enum {
  B_KF = 0,              // [2] a block's K loaded (bytes)
  B_KE = 2,              // [2] read (commit)
  B_QF = 4,              // [kQRing] a Q tile loaded (bytes)
  B_QE = B_QF + kQRing,  // [kQRing] read (commit)
  B_LF = B_QE + kQRing,  // [kQRing] its rows' lse in shared memory (warp 2)
  B_LE = B_LF + kQRing,  // [kQRing] read (16 warps)
  B_SF = B_LE + kQRing,  // [t][2] S^T in tensor memory (commit)
  B_SC = B_SF + 4,       // [t][2] read (8 warps)
  B_JF = B_SC + 4,       // [t] half 1's sums in shared memory (4 warps)
  B_JE = B_JF + 2,       // [t] read (4 warps)
  B_DRAIN = B_JE + 2,
  B_COUNT
};
constexpr int kSmem = 232448, kLayout = 2 * 2 * kTile + kQRing * kTile + kQRing * 512 + 1024 + 8 * B_COUNT + 16;
static_assert(kLayout <= kSmem, "shared memory");

// A stream's units.  Row tile rt holds tokens [rt qt, ...); key block jt is
// seen from the first token that sees its first key on, by all tiles after that.
struct Stream {
  SeqView v;
  int n_kb, n_rt;  // key blocks, row tiles; 0 where nothing is to be summed
  __device__ Stream() {}
  __device__ Stream(const PagedSeqs& s, int b, int qt, uint32_t* err) : v(load_seq(s, b, err)) {
    const bool some = v.n > 0 && v.kv > 0;
    n_kb = some ? (v.kv + kKeys - 1) / kKeys : 0;
    n_rt = some ? (v.n + qt - 1) / qt : 0;
  }
  // the first token that sees key j
  __device__ int first_token(const FastDiv& mask, int j) const {
    if (mask.by <= 0) return 0;
    const int past = j - (v.kv - v.n);
    return past < mask.by ? 0 : past - mask.mod(past);
  }
  __device__ int first_tile(const PagedWeightParams& p, int jt) const {
    return p.per_tile.div(first_token(p.mask, jt * kKeys));
  }
  __device__ long long units(const PagedWeightParams& p) const {
    if (n_kb == 0) return 0;
    if (p.mask_block <= 0) return (long long)n_kb * n_rt;
    const long long all = (long long)(v.kv - v.n) + p.mask_block;  // blocks that begin below it are seen by every tile
    long long full = all <= 0 ? 0 : (all + kKeys - 1) / kKeys;
    if (full > n_kb) full = n_kb;
    long long sum = full * n_rt;
    for (int jt = int(full); jt < n_kb; ++jt) sum += n_rt - first_tile(p, jt);
    return sum;
  }
};

struct Unit {
  int b, hk, jt, rt;
  bool first, last;    // of the block's units, within this CTA's range
  bool starts, ends;   // the range has the block's very first unit; this is its very last
  bool head;           // of the range's first block
};

// The units of a CTA's range in order.
struct Walk {
  Stream s;
  Unit u;
  long long left;
  bool begun, fresh;
  __device__ bool next(const PagedWeightParams& p, int qt) {
    if (left <= 0) return false;
    if (!begun) {
      s = Stream(p.s, u.b, qt, nullptr);
      begun = u.head = true;
    } else if (++u.rt >= s.n_rt) {
      if (++u.jt >= s.n_kb) {
        u.jt = 0;
        if (++u.hk >= p.kv_heads) {
          u.hk = 0;
          do {
            if (++u.b >= p.s.n_seqs) return false;  // (cannot happen: the range lies inside the units)
            s = Stream(p.s, u.b, qt, nullptr);
          } while (s.n_kb == 0);
        }
      }
      u.rt = s.first_tile(p, u.jt);
      fresh = true;
      u.head = false;
    }
    --left;
    u.first = fresh;
    if (fresh) u.starts = u.rt == s.first_tile(p, u.jt);
    fresh = false;
    u.ends = u.rt == s.n_rt - 1;
    u.last = u.ends || left == 0;
    return true;
  }
  __device__ int rows(const PagedWeightParams& p, int qt) const { return min(qt, s.v.n - u.rt * qt) * p.group; }
};

// Sum of c over threads below this one (its own not counted), and the total.
__device__ __forceinline__ long long scan(long long c, long long* sh, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = c;
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  long long before = 0;
  total = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += sh[i];
    total += sh[i];
  }
  return before + inc - c;
}

// Where the CTA's range begins.  sh: 32 shared words.
__device__ __forceinline__ Walk find_range(const PagedWeightParams& p, int qt, long long* sh) {
  const int tid = threadIdx.x;
  Walk w;
  w.left = 0, w.begun = false, w.fresh = true;
  auto cost = [&](int b, uint32_t* err) {
    return b < p.s.n_seqs ? Stream(p.s, b, qt, err).units(p) * p.kv_heads : 0;
  };
  long long first = cost(tid, p.err), mine = first, total;
  for (int b = tid + kThreads; b < p.s.n_seqs; b += kThreads) mine += cost(b, p.err);
  scan(mine, sh, total);
  const int ctas = total < gridDim.x ? int(total) : int(gridDim.x), cta = blockIdx.x;
  if (cta >= ctas) return w;
  const long long u0 = total * cta / ctas;
  w.left = total * (cta + 1) / ctas - u0;
  long long base = 0;
  for (int b0 = 0; b0 < p.s.n_seqs; b0 += kThreads) {
    const long long c = b0 == 0 ? first : cost(b0 + tid, nullptr);
    long long all;
    const long long beg = base + scan(c, sh, all);
    if (c > 0 && u0 >= beg && u0 < beg + c) {
      sh[24] = b0 + tid;
      sh[25] = u0 - beg;
    }
    __syncthreads();
    base += all;
    if (u0 < base) break;
  }
  w.u.b = int(sh[24]);
  const Stream s(p.s, w.u.b, qt, nullptr);
  const long long per = s.units(p);
  w.u.hk = int(sh[25] / per);
  const long long off = sh[25] % per;
  // the key block: a second search over the stream's blocks
  base = 0;
  for (int j0 = 0; j0 < s.n_kb; j0 += kThreads) {
    const int jt = j0 + tid, r0 = jt < s.n_kb ? s.first_tile(p, jt) : 0;
    const long long c = jt < s.n_kb ? s.n_rt - r0 : 0;
    long long all;
    const long long beg = base + scan(c, sh, all);
    if (c > 0 && off >= beg && off < beg + c) {
      sh[26] = jt;
      sh[27] = r0 + (off - beg);
    }
    __syncthreads();
    base += all;
    if (off < base) break;
  }
  w.u.jt = int(sh[26]);
  w.u.rt = int(sh[27]);
  __syncthreads();
  return w;
}

// Which slot of the Q ring a unit reads: units of neighbouring blocks that
// read the same tile (single tokens) share a slot.
struct QSlot {
  int b = -1, hk = 0, rt = 0;
  uint32_t count = 0;  // tiles so far; the current one is count - 1
  __device__ bool step(const Unit& u) {  // true: a new tile
    if (u.b == b && u.hk == hk && u.rt == rt) return false;
    b = u.b, hk = u.hk, rt = u.rt;
    ++count;
    return true;
  }
  __device__ uint32_t slot() const { return (count - 1) % kQRing; }
  __device__ uint32_t parity() const { return ((count - 1) / kQRing) & 1; }
};

__device__ __forceinline__ void load_role(const PagedWeightParams& p, const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                                          Walk walk, int qt, uint64_t* bars, uint8_t* sK, uint8_t* sQ,
                                          const WaitCtl& w) {
  const int lane = threadIdx.x & 31;
  QSlot q;
  uint32_t blocks = 0;
  bool more = walk.next(p, qt);
  while (more) {  // a (stream, key head) at a time: its key tiles lie in a row
    const int b = walk.u.b, hk = walk.u.hk;
    BoxRows<128> rows(p.s, b, walk.s.v.kv, hk, p.kv_heads, 2 * walk.u.jt, 2 * walk.s.n_kb, p.err);
    for (; more && walk.u.b == b && walk.u.hk == hk; more = walk.next(p, qt)) {
      const Unit& u = walk.u;
      if (u.first) {
        const uint32_t i = blocks & 1;
        if (blocks >= 2 && !warp_wait(&bars[B_KE + i], ((blocks >> 1) - 1) & 1, w)) return;
        if (lane == 0) mbar_expect_tx(&bars[B_KF + i], 2 * kTile);
        __syncwarp();
#pragma unroll
        for (int t = 0; t < 2; ++t) rows.load(2 * u.jt + t, sK + (2 * i + t) * kTile, tm_k, &bars[B_KF + i]);
        __syncwarp();
        ++blocks;
      }
      if (q.step(u)) {
        if (q.count > kQRing && !warp_wait(&bars[B_QE + q.slot()], q.parity() ^ 1, w)) return;
        if (lane == 0) {
          mbar_expect_tx(&bars[B_QF + q.slot()], 2u * uint32_t(qt * p.group) * 128u);
          for (int h = 0; h < 2; ++h)
            tma_load_3d(sQ + q.slot() * kTile + h * kHalfTile, tm_q, &bars[B_QF + q.slot()], h * 64, hk * p.group,
                        walk.s.v.q0 + u.rt * qt);
        }
        __syncwarp();
      }
    }
  }
}

// One warp (see elect_one).
__device__ __forceinline__ void mma_role(const PagedWeightParams& p, Walk walk, int qt, uint64_t* bars, uint8_t* sK,
                                         uint8_t* sQ, uint32_t tmem, const WaitCtl& w) {
  const uint32_t dk = desc_lo(sK, 16), dq = desc_lo(sQ, 16);
  const uint32_t el = elect_one();
  QSlot q;
  uint32_t blocks = 0, g = 0, old = 0;
  while (walk.next(p, qt)) {
    const Unit& u = walk.u;
    if (u.first) {
      if (!warp_wait(&bars[B_KF + (blocks & 1)], (blocks >> 1) & 1, w)) return;
      ++blocks;
    }
    const uint32_t i = (blocks - 1) & 1;
    if (q.step(u)) {
      if (q.count > 1) mma_commit_el(&bars[B_QE + old], el);
      old = q.slot();
      if (!warp_wait(&bars[B_QF + old], q.parity(), w)) return;
    }
    const int rows = walk.rows(p, qt);
    const uint32_t id = idesc_bf16(128, (rows + 15) & ~15, 0, 0), buf = g & 1;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (g >= 2 && !warp_wait(&bars[B_SC + 2 * t + buf], ((g >> 1) - 1) & 1, w)) return;
      tc_fence_after();
      mma_tile<128>(tmem + (2 * t + buf) * 128, dk + (2 * i + t) * (kTile >> 4), dq + old * (kTile >> 4), id, el);
      mma_commit_el(&bars[B_SF + 2 * t + buf], el);
    }
    if (u.last) mma_commit_el(&bars[B_KE + i], el);
    ++g;
  }
}

// Rows' -lse log2(e), a tile ahead of their use; -inf where a row adds nothing.
__device__ __forceinline__ void lse_role(const PagedWeightParams& p, Walk walk, int qt, uint64_t* bars, float* sL,
                                         const WaitCtl& w) {
  const int lane = threadIdx.x & 31;
  QSlot q;
  while (walk.next(p, qt)) {
    const Unit& u = walk.u;
    if (!q.step(u)) continue;
    const int rows = walk.rows(p, qt);
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = lane + 32 * i, t = p.per_group.div(r);
      x[i] = -INFINITY;
      if (r < rows)
        x[i] = p.lse[int64_t(walk.s.v.q0 + u.rt * qt + t) * p.heads + u.hk * p.group + (r - t * p.group)];
    }
    if (q.count > kQRing && !warp_wait(&bars[B_LE + q.slot()], q.parity() ^ 1, w)) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sL[q.slot() * 128 + lane + 32 * i] = x[i] == -INFINITY ? x[i] : -1.4426950408889634f * x[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[B_LF + q.slot()]);
  }
}

// Pairs of 16 whose exponentials run on the FMA pipe.
constexpr int kPolyPairs = 5;

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
      const bool poly = !kMask && (x + y) % 3 == 1 && (x + y) / 3 < kPolyPairs;
      e = poly ? exp2_fma_pair5(e) : make_float2(fast_exp2(e.x), fast_exp2(e.y));
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
__device__ __forceinline__ void sum_role(const PagedWeightParams& p, Walk walk, int qt, uint64_t* bars, const float* sL,
                                         float* sJ, uint32_t tmem, int t, int half, const WaitCtl& w) {
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, row = quarter * 32 + lane;
  const uint32_t tS = tmem + t * 256 + half * 64 + (uint32_t(quarter * 32) << 16);
  const float2 sc = make_float2(p.scale_log2, p.scale_log2);
  QSlot q;
  uint32_t g = 0, old = 0, blocks = 0;
  float sum = 0.f;
  while (walk.next(p, qt)) {
    const Unit& u = walk.u;
    if (q.step(u)) {
      if (q.count > 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_LE + old]);
      }
      old = q.slot();
      if (!warp_wait(&bars[B_LF + old], q.parity(), w)) return;
    }
    const int key = u.jt * kKeys + t * 128 + row, rows = walk.rows(p, qt);
    // the key is seen by the tile's columns [lo, rows)
    const long long from = (long long)(walk.s.first_token(p.mask, key) - u.rt * qt) * p.group;
    const int lo = from < 0 ? 0 : from > 128 ? 128 : int(from);
    const bool masked = __any_sync(0xffffffffu, lo > 0) || rows < 128;
    const uint32_t buf = g & 1;
    if (!warp_wait(&bars[B_SF + 2 * t + buf], (g >> 1) & 1, w)) return;
    ++g;
    tc_fence_after();
    const float4* nl = reinterpret_cast<const float4*>(sL + old * 128 + half * 64);
    float2 acc = make_float2(0.f, 0.f);
    // (columns from the product's width on hold an older product, and are masked)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t r[32];
      const bool some = half * 64 + 32 * c < rows;
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
        acc = sum_chunk<false>(r, nl + 8 * c, sc, 0, 0, 0, acc);
      else if (some)
        acc = sum_chunk<true>(r, nl + 8 * c, sc, half * 64 + 32 * c, lo, rows, acc);
    }
    sum += acc.x + acc.y;
    if (u.last) {
      if (half == 1) {
        if (blocks > 0 && !warp_wait(&bars[B_JE + t], (blocks - 1) & 1, w)) return;
        sJ[t * 128 + row] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_JF + t]);
      } else {
        if (!warp_wait(&bars[B_JF + t], blocks & 1, w)) return;
        sum += sJ[t * 128 + row];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_JE + t]);
        const bool whole = u.starts && u.ends;
        const int piece = 2 * blockIdx.x + (u.head ? 0 : 1);
        if (whole) {
          const int64_t at = (int64_t(u.b) * p.kv_heads + u.hk) * p.w_ld + key;
          if (key < walk.s.v.kv) p.w_out[at] = fmaf(p.decay, p.w_in[at], sum);
        } else {
          p.part_w[piece * kKeys + t * 128 + row] = sum;
          if (t == 0 && row == 0) p.rec[piece] = make_int4(u.b, u.hk, u.jt, (u.starts ? 1 : 0) | (u.ends ? 2 : 0));
        }
      }
      ++blocks;
      sum = 0.f;
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
  uint64_t* bars = reinterpret_cast<uint64_t*>(sJ + 256);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, qt = 128 / p.group;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i)
      mbar_init(&bars[i], i >= B_LE && i < B_LE + kQRing ? 16 : i >= B_SC && i < B_JF ? 8 : i >= B_JF && i < B_DRAIN ? 4 : 1);
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
  if (threadIdx.x < 2) p.rec[2 * blockIdx.x + threadIdx.x] = make_int4(-1, 0, 0, 0);
  const Walk walk = find_range(p, qt, reinterpret_cast<long long*>(sL));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitCtl w{abort_flag, p.err, p.wait_limit_ns};
  if (warp == 0) {
    load_role(p, &tm_q, &tm_k, walk, qt, bars, sK, sQ, w);
  } else if (warp == 1) {
    mma_role(p, walk, qt, bars, sK, sQ, tmem, w);
  } else if (warp == 2) {
    lse_role(p, walk, qt, bars, sL, w);
  } else if (warp >= 4) {
    const int wg = (warp >> 2) - 1;
    sum_role(p, walk, qt, bars, sL, sJ, tmem, wg & 1, wg >> 1, w);
  }
  // shared and tensor memory are released once a commit behind every product has arrived
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

// The first `ctas` blocks join the pieces of a key block that CTA ranges cut
// (that of the CTA which holds its first unit, and slots 0 of the CTAs after it
// up to the one that ends it); the others clear the rows past kv_len, and fade
// the weights of streams without new tokens.
constexpr int kTail = 4096;
__global__ void __launch_bounds__(kKeys) paged_weights_finish_kernel(const PagedWeightParams p, int ctas) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x;
  if (int(blockIdx.x) < ctas) {
    const int c = blockIdx.x;
    int slot = -1;
    int4 rec = p.rec[2 * c];
    if (rec.x >= 0 && rec.w == 1) slot = 0;
    if (slot < 0) {
      rec = p.rec[2 * c + 1];
      if (rec.x >= 0 && rec.w == 1) slot = 1;
    }
    if (slot < 0) return;
    float sum = p.part_w[(2 * c + slot) * kKeys + tid];
    for (int i = c + 1; i < ctas; ++i) {
      sum += p.part_w[2 * i * kKeys + tid];
      if (p.rec[2 * i].w & 2) break;
    }
    const int key = rec.z * kKeys + tid;
    const int64_t at = (int64_t(rec.x) * p.kv_heads + rec.y) * p.w_ld + key;
    if (key < p.s.kv_len[rec.x]) p.w_out[at] = fmaf(p.decay, p.w_in[at], sum);
    return;
  }
  const long long per_row = (p.w_ld + kTail - 1) / kTail, items = per_row * p.s.n_seqs * p.kv_heads;
  for (long long it = blockIdx.x - ctas; it < items; it += gridDim.x - ctas) {
    const long long row = it / per_row, j0 = it % per_row * kTail;
    const SeqView v = load_seq(p.s, int(row / p.kv_heads), nullptr);
    if (v.n < 0) continue;
    const long long j1 = min((long long)p.w_ld, j0 + kTail);
    if (j1 <= v.kv && v.n > 0) continue;
    for (long long j = j0 + tid; j < j1; j += kKeys) {
      const int64_t at = row * p.w_ld + j;
      if (j >= v.kv)
        p.w_out[at] = 0.f;
      else if (v.n == 0)
        p.w_out[at] = p.decay * p.w_in[at];
    }
  }
}

}  // namespace

cudaError_t launch_paged_weights_bf16(const PagedWeightParams& p, const CUtensorMap& tk, int sms, cudaStream_t st) {
  static unsigned done = 0;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(paged_weights_bf16_kernel), kSmem, &done);
  if (e != cudaSuccess) return e;
  int ctas = 0;
  if (p.s.tokens > 0 && p.s.max_q > 0 && p.s.max_kv > 0) {
    CUtensorMap tq;
    if (!paged_query_map(&tq, p.q, p.s.tokens, p.heads, p.group, p.ld_q)) return cudaErrorInvalidValue;
    ctas = sms;
    e = launch_overlapped(paged_weights_bf16_kernel, dim3(unsigned(ctas)), kThreads, kSmem, st, 0, tq, tk, p);
    if (e != cudaSuccess) return e;
  }
  const long long items = (p.w_ld + kTail - 1) / kTail * p.s.n_seqs * p.kv_heads;
  return launch_overlapped(paged_weights_finish_kernel, dim3(unsigned(ctas + (items < 65536 ? items : 65536))), kKeys, 0, st,
                           0, p, ctas);
}

}  // namespace arl2
