// Eviction from the paged cache by accumulated weight: which keys stay, and
// the copy of their K and V rows to the pages of another table.
//
// Per stream and key head, of the kv keys between the first `sink` and the
// last `recent` the m = budget - sink - recent with the largest weights stay.
// Weights become whole numbers in the same order (NaN lowest, -0 equal to 0);
// their m-th largest, T, is found by digits of 11, 11 and 10 bits from the top,
// and keys above T stay, and as many of those equal to T as are left, lowest
// index first.  A cluster of CTAs takes a (stream, key head), a slice of its keys
// each: a digit's histograms are summed by every CTA out of all the cluster's
// shared memories, so that a digit costs one cluster barrier.  Then the copy,
// bound by bytes: each kept row in and out once.

#include "paged.h"
#include "sm100.cuh"

namespace arl2 {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kCopyRows = 32, kCopyThreads = 256;
constexpr int kBins = 2048;

__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int2 warp_scan(int2 v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) v.x += x, v.y += y;
  }
  return v;
}
// Sum over the block's threads below this one, and the whole sum.
__device__ __forceinline__ int2 block_scan(int2 v, int2* sh, int2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int2 inc = warp_scan(v);
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  const int2 mine = sh[lane], sums = warp_scan(mine);  // (32 warps, a lane each)
  static_assert(kWarps == 32, "a lane a warp");
  total = make_int2(__shfl_sync(0xffffffffu, sums.x, 31), __shfl_sync(0xffffffffu, sums.y, 31));
  const int bx = __shfl_sync(0xffffffffu, sums.x - mine.x, warp), by = __shfl_sync(0xffffffffu, sums.y - mine.y, warp);
  __syncthreads();
  return make_int2(bx + inc.x - v.x, by + inc.y - v.y);
}

constexpr int kHeld = 4;                      // keys a thread keeps in registers
constexpr int kChunk = kThreads * kHeld;      // keys of a round
constexpr int kMaxCluster = 8;

// Two words of another CTA's shared memory (no barrier is passed on the way, so
// that the loads of several CTAs' are in flight together).
__device__ __forceinline__ int2 remote_int2(const int* p, uint32_t rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(cluster_map(smem_u32(p), rank)));
  return v;
}

// One cluster per (stream, key head).
__global__ void __launch_bounds__(kThreads) paged_select_kernel(const PagedEvictParams p, int cluster) {
  __shared__ __align__(8) int hist[3][kBins];
  __shared__ int2 sh[kWarps];
  __shared__ int found[2];
  __shared__ __align__(8) int counts[2];
  const int item = blockIdx.x / cluster, rank = blockIdx.x - item * cluster, tid = threadIdx.x;
  const int b = item / p.kv_heads, hk = item - b * p.kv_heads;
  grid_dependency_wait();
  allow_dependent_launch();
  const int kv = max(0, load_kv_len(p.s, b, p.err));  // (a stream that breaks a bound has no keys afterwards)
  const int64_t row = int64_t(b) * p.kv_heads + hk;
  const float* w = p.w_in + row * p.w_ld;
  float* wo = p.w_out + row * p.w_ld;
  int32_t* kept = p.kept + row * p.budget;
  const int step = cluster * kThreads, me = rank * kThreads + tid;
  if (hk == 0 && me == 0) p.kv_len_out[b] = kv < p.budget ? kv : p.budget;
  if (kv <= p.budget) {
    for (int j = me; j < p.budget; j += step) kept[j] = j < kv ? j : -1;
    for (int j = me; j < p.w_ld; j += step) wo[j] = j < kv ? w[j] : 0.f;
    return;
  }
  const int lo = p.sink, hi = kv - p.recent;
  // this CTA's keys, a run of whole rounds; the first round's stay in registers, four in a row a thread
  const int rounds = (kv + kChunk * cluster - 1) / (kChunk * cluster);
  const int per = rounds > 1 ? rounds * kChunk : (kv + cluster - 1) / cluster;
  const int j_lo = min(kv, rank * per), j_hi = min(kv, j_lo + per);
  float held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int j = j_lo + tid * kHeld + i;
    held[i] = j < j_hi ? w[j] : 0.f;
  }
  // The weights of a round, thread by thread in order of their keys.
  auto round_keys = [&](int r, auto&& use) {
    const int j0 = j_lo + r * kChunk + tid * kHeld;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (j0 + i < j_hi) use(j0 + i, r == 0 ? held[i] : w[j0 + i], i);
  };
  int need = p.budget - p.sink - p.recent;  // of the keys [lo, hi), hi - lo > need
  const bool any = need > 0;
  uint32_t T = 0, mask = 0;
  if (any) {
    for (int i = tid; i < 3 * kBins; i += kThreads) hist[0][i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digit = pass == 2 ? 1023u : 2047u;
      int* h = hist[pass];
      for (int r = 0; r < rounds; ++r)
        round_keys(r, [&](int j, float x, int) {
          const uint32_t k = order_key(x);
          if (j >= lo && j < hi && (k & mask) == T) atomicAdd(&h[(k >> shift) & digit], 1);
        });
      cluster_barrier();
      // the digit in which the need-th largest lies: bins from the top, two a thread
      const int b0 = kBins - 1 - 2 * tid;
      int c0 = 0, c1 = 0;
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        if (q < cluster) {
          const int2 c = remote_int2(&h[b0 - 1], q);
          c0 += c.y, c1 += c.x;
        }
      }
      int2 total;
      const int above = block_scan(make_int2(c0 + c1, 0), sh, total).x;
      if (above < need && above + c0 + c1 >= need) {
        const bool first = above + c0 >= need;
        found[0] = first ? b0 : b0 - 1;
        found[1] = need - above - (first ? 0 : c0);
      }
      __syncthreads();
      T |= uint32_t(found[0]) << shift;
      mask |= digit << shift;
      need = found[1];
      __syncthreads();
    }
  }
  // each CTA's kept keys (for their place, or above T) and those equal to T, then their places
  auto kind = [&](int j, float x) {
    if (j < lo || j >= hi) return make_int2(1, 0);
    const uint32_t k = order_key(x);
    return any ? make_int2(k > T, k == T) : make_int2(0, 0);
  };
  int2 sum = make_int2(0, 0), total;
  for (int r = 0; r < rounds; ++r)
    round_keys(r, [&](int j, float x, int) {
      const int2 c = kind(j, x);
      sum.x += c.x, sum.y += c.y;
    });
  block_scan(sum, sh, total);
  if (tid < 2) counts[tid] = tid == 0 ? total.x : total.y;
  cluster_barrier();
  int2 before = make_int2(0, 0);
#pragma unroll
  for (int q = 0; q < kMaxCluster; ++q) {
    if (q < rank) {
      const int2 c = remote_int2(counts, q);
      before.x += c.x, before.y += c.y;
    }
  }
  for (int r = 0; r < rounds; ++r) {
    int2 mine = make_int2(0, 0);
    round_keys(r, [&](int j, float x, int) {
      const int2 c = kind(j, x);
      mine.x += c.x, mine.y += c.y;
    });
    int2 at = block_scan(mine, sh, total);
    at.x += before.x, at.y += before.y;
    round_keys(r, [&](int j, float x, int) {
      const int2 c = kind(j, x);
      if (c.x || (c.y && at.y < need)) {
        const int i = at.x + min(at.y, need);
        kept[i] = j;
        wo[i] = x;
      }
      at.x += c.x, at.y += c.y;
    });
    before.x += total.x, before.y += total.y;
  }
  for (int j = p.budget + me; j < p.w_ld; j += step) wo[j] = 0.f;
  cluster_barrier();  // the counts are read
}

// Rows [j0, j0 + 32) of the kept keys of one stream and key head per block.
__global__ void __launch_bounds__(kCopyThreads) paged_move_kernel(const PagedEvictParams p, int n_tiles) {
  __shared__ int64_t src[kCopyRows], dst[kCopyRows];
  __shared__ int own[kCopyRows];  // destination page of each row, or -1
  const int tid = threadIdx.x;
  const int chunks = p.row_bytes / 16;
  const long long items = (long long)p.s.n_seqs * p.kv_heads * n_tiles;
  grid_dependency_wait();
  allow_dependent_launch();
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int tile = int(it % n_tiles), hk = int(it / n_tiles % p.kv_heads), b = int(it / n_tiles / p.kv_heads);
    const int kv = load_kv_len(p.s, b, p.err);
    const int m = kv < p.budget ? kv : p.budget, j0 = tile * kCopyRows;
    if (j0 >= m) continue;  // (also a stream that is left out)
    const int rows = min(kCopyRows, m - j0);
    __syncthreads();
    if (tid < kCopyRows) {
      own[tid] = -1;
      dst[tid] = -1;
      src[tid] = -1;
      if (tid < rows) {
        const int j = j0 + tid, slot = j / p.s.page_size;
        int pg = slot < p.dst_ld ? p.dst_pages[int64_t(b) * p.dst_ld + slot] : -1;
        if (unsigned(pg) >= unsigned(p.s.n_pages)) {
          record_error(p.err, kDevPage);
          pg = -1;
        }
        own[tid] = pg;
        if (pg >= 0) dst[tid] = (int64_t(pg) * p.kv_heads + hk) * p.s.page_size + j % p.s.page_size;
        const int from = p.kept[(int64_t(b) * p.kv_heads + hk) * p.budget + j];
        const int sp = page_of(p.s, b, from, p.err);
        if (sp >= 0) src[tid] = (int64_t(sp) * p.kv_heads + hk) * p.s.page_size + from % p.s.page_size;
      }
    }
    __syncthreads();
    // a destination that the stream reads is not written
    const int n_src = (kv + p.s.page_size - 1) / p.s.page_size;
    for (int i = tid; i < n_src; i += kCopyThreads) {
      const int sp = p.s.pages[int64_t(b) * p.s.pages_ld + i];
      for (int r = 0; r < rows;) {
        if (own[r] == sp && sp >= 0) {
          record_error(p.err, kDevPage);
          for (int x = r; x < rows && own[x] == sp; ++x) dst[x] = -1;
        }
        r += p.s.page_size - (j0 + r) % p.s.page_size;  // the next page's first row
      }
    }
    __syncthreads();
    const int n = rows * chunks;
#pragma unroll 4
    for (int i = tid; i < n; i += kCopyThreads) {
      const int r = i / chunks, c = i - r * chunks;
      const int64_t from = src[r] * p.row_bytes, to = dst[r] * p.row_bytes;
      if (to < 0) continue;
      uint4 k = make_uint4(0, 0, 0, 0), v = k;
      if (from >= 0) {
        k = reinterpret_cast<const uint4*>(static_cast<const char*>(p.k_pool) + from)[c];
        v = reinterpret_cast<const uint4*>(static_cast<const char*>(p.v_pool) + from)[c];
      }
      reinterpret_cast<uint4*>(static_cast<char*>(p.k_pool) + to)[c] = k;
      reinterpret_cast<uint4*>(static_cast<char*>(p.v_pool) + to)[c] = v;
    }
  }
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictParams& p, int sms, cudaStream_t st) {
  const unsigned items = unsigned(p.s.n_seqs) * unsigned(p.kv_heads);
  // A cluster as large as the longest stream has rounds, up to 8 CTAs.
  int cluster = 1;
  while (cluster < kMaxCluster && cluster * kChunk < p.s.max_kv) cluster *= 2;
  if ((long long)items * cluster >= (1LL << 31)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_overlapped(paged_select_kernel, dim3(items * unsigned(cluster)), kThreads, 0, st, cluster, p,
                                          cluster);
  if (e != cudaSuccess) return e;
  const int most = p.budget < p.s.max_kv ? p.budget : p.s.max_kv;
  const int n_tiles = (most + kCopyRows - 1) / kCopyRows;
  const long long moves = (long long)n_tiles * items, cap = 64LL * sms;
  if (moves < 1) return cudaSuccess;
  return launch_overlapped(paged_move_kernel, dim3(unsigned(moves < cap ? moves : cap)), kCopyThreads, 0, st, 0, p, n_tiles);
}

}  // namespace arl2
