// Eviction from the paged cache by accumulated weight: which keys stay, and
// the copy of their K and V rows to the pages of another table.
//
// Per stream and key head, of the kv keys between the first `sink` and the
// last `recent` the m = budget - sink - recent with the largest weights stay.
// Weights become whole numbers in the same order (NaN lowest, -0 equal to 0);
// their m-th largest, T, is found by digits of 11, 11 and 10 bits from the top
// (a histogram each, in shared memory), and keys above T stay, and as many of
// those equal to T as are left, lowest index first.  The copy is bound by
// bytes: each kept row in and out once.

#include "paged.h"
#include "sm100.cuh"

namespace arl2 {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kCopyRows = 64, kCopyThreads = 256;
constexpr int kBins = 2048;

__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum over the block's threads below this one, and the whole sum.
__device__ __forceinline__ int2 block_scan(int2 v, int2* sh, int2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 inc = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc.x, o), y = __shfl_up_sync(0xffffffffu, inc.y, o);
    if (lane >= o) inc.x += x, inc.y += y;
  }
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  int2 base = make_int2(0, 0);
  total = make_int2(0, 0);
  for (int w = 0; w < kWarps; ++w) {
    const int2 s = sh[w];
    if (w < warp) base.x += s.x, base.y += s.y;
    total.x += s.x, total.y += s.y;
  }
  __syncthreads();
  return make_int2(base.x + inc.x - v.x, base.y + inc.y - v.y);
}

// One block per (stream, key head).
__global__ void __launch_bounds__(kThreads) paged_select_kernel(const PagedEvictParams p) {
  __shared__ int hist[kBins];
  __shared__ int2 sh[kWarps];
  __shared__ int found[2];
  const int b = blockIdx.x / p.kv_heads, hk = blockIdx.x % p.kv_heads, tid = threadIdx.x;
  const int kv = load_kv_len(p.s, b, p.err);
  if (kv < 0) return;
  const int64_t row = int64_t(b) * p.kv_heads + hk;
  const float* w = p.w_in + row * p.w_ld;
  float* wo = p.w_out + row * p.w_ld;
  int32_t* kept = p.kept + row * p.budget;
  if (hk == 0 && tid == 0) p.kv_len_out[b] = kv < p.budget ? kv : p.budget;
  if (kv <= p.budget) {
    for (int j = tid; j < p.budget; j += kThreads) kept[j] = j < kv ? j : -1;
    for (int64_t j = tid; j < p.w_ld; j += kThreads) wo[j] = j < kv ? w[j] : 0.f;
    return;
  }
  const int lo = p.sink, hi = kv - p.recent;
  int need = p.budget - p.sink - p.recent;  // of the keys [lo, hi), hi - lo > need
  uint32_t T = 0, mask = 0;
  if (need > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kThreads) {
        const uint32_t k = order_key(w[j]);
        if ((k & mask) == T) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
      }
      __syncthreads();
      // the digit in which the need-th largest lies: bins from the top
      const int b0 = kBins - 1 - 2 * tid, c0 = hist[b0], c1 = hist[b0 - 1];
      int2 total;
      const int above = block_scan(make_int2(c0 + c1, 0), sh, total).x;
      if (above < need && above + c0 + c1 >= need) {
        const bool first = above + c0 >= need;
        found[0] = first ? b0 : b0 - 1;
        found[1] = need - above - (first ? 0 : c0);
      }
      __syncthreads();
      T |= uint32_t(found[0]) << shift;
      mask |= ((1u << bits) - 1) << shift;
      need = found[1];
      __syncthreads();
    }
  }
  // keys in order, a block's width at a time
  int2 before = make_int2(0, 0);  // kept for their place or above T; equal to T
  const bool any = p.budget > p.sink + p.recent;
  for (int j0 = 0; j0 < kv; j0 += kThreads) {
    const int j = j0 + tid;
    int2 c = make_int2(0, 0);
    float x = 0.f;
    if (j < kv) {
      x = w[j];
      if (j < lo || j >= hi) {
        c.x = 1;
      } else if (any) {
        const uint32_t k = order_key(x);
        c.x = k > T;
        c.y = k == T;
      }
    }
    int2 total;
    const int2 at = block_scan(c, sh, total);
    const int eq = before.y + at.y;
    if (c.x || (c.y && eq < need)) {
      const int i = before.x + at.x + (eq < need ? eq : need);
      kept[i] = j;
      wo[i] = x;
    }
    before.x += total.x;
    before.y += total.y;
  }
  for (int64_t j = p.budget + tid; j < p.w_ld; j += kThreads) wo[j] = 0.f;
}

// Rows [j0, j0 + 64) of the kept keys of one stream and key head per block.
__global__ void __launch_bounds__(kCopyThreads) paged_move_kernel(const PagedEvictParams p, int n_tiles) {
  __shared__ int64_t src[kCopyRows], dst[kCopyRows];
  __shared__ int own[kCopyRows];  // destination page of each row, or -1
  const int tid = threadIdx.x;
  const int chunks = p.row_bytes / 16;
  const long long items = (long long)p.s.n_seqs * p.kv_heads * n_tiles;
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
    const char* in[2] = {static_cast<const char*>(p.k_pool), static_cast<const char*>(p.v_pool)};
    char* out[2] = {static_cast<char*>(p.k_pool), static_cast<char*>(p.v_pool)};
    const int n = rows * chunks;
    for (int x = 0; x < 2; ++x) {
#pragma unroll 4
      for (int i = tid; i < n; i += kCopyThreads) {
        const int r = i / chunks, c = i - r * chunks;
        if (dst[r] < 0) continue;
        const uint4 v = src[r] < 0 ? make_uint4(0, 0, 0, 0)
                                   : reinterpret_cast<const uint4*>(in[x] + src[r] * p.row_bytes)[c];
        reinterpret_cast<uint4*>(out[x] + dst[r] * p.row_bytes)[c] = v;
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictParams& p, int sms, cudaStream_t st) {
  paged_select_kernel<<<unsigned(p.s.n_seqs) * unsigned(p.kv_heads), kThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int most = p.budget < p.s.max_kv ? p.budget : p.s.max_kv;
  const int n_tiles = (most + kCopyRows - 1) / kCopyRows;
  const long long items = (long long)n_tiles * p.s.n_seqs * p.kv_heads;
  if (items < 1) return cudaSuccess;
  const long long cap = 64LL * sms;
  paged_move_kernel<<<unsigned(items < cap ? items : cap), kCopyThreads, 0, st>>>(p, n_tiles);
  return cudaGetLastError();
}

}  // namespace arl2
