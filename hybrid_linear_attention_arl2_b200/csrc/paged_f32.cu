// Paged KV cache on CUDA cores (float32 tensors): attention of new tokens over
// the pages, and the weights the cached keys received.
//
//   O = softmax(Q K^T scale) V over the visible keys,  lse = log sum exp,
//   w_out[j] = decay w_in[j] + sum over rows of exp(s_j - lse)
//
// One pass over the keys with the running maximum and sum of each row (Q K^T
// in units of log2).  A CTA holds 64 query rows (token, head of the group) of
// one key head and takes tiles of 64 keys; S and O are 4 x 4 and 4 x d/16
// register tiles a thread, P passes through shared memory.  The f32 path is
// bound by the FMA pipe: 4 d FMAs a (row, key) pair.

#include <cuda_bf16.h>

#include "paged.h"
#include "paged_join.cuh"
#include "params.h"
#include "sm100.cuh"

namespace arl2 {

namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 256;
using Plan = PagedPlan<1, kKeys, 1>;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

// Rows of keys [k0, k0 + 64) of stream b and head hk into dst[64][ld] as
// float; keys at or past `end` and keys of pages that are none read as zeros.
__device__ __forceinline__ void load_keys(float* dst, int ld, const float* pool, const PagedSeqs& s, int b, int hk,
                                          int kv_heads, int d, int k0, int end, uint32_t* err) {
  const int v4 = d >> 2;
  for (int i = threadIdx.x; i < kKeys * v4; i += kThreads) {
    const int r = i / v4, c = (i - r * v4) * 4, j = k0 + r;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (j < end) {
      const int pg = page_of(s, b, j, err);
      if (pg >= 0) v = load4(pool + ((int64_t(pg) * kv_heads + hk) * s.page_size + s.page.mod(j)) * d + c);
    }
    store4(dst + r * ld + c, v);
  }
}

// S = Q K^T for this thread's 4 rows (4 ty ..) x 4 keys (tx + 16 i).
__device__ __forceinline__ void scores(const float* sQ, const float* sK, int ld, int d, int ty, int tx,
                                       float (&acc)[4][4]) {
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[a][i] = 0.f;
  for (int c = 0; c < d; c += 4) {
    float4 q[4], k[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) q[a] = *reinterpret_cast<const float4*>(sQ + (4 * ty + a) * ld + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) k[i] = *reinterpret_cast<const float4*>(sK + (tx + 16 * i) * ld + c);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[a][i] = dot4(q[a], k[i], acc[a][i]);
  }
}

__host__ __device__ inline size_t smem_floats(int d) {
  return size_t(2 * kRows + kKeys) * (d + 4) + size_t(kKeys) * (kRows + 4);
}

// DC: 64-column chunks of the head dimension a thread accumulates (d <= 64 DC).
template <int DC>
__global__ void __launch_bounds__(kThreads)
paged_attn_f32_kernel(const PagedAttnParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  extern __shared__ float sm[];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, d = p.d, ld = d + 4;
  float* sQ = sm;
  float* sK = sQ + kRows * ld;
  float* sV = sK + kKeys * ld;
  float* sP = sV + kKeys * ld;  // [key][row], pitch 68
  constexpr int kPl = kRows + 4;
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
    const int rows = s.blk.n_tok * p.group, b = p.per_blk.div(s.f);
    // query rows, and each of this thread's rows' visible keys
    for (int i = tid; i < kRows * (d >> 2); i += kThreads) {
      const int r = i / (d >> 2), c = (i - r * (d >> 2)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        v = load4(q + int64_t(s.blk.row0 + p.per_group.div(r)) * p.ld_q + (s.hk * p.group + p.per_group.mod(r)) * d + c);
      store4(sQ + r * ld + c, v);
    }
    int lim[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = 4 * ty + a;
      lim[a] = r < rows ? visible_keys(s.blk.view(), p.mask, s.blk.t0 + p.per_group.div(r)) : 0;
    }
    float m[4], l[4], o[4][4 * DC];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      m[a] = -INFINITY;
      l[a] = 0.f;
#pragma unroll
      for (int c = 0; c < 4 * DC; ++c) o[a][c] = 0.f;
    }
    for (int j = s.u0; j < s.u1; ++j) {
      const int k0 = j * kKeys;
      __syncthreads();
      load_keys(sK, ld, static_cast<const float*>(p.k_pool), p.s, b, s.hk, p.kv_heads, d, k0, s.blk.kv, p.err);
      load_keys(sV, ld, static_cast<const float*>(p.v_pool), p.s, b, s.hk, p.kv_heads, d, k0, s.blk.kv, p.err);
      __syncthreads();
      float acc[4][4];
      scores(sQ, sK, ld, d, ty, tx, acc);
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
        for (int c = 0; c < 4 * DC; ++c) o[a][c] *= corr;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(sP + (tx + 16 * i) * kPl + 4 * ty) =
            make_float4(acc[0][i], acc[1][i], acc[2][i], acc[3][i]);
      __syncthreads();
#pragma unroll 4
      for (int k = 0; k < kKeys; ++k) {
        const float4 pk = *reinterpret_cast<const float4*>(sP + k * kPl + 4 * ty);
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          const int col = tx * 4 + 64 * c;
          if (col < d) {
            const float4 v = *reinterpret_cast<const float4*>(sV + k * ld + col);
            const float pr[4] = {pk.x, pk.y, pk.z, pk.w};
#pragma unroll
            for (int a = 0; a < 4; ++a) {
              o[a][4 * c] = fmaf(pr[a], v.x, o[a][4 * c]);
              o[a][4 * c + 1] = fmaf(pr[a], v.y, o[a][4 * c + 1]);
              o[a][4 * c + 2] = fmaf(pr[a], v.z, o[a][4 * c + 2]);
              o[a][4 * c + 3] = fmaf(pr[a], v.w, o[a][4 * c + 3]);
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
        const float4 x = make_float4(o[a][4 * c] * inv, o[a][4 * c + 1] * inv, o[a][4 * c + 2] * inv,
                                     o[a][4 * c + 3] * inv);
        if (whole)
          store4(static_cast<float*>(p.o) + orow * d + col, x);
        else
          store4(p.part_o + (int64_t(piece) * kRows + r) * d + col, x);
      }
      if (tx == 0) {
        if (!whole)
          p.part_ml[int64_t(piece) * kRows + r] = make_float2(m[a], l[a]);
        else if (p.lse)
          p.lse[orow] = l[a] > 0.f ? (m[a] + log2f(l[a])) * 0.69314718055994531f : -INFINITY;
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) join = last_piece(p.joined + 8 * s.owner, s.pieces);
      __syncthreads();
      if (join) {
        constexpr int kWarps = kThreads / 32;
        const int n = (rows + kWarps - 1) / kWarps, r0 = (tid >> 5) * n;
        join_rows<float, kRows, false>(p, s.owner, s.owner_slot, s.pieces, r0, min(rows - r0, n), out_row);
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
// One CTA per (stream, key head, 64 keys): every new token's rows go past in
// tiles of 64, a thread sums its 4 rows' weights of its 4 keys.
__global__ void __launch_bounds__(kThreads)
paged_weights_f32_kernel(const PagedWeightParams p, int n_kt) {
  grid_dependency_wait();
  allow_dependent_launch();
  extern __shared__ float sm[];
  __shared__ float part[16][kKeys];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, d = p.d, ld = d + 4;
  float* sQ = sm;
  float* sK = sQ + kRows * ld;
  const float* q = static_cast<const float*>(p.q);
  const int qt = kRows / p.group;
  const long long items = (long long)p.s.n_seqs * p.kv_heads * n_kt;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int jt = int(it % n_kt), hk = int(it / n_kt % p.kv_heads), b = int(it / n_kt / p.kv_heads);
    const SeqView v = load_seq(p.s, b, p.err);
    const int k0 = jt * kKeys;
    if (v.n < 0) continue;
    float* out = p.w_out + (int64_t(b) * p.kv_heads + hk) * p.w_ld;
    const float* in = p.w_in + (int64_t(b) * p.kv_heads + hk) * p.w_ld;
    if (k0 < v.kv) {
      __syncthreads();
      load_keys(sK, ld, static_cast<const float*>(p.k_pool), p.s, b, hk, p.kv_heads, d, k0, v.kv, p.err);
      float w[4] = {0.f, 0.f, 0.f, 0.f};
      for (int t0 = 0; t0 < v.n; t0 += qt) {
        const int rows = min(qt, v.n - t0) * p.group;
        if (visible_keys(v, p.mask, min(t0 + qt, v.n) - 1) <= k0) continue;  // no row of the tile sees the keys
        __syncthreads();
        for (int i = tid; i < kRows * (d >> 2); i += kThreads) {
          const int r = i / (d >> 2), c = (i - r * (d >> 2)) * 4;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (r < rows) x = load4(q + int64_t(v.q0 + t0 + r / p.group) * p.ld_q + (hk * p.group + r % p.group) * d + c);
          store4(sQ + r * ld + c, x);
        }
        __syncthreads();
        float acc[4][4];
        scores(sQ, sK, ld, d, ty, tx, acc);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int r = 4 * ty + a;
          if (r >= rows) continue;
          const int t = t0 + r / p.group, lim = visible_keys(v, p.mask, t);
          const float lse = p.lse[int64_t(v.q0 + t) * p.heads + hk * p.group + r % p.group];
          if (lse == -INFINITY) continue;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (k0 + tx + 16 * i < lim) w[i] += exp2f(fmaf(acc[a][i], p.scale_log2, -1.4426950408889634f * lse));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) part[ty][tx + 16 * i] = w[i];
      __syncthreads();
      if (tid < kKeys && k0 + tid < v.kv) {
        float sum = 0.f;
        for (int y = 0; y < 16; ++y) sum += part[y][tid];
        out[k0 + tid] = fmaf(p.decay, in[k0 + tid], sum);
      }
      __syncthreads();
    }
    if (tid < kKeys && k0 + tid >= v.kv && k0 + tid < p.w_ld) out[k0 + tid] = 0.f;
  }
}

template <int DC>
cudaError_t launch_attn(PagedAttnParams p, int grid, cudaStream_t st) {
  static unsigned done = 0;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(paged_attn_f32_kernel<DC>),
                                   int(smem_floats(128) * sizeof(float)), &done);
  if (e != cudaSuccess) return e;
  return launch_overlapped(paged_attn_f32_kernel<DC>, dim3(unsigned(grid)), kThreads, smem_floats(p.d) * sizeof(float), st, 0,
                           p);
}

}  // namespace

cudaError_t launch_paged_attn_f32(PagedAttnParams p, int grid, cudaStream_t st) {
  return p.d <= 64 ? launch_attn<1>(p, grid, st) : launch_attn<2>(p, grid, st);
}

cudaError_t launch_paged_weights_f32(const PagedWeightParams& p, cudaStream_t st) {
  const int bytes = int(size_t(kRows + kKeys) * (p.d + 4) * sizeof(float));
  static unsigned done = 0;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(paged_weights_f32_kernel),
                                   int(size_t(kRows + kKeys) * 132 * sizeof(float)), &done);
  if (e != cudaSuccess) return e;
  const long long n_kt = (p.w_ld + kKeys - 1) / kKeys;
  const long long items = n_kt * p.s.n_seqs * p.kv_heads;
  const unsigned grid = unsigned(items < (1 << 20) ? items : (1 << 20));
  return launch_overlapped(paged_weights_f32_kernel, dim3(grid), kThreads, size_t(bytes), st, 0, p, int(n_kt));
}

}  // namespace arl2
