// Norm of queries and keys for each head with the position rotation in the
// same pass, alone or storing K and V into the pages of a cache:
//
//   y = x * rsqrt(mean(x^2) + eps) * w;   (y0, y1) -> (y0 cos a - y1 sin a, y0 sin a + y1 cos a)
//
// A row (one token, one head) is held by a group of lanes, 16 bytes a lane:
// the sum of squares is a few shuffles, pairs of neighbours lie in one lane and
// pairs R/2 apart in two (one shuffle a channel).  The angles of a token are
// the same for all its heads: the block computes them once, one thread a pair,
// while its first rows are on their way.  An angle is pos * freq with freq a
// 64-bit fraction of a turn: the product modulo 2^64 is the fraction of the
// turn exactly up to pos * 2^-65, so no position loses bits to range reduction;
// its upper 32 bits go to sincospif.  Bound: bytes (each row in and out once).

#include <cuda_bf16.h>

#include "paged.h"
#include "sm100.cuh"

namespace arl2 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;  // tokens of a block at most

template <typename T>
struct Vec {  // 16 bytes of a row
  static constexpr int N = 16 / sizeof(T);
  float v[N];
};
__device__ __forceinline__ void unpack(uint4 u, Vec<float>& x) {
  x.v[0] = __uint_as_float(u.x), x.v[1] = __uint_as_float(u.y), x.v[2] = __uint_as_float(u.z),
  x.v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(uint4 u, Vec<__nv_bfloat16>& x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x.v[2 * i] = __uint_as_float(w[i] << 16);
    x.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack(const Vec<float>& x) {
  return make_uint4(__float_as_uint(x.v[0]), __float_as_uint(x.v[1]), __float_as_uint(x.v[2]),
                    __float_as_uint(x.v[3]));
}
__device__ __forceinline__ uint4 pack(const Vec<__nv_bfloat16>& x) {
  return make_uint4(pack_bf16x2(x.v[0], x.v[1]), pack_bf16x2(x.v[2], x.v[3]), pack_bf16x2(x.v[4], x.v[5]),
                    pack_bf16x2(x.v[6], x.v[7]));
}

// LPR: lanes of a row (a power of two >= d * sizeof(T) / 16).  A block takes
// `tpb` tokens; blockIdx.y takes rows y, y + gridDim.y, ... of them in steps of
// the block's row groups, which spreads few tokens over more SMs.
template <typename T, int LPR, bool kAppend>
__global__ void __launch_bounds__(kThreads)
prep_kernel(const __grid_constant__ PrepParams p, int tpb) {
  constexpr int N = Vec<T>::N, kGroups = kThreads / LPR, kUnroll = 2;
  __shared__ float2 turn[kMaxTokens][64];  // (cos, sin)
  __shared__ int2 dst[kMaxTokens];         // append: stream's page (or -1) and row in it
  grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x, lane = tid % LPR, group = tid / LPR;
  const int64_t t0 = int64_t(blockIdx.x) * tpb;
  const int nt = int(min(int64_t(tpb), p.tokens - t0));
  const int H = p.heads, Hk = p.kv_heads, nq = p.q_out ? H : 0;
  const int per_tok = nq + Hk + (kAppend ? Hk : 0), rows = nt * per_tok;
  const bool on = lane * N < p.d;
  const int step = kGroups * int(gridDim.y);

  auto src = [&](int r) -> const uint4* {
    const int t = r / per_tok, i = r - t * per_tok;
    const T* base = i < nq        ? static_cast<const T*>(p.q) + (t0 + t) * p.ld_q + int64_t(i) * p.d
                    : i < nq + Hk ? static_cast<const T*>(p.k) + (t0 + t) * p.ld_k + int64_t(i - nq) * p.d
                                  : static_cast<const T*>(p.v) + (t0 + t) * p.ld_v + int64_t(i - nq - Hk) * p.d;
    return reinterpret_cast<const uint4*>(base) + lane;
  };
  int r = int(blockIdx.y) * kGroups + group;
  uint4 in[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) in[u] = on && r + u * step < rows ? *src(r + u * step) : make_uint4(0, 0, 0, 0);
  Vec<T> wq, wk;
  if (p.norm && on) {
    unpack(reinterpret_cast<const uint4*>(p.w_q)[lane], wq);
    unpack(reinterpret_cast<const uint4*>(p.w_k)[lane], wk);
  }
  // the block's angles
  const int pairs = p.rot / 2;
  for (int i = tid; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, pr = i - t * pairs;
    const int e0 = p.axis_dim[0] >> 1, e1 = e0 + (p.n_axes > 1 ? p.axis_dim[1] >> 1 : 0);
    const int axis = pr < e0 ? 0 : pr < e1 ? 1 : 2;
    const int pos = p.pos[(t0 + t) * p.n_axes + axis];
    const uint64_t turns = uint64_t(int64_t(pos)) * p.freq[pr];
    float sn, cs;
    sincospif(float(int(turns >> 32)) * (1.f / 2147483648.f), &sn, &cs);  // pi * (turns * 2^-63)
    turn[t][pr] = make_float2(cs, sn);
  }
  if (kAppend) {
    // A token's stream: the number of streams that end at or before it.
    int b[kMaxTokens];
#pragma unroll
    for (int t = 0; t < kMaxTokens; ++t) b[t] = 0;
    for (int s0 = 0; s0 < p.s.n_seqs; s0 += kThreads) {
      const int e = s0 + tid < p.s.n_seqs ? p.s.q_start[s0 + tid + 1] : 0x7fffffff;
#pragma unroll
      for (int t = 0; t < kMaxTokens; ++t) b[t] += __syncthreads_count(int64_t(e) <= t0 + t);
    }
    if (tid < nt) {
      int bt = 0;
#pragma unroll
      for (int t = 0; t < kMaxTokens; ++t)
        if (tid == t) bt = b[t];
      int2 d2 = make_int2(-2, 0);  // no stream's token: nothing of it is written
      if (bt < p.s.n_seqs) {
        const SeqView v = load_seq(p.s, bt, p.err);
        const int64_t t = t0 + tid - v.q0;
        if (v.n >= 0 && t >= 0 && t < v.n) {
          const int64_t j = int64_t(v.kv) - v.n + t;
          d2.x = -1;  // its Q is written, its K and V have no row
          if (j >= 0) {
            const int pg = page_of(p.s, bt, int(j), p.err);
            if (pg >= 0) d2 = make_int2(pg, int(j) % p.s.page_size);
          } else {
            record_error(p.err, kDevPage);
          }
        }
      }
      dst[tid] = d2;
    }
  }
  __syncthreads();

  for (; __any_sync(0xffffffffu, r < rows); r += kUnroll * step) {  // (whole warps leave together)
    uint4 cur[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      cur[u] = in[u];
      const int rn = r + (kUnroll + u) * step;
      if (on && rn < rows) in[u] = *src(rn);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int ru = r + u * step;
      const bool live = ru < rows;
      const int t = live ? ru / per_tok : 0, i = live ? ru - t * per_tok : 0;
      const bool is_q = i < nq, is_v = i >= nq + Hk;
      Vec<T> x;
      unpack(cur[u], x);
      if (p.norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) ss = fmaf(x.v[e], x.v[e], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss / float(p.d) + p.eps);
#pragma unroll
        for (int e = 0; e < N; ++e) x.v[e] = is_v ? x.v[e] : x.v[e] * inv * (is_q ? wq.v[e] : wk.v[e]);
      }
      if (p.rot > 0) {
        const int c = lane * N, half = p.rot / 2;
        if (p.halves) {
          // the partner holds channels half before or after; half is a multiple of N
          const bool lo = c < half, in_rot = c < p.rot;
          const int other = in_rot ? (lo ? lane + half / N : lane - half / N) : lane;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float y = __shfl_sync(0xffffffffu, x.v[e], other, LPR);
            if (in_rot && !is_v) {
              const float2 a = turn[t][lo ? c + e : c - half + e];
              x.v[e] = lo ? x.v[e] * a.x - y * a.y : y * a.y + x.v[e] * a.x;
            }
          }
        } else if (!is_v) {
#pragma unroll
          for (int e = 0; e < N; e += 2) {
            if (c + e < p.rot) {
              const float2 a = turn[t][(c + e) >> 1];
              const float y0 = x.v[e], y1 = x.v[e + 1];
              x.v[e] = y0 * a.x - y1 * a.y;
              x.v[e + 1] = y0 * a.y + y1 * a.x;
            }
          }
        }
      }
      if (!live || !on) continue;
      T* out;
      if (kAppend) {
        const int2 d2 = dst[t];
        if (is_q) {
          if (d2.x == -2) continue;
          out = static_cast<T*>(p.q_out) + (t0 + t) * p.ld_qo + int64_t(i) * p.d;
        } else {
          if (d2.x < 0) continue;
          const int hk = is_v ? i - nq - Hk : i - nq;
          out = static_cast<T*>(is_v ? p.v_pool : p.k_pool) +
                ((int64_t(d2.x) * Hk + hk) * p.s.page_size + d2.y) * p.d;
        }
      } else {
        out = is_q ? static_cast<T*>(p.q_out) + (t0 + t) * p.ld_qo + int64_t(i) * p.d
                   : static_cast<T*>(p.k_out) + (t0 + t) * p.ld_ko + int64_t(i - nq) * p.d;
      }
      reinterpret_cast<uint4*>(out)[lane] = is_v ? cur[u] : pack(x);
    }
  }
}

template <typename T, int LPR>
cudaError_t launch(const PrepParams& p, bool append, dim3 grid, int tpb, cudaStream_t st) {
  return launch_overlapped(append ? prep_kernel<T, LPR, true> : prep_kernel<T, LPR, false>, grid, kThreads, 0, st, 0, p, tpb);
}

}  // namespace

cudaError_t launch_prep(const PrepParams& p, int dtype, bool append, int sms, cudaStream_t st) {
  if (p.tokens < 1) return cudaSuccess;
  const int chunks = p.d * (dtype == ARL2_BF16 ? 2 : 4) / 16;
  int lpr = 1;
  while (lpr < chunks) lpr *= 2;
  const int groups = kThreads / lpr, per_tok = (p.q_out ? p.heads : 0) + p.kv_heads * (append ? 2 : 1);
  // Few tokens: one a block, its rows spread over blocks.  Many: four a block,
  // whose rows keep loads in flight while the angles are computed once.
  const int tpb = p.tokens >= 4LL * sms ? kMaxTokens : 1;
  int y = 1;
  if (p.tokens < sms) {
    y = (per_tok + groups - 1) / groups;
    if (y > 64) y = 64;
  }
  const int64_t x = (p.tokens + tpb - 1) / tpb;
  const dim3 grid{unsigned(x), unsigned(y)};
  if (dtype == ARL2_BF16) {
    switch (lpr) {
      case 1: return launch<__nv_bfloat16, 1>(p, append, grid, tpb, st);
      case 2: return launch<__nv_bfloat16, 2>(p, append, grid, tpb, st);
      case 4: return launch<__nv_bfloat16, 4>(p, append, grid, tpb, st);
      case 8: return launch<__nv_bfloat16, 8>(p, append, grid, tpb, st);
      default: return launch<__nv_bfloat16, 16>(p, append, grid, tpb, st);
    }
  } else {
    switch (lpr) {
      case 1: return launch<float, 1>(p, append, grid, tpb, st);
      case 2: return launch<float, 2>(p, append, grid, tpb, st);
      case 4: return launch<float, 4>(p, append, grid, tpb, st);
      case 8: return launch<float, 8>(p, append, grid, tpb, st);
      case 16: return launch<float, 16>(p, append, grid, tpb, st);
      default: return launch<float, 32>(p, append, grid, tpb, st);
    }
  }
}

}  // namespace arl2
