// Norm of queries and keys for each head with the position rotation in the
// same pass, alone or storing K and V into the pages of a cache:
//
//   y = x * rsqrt(mean(x^2) + eps) * w;   (y0, y1) -> (y0 cos a - y1 sin a, y0 sin a + y1 cos a)
//
// A group of lanes takes a token, 16 bytes of a row a lane, and goes through
// its rows (heads of Q, K and, appending, V), six in flight: the sum of squares
// is a few shuffles, pairs of neighbours lie in one lane and pairs R/2 apart in
// two (one shuffle a channel).  The angles are the token's: a block computes
// them once, a thread a pair, and a lane keeps those of its channels.
// An angle is pos * freq with freq a 64-bit fraction of a turn: the product
// modulo 2^64 is the fraction of the turn exactly up to pos * 2^-65, so no
// position loses bits to range reduction; its upper 32 bits go to sincospif.
// Few tokens: a token's rows are split over several groups, so that every SM
// has loads in flight.  Bound: bytes (each row in and out once).

#include <cuda_bf16.h>

#include "paged.h"
#include "sm100.cuh"

namespace arl2 {

namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 6;  // rows in flight of a group

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

// LPR: lanes of a row (a power of two >= d * sizeof(T) / 16).  A token's rows
// are split over `parts` groups of LPR lanes.
template <typename T, int LPR, bool kAppend>
__global__ void __launch_bounds__(kThreads)
prep_kernel(const __grid_constant__ PrepParams p, int parts) {
  constexpr int N = Vec<T>::N;
  grid_dependency_wait();
  allow_dependent_launch();
  // groups of a block: kThreads / LPR, `parts` (a power of two) to a token
  constexpr int kGroups = kThreads / LPR;
  __shared__ float2 turn[kThreads * N / 2];  // (cos, sin) of the block's tokens' pairs
  const int lane = threadIdx.x % LPR, c = lane * N, group = threadIdx.x / LPR;
  const int tokens = kGroups / parts, mine = group / parts, part = group - mine * parts;
  const int64_t t0 = int64_t(blockIdx.x) * tokens;
  const bool have = t0 + mine < p.tokens, on = have && c < p.d;
  const int64_t t = have ? t0 + mine : p.tokens - 1;  // (a group without a token keeps step with its warp)
  const int row4 = p.d / N;  // 16-byte words of a row
  // Rows part + r0, part + r0 + parts, ... of n, kAhead of them.
  auto fetch = [&](uint4 (&x)[kAhead], const T* src, int n, int r0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + part + i * parts;
      x[i] = make_uint4(0, 0, 0, 0);
      if (on && r < n) x[i] = reinterpret_cast<const uint4*>(src)[r * row4 + lane];
    }
  };
  const T* q = static_cast<const T*>(p.q) + t * p.ld_q;
  const T* k = static_cast<const T*>(p.k) + t * p.ld_k;
  const int nq = p.q_out ? p.heads : 0;
  uint4 first_q[kAhead], first_k[kAhead];
  fetch(first_q, q, nq, 0);
  fetch(first_k, k, p.kv_heads, 0);
  // the block's angles, a thread a pair; then each lane takes those of its channels
  const int half = p.rot / 2;
  const bool in_rot = c < p.rot, lo = c < half;
  float cs[N], sn[N];
  if (half > 0) {
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
      const int j = i / half, pr = i - j * half;
      const int e0 = p.axis_dim[0] >> 1, e1 = e0 + (p.axis_dim[1] >> 1);
      if (t0 + j < p.tokens) {
        const int pos = p.pos[(t0 + j) * p.n_axes + (pr < e0 ? 0 : pr < e1 ? 1 : 2)];
        const uint64_t turns = uint64_t(int64_t(pos)) * p.freq[pr];
        float2 a;
        sincospif(float(int(turns >> 32)) * (1.f / 2147483648.f), &a.y, &a.x);  // pi * (turns * 2^-63)
        turn[i] = a;
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (!p.halves && (e & 1)) continue;
      const int pr = p.halves ? (lo ? c + e : c - half + e) : (c + e) >> 1;
      const float2 a = (p.halves ? in_rot : c + e < p.rot) && have ? turn[mine * half + pr] : make_float2(1.f, 0.f);
      cs[e] = a.x, sn[e] = a.y;
    }
  }
  // append: the row of the token's K and V in the pools
  int64_t dst = -1;
  bool used = true;  // the token belongs to a stream
  if (kAppend) {
    // its stream: as many as end at or before it come first
    int b = 0;
    const unsigned mask = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1u) << (threadIdx.x % 32 / LPR * LPR);
    for (int s0 = 0; s0 < p.s.n_seqs; s0 += LPR) {
      const bool before = s0 + lane < p.s.n_seqs && p.s.q_start[s0 + lane + 1] <= t;
      b += __popc(__ballot_sync(0xffffffffu, before) & mask);
    }
    used = b < p.s.n_seqs;
    if (used) {
      const SeqView sv = load_seq(p.s, b, lane == 0 ? p.err : nullptr);
      const int64_t i = t - sv.q0;
      used = sv.n >= 0 && i >= 0 && i < sv.n;
      if (used) {
        const int64_t j = int64_t(sv.kv) - sv.n + i;
        if (j >= 0) {
          const int pg = page_of(p.s, b, int(j), lane == 0 ? p.err : nullptr);
          if (pg >= 0) dst = int64_t(pg) * p.kv_heads * p.s.page_size + p.s.page.mod(int(j));
        } else if (lane == 0) {
          record_error(p.err, kDevPage);
        }
      }
    }
  }
  const bool part_rot = p.rot < p.d;
  const int other = in_rot ? (lo ? lane + half / N : lane - half / N) : lane;  // (halves; half is a multiple of N)
  // Norm and rotation of n rows, as many rounds in every group.
  auto turned = [&](uint4 (&x)[kAhead], const void* weights, const T* src, int n, T* out, int pitch, bool write) {
    Vec<T> w;
#pragma unroll
    for (int e = 0; e < N; ++e) w.v[e] = 1.f;
    if (p.norm && c < p.d) unpack(reinterpret_cast<const uint4*>(weights)[lane], w);
    for (int r0 = 0; r0 < n; r0 += kAhead * parts) {
      if (r0 > 0) fetch(x, src, n, r0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (r0 + i * parts >= n) continue;  // (no group has one)
        const int r = r0 + part + i * parts;
        Vec<T> y;
        unpack(x[i], y);
        if (p.norm) {
          float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < N; e += 2) s2 = __ffma2_rn(make_float2(y.v[e], y.v[e + 1]), make_float2(y.v[e], y.v[e + 1]), s2);
          float ss = s2.x + s2.y;
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float inv = rsqrtf(fmaf(ss, p.inv_d, p.eps));
#pragma unroll
          for (int e = 0; e < N; e += 2) {
            const float2 m = __fmul2_rn(make_float2(w.v[e], w.v[e + 1]), make_float2(inv, inv));
            const float2 z = __fmul2_rn(make_float2(y.v[e], y.v[e + 1]), m);
            y.v[e] = z.x, y.v[e + 1] = z.y;
          }
        }
        if (p.halves && half > 0) {
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float z = __shfl_sync(0xffffffffu, y.v[e], other, LPR);
            if (in_rot) y.v[e] = lo ? y.v[e] * cs[e] - z * sn[e] : z * sn[e] + y.v[e] * cs[e];
          }
        } else if (half > 0) {
#pragma unroll
          for (int e = 0; e < N; e += 2) {
            if (part_rot && c + e >= p.rot) continue;
            const float2 z = __fmul2_rn(make_float2(y.v[e + 1], y.v[e]), make_float2(-sn[e], sn[e]));
            const float2 o = __ffma2_rn(make_float2(y.v[e], y.v[e + 1]), make_float2(cs[e], cs[e]), z);
            y.v[e] = o.x, y.v[e + 1] = o.y;
          }
        }
        if (write && on && r < n) reinterpret_cast<uint4*>(out + int64_t(r) * pitch)[lane] = pack(y);
      }
    }
  };
  if (kAppend) {  // V as it is
    const T* v = static_cast<const T*>(p.v) + t * p.ld_v;
    T* out = static_cast<T*>(p.v_pool) + dst * p.d;
    const int64_t pitch = int64_t(p.s.page_size) * p.d;
    for (int r0 = 0; r0 < p.kv_heads; r0 += kAhead * parts) {
      uint4 x[kAhead];
      fetch(x, v, p.kv_heads, r0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int r = r0 + part + i * parts;
        if (dst >= 0 && on && r < p.kv_heads) reinterpret_cast<uint4*>(out + r * pitch)[lane] = x[i];
      }
    }
  }
  if (nq > 0) turned(first_q, p.w_q, q, nq, static_cast<T*>(p.q_out) + t * p.ld_qo, p.d, used);
  if (kAppend)
    turned(first_k, p.w_k, k, p.kv_heads, static_cast<T*>(p.k_pool) + dst * p.d, p.s.page_size * p.d, dst >= 0);
  else
    turned(first_k, p.w_k, k, p.kv_heads, static_cast<T*>(p.k_out) + t * p.ld_ko, p.d, true);
}

template <typename T, int LPR>
cudaError_t launch(const PrepParams& p, bool append, int parts, cudaStream_t st) {
  const int64_t tokens = kThreads / LPR / parts;  // of a block
  const dim3 grid{unsigned((p.tokens + tokens - 1) / tokens)};
  return launch_overlapped(append ? prep_kernel<T, LPR, true> : prep_kernel<T, LPR, false>, grid, kThreads, 0, st, 0, p, parts);
}

}  // namespace

cudaError_t launch_prep(const PrepParams& p, int dtype, bool append, int sms, cudaStream_t st) {
  if (p.tokens < 1) return cudaSuccess;
  const int chunks = p.d * (dtype == ARL2_BF16 ? 2 : 4) / 16;
  int lpr = 1;
  while (lpr < chunks) lpr *= 2;
  // Parts, a power of two up to a block's groups, until an SM has 256 threads:
  // a single token's rows go to all of a block's groups, 25000 tokens take one.
  const int groups = kThreads / lpr;
  int parts = 1;
  while (parts < groups && p.tokens * parts * lpr < int64_t(sms) * 256) parts *= 2;
  if (dtype == ARL2_BF16) {
    switch (lpr) {
      case 1: return launch<__nv_bfloat16, 1>(p, append, parts, st);
      case 2: return launch<__nv_bfloat16, 2>(p, append, parts, st);
      case 4: return launch<__nv_bfloat16, 4>(p, append, parts, st);
      case 8: return launch<__nv_bfloat16, 8>(p, append, parts, st);
      default: return launch<__nv_bfloat16, 16>(p, append, parts, st);
    }
  } else {
    switch (lpr) {
      case 1: return launch<float, 1>(p, append, parts, st);
      case 2: return launch<float, 2>(p, append, parts, st);
      case 4: return launch<float, 4>(p, append, parts, st);
      case 8: return launch<float, 8>(p, append, parts, st);
      case 16: return launch<float, 16>(p, append, parts, st);
      default: return launch<float, 32>(p, append, parts, st);
    }
  }
}

}  // namespace arl2
