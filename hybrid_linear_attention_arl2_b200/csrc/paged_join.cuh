// Joins the pieces of an attention item that several CTAs share (paged.h's work
// division): with M the largest of their maxima, O = sum 2^(m_i - M) O_i /
// sum 2^(m_i - M) l_i, in the same order whoever joins them.  The CTA that comes
// last does it, told by a count; nobody waits.
#pragma once

#include <cuda_bf16.h>

#include "paged.h"
#include "sm100.cuh"

namespace arl2 {

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// Whether the caller's piece is the last of `pieces`; what the others wrote is
// visible to it then.  One thread calls it, after a fence by every writer.
__device__ __forceinline__ bool last_piece(uint32_t* count, int pieces) {
  if (atomicAdd(count, 1u) + 1u != uint32_t(pieces)) return false;
  *count = 0;  // for the next launch
  __threadfence();
  return true;
}

// Where eight columns (32 bytes) of a row of a 256-row piece of 128 columns
// lie, in floats: the rows of a warp side by side, so that a thread that holds
// a row stores and loads full lines with its warp.  `first`: the piece's first
// row among all pieces' rows.
__device__ __forceinline__ int64_t piece_at(int64_t first, int row, int col8) {
  return first * 128 + (col8 * 256 + row) * 8;
}

// bf16: rows [r0, r0 + n) of the pieces' 256 (piece_at), n <= 32, by one warp: the
// lanes hold the rows' statistics; then kRows rows at a time, a lane's four
// columns each, kUnroll pieces in flight.  `out(r)`: row r's index in O's [token,
// head] rows.
template <int kRows, int kUnroll, class Out>
__device__ __forceinline__ void join_some(const PagedAttnParams& p, int owner, int owner_slot, int pieces, int r0, int n,
                                          const Out& out) {
  const int lane = threadIdx.x & 31;
  auto piece = [&](int k) { return int64_t(k == 0 ? 2 * owner + owner_slot : 2 * (owner + k)) * 256 + r0; };
  float M = -INFINITY, L = 0.f;
  if (kRows == 2) {  // the lanes share the pieces, 32 at a time
    float mine[2] = {-INFINITY, -INFINITY};
    for (int k = lane; k < pieces; k += 32) {
      mine[0] = fmaxf(mine[0], __ldcg(&p.part_ml[piece(k)].x));
      if (n > 1) mine[1] = fmaxf(mine[1], __ldcg(&p.part_ml[piece(k) + 1].x));
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      mine[0] = fmaxf(mine[0], __shfl_xor_sync(0xffffffffu, mine[0], x));
      mine[1] = fmaxf(mine[1], __shfl_xor_sync(0xffffffffu, mine[1], x));
    }
    M = lane == 0 ? mine[0] : lane == 1 ? mine[1] : -INFINITY;
  } else if (lane < n) {
#pragma unroll 4
    for (int k = 0; k < pieces; ++k) M = fmaxf(M, __ldcg(&p.part_ml[piece(k) + lane].x));
  }
  if (M == -INFINITY) M = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kRows) {
    float4 acc[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    L = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < pieces; k0 += kUnroll) {
      float2 ml[kUnroll];
      float4 v[kUnroll][kRows];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t at = piece(k0 + u);
        ml[u] = make_float2(-INFINITY, 0.f);
        if (lane < n && k0 + u < pieces) ml[u] = __ldcg(&p.part_ml[at + lane]);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          v[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i0 + i < n && k0 + u < pieces)
            v[u][i] = __ldcg(reinterpret_cast<const float4*>(
                p.part_o + piece_at(at - r0, r0 + i0 + i, lane >> 1) + (lane & 1) * 4));
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const float mine = exp2f(ml[u].x - M);
        L = fmaf(ml[u].y, mine, L);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const float w = __shfl_sync(0xffffffffu, mine, (i0 + i) & 31);
          acc[i] = make_float4(fmaf(v[u][i].x, w, acc[i].x), fmaf(v[u][i].y, w, acc[i].y), fmaf(v[u][i].z, w, acc[i].z),
                               fmaf(v[u][i].w, w, acc[i].w));
        }
      }
    }
    const float rcp = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float inv = __shfl_sync(0xffffffffu, rcp, (i0 + i) & 31);
      if (i0 + i < n)
        store4(static_cast<__nv_bfloat16*>(p.o) + out(r0 + i0 + i) * 128 + lane * 4,
               make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv));
    }
  }
  if (lane < n && p.lse) p.lse[out(r0 + lane)] = row_lse(M, L);
}

// The same, with more pieces in flight where the rows are few: one token of 16
// heads on 20000 keys (74 pieces a key head) took 90 us when one warp joined
// all rows, four pieces' statistics and two pieces' rows at a time; 28 us so.
template <class Out>
__device__ __forceinline__ void join_rows(const PagedAttnParams& p, int owner, int owner_slot, int pieces, int r0, int n,
                                          const Out& out) {
  if (n <= 2)
    join_some<2, 8>(p, owner, owner_slot, pieces, r0, n, out);
  else
    join_some<8, 2>(p, owner, owner_slot, pieces, r0, n, out);
}

}  // namespace arl2
