// Joins the pieces of attention items that several CTAs share (paged.h's work
// division), for the float32 and the bf16 kernel.
#pragma once

#include <cuda_bf16.h>

#include "paged.h"
#include "sm100.cuh"

namespace arl2 {

namespace {

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// The pieces of an item that several CTAs share, in key order: with M the
// largest of their maxima, O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.  The
// CTA whose range the item starts in owns it (at most one per CTA); its
// continuations are the next CTAs' slots 0.  A warp per row; reads are the
// pieces, just written, from L2.
constexpr int kCombineRows = 32;

template <typename T, class P, int kPieceRows, int kTileRows>
__global__ void __launch_bounds__(256)
paged_combine_kernel(const PagedAttnParams p, int ctas) {
  grid_dependency_wait();
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int slot = -1;
  int4 rec = p.rec[2 * c];
  if (rec.x >= 0 && rec.z && !rec.w) slot = 0;
  if (slot < 0) {
    rec = p.rec[2 * c + 1];
    if (rec.x >= 0 && rec.z && !rec.w) slot = 1;
  }
  if (slot < 0) return;
  int n = 1;  // pieces: this one, then slots 0 of the CTAs after it up to the one that ends the item
  for (int base = c + 1; base < ctas; base += 32) {
    const bool end = base + lane < ctas && p.rec[2 * (base + lane)].w != 0;
    const unsigned b = __ballot_sync(0xffffffffu, end);
    if (b) {
      n = base - c + __ffs(b);
      break;
    }
  }
  const int f = rec.x, hk = rec.y;
  const typename P::Block blk = P::block(p.s, f / p.n_qblk, f % p.n_qblk, p.group, p.mask_block, nullptr);
  const int qt = P::tile_tokens(p.group);
  for (int i = warp; i < kCombineRows; i += 8) {
    const int r = blockIdx.y * kCombineRows + i;
    const int tile = r / kTileRows, rr = r % kTileRows, tt = tile * qt + rr / p.group;
    if (r >= kPieceRows || rr >= qt * p.group || tt >= blk.n_tok) continue;
    auto piece = [&](int k) { return int64_t(k == 0 ? 2 * c + slot : 2 * (c + k)) * kPieceRows + r; };
    float M = -INFINITY;
    for (int k = lane; k < n; k += 32) M = fmaxf(M, p.part_ml[piece(k)].x);
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    if (M != -INFINITY) {
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        const float2 ml = p.part_ml[piece(k)];
        const float w = exp2f(ml.x - M);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane * 4 < p.d) v = load4(p.part_o + piece(k) * p.d + lane * 4);
        L = fmaf(ml.y, w, L);
        acc = make_float4(fmaf(v.x, w, acc.x), fmaf(v.y, w, acc.y), fmaf(v.z, w, acc.z), fmaf(v.w, w, acc.w));
      }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    const int64_t orow = int64_t(blk.q0 + blk.t0 + tt) * p.heads + hk * p.group + rr % p.group;
    if (lane * 4 < p.d)
      store4(static_cast<T*>(p.o) + orow * p.d + lane * 4,
             make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (lane == 0 && p.lse) p.lse[orow] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
  }
}

template <typename T, int kTiles, int kTileRows, int kKeysOf>
cudaError_t launch_combine(const PagedAttnParams& p, int grid, cudaStream_t st) {
  constexpr int kPiece = kTiles * kTileRows;
  // rows of a piece: the streams' own where they fit one tile
  const int rows = p.s.max_q <= kTileRows / p.group ? p.s.max_q * p.group : kPiece;
  const int y = (rows + kCombineRows - 1) / kCombineRows;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(grid), unsigned(y < 1 ? 1 : y));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel<T, PagedPlan<kTiles, kTileRows, kKeysOf>, kPiece, kTileRows>, p,
                            grid);
}

}  // namespace

}  // namespace arl2
