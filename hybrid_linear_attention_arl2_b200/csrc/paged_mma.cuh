// What the paged cache's bf16 kernels share: single-CTA tensor-core
// instructions with a tensor-memory operand, tiles of keys gathered from pages
// by TMA, exponentials, and full-sector stores.
#pragma once

#include <cuda.h>

#include "paged.h"
#include "sm100.cuh"

namespace arl2 {

constexpr uint32_t kTile = 32768;  // 128 rows x 128 bf16: two boxes of 64 columns
constexpr uint32_t kHalfTile = 16384;

// D (+)= A B, A in tensor memory (bf16 pairs), B MN-major in shared memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc));
}

// D = A B^T over K = 128, both K-major tiles of 128 rows.
__device__ __forceinline__ void mma_tile(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = (kk >> 2) * (kHalfTile >> 4) + (kk & 3) * 2;
    mma_ss(d, a + off, b + off, idesc, kk > 0);
  }
}

// 32 lanes x 16 columns of 32-bit values.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 32 bytes of a row, one sector, 32-byte aligned.
__device__ __forceinline__ void store_sector(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Keys per TMA box: boxes of a 128-key tile lie inside pages.
__host__ __device__ __forceinline__ int box_keys(int page_size) {
  int a = page_size, b = 128;
  while (b) {
    const int t = a % b;
    a = b, b = t;
  }
  return a;
}

// The pool row of the box at keys [k, k + box) of a stream, for the lane that
// loads it; the row past the pool's last (zeros) where the stream has no key
// there or its table no page.
__device__ __forceinline__ int box_row(const PagedSeqs& s, int b, int k, int kv, int hk, int kv_heads, uint32_t* err) {
  const int none = s.n_pages * kv_heads * s.page_size;
  if (k >= kv) return none;
  const int pg = page_of(s, b, k, err);
  return pg < 0 ? none : (pg * kv_heads + hk) * s.page_size + k % s.page_size;
}

// 2^x for a pair on the FMA pipe: x = n + f, n = round(x) in the low mantissa
// bits after adding 1.5 * 2^23, 2^f by the polynomial of degree 4 through the
// five Chebyshev nodes of [-1/2, 1/2] (gen_exp2_poly.py 4; relative error below
// 3.6e-6), 2^n added to the exponent field.  x is clamped below at -125.
__device__ __forceinline__ float2 exp2_fma_pair(float2 x) {
  constexpr float kRound = 12582912.f;
  constexpr float c0 = 1.f, c1 = 0.693121016f, c2 = 0.240223497f, c3 = 0.0559219755f, c4 = 0.00966636837f;
  x.x = fmaxf(x.x, -125.f);
  x.y = fmaxf(x.y, -125.f);
  const float2 t = __fadd2_rn(x, make_float2(kRound, kRound));
  const float2 f = __fadd2_rn(x, __fadd2_rn(make_float2(kRound, kRound), make_float2(-t.x, -t.y)));
  float2 q = __ffma2_rn(make_float2(c4, c4), f, make_float2(c3, c3));
  q = __ffma2_rn(q, f, make_float2(c2, c2));
  q = __ffma2_rn(q, f, make_float2(c1, c1));
  q = __ffma2_rn(q, f, make_float2(c0, c0));
  return make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + __float_as_uint(q.x)),
                     __uint_as_float((__float_as_uint(t.y) << 23) + __float_as_uint(q.y)));
}

// The same with the polynomial of degree 5 (gen_exp2_poly.py 5; relative error
// below 1.1e-7): where the sum is kept in float32.
__device__ __forceinline__ float2 exp2_fma_pair5(float2 x) {
  constexpr float kRound = 12582912.f;
  constexpr float c0 = 1.00000012f, c1 = 0.693147182f, c2 = 0.240221068f, c3 = 0.0555035695f, c4 = 0.00967603177f,
                  c5 = 0.00133908633f;
  x.x = fmaxf(x.x, -125.f);
  x.y = fmaxf(x.y, -125.f);
  const float2 t = __fadd2_rn(x, make_float2(kRound, kRound));
  const float2 f = __fadd2_rn(x, __fadd2_rn(make_float2(kRound, kRound), make_float2(-t.x, -t.y)));
  float2 q = __ffma2_rn(make_float2(c5, c5), f, make_float2(c4, c4));
  q = __ffma2_rn(q, f, make_float2(c3, c3));
  q = __ffma2_rn(q, f, make_float2(c2, c2));
  q = __ffma2_rn(q, f, make_float2(c1, c1));
  q = __ffma2_rn(q, f, make_float2(c0, c0));
  return make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + __float_as_uint(q.x)),
                     __uint_as_float((__float_as_uint(t.y) << 23) + __float_as_uint(q.y)));
}

}  // namespace arl2
