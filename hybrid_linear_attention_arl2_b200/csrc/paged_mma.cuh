// What the paged cache's bf16 kernels share: single-CTA tensor-core
// instructions with a tensor-memory operand, tiles of keys gathered from pages
// by TMA, and full-sector stores.
#pragma once

#include <cuda.h>

#include "paged.h"
#include "sm100.cuh"

namespace arl2 {

constexpr uint32_t kTile = 32768;  // 128 rows x 128 bf16: two boxes of 64 columns
constexpr uint32_t kHalfTile = 16384;

// The issuing warp runs its loop as one, so that descriptors stay in uniform
// registers, and one lane of it issues: `el` is 1 in that lane.  (Issued from a
// branch of one lane, the moves of the operands took longer than the products:
// 85 to 125 clocks each where 64 suffice.)
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t el;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(el));
  return el;
}
// A condition that is the same in all lanes, told to the compiler: what changes
// under it stays in uniform registers.
__device__ __forceinline__ bool uniform(bool x) { return __any_sync(0xffffffffu, x); }

// Shared-memory descriptors of 128-byte-swizzled tiles as (low word, shared high
// word): the low word holds the address in units of 16 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(const void* smem, uint32_t lbo) {
  return (smem_u32(smem) & 0x3FFFF) >> 4 | (lbo >> 4) << 16;
}

// D (+)= A B^T, both in shared memory, for the elected lane.
__device__ __forceinline__ void mma_ss_el(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc,
                                          uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 e, %6, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(acc), "r"(el));
}
// D (+)= A B, A in tensor memory (bf16 pairs), B MN-major in shared memory.
__device__ __forceinline__ void mma_ts_el(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc,
                                          uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 e, %6, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(acc), "r"(el));
}
__device__ __forceinline__ void mma_commit_el(uint64_t* bar, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(el)
      : "memory");
}

// D = A B^T over K = 128, both K-major tiles in two boxes of 64 columns: A of
// 128 rows, B of kRowsB.
template <int kRowsB>
__device__ __forceinline__ void mma_tile(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t el) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ss_el(d, a + (kk >> 2) * (kHalfTile >> 4) + (kk & 3) * 2, b + (kk >> 2) * (kRowsB * 128 >> 4) + (kk & 3) * 2, idesc,
              kk > 0, el);
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& w) {
  const bool ok = mbar_wait(bar, parity, w);
  return __all_sync(0xffffffffu, ok);
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

// The pool rows of a run of a stream's key tiles, fetched ahead: a warp's lanes
// hold the boxes of 32 / boxes tiles in a row, and the page numbers of the ones
// after them are on their way while these are used.  A box without a key, or
// whose table entry is no page, gets the row past the pool's last, which reads
// as zeros.
template <int kKeys>  // of a tile
struct BoxRows {
  const int32_t* table;
  FastDiv page;
  int box, boxes, per, kv, n_pages, hk, kv_heads;
  int first, end;  // tiles held, [first, first + per); none from end on
  int row, ahead;  // this lane's box; the page number of its box `per` tiles on
  uint32_t* err;

  __device__ int key_of(int tile0) const {
    const int lane = threadIdx.x & 31;
    return lane < per * boxes ? tile0 * kKeys + lane * box : 0x7fffffff;
  }
  __device__ int fetch(int tile0) const {
    const int k = key_of(tile0);
    return tile0 < end && k < kv ? table[page.div(k)] : -1;
  }
  __device__ void turn(int tile0, int pg) {
    const int k = key_of(tile0);
    row = n_pages * kv_heads * page.by;
    if (tile0 < end && k < kv) {
      if (unsigned(pg) < unsigned(n_pages))
        row = (pg * kv_heads + hk) * page.by + page.mod(k);
      else
        record_error(err, kDevPage);
    }
    first = tile0;
  }
  __device__ BoxRows() {}
  // tiles [tile0, tile1) of stream b
  __device__ BoxRows(const PagedSeqs& s, int b, int kv_, int hk_, int kv_heads_, int tile0, int tile1, uint32_t* err_)
      : table(s.pages + int64_t(b) * s.pages_ld), page(s.page), box(s.box), boxes(kKeys / s.box), per(32 / boxes), kv(kv_),
        n_pages(s.n_pages), hk(hk_), kv_heads(kv_heads_), end(tile1), err(err_) {
    const int pg = fetch(tile0);
    ahead = fetch(tile0 + per);
    turn(tile0, pg);
  }
  // Loads a tile (tiles are asked for in order) into dst: two boxes of 64
  // columns for each run of keys, by the lanes that hold them.
  __device__ void load(int tile, uint8_t* dst, const CUtensorMap* tm, uint64_t* bar) {
    if (tile >= first + per) {
      turn(first + per, ahead);
      ahead = fetch(first + per);
    }
    const int i = int(threadIdx.x & 31) - (tile - first) * boxes;
    if (i >= 0 && i < boxes) {
      uint8_t* d = dst + i * box * 128;
      tma_load_3d(d, tm, bar, 0, row, 0);
      tma_load_3d(d + kKeys * 128, tm, bar, 64, row, 0);
    }
  }
};

}  // namespace arl2
