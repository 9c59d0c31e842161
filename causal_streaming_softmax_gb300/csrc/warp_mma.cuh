// warp_mma.cuh - warp-level matrix products m16n8k16 (binary16 or bfloat16 in,
// binary32 sums) and the shared-memory fragment loads that feed them.
#pragma once

#include <stdint.h>

#include "sm103.cuh"

namespace css {

// Four 8x8 matrices of 16-bit values; lane l gives the address of row l % 8 of
// matrix l / 8, and holds of each the two values at row l / 4, columns
// 2 (l % 4) and the next.
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// The same with each matrix transposed.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// d += a b: a 16x16 (rows l / 4 and l / 4 + 8), b 16x8, d 16x8.
template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two binary32 values as a 16-bit pair of the operands' type, to nearest even.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return BF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}

template <bool BF16>
__device__ __forceinline__ float half_to_f32(uint16_t h) {
  return BF16 ? __uint_as_float((uint32_t)h << 16) : f16_bits_to_f32(h);
}

// A pair of two consecutive keys' values with those at or past `left` keys
// replaced by zero.
__device__ __forceinline__ uint32_t drop_keys(uint32_t pair, int left) {
  return left >= 2 ? pair : (left == 1 ? pair & 0xffffu : 0u);
}

// Replaces the infinities and NaN of a pair by zero; nonzero if there were any.
template <bool BF16>
__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t* pair) {
  constexpr uint32_t e = BF16 ? 0x7f80u : 0x7c00u;  // exponent bits of one value
  uint32_t drop = 0;
  if ((*pair & e) == e) drop |= 0xffffu;
  if ((*pair & (e << 16)) == (e << 16)) drop |= 0xffff0000u;
  *pair &= ~drop;
  return drop;
}

}  // namespace css
