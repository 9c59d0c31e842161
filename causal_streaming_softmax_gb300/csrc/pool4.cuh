// pool4.cuh - the rows of a 4-bit cache.
//
// The block rule, a group's signed extremum over -8 as its scale and codes -8..7, is that
// of the published 4-bit block format Q4_0 of open model files; the scale's bits, cut so
// that products are exact, and the unit's layout are this cache's own.  Small whole numbers
// through the bits of 1024 + x (binary16) or 16 + x (bfloat16) are the old device of adding
// 2^23 to read a number off a significand, as Kim et al. (2022, on serving mixtures of
// experts) use it for weights of few bits.
//
// A row of 64 channels is 32 bytes of codes and two 16-bit scales.  Byte c holds
// channel c in its low half and channel c + 32 in its high half, each as code + 8
// with code in -8..7; the value is code * scale of the channel's group (0..31,
// 32..63).  A scale has three significant bits fewer than the cache's type, so
// that code * scale is exact in that type: the attention kernels form the 16-bit
// operands of their matrix products without rounding, and a row read back is the
// row that they see.
//
// Eight rows make a unit of 288 bytes, their codes before their scales: any run of
// units in a page is one contiguous copy, and the shared-memory layout of a key
// tile does not depend on the page size.
#pragma once

#include <math.h>
#include <stdint.h>

#include "sm103.cuh"
#include "warp_mma.cuh"

namespace css {

constexpr int kUnitBytes = 288, kUnitScales = 256;

// Bytes of a page of one K/V head.
__host__ __device__ constexpr int page4_bytes(int shift) { return (kUnitBytes / 8) << shift; }

// Where row r of a page has its codes; its scales.
__device__ __forceinline__ int code_at(int r) { return (r >> 3) * kUnitBytes + (r & 7) * 32; }
__device__ __forceinline__ int scale_at(int r) {
  return (r >> 3) * kUnitBytes + kUnitScales + (r & 7) * 4;
}

// max and min of three that keep a NaN.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The scale of a group with the largest value mx and the smallest mn, as 16 bits of
// the type: -e / 8 for the extremum e, which then has the code -8, to nearest (its
// code comes out between -8.25 and -7.75, so cutting it off at -8 costs less than a
// rounding).  The largest scale keeps 8 s (binary16) and 24 s (bfloat16, where the
// attention kernels form that) finite.  A group that holds an infinity or a NaN has
// the scale NaN and reads as NaN throughout.
template <bool BF16>
__device__ __forceinline__ uint32_t group_scale(float mx, float mn) {
  constexpr int kDrop = BF16 ? 19 : 16;  // significand bits left out, of 24
  constexpr float kMost = BF16 ? 0x1p123f : 8160.f;
  const float e = (mx > -mn ? -mx : -mn) * 0.125f + 0.f;  // a group of zeros: +0
  const float s = __uint_as_float((__float_as_uint(e) + (1u << (kDrop - 1))) & (~0u << kDrop));
  const uint32_t h = pack2<BF16>(fminf(fmaxf(s, -kMost), kMost), 0.f) & 0xffffu;
  return fabsf(mx) < INFINITY && fabsf(mn) < INFINITY ? h : (BF16 ? 0x7fc0u : 0x7e00u);
}

// The quotients of a group's values by its scale, correctly rounded: a tie between
// two codes is common with so few bits on both sides, and goes to the even one.  After
// Markstein (1990): with y = 1 / s correctly rounded, q0 = x y and r = x - q0 s, the
// sum q0 + r y is.  That wants s away from the smallest numbers: there both sides are
// first multiplied by 2^64.
struct Quotient {
  float s, y, up;
  // code + 8 of two values in the low bytes
  __device__ __forceinline__ uint2 codes(float2 x) const {
    const float2 y2 = make_float2(y, y);
    x = __fmul2_rn(x, make_float2(up, up));
    float2 q = __fmul2_rn(x, y2);
    q = __ffma2_rn(__ffma2_rn(q, make_float2(-s, -s), x), y2, q);
    // 1.5 2^23 + 8: the sum's last bit counts one, halves go to even
    q = __fadd2_rn(make_float2(fminf(fmaxf(q.x, -8.f), 7.f), fminf(fmaxf(q.y, -8.f), 7.f)),
                   make_float2(12582920.f, 12582920.f));
    return make_uint2(__float_as_uint(q.x), __float_as_uint(q.y));
  }
  // four of them, a byte each; 8 in a group that is zero or reads as NaN
  __device__ __forceinline__ uint32_t codes(float2 a, float2 b) const {
    const uint2 u = codes(a), v = codes(b);
    const uint32_t w =
        __byte_perm(__byte_perm(u.x, u.y, 0x0040), __byte_perm(v.x, v.y, 0x0040), 0x5410);
    return fabsf(y) < INFINITY ? w : 0x08080808u;
  }
};
__device__ __forceinline__ Quotient quotient(float s) {
  const float up = fabsf(s) < 0x1p-60f ? 0x1p64f : 1.f;
  return Quotient{s * up, __fdiv_rn(1.f, s * up), up};
}

template <bool BF16>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (BF16)
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  if (BF16)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  else
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// The bits of 16 + code of the half bytes that a shift brought to bits 3..6 of each
// 16-bit half, as bfloat16.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
  return (w & 0x00780078u) | 0x41804180u;
}

// A word of codes as pairs of code * scale: the low and high halves of bytes 0 and
// 2, then of bytes 1 and 3.
template <bool BF16>
__device__ __forceinline__ void scaled_codes(uint32_t w, uint32_t s_lo, uint32_t s_hi,
                                             uint32_t& lo0, uint32_t& hi0, uint32_t& lo1,
                                             uint32_t& hi1) {
  if (BF16) {
    // (16 + code') s - 24 s: both exact, as s has five significant bits
    const uint32_t z_lo = mul2<true>(s_lo, 0xc1c0c1c0u), z_hi = mul2<true>(s_hi, 0xc1c0c1c0u);
    lo0 = fma2<true>(codes_bf16(w << 3), s_lo, z_lo);
    hi0 = fma2<true>(codes_bf16(w >> 1), s_hi, z_hi);
    lo1 = fma2<true>(codes_bf16(w >> 5), s_lo, z_lo);
    hi1 = fma2<true>(codes_bf16(w >> 9), s_hi, z_hi);
  } else {
    // 1024 + code' - 1032 and (1024 + 16 code') / 16 - 72, then times s
    constexpr uint32_t kOne = 0x3c003c00u, kSixteenth = 0x2c002c00u, kM = 0x64006400u,
                       k1032 = 0xe408e408u, k72 = 0xd480d480u;
    const uint32_t v = w >> 8;
    lo0 = mul2<false>(fma2<false>((w & 0x000f000fu) | kM, kOne, k1032), s_lo);
    hi0 = mul2<false>(fma2<false>((w & 0x00f000f0u) | kM, kSixteenth, k72), s_hi);
    lo1 = mul2<false>(fma2<false>((v & 0x000f000fu) | kM, kOne, k1032), s_lo);
    hi1 = mul2<false>(fma2<false>((v & 0x00f000f0u) | kM, kSixteenth, k72), s_hi);
  }
}

}  // namespace css
