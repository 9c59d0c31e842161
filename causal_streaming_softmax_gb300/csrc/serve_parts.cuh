// serve_parts.cuh - sharing a list of key tiles out over blocks, and the parts
// of rows whose keys were split between blocks.
//
// The list holds the tiles of every work item (a request's block of rows and a
// K/V head) one item behind the other.  The n blocks take equal runs of it (to one
// position), so that at most its first and its last item are
// shared with other blocks.  Of a shared item each block writes the running
// maximum m, the sum l and the unscaled O in binary32: the block that starts
// the item into its tail part, the later ones into their head parts.  The
// joining kernel adds them in the order of the keys, so results do not depend
// on timing.
#pragma once

#include <math.h>
#include <stdint.h>

#include "serve_index.h"
#include "serve_internal.h"
#include "sm103.cuh"
#include "warp_mma.cuh"

namespace css {

__device__ __forceinline__ long long part_row(const PartArgs& p, int block, bool tail, int row) {
  return ((long long)block * 2 + (tail ? 1 : 0)) * p.rows + row;
}

// The description that block c left, read once a warp: what is checked is what
// is used, and a warp's lanes agree on it whatever else writes there.
__device__ __forceinline__ PartDesc part_desc(const PartArgs& p, int c) {
  static_assert(sizeof(PartDesc) == 16, "one load");
  PartDesc d;
  asm volatile("ld.global.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(d.q0), "=r"(d.kv), "=r"(d.rows), "=r"(d.last)
               : "l"(p.desc + c)
               : "memory");
  d.q0 = __shfl_sync(0xffffffffu, d.q0, 0);
  d.kv = __shfl_sync(0xffffffffu, d.kv, 0);
  d.rows = __shfl_sync(0xffffffffu, d.rows, 0);
  d.last = __shfl_sync(0xffffffffu, d.last, 0);
  return d;
}

// Eight columns of a row's part; the thread of column 0 writes m and l.
__device__ __forceinline__ void store_part(const PartArgs& p, int block, bool tail, int row,
                                           int c0, const float (&acc)[8], float m, float l) {
  const long long at = part_row(p, block, tail, row);
  float4* const d = reinterpret_cast<float4*>(p.o + at * 64 + c0);
  d[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  d[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  if (c0 == 0) p.ml[at] = make_float2(m, l);
}

// Eight columns of a finished row: O / l, and L = m + log2 l from column 0's
// thread.  A row that saw no key (l = 0) gives 0 and -inf.
template <bool BF16>
__device__ __forceinline__ void write_row(const RowsArg& o, float* lse, int tokens, int tok, int h,
                                          int c0, const float (&acc)[8], float m, float l) {
  const bool some = l > 0.f || l != l;
  const float inv = some ? 1.0f / l : 0.f;
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = some ? pack2<BF16>(acc[2 * e] * inv, acc[2 * e + 1] * inv) : 0u;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.p) + (long long)tok * o.t +
                            (long long)h * o.h + c0) = make_uint4(w[0], w[1], w[2], w[3]);
  if (lse && c0 == 0)
    lse[(long long)h * tokens + tok] = some ? m + lg2_approx(l) : -INFINITY;
}

}  // namespace css
