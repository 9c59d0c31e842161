// paged_fwd.cu - attn_paged_fwd: which kernels a call runs, its workspace, and
// the kernel that joins the parts of split rows.
#include <mutex>

#include "serve_internal.h"
#include "serve_parts.cuh"
#include "sm103.cuh"

namespace css {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kJoinSlots = kJoinThreads / 8;  // eight threads a row
constexpr int kJoinRows = 16;                 // rows of a block

// O = sum_i O_i 2^(m_i - m) / sum_i l_i 2^(m_i - m).  The first n1 blocks join
// the items whose tail parts the blocks of the first kernel wrote, the others
// 16 rows each of those of the second (`chunks` blocks an item).  Latency
// bound, the parts lie in L2: the slots that rows leave free take every g-th
// part of a row; the g sums are added in order, so the result does not depend
// on timing.
template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads)
    join_kernel(const PartArgs p1, int n1, const PartArgs p2, int n2, int chunks, const RowsArg o,
                float* lse, int tokens, int Hkv, int G, uint32_t* err) {
  __shared__ float s_sum[kJoinSlots][8][9];
  griddep_launch_dependents();
  griddep_wait();
  const bool one = (int)blockIdx.x < n1;
  const PartArgs& p = one ? p1 : p2;
  const int at_2 = blockIdx.x - n1, c = one ? blockIdx.x : at_2 / chunks;
  const PartDesc d = part_desc(p, c);
  if (d.rows == 0) return;  // block c left no part to join
  if (!part_ok(d.q0, d.kv, d.rows, d.last, c, one ? n1 : n2, p.rows, tokens, Hkv, G)) {
    // two calls share a workspace: wrong rows, but no access outside the tensors
    if (threadIdx.x == 0) atomicOr(err, kErrIndex);
    return;
  }
  const int row0 = one ? 0 : at_2 % chunks * kJoinRows, rows = min(d.rows - row0, kJoinRows);
  if (rows <= 0) return;
  int span = 1;  // rows rounded up to a power of two
  while (span < rows) span <<= 1;
  const int slot = threadIdx.x >> 3, lane = threadIdx.x & 7, c0 = lane * 8;
  const int at_row = slot & (span - 1), group = slot / span, groups = kJoinSlots / span;
  const int row = row0 + at_row;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, l = 0.f, m = -INFINITY;
  if (at_row < rows) {
    // part i of n: the tail part of block c, then head parts
    const unsigned mask = 0xffu << (threadIdx.x & 24);
    const int n = d.last - c + 1;
    for (int i = lane; i < n; i += 8) m = fmaxf(m, p.ml[part_row(p, c + i, i == 0, row)].x);
#pragma unroll
    for (int by = 1; by < 8; by <<= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, by));
#pragma unroll 4
    for (int i = group; i < n; i += groups) {
      const long long at = part_row(p, c + i, i == 0, row);
      const float2 ml = p.ml[at];
      const float4* const s = reinterpret_cast<const float4*>(p.o + at * 64 + c0);
      const float4 x = s[0], y = s[1];
      if (ml.x == -INFINITY && ml.y == 0.f) continue;  // no key of this part is seen
      const float f = ex2_approx(ml.x - m);
      l = fmaf(ml.y, f, l);
      acc[0] = fmaf(x.x, f, acc[0]);
      acc[1] = fmaf(x.y, f, acc[1]);
      acc[2] = fmaf(x.z, f, acc[2]);
      acc[3] = fmaf(x.w, f, acc[3]);
      acc[4] = fmaf(y.x, f, acc[4]);
      acc[5] = fmaf(y.y, f, acc[5]);
      acc[6] = fmaf(y.z, f, acc[6]);
      acc[7] = fmaf(y.w, f, acc[7]);
    }
  }
  float* const mine = s_sum[slot][lane];
#pragma unroll
  for (int e = 0; e < 8; ++e) mine[e] = acc[e];
  mine[8] = l;
  __syncthreads();
  if (group != 0 || at_row >= rows) return;
  for (int g = 1; g < groups; ++g) {
    const float* const other = s_sum[g * span + at_row][lane];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += other[e];
    l += other[8];
  }
  write_row<BF16>(o, lse, tokens, d.q0 + row / G, d.kv * G + row % G, c0, acc, m, l);
}

int launch_join(const PagedDims& d, const DevCtx& ctx, const PartArgs& p1, int n1,
                const PartArgs& p2, int n2, const RowsArg& o, float* lse, cudaStream_t stream) {
  static_assert(kDecodeRows <= kJoinRows && kItemRows % kJoinRows == 0, "rows of a block");
  // no item has more rows than the largest request, nor than its tiles hold
  const long long most = (long long)d.max_new * d.G;
  const int rows = most < kItemRows ? (int)most : kItemRows;
  const int chunks = (rows + kJoinRows - 1) / kJoinRows;
  return cuda_status(launch_dependent(d.bf16 ? join_kernel<true> : join_kernel<false>,
                                      dim3(n1 + n2 * chunks), dim3(kJoinThreads), 0, stream, p1,
                                      n1, p2, n2, chunks, o, lse, d.tokens, d.Hkv, d.G, ctx.err));
}

// The largest grid of the split kernels on any device this library runs on:
// the workspace's size must not depend on the current device.
constexpr int kMaxSm = 160;

}  // namespace

int allow_smem(int which, const void* kernel, size_t bytes) {
  static std::once_flag once[kSmemKernels][64];
  static cudaError_t status[kSmemKernels][64];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e);
  std::call_once(once[which][dev & 63], [&] {
    status[which][dev & 63] = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  });
  return cuda_status(status[which][dev & 63]);
}

namespace {

// A workspace of parts for `blocks` blocks of `rows` rows; 16-byte aligned.
constexpr size_t parts_bytes(size_t blocks, size_t rows) {
  return blocks * sizeof(PartDesc) + blocks * 2 * rows * (64 * 4 + 8);
}

PartArgs parts_at(void* ws, size_t blocks, int rows, int min_tiles) {
  PartArgs p;
  p.desc = static_cast<PartDesc*>(ws);
  p.o = reinterpret_cast<float*>(p.desc + blocks);
  p.ml = reinterpret_cast<float2*>(p.o + blocks * 2 * rows * 64);
  p.rows = rows;
  p.min_tiles = min_tiles;
  return p;
}

// A block takes at least so many tiles: below, starting it and joining its
// parts costs more than its tiles.  Few rows (64-key tiles), us with at least
// 1 / 2 / 4: one request of 100 keys 6.6 / 5.8 / 7.7, of 777 7.8 / 7.8 / 9.0, of
// 4000 11.2 / 9.5 / 10.6, eight of 256 7.7 / 7.9 / 7.3, 64 of 60 7.8 / 7.7 / 11.1.
constexpr int kLeastFew = 2, kLeastRows = 2;

}  // namespace

size_t paged_workspace_bytes(const PagedDims& d) {
  const int ntok = decode_tokens(d.G);
  return (ntok > 0 ? parts_bytes(2 * kMaxSm, kDecodeRows) : 0) +
         (d.max_new > ntok ? parts_bytes(kMaxSm, kItemRows) : 0);
}

int launch_paged_fwd(const PagedDims& d, const DevCtx& ctx, const RowsArg& q, const PoolArg& kc,
                     const PoolArg& vc, const int32_t* table, const int32_t* cu,
                     const int32_t* lens, void* ws, const RowsArg& o, float* lse,
                     cudaStream_t stream) {
  const int ntok = decode_tokens(d.G);
  const int sms = ctx.sm_count < kMaxSm ? ctx.sm_count : kMaxSm;
  uint8_t* at = static_cast<uint8_t*>(ws);
  PartArgs few{}, rows{};
  int n_few = 0, n_rows = 0, rc;
  if (ntok > 0) {
    few = parts_at(at, 2 * kMaxSm, kDecodeRows, kLeastFew);
    at += parts_bytes(2 * kMaxSm, kDecodeRows);
    rc = launch_paged_decode(d, ctx, q, kc, vc, table, cu, lens, few, 2 * sms, o, lse, stream);
    if (rc != ATTN_OK) return rc;
    if (!decode_whole(d, ctx.sm_count)) n_few = 2 * sms;
  }
  if (d.max_new > ntok) {
    rows = parts_at(at, kMaxSm, kItemRows, kLeastRows);
    n_rows = sms;
    rc = launch_paged_rows(d, ctx, q, kc, vc, table, cu, lens, rows, n_rows, ntok, o, lse, stream);
    if (rc != ATTN_OK) return rc;
  }
  if (n_few + n_rows == 0) return ATTN_OK;
  return launch_join(d, ctx, few, n_few, rows, n_rows, o, lse, stream);
}

}  // namespace css
