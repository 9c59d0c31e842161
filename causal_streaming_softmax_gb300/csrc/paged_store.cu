// paged_store.cu - the new tokens' K and V rows into their slots of the paged
// cache: a copy, bound by memory bandwidth (2 x 128 B read and written per
// token and K/V head).
//
// A thread moves 16 bytes of K and the same 16 bytes of V of one (token,
// head); eight threads cover a row, so that a warp's loads and stores are
// whole 128-byte lines whatever the strides.  Rows are read before their
// slots are known, and with many rows a thread has two such moves under way:
// 36,000 tokens of 8 heads (149 MB) take 23.0 us, 96% of the measured copy
// rate; one move a thread 24.1, the slot before the row 25.0, four moves 25.3.
#include "serve_index.h"
#include "serve_internal.h"
#include "sm103.cuh"

namespace css {
namespace {

constexpr int kThreads = 256;

struct StoreArgs {
  int tokens, Hkv, pages, shift;
  RowsArg k, v;
  PoolArg kc, vc;
  const int32_t* slots;
  uint32_t* err;
};

// kMoves: moves of a thread in one round.
template <int kMoves>
__global__ void __launch_bounds__(kThreads) paged_store_kernel(const StoreArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const long long n = (long long)a.tokens * a.Hkv * 8;
  const long long step = (long long)gridDim.x * kThreads * kMoves;
  bool bad = false;
  for (long long i0 = (long long)blockIdx.x * kThreads * kMoves + threadIdx.x; i0 < n; i0 += step) {
    uint4 kw[kMoves], vw[kMoves];
    long long k_at[kMoves], v_at[kMoves];
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      const long long i = i0 + u * kThreads;
      k_at[u] = -1;
      if (i >= n) continue;
      const int c = (int)(i & 7) * 8;
      const long long row = i >> 3;
      const int t = (int)(row / a.Hkv), h = (int)(row - (long long)t * a.Hkv);
      const int slot = a.slots[t];
      kw[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.k.p) + t * a.k.t +
                                              h * a.k.h + c);
      vw[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.v.p) + t * a.v.t +
                                              h * a.v.h + c);
      if (slot < 0) continue;
      const int page = slot >> a.shift, r = slot & ((1 << a.shift) - 1);
      if (!page_ok(page, a.pages)) {
        bad = true;
        continue;
      }
      k_at[u] = page * a.kc.pg + h * a.kc.h + r * a.kc.r + c;
      v_at[u] = page * a.vc.pg + h * a.vc.h + r * a.vc.r + c;
    }
#pragma unroll
    for (int u = 0; u < kMoves; ++u)
      if (k_at[u] >= 0) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.kc.p) + k_at[u]) = kw[u];
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.vc.p) + v_at[u]) = vw[u];
      }
  }
  if (bad) atomicOr(a.err, kErrIndex);
}

}  // namespace

int launch_paged_store(const PagedDims& d, const DevCtx& ctx, const RowsArg& k, const RowsArg& v,
                       const int32_t* slots, const PoolArg& kc, const PoolArg& vc,
                       cudaStream_t stream) {
  const long long moves = (long long)d.tokens * d.Hkv * 8;
  const StoreArgs args{d.tokens, d.Hkv, d.pages, d.shift, k, v, kc, vc, slots, ctx.err};
  // two moves a thread once that fills every SM (eight blocks each); below, one
  // move finds its SM sooner (64 tokens 1.9 us against 2.2)
  const bool two = moves >= 2LL * kThreads * 8 * ctx.sm_count;
  const long long per = (two ? 2 : 1) * kThreads, most = 16LL * ctx.sm_count;
  const long long blocks = (moves + per - 1) / per;
  return cuda_status(launch_dependent(two ? paged_store_kernel<2> : paged_store_kernel<1>,
                                      dim3((unsigned)(blocks > most ? most : blocks)),
                                      dim3(kThreads), 0, stream, args));
}

}  // namespace css
