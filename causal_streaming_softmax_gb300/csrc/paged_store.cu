// paged_store.cu - the new tokens' K and V rows into their slots of the paged
// cache: a copy, bound by memory bandwidth (2 x 128 B read and written per
// token and K/V head).
//
// A thread moves 16 bytes of K and the same 16 bytes of V of one (token,
// head); eight threads cover a row, so that a warp's loads and stores are
// whole 128-byte lines whatever the strides.
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

__global__ void __launch_bounds__(kThreads) paged_store_kernel(const StoreArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const long long n = (long long)a.tokens * a.Hkv * 8;
  const long long step = (long long)gridDim.x * kThreads;
  bool bad = false;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
    const int c = (int)(i & 7) * 8;
    const long long row = i >> 3;
    const int t = (int)(row / a.Hkv), h = (int)(row - (long long)t * a.Hkv);
    const int slot = a.slots[t];
    if (slot < 0) continue;
    const int page = slot >> a.shift, r = slot & ((1 << a.shift) - 1);
    if (!page_ok(page, a.pages)) {
      bad = true;
      continue;
    }
    const uint4 kw = *reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(a.k.p) + t * a.k.t + h * a.k.h + c);
    const uint4 vw = *reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(a.v.p) + t * a.v.t + h * a.v.h + c);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.kc.p) + page * a.kc.pg + h * a.kc.h +
                              r * a.kc.r + c) = kw;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.vc.p) + page * a.vc.pg + h * a.vc.h +
                              r * a.vc.r + c) = vw;
  }
  if (bad) atomicOr(a.err, kErrIndex);
}

}  // namespace

int launch_paged_store(const PagedDims& d, const DevCtx& ctx, const RowsArg& k, const RowsArg& v,
                       const int32_t* slots, const PoolArg& kc, const PoolArg& vc,
                       cudaStream_t stream) {
  const long long blocks = ((long long)d.tokens * d.Hkv * 8 + kThreads - 1) / kThreads;
  const long long most = 64LL * ctx.sm_count;
  const StoreArgs args{d.tokens, d.Hkv, d.pages, d.shift, k, v, kc, vc, slots, ctx.err};
  return cuda_status(launch_dependent(paged_store_kernel,
                                      dim3((unsigned)(blocks > most ? most : blocks)),
                                      dim3(kThreads), 0, stream, args));
}

}  // namespace css
