// serve_decode.cuh - what the kernels of a request's few new rows share: the list
// of key tiles of all requests and K/V heads, and the places in it.
#pragma once

#include "serve_index.h"
#include "serve_internal.h"
#include "sm103.cuh"

namespace css {

struct DecodeArgs {
  int batch, tokens, H, Hkv, G, ntok, max_new, pages, width, shift;
  float c;
  const int32_t *cu, *lens, *table;
  RowsArg o;
  float* lse;
  PartArgs part;
  uint32_t* err;
  uint64_t wait_ns;
  int split;  // 4 bits: tokens of an item, at most (all of a request unless C::kSplit)
  int drop;   // 4 bits: binary orders that scores of the edge's walk are down by,
  float c_drop;  // and c times as much
};

// A request's rows and keys; n_new 0 for one that this kernel does not take.
struct Request {
  int q0, n_new, n_keys;
};

__device__ __forceinline__ Request request_at(const DecodeArgs& a, int i, bool* bad) {
  const RowRange r = row_range(a.cu[i], a.cu[i + 1], a.tokens);
  bool b;
  Request q{r.begin, r.end - r.begin, key_count(a.lens[i], a.width, a.shift, &b)};
  *bad = r.bad || b || q.n_new > a.max_new;
  if (q.n_new > min(a.ntok, a.max_new)) q.n_new = 0;
  return q;
}

template <class C>
__device__ __forceinline__ int tiles_of(int n_keys) {
  return n_keys <= 0 ? 1 : (n_keys - 1) / C::kTileKeys + 1;
}

// C::kSplit: a request with more tokens than an item has rows for is several: its
// first `split` tokens over the keys that they see, and so on.
template <class C>
__device__ __forceinline__ int sub_count(const DecodeArgs& a, const Request& r) {
  return C::kSplit ? (r.n_new + a.split - 1) / a.split : 1;
}
template <class C>
__device__ __forceinline__ Request sub_request(const DecodeArgs& a, const Request& r, int i) {
  if (!C::kSplit) return r;
  const int first = i * a.split, n = min(a.split, r.n_new - first);
  return Request{r.q0 + first, n, r.n_keys - (r.n_new - first - n)};
}

// A place in the tile list: tile t0 of nt of a request and K/V head.
struct Place {
  Request r;
  int req, kv, t0, nt;
  Request all;  // C::kSplit: r is part `sub` of it
  int sub;
};

// What the producer hands the consumers beside an item's Q: they read no device
// array themselves, so that the warps agree on an item whatever those hold.
struct Item {
  Request r;
  int kv, t0, t1;
  int whole;  // its rows are finished here; else a part
};

// The place at position pos.  pre[i] counts the tiles (whole: the items) of one
// head of the requests before i.
template <class C>
__device__ __forceinline__ Place place_at(const DecodeArgs& a, const long long* pre,
                                          long long pos) {
  int lo = 0, hi = a.batch;  // the last i with pre[i] * Hkv <= pos: never an empty request
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] * a.Hkv <= pos)
      lo = mid + 1;
    else
      hi = mid;
  }
  Place p;
  p.req = lo - 1;
  const long long off = pos - pre[p.req] * a.Hkv;
  bool b;
  p.all = request_at(a, p.req, &b);
  p.sub = 0;
  p.r = sub_request<C>(a, p.all, 0);
  p.nt = tiles_of<C>(p.r.n_keys);
  const int subs = sub_count<C>(a, p.all);
  long long per = p.nt;  // tiles of a head
  if (C::kSplit)
    for (int i = 1; i < subs; ++i) per += tiles_of<C>(sub_request<C>(a, p.all, i).n_keys);
  const long long kv = C::kWhole ? off : quot(off, per);
  p.t0 = C::kWhole ? 0 : (int)(off - kv * per);
  p.kv = (int)min(kv, a.Hkv - 1ll);  // less already, unless lens changed meanwhile
  if (C::kSplit)
    while (p.t0 >= p.nt && p.sub + 1 < subs) {
      p.t0 -= p.nt;
      p.r = sub_request<C>(a, p.all, ++p.sub);
      p.nt = tiles_of<C>(p.r.n_keys);
    }
  return p;
}

// The place behind an item: the next head or the next request with rows.
// Called only where the list goes on; never past the last request, also where
// lens changed meanwhile.
template <class C>
__device__ __forceinline__ void next_place(const DecodeArgs& a, const long long* pre, Place* p) {
  p->t0 = 0;
  if (C::kSplit && sub_count<C>(a, p->all) > 1) {
    if (++p->sub == sub_count<C>(a, p->all)) p->sub = 0, ++p->kv;
    if (p->kv < a.Hkv) {
      p->r = sub_request<C>(a, p->all, p->sub);
      p->nt = tiles_of<C>(p->r.n_keys);
      return;
    }
  } else if (++p->kv < a.Hkv) {
    return;
  }
  p->kv = 0;
  do {
    p->req = min(p->req + 1, a.batch - 1);
  } while (pre[p->req + 1] == pre[p->req] && p->req + 1 < a.batch);
  bool b;
  p->all = request_at(a, p->req, &b);
  p->sub = 0;
  p->r = sub_request<C>(a, p->all, 0);
  p->nt = tiles_of<C>(p->r.n_keys);
}

// Tiles (whole: items) of one head before each request, every block for itself:
// s_pre [batch + 1].  Called by all threads of the block.
template <class C>
__device__ __forceinline__ void tiles_before_each(const DecodeArgs& a, long long* s_pre,
                                                  long long* s_scan) {
  constexpr int kThreads = C::kThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int i0 = tid * per, i1 = min(a.batch, i0 + per);
  long long sum = 0;
  bool bad = false;
  for (int i = i0; i < i1; ++i) {
    bool b;
    const Request r = request_at(a, i, &b);
    bad |= b;
    int subs = r.n_new > 0 ? sub_count<C>(a, r) : 0;
    while (--subs >= 0)
      sum += C::kWhole ? 1 : tiles_of<C>(sub_request<C>(a, r, subs).n_keys);
    s_pre[i + 1] = sum;
  }
  if (bad && blockIdx.x == 0) atomicOr(a.err, kErrIndex);
  long long upto = sum;
#pragma unroll
  for (int by = 1; by < 32; by <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, by);
    if (lane >= by) upto += x;
  }
  if (lane == 31) s_scan[warp] = upto;
  __syncthreads();
  long long before = upto - sum;
  for (int w = 0; w < warp; ++w) before += s_scan[w];
  for (int i = i0; i < i1; ++i) s_pre[i + 1] += before;
  if (tid == 0) s_pre[0] = 0;
  __syncthreads();
}

}  // namespace css
