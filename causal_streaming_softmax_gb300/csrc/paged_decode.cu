// paged_decode.cu - attention of a request's few new rows (new tokens x heads
// of a group <= 16) over its pages: the token step of a server.
//
// For each request and K/V head: S = Q K^T, t = S c in base 2, per key block
// m' = max(m, max t), P = 2^(t - m'), l = l 2^(m - m') + sum P (binary32, P
// unrounded), O = O 2^(m - m') + P V with P rounded to the operands' type;
// O / l and L = m + log2 l.  P is rounded because the matrix product takes
// 16-bit operands, as in every forward pass of the library; next to the rounding
// of O that adds up to a tenth to the error against 64 bits (binary16 2.2e-4,
// bfloat16 1.8e-3, relative to the outputs' norm).
//
// Bound by memory: 256 bytes of K and V a key and K/V head, 4 * 64 * 16
// operations on a padded 16-row tile, a twentieth of what the matrix units
// could do in that time.  So the design is about keeping loads in flight:
//  * the keys of all requests and heads form one list of 64-key tiles, which
//    the blocks share out in equal runs whatever the requests' lengths (a
//    request that crosses a border is joined by a second kernel from binary32
//    parts, in a fixed order);
//  * a producer warp copies tiles by TMA into a ring of stages, its page ids
//    read 32 at a time ahead of their use; two blocks a SM keep 2 x 5 x 16 KB
//    under way.  The 8 bytes a request of the tile counts (s_pre) end that
//    between 1,024 and 1,280 requests, from where one block fits: 6.7 TB/s at
//    1,024 requests of 512..3500 keys (32 / 4 heads), 3.9 at 1,280 and at 4,096;
//  * four consumer warps (eight where a block takes whole items) take 16 keys
//    each of every tile with their own running maximum, in registers from S to
//    O (warp-level matrix products: with 16 rows and a handful of keys a warp, a
//    tensor-memory round trip would be the longer path), and meet once a work
//    item, which the producer describes to them beside its Q;
//  * the next item's request and page ids are read while this one's tiles
//    arrive, so that short requests do not wait for them.
//
// Measured (GB300, join included; boxes differ by 2%): 256 requests over
// 1024..16384 keys, 32 / 4 heads 310 to 317 us = 6.7 to 6.8 TB/s, 98 to 101% of
// the measured copy rate; 64 over 17..8192, 32 / 8 heads 93 us = 5.97 TB/s; 2 over
// 50000..65536, 16 / 16 heads 75 us = 6.25 TB/s; one over 777 keys 7.9 us, nearly
// all of it two launches and the chain of loads lengths -> page ids -> pages ->
// parts.
#include <math.h>

#include "serve_index.h"
#include "serve_internal.h"
#include "serve_parts.cuh"
#include "sm103.cuh"
#include "warp_mma.cuh"

namespace css {
namespace {

// A block's shape: consumer warps of 16 keys each, stages, and its shared
// memory.  kWhole: a block takes whole items, so that nothing is joined.
template <int CONSUMERS, int STAGES, bool WHOLE>
struct Config {
  static constexpr bool kWhole = WHOLE;
  static constexpr int kMaxBatch = WHOLE ? 1024 : kMaxPagedBatch;  // whole: <= the SMs
  static constexpr int kConsumers = CONSUMERS, kStages = STAGES;
  static constexpr int kThreads = 32 * (CONSUMERS + 1);
  static constexpr int kTileKeys = 16 * CONSUMERS;
  static constexpr uint32_t kHalf = kTileKeys * 128;  // K (or V) of a stage
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr uint32_t kQ = kDecodeRows * 128;
  static constexpr uint32_t kSmemQ = kStages * kStage;
  static constexpr uint32_t kSmemJoin = kSmemQ + 2 * kQ;
  static constexpr uint32_t kSmemMl = kSmemJoin + kConsumers * kDecodeRows * 68 * 4;
  static constexpr uint32_t kSmemBar = kSmemMl + kConsumers * kDecodeRows * 8;
  static constexpr uint32_t kSmemPre = kSmemBar + 128;  // + 8 (batch + 1), + alignment slack
  // barriers
  static constexpr int kFull = 0, kEmpty = kStages, kQFull = 2 * kStages, kQFree = kQFull + 2;
  static_assert((kQFree + 2) * 8 <= 128, "barrier area");
};
using Split = Config<4, 5, false>;
using Whole = Config<8, 4, true>;
static_assert(Split::kSmemPre + 8 * (Split::kMaxBatch + 1) + 1024 <= 227 * 1024 - 2048 &&
                  Whole::kSmemPre + 8 * (Whole::kMaxBatch + 1) + 1024 <= 227 * 1024 - 2048,
              "shared memory of a block");
constexpr int kLd = 68;  // floats a row of the joining buffer (bank spread)

struct DecodeArgs {
  int batch, tokens, H, Hkv, G, ntok, max_new, pages, width, shift;
  float c;
  const int32_t *cu, *lens, *table;
  RowsArg o;
  float* lse;
  PartArgs part;
  uint32_t* err;
  uint64_t wait_ns;
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

// A place in the tile list: tile t0 of nt of a request and K/V head.
struct Place {
  Request r;
  int req, kv, t0, nt;
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
  p.r = request_at(a, p.req, &b);
  p.nt = tiles_of<C>(p.r.n_keys);
  const long long kv = C::kWhole ? off : quot(off, p.nt);
  p.t0 = C::kWhole ? 0 : (int)(off - kv * p.nt);
  p.kv = (int)min(kv, a.Hkv - 1ll);  // less already, unless lens changed meanwhile
  return p;
}

// The place behind an item: the next head or the next request with rows.
// Called only where the list goes on; never past the last request, also where
// lens changed meanwhile.
template <class C>
__device__ __forceinline__ void next_place(const DecodeArgs& a, const long long* pre, Place* p) {
  p->t0 = 0;
  if (++p->kv < a.Hkv) return;
  p->kv = 0;
  do {
    p->req = min(p->req + 1, a.batch - 1);
  } while (pre[p->req + 1] == pre[p->req] && p->req + 1 < a.batch);
  bool b;
  p->r = request_at(a, p->req, &b);
  p->nt = tiles_of<C>(p->r.n_keys);
}

template <bool BF16, class C>
__global__ void __launch_bounds__(C::kThreads, C::kWhole ? 1 : 2)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const DecodeArgs a) {
  constexpr int kConsumers = C::kConsumers, kStages = C::kStages, kThreads = C::kThreads,
                kTileKeys = C::kTileKeys;
  constexpr uint32_t kHalf = C::kHalf, kStage = C::kStage, kQ = C::kQ, kSmemQ = C::kSmemQ;
  constexpr int BAR_FULL = C::kFull, BAR_EMPTY = C::kEmpty, BAR_Q = C::kQFull,
                BAR_Q_FREE = C::kQFree;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int s_abort;
  __shared__ Item s_item[2];  // [Q buffer]
  __shared__ long long s_scan[kThreads / 32];
  griddep_launch_dependents();
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (sbase - smem_u32(smem_raw));
  float* const s_join = reinterpret_cast<float*>(smem + C::kSmemJoin);
  float2* const s_ml = reinterpret_cast<float2*>(smem + C::kSmemMl);
  long long* const s_pre = reinterpret_cast<long long*>(smem + C::kSmemPre);
  const uint32_t bar0 = sbase + C::kSmemBar;
#define BAR(i) (bar0 + 8u * (uint32_t)(i))
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const WaitCtl wc{a.err, a.wait_ns, &s_abort};

  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(BAR(BAR_FULL + s), 1);
      mbar_init(BAR(BAR_EMPTY + s), kConsumers);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(BAR(BAR_Q + s), 1);
      mbar_init(BAR(BAR_Q_FREE + s), kConsumers);
    }
    fence_mbarrier_init();
  }
  // rows of the query tile that no copy fills read as zero
  for (int i = tid; i < (int)(2 * kQ / 16); i += kThreads)
    reinterpret_cast<uint4*>(smem + kSmemQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_shared();
  griddep_wait();

  // tiles of one head before each request, every block for itself
  {
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int i0 = tid * per, i1 = min(a.batch, i0 + per);
    long long sum = 0;
    bool bad = false;
    for (int i = i0; i < i1; ++i) {
      bool b;
      const Request r = request_at(a, i, &b);
      bad |= b;
      s_pre[i + 1] = sum += r.n_new > 0 ? (C::kWhole ? 1 : tiles_of<C>(r.n_keys)) : 0;
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
  const Share share = share_of(s_pre[a.batch] * a.Hkv, C::kWhole ? 1 : a.part.min_tiles, gridDim.x, blockIdx.x);

  if (warp == kConsumers) {
    // ---------------- producer ----------------
    const int box = min(1 << a.shift, kTileKeys);         // rows a copy
    const int boxes = kTileKeys / box;                    // copies a tile of K (and of V)
    const int per_tile = (1 << a.shift) >= kTileKeys ? 0 : boxes;
    int it = 0, nq = 0;
    bool ok = true, bad = false, tail = false;
    // page ids go 32 at a time: lane l of group g has page first + 32 g + l.
    // The first two groups of the next item are read while this one runs.
    Place nx{};
    int nx_ids = 0, nx_next = 0;
    const auto read_ids = [&] {
      const int32_t* const row = a.table + (long long)nx.req * a.width;
      const int at = (int)(((long long)nx.t0 * kTileKeys) >> a.shift) + lane;
      const int n = (int)pages_for(nx.r.n_keys, a.shift);
      nx_ids = at < n ? row[at] : a.pages;
      nx_next = at + 32 < n ? row[at + 32] : a.pages;
    };
    if (share.begin < share.end) {
      nx = place_at<C>(a, s_pre, share.begin);
      read_ids();
    }
    for (long long pos = share.begin; ok && pos < share.end;) {
      const Place sg = nx;
      const Request r = sg.r;
      const int t1 = C::kWhole ? sg.nt : (int)min((long long)sg.nt, sg.t0 + (share.end - pos));
      const int32_t* const row = a.table + (long long)sg.req * a.width;
      const int n_pages = (int)pages_for(r.n_keys, a.shift);
      int base = (int)(((long long)sg.t0 * kTileKeys) >> a.shift);
      int ids = nx_ids, next = nx_next;
      const long long last = pos - sg.t0 + sg.nt - 1;  // the item's last position
      pos += C::kWhole ? 1 : t1 - sg.t0;
      if (pos < share.end) {
        next_place<C>(a, s_pre, &nx);
        read_ids();
      }
      const int qbuf = nq & 1;
      ok = !(nq >= 2) || mbar_wait_warp(BAR(BAR_Q_FREE + qbuf), ((nq >> 1) - 1) & 1, wc);
      if (!ok) break;
      if (lane == 0) {
        s_item[qbuf] = Item{r, sg.kv, sg.t0, t1, C::kWhole || (sg.t0 == 0 && t1 == sg.nt)};
        mbar_arrive_expect_tx(BAR(BAR_Q + qbuf), a.ntok * a.G * 128);
        tma_load_4d(sbase + kSmemQ + qbuf * kQ, &tm_q, BAR(BAR_Q + qbuf), 0, 0, sg.kv, r.q0);
      }
      ++nq;
      for (int t = sg.t0; t < t1; ++t, ++it) {
        const int s = it % kStages;
        if (it >= kStages && !mbar_wait_warp(BAR(BAR_EMPTY + s), (it / kStages - 1) & 1, wc)) {
          ok = false;
          break;
        }
        const int k0 = t * kTileKeys;
        const int page = k0 >> a.shift;  // the tile's first page
        if (page - base >= 32) {
          base += 32;
          ids = next;
          next = base + 32 + lane < n_pages ? row[base + 32 + lane] : a.pages;
        }
        // boxes that hold keys below n_keys; the rest of the stage is masked
        const int live = r.n_keys <= k0 ? 0 : min(boxes, (r.n_keys - k0 - 1) / box + 1);
        if (lane == 0) mbar_arrive_expect_tx(BAR(BAR_FULL + s), 2 * live * box * 128);
        __syncwarp();
#pragma unroll
        for (int b0 = 0; b0 < kTileKeys / 8; b0 += 16) {  // pages of 8 tokens make the most boxes
          if (b0 >= boxes) break;
          const int bx = b0 + (lane & 15);
          const int id = __shfl_sync(0xffffffffu, ids, (page - base + (per_tile ? bx : 0)) & 31);
          const bool fine = page_ok(id, a.pages);
          if (bx < live) {
            bad |= !fine;
            tma_load_4d(sbase + s * kStage + (lane >> 4) * kHalf + bx * box * 128,
                        lane < 16 ? &tm_k : &tm_v, BAR(BAR_FULL + s), 0,
                        per_tile ? 0 : k0 & ((1 << a.shift) - 1), sg.kv,
                        fine ? id : a.pages);  // past the pool: reads as zero
          }
        }
      }
      if (!C::kWhole && sg.t0 == 0 && t1 < sg.nt) {
        tail = true;
        if (lane == 0)
          a.part.desc[blockIdx.x] = PartDesc{r.q0, sg.kv, r.n_new * a.G, last_block(share, last)};
      }
    }
    if (!C::kWhole && lane == 0 && !tail) a.part.desc[blockIdx.x] = PartDesc{0, 0, 0, 0};
    if (bad) atomicOr(a.err, kErrIndex);
    // no copy may still be landing when the block exits (matters only when a
    // wait gave up)
    if (lane == 0) {
      for (int q = 0; q < 2 && q < nq; ++q) drain_wait(BAR(BAR_Q + q), ((nq - q + 1) / 2 - 1) & 1);
      for (int k = it > kStages ? it - kStages : 0; k < it; ++k)
        drain_wait(BAR(BAR_FULL + k % kStages), (k / kStages) & 1);
    }
  } else {
    // ---------------- consumers ----------------
    const int g = lane >> 2, tq = lane & 3;
    const int mi = lane >> 3, mr = lane & 7;
    int it = 0, nq = 0;
    for (long long pos = share.begin; pos < share.end;) {
      const int qbuf = nq & 1;
      uint32_t q[4][4];
      Item sg{};
      bool ok = mbar_wait_warp(BAR(BAR_Q + qbuf), (nq >> 1) & 1, wc);
      if (ok) {
        sg = s_item[qbuf];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          ldmatrix_x4(sbase + kSmemQ + qbuf * kQ +
                          sw128_offset((mi & 1) * 8 + mr, 2 * kk + (mi >> 1)),
                      q[kk]);
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(BAR_Q_FREE + qbuf));
      }
      ++nq;
      const Request r = sg.r;
      const int t1 = sg.t1, rows = r.n_new * a.G;
      pos += C::kWhole ? 1 : t1 - sg.t0;
      // keys that this thread's two rows see
      const int first_lim = row_limit(r.n_keys, r.n_new, 0);
      const int lim0 = row_limit(r.n_keys, r.n_new, g / a.G),
                lim1 = row_limit(r.n_keys, r.n_new, (g + 8) / a.G);
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      float o[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

      for (int t = sg.t0; t < t1; ++t, ++it) {
        const int s = it % kStages;
        ok = mbar_wait_warp(BAR(BAR_FULL + s), (it / kStages) & 1, wc);
        if (!ok) break;
        const uint32_t ks = sbase + s * kStage + warp * 16 * 128, vs = ks + kHalf;
        const int k0 = t * kTileKeys + warp * 16;
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint32_t kf[4];
          ldmatrix_x4(ks + sw128_offset((mi >> 1) * 8 + mr, 2 * kk + (mi & 1)), kf);
          mma_16816<BF16>(sc[0], q[kk], kf[0], kf[1]);
          mma_16816<BF16>(sc[1], q[kk], kf[2], kf[3]);
        }
        const bool edge = past_limit(k0, 16, first_lim);  // some row does not see every key
        if (edge) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = k0 + n * 8 + tq * 2 + e;
              if (key >= lim0) sc[n][e] = -INFINITY;
              if (key >= lim1) sc[n][2 + e] = -INFINITY;
            }
        }
        float x0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
        float x1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
        const float n0 = fmaxf(m0, x0 * a.c), n1 = fmaxf(m1, x1 * a.c);
        const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
        const float al0 = ex2_approx(m0 - u0), al1 = ex2_approx(m1 - u1);
        m0 = n0;
        m1 = n1;
        float p[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          p[n][0] = ex2_approx(fmaf(sc[n][0], a.c, -u0));
          p[n][1] = ex2_approx(fmaf(sc[n][1], a.c, -u0));
          p[n][2] = ex2_approx(fmaf(sc[n][2], a.c, -u1));
          p[n][3] = ex2_approx(fmaf(sc[n][3], a.c, -u1));
        }
        l0 = l0 * al0 + ((p[0][0] + p[0][1]) + (p[1][0] + p[1][1]));
        l1 = l1 * al1 + ((p[0][2] + p[0][3]) + (p[1][2] + p[1][3]));
        if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i][0] *= al0;
            o[i][1] *= al0;
            o[i][2] *= al1;
            o[i][3] *= al1;
          }
        }
        const uint32_t pf[4] = {pack2<BF16>(p[0][0], p[0][1]), pack2<BF16>(p[0][2], p[0][3]),
                                pack2<BF16>(p[1][0], p[1][1]), pack2<BF16>(p[1][2], p[1][3])};
        uint32_t odd = 0;  // V values of the edge that are not finite
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
          uint32_t vf[4];
          ldmatrix_x4_trans(vs + sw128_offset((mi & 1) * 8 + mr, c + (mi >> 1)), vf);
          if (edge) {
            // keys that no row sees count as zero whatever stands there, and
            // so, for now, does a value that is not finite
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              vf[j] = drop_keys(vf[j], r.n_keys - (k0 + (j & 1) * 8 + tq * 2));
              odd |= drop_nonfinite<BF16>(&vf[j]);
            }
          }
          mma_16816<BF16>(o[c], pf, vf[0], vf[1]);
          mma_16816<BF16>(o[c + 1], pf, vf[2], vf[3]);
        }
        if (edge && __any_sync(0xffffffffu, odd != 0)) {
          // add what the dropped values give the rows that see them
          for (int key = 0; key < 16; ++key) {
            const int src = (lane & ~3) | ((key & 7) >> 1);
            const float pe0 = key & 8 ? p[1][0] : p[0][0], po0 = key & 8 ? p[1][1] : p[0][1];
            const float pe1 = key & 8 ? p[1][2] : p[0][2], po1 = key & 8 ? p[1][3] : p[0][3];
            const float w0 = __shfl_sync(0xffffffffu, key & 1 ? po0 : pe0, src);
            const float w1 = __shfl_sync(0xffffffffu, key & 1 ? po1 : pe1, src);
            if (k0 + key >= r.n_keys) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint16_t h = *reinterpret_cast<const uint16_t*>(
                    smem + (vs - sbase) + sw128_offset(key, i) + (tq * 2 + e) * 2);
                const float v = half_to_f32<BF16>(h);
                if (!isfinite(v)) {
                  if (k0 + key < lim0) o[i][e] = fmaf(w0, v, o[i][e]);
                  if (k0 + key < lim1) o[i][2 + e] = fmaf(w1, v, o[i][2 + e]);
                }
              }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(BAR_EMPTY + s));
      }

      // ---------------- the consumer warps meet ----------------
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      if (tq == 0) {
        s_ml[warp * kDecodeRows + g] = make_float2(m0, l0);
        s_ml[warp * kDecodeRows + g + 8] = make_float2(m1, l1);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float* const d = s_join + (warp * kDecodeRows + g) * kLd + i * 8 + tq * 2;
        *reinterpret_cast<float2*>(d) = make_float2(o[i][0], o[i][1]);
        *reinterpret_cast<float2*>(d + 8 * kLd) = make_float2(o[i][2], o[i][3]);
      }
      // where a wait gave up, all leave together
      if (named_barrier_any(1, kConsumers * 32, !ok)) break;
      const int row = tid >> 3, c0 = (tid & 7) * 8;
      if (row < rows) {  // the first 128 threads have a row
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) m = fmaxf(m, s_ml[w * kDecodeRows + row].x);
        // a NaN anywhere in the row's scores stays one
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, l = 0.f;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) {
          const float2 ml = s_ml[w * kDecodeRows + row];
          if (ml.x == -INFINITY && ml.y == 0.f) continue;
          const float f = ex2_approx(ml.x - m);
          l = fmaf(ml.y, f, l);
          const float* const d = s_join + (w * kDecodeRows + row) * kLd + c0;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = fmaf(d[e], f, acc[e]);
        }
        const int tok = r.q0 + row / a.G, h = sg.kv * a.G + row % a.G;
        if (sg.whole)
          write_row<BF16>(a.o, a.lse, a.tokens, tok, h, c0, acc, m, l);
        else
          store_part(a.part, blockIdx.x, sg.t0 == 0, row, c0, acc, m, l);
      }
      named_barrier_sync(1, kConsumers * 32);
    }
  }
#undef BAR
}

}  // namespace

constexpr int kWholeKeys = 256;

int decode_tokens(int G) { return G > kDecodeRows ? 0 : kDecodeRows / G; }


namespace {

template <class C>
int launch(const PagedDims& d, const DevCtx& ctx, const RowsArg& q, const PoolArg& kc,
           const PoolArg& vc, const DecodeArgs& args, int blocks, int which, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  const uint32_t box = (1u << d.shift) < C::kTileKeys ? (1u << d.shift) : C::kTileKeys;
  const uint64_t P = 1ull << d.shift;
  if (!encode_tmap_4d(&tq, d.bf16, q.p, d.G, d.Hkv, d.tokens, q.h, q.h * d.G, q.t, d.G, 1,
                      args.ntok) ||
      !encode_tmap_4d(&tk, d.bf16, kc.p, P, d.Hkv, d.pages, kc.r, kc.h, kc.pg, box, 1, 1) ||
      !encode_tmap_4d(&tv, d.bf16, vc.p, P, d.Hkv, d.pages, vc.r, vc.h, vc.pg, box, 1, 1))
    return ATTN_ERR_CUDA;
  const size_t smem = C::kSmemPre + 8 * (size_t)(d.batch + 1) + 1024;
  auto* kernel = d.bf16 ? paged_decode_kernel<true, C> : paged_decode_kernel<false, C>;
  const int rc = allow_smem(which + d.bf16, reinterpret_cast<const void*>(kernel),
                            C::kSmemPre + 8 * (C::kMaxBatch + 1) + 1024);
  if (rc != ATTN_OK) return rc;
  return cuda_status(launch_dependent(kernel, dim3(blocks), dim3(C::kThreads), smem, stream, tq,
                                      tk, tv, args));
}

}  // namespace

// Whole items where every item finds an SM and the table leaves room for no
// more than kWholeKeys keys a request: eight warps are through with an item in
// two steps, and the parts and the second launch fall away.  Split / whole, us:
// one request of 100 keys 5.8 / 4.4, of 250 7.2 / 5.4, of 777 7.8 / 9.6, of 4000
// 9.5 / 32; eight of 256 7.9 / 5.5; 64 of 60 (512 items) 7.7 / 16.7.  The width
// stands for the lengths, which the host does not see: short requests in a wide
// table take the split form and its 1.4 to 3 us.
bool decode_whole(const PagedDims& d, int sm_count) {
  return (long long)d.batch * d.Hkv <= sm_count && ((long long)d.width << d.shift) <= kWholeKeys;
}

int launch_paged_decode(const PagedDims& d, const DevCtx& ctx, const RowsArg& q,
                        const PoolArg& kc, const PoolArg& vc, const int32_t* table,
                        const int32_t* cu, const int32_t* lens, const PartArgs& part, int blocks,
                        const RowsArg& o, float* lse, cudaStream_t stream) {
  const DecodeArgs args{d.batch, d.tokens, d.H, d.Hkv, d.G,  decode_tokens(d.G), d.max_new,
                        d.pages, d.width,  d.shift, d.c, cu, lens, table, o, lse, part, ctx.err,
                        ctx.wait_ns};
  if (decode_whole(d, ctx.sm_count))
    return launch<Whole>(d, ctx, q, kc, vc, args, d.batch * d.Hkv, kSmemWholeF16, stream);
  return launch<Split>(d, ctx, q, kc, vc, args, blocks, kSmemDecodeF16, stream);
}

}  // namespace css
