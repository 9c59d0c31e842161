// paged_decode4.cu - attention of a request's few new rows (new tokens x heads of
// a group <= 16) over the pages of a 4-bit cache: the token step of a server.
//
// The arithmetic is that of the 16-bit kernel (S = Q K^T, P = 2^(S c - m), running
// maximum m and sum l in binary32, O += P V) over values code * scale, which are exact
// in 16 bits (pool4.cuh); what is rounded to 16 bits is q, once an item, and P times V's
// scales, both to binary16 whatever the cache's type.
//
// 72 bytes a key and K/V head come from memory where the 16-bit cache has 256, so
// the same arithmetic has less than a third of the time: for 16 keys of a K/V head
// the schedulers of a SM have some 200 issue slots at the copy rate, and the kernel
// takes about 140.  Hence:
//  * S^T = K Q^T and O^T = V^T P^T: the 16-row side of the warp-level product holds
//    keys and channels, the 8-column side the query rows, so that a group of up to
//    eight rows pads nothing and half the products, maxima and exponentials of the
//    other way round remain.  9 to 16 rows take two column tiles;
//  * a lane reads a quarter of a key's codes (eight bytes) and has in them the
//    channels that its places in two fragments of either half stand for, in an order
//    of its own that Q's fragments follow: no shuffle between code and product;
//  * ldmatrix takes V's codes two bytes at a time as 16-bit elements and transposes
//    them, which puts the same channel of two keys side by side in a word: the four
//    codes of an element are the four channel tiles of O^T;
//  * all products take binary16: the bits of code + 8 are the subnormal number
//    (code + 8) 2^-24 (2^-20 in the high half of a byte), which costs an AND and no
//    conversion.  q goes in with its row's largest element at 2^9 (low channels 2^13).
//    K's scale is applied to the scores, the offset of 8 times the sum of q is where they
//    start.  V's scale, which varies along the sum, goes into the weights, the offset
//    comes off V's codes (left in, it would be taken off a sum ten times the result);
//  * weights times V's scales are binary16 too, a weight of 1 counting 2^kBias and the
//    scales in a unit near the largest so far: spacing 2^-34 of that;
//  * m and the units are followed only when a lane's sum of a step's weights passes
//    kMost or a scale leaves its unit's range: one vote a step, no maximum over the keys'
//    lanes;
//  * the two channel groups have units of their own, which the keys that every row of
//    the item sees set.  In a tile whose scales lie further apart than binary16 weights
//    hold, weights times scales go in as the sum of two bfloat16 numbers: 16 bits, and
//    binary32's range (twice the products of V);
//  * a lane converts the scales of two keys and passes them on through shared memory,
//    each twice, as operands of the paired binary32 instructions.
// Tiles of 64 keys go round four consumer warps a block, each with a ring of three (with
// two column tiles four); the producer hands out four at a time, eight lanes each.
// Items, places and the joining of parts are those of the 16-bit kernel
// (serve_decode.cuh, serve_parts.cuh).
//
// Measured (GB300, join included): 256 requests over 1024..16384 keys, 32 / 4 heads,
// 132 us = 4.7 TB/s, 69% of the measured copy rate; 2 over 50000..65536, 16 / 16 heads,
// 38 us = 3.75 TB/s; one over 777 keys 8.7 us.  (The ranges of V and q cost 1 to 2% of
// that, or nothing, from one arrangement of the same instructions to the next; edge tiles
// always with two terms of weights 141, zeros told apart in the full walk 132 to 141.)
// Before them the copies alone took 105 us of 130
// with two blocks a SM and rings of five (copies of 2304 bytes, 26 clocks each beside
// their bytes: pages of 16 rows 1.3 times the time of pages of 64), the arithmetic alone
// about 100: neither hides all of the other.  What was slower: 8 warps of 32 keys in
// step 163 us; seven warps a block, two blocks, 151; four, two blocks, rings of five 140;
// a product of its own for the offset of 8 147; the scores of one tile beside the
// product of the one before 144; both operands as code * scale, exact, 201.
#include <math.h>

#include <type_traits>

#include "pool4.cuh"
#include "serve_decode.cuh"
#include "serve_index.h"
#include "serve_internal.h"
#include "serve_parts.cuh"
#include "sm103.cuh"
#include "warp_mma.cuh"

namespace css {
namespace {

// A weight counts 2^kBias where the score is m, so that binary16 holds small ones
// too.  What a lane's weights of a row in a step may add up to, and what a scale of V
// may reach in its unit, before m and the unit are followed: a weight times a scale
// stays at or below 2^15.  A scale of kVLeast units is the least for the binary16
// product: there a weight of 1 counts 1, so that what binary16 leaves out of a weight
// times a scale is at most 2^-25 of the key's value, as where weights alone are held in it.
constexpr float kBias = 10.f, kMost = 0x1p13f, kVMost = 4.f, kVLeast = 0x1p-10f;
// The bfloat16 product: what a scale may reach in its unit, so that sums stay inside
// binary32.  A tile for it sets a unit at its least scale, or kVFar of its largest: units
// only go up, as sums that are carried to a higher one shrink and cannot overflow.
constexpr float kVTop = 0x1p60f, kVFar = 0x1p-40f;
constexpr float kVNone = 0x1p126f;  // the inverse before a group has a scale above zero
// Scores: q goes in with one power of two for a row, which does not serve where a
// channel group lies kQApart below the other, or where the row's largest element, or c
// times it, is beyond kFar or its inverse.  Such items go through the edge's walk with a
// power of two for each group; that scales the groups' products one by one, to scores
// times 2^-kDrop, and takes c 2^kDrop from there, so that a score stays inside binary32
// where sum q k does, whatever q, K and c are by themselves.
constexpr float kQApart = 0x1p-12f, kFar = 0x1p100f;
constexpr int kDrop = 12;
constexpr int kTileKeys = 64;
constexpr int kGroup = 4;  // tiles that the producer hands out at a time, eight lanes each
// Pages of so many rows (their logarithm) are copied by tensor maps, whose boxes have
// to start on 128 bytes of shared memory: four units.  Smaller ones are plain copies.
constexpr int kTiledShift = 5;
static_assert(kTiledShift >= 5 && (32 / 8 * kUnitBytes) % 128 == 0, "a box of 32 rows");
constexpr int kLd = 68;  // floats a row of the joining buffer (bank spread)

// A block's shape.  COLS: column tiles of eight query rows.  WHOLE: a block takes
// whole items, so that nothing is joined.  SPLIT: a request may be several items.
template <int COLS, bool WHOLE, bool SPLIT = false>
struct Config {
  static constexpr bool kWhole = WHOLE, kSplit = SPLIT;
  static_assert(!(WHOLE && SPLIT), "a block for each item of a batch");
  static constexpr int kTileKeys = css::kTileKeys;
  static constexpr int kCols = COLS, kRows = 8 * COLS;
  static constexpr int kBlocks = COLS == 1 ? 3 : 2;  // a SM
  // The tiles go round the consumer warps, each with a ring of its own: the phases of
  // a stage's barriers are told apart by their parity, so a warp may look at a stage
  // only in the order in which it is used.
  static constexpr int kConsumers = 4, kRing = COLS == 1 ? 3 : 4;
  static constexpr int kStages = kConsumers * kRing;
  static constexpr int kThreads = 32 * (kConsumers + 1);
  static constexpr uint32_t kHalf = kTileKeys / 8 * kUnitBytes;  // K (or V) of a stage
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr uint32_t kQ = kDecodeRows * 128;
  static constexpr uint32_t kSmemStage = 2 * kQ;  // behind two Q buffers
  static constexpr uint32_t kSmemJoin = kSmemStage + kStages * kStage;
  // a warp's place in the joining buffer holds its scales before
  static constexpr uint32_t kScales = kTileKeys * 32;
  static constexpr uint32_t kJoin = kRows * kLd * 4 > kScales ? kRows * kLd * 4 : kScales;
  static constexpr uint32_t kSmemMl = kSmemJoin + kConsumers * kJoin;
  static constexpr uint32_t kSmemBar = kSmemMl + kConsumers * kRows * 8;
  // barriers
  static constexpr int kFull = 0, kEmpty = kStages, kQFull = 2 * kStages, kQFree = kQFull + 2;
  static constexpr uint32_t kSmemPre = kSmemBar + 8 * (kQFree + 2);  // + 8 (batch + 1), + slack
  static_assert(kConsumers >= kGroup, "a group goes round the warps once at most");
  static_assert(kSmemStage % 128 == 0 && kHalf % 128 == 0, "boxes start on 128 bytes");
  static_assert(kSmemMl % 16 == 0 && kSmemBar % 16 == 0, "layout");
  static_assert(kSmemPre + 8 * (kMaxPagedBatch + 1) + 1024 <= 227 * 1024 - 2048,
                "shared memory of a block");
};

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(at) : "memory");
  return r;
}

// Transposes an 8x8 matrix of 16-bit values held two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// d = a b + c on the tensor cores, binary16 in, binary32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4],
                                        const uint32_t (&b)[2], const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(c[0]), "f"(c[1]),
        "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t add_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A word of codes as pairs of binary16 operands: the low and high halves of bytes 0
// and 2, then of bytes 1 and 3, as the subnormal numbers (code + 8) 2^-24 and
// (code + 8) 2^-20.
__device__ __forceinline__ void raw_codes(uint32_t w, uint32_t& lo0, uint32_t& hi0, uint32_t& lo1,
                                          uint32_t& hi1) {
  const uint32_t v = w >> 8;
  lo0 = w & 0x000f000fu;
  hi0 = w & 0x00f000f0u;
  lo1 = v & 0x000f000fu;
  hi1 = v & 0x00f000f0u;
}
constexpr float kLoZero = 0x1p-21f, kHiZero = 0x1p-17f;  // what stands for code 0
constexpr uint32_t kLoUnit = 0x33803380u, kHiUnit = 0x35803580u;  // pairs of bfloat16 2^-24, 2^-20

// The same as code 2^-24 and code 2^-20.
__device__ __forceinline__ void signed_codes(uint32_t w, uint32_t& lo0, uint32_t& hi0,
                                             uint32_t& lo1, uint32_t& hi1) {
  raw_codes(w, lo0, hi0, lo1, hi1);
  lo0 = add_f16(lo0, 0x80088008u);
  hi0 = add_f16(hi0, 0x80808080u);
  lo1 = add_f16(lo1, 0x80088008u);
  hi1 = add_f16(hi1, 0x80808080u);
}

// A row's m follows its largest score x (in units of `unit`) where that is higher;
// f: what its sums are multiplied by.
__device__ __forceinline__ void follow(float x, float unit, float* neg_m, float* most, float* l,
                                       float* f) {
  const float to = kBias - x * unit;
  if (x > -INFINITY && (*most < 0.f || to < *neg_m)) {
    *f = *most < 0.f ? 0.f : ex2_approx(to - *neg_m);
    *neg_m = to;
    *most = kMost;
    *l *= *f;
  }
}

// Whether one of the two scales of a row is an infinity or NaN.
template <bool BF16>
__device__ __forceinline__ bool odd_scale(uint32_t s) {
  constexpr uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
  return (s & e) == e || (s & (e << 16)) == (e << 16);
}

// The magnitudes of a row's two scales.
template <bool BF16>
__device__ __forceinline__ float2 magnitudes(uint32_t s) {
  return make_float2(half_to_f32<BF16>((uint16_t)(s & 0x7fffu)),
                     half_to_f32<BF16>((uint16_t)(s >> 16 & 0x7fffu)));
}

// 2^e, -126 <= e <= 127; the binary order of x >= 0 (-127 below 2^-126).
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ int order(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }
// The inverse of a power of two between 2^-126 and 2^126.
__device__ __forceinline__ float inverse2(float x) {
  return __uint_as_float((254u << 23) - __float_as_uint(x));
}
// That of the power of two at x, or the next below it (from 2^-125 on).
__device__ __forceinline__ float inverse_unit(float x) {
  return inverse2(fmaxf(__uint_as_float(__float_as_uint(x) & 0x7f800000u), 0x1p-125f));
}

template <bool BF16, class C>
__global__ void __launch_bounds__(C::kThreads, C::kBlocks)
    paged_decode4_kernel(const __grid_constant__ CUtensorMap tm_q,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const DecodeArgs a,
                         const PoolArg kc, const PoolArg vc) {
  constexpr int kConsumers = C::kConsumers, kStages = C::kStages, kThreads = C::kThreads,
                kCols = C::kCols, kRows = C::kRows, kRing = C::kRing,
                kSteps = kTileKeys / 16;
  constexpr uint32_t kHalf = C::kHalf, kStage = C::kStage, kQ = C::kQ;
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
  // [warp][row] an item's m and l; while its tiles are walked, what products of q's low
  // and high channels count
  float2* const s_ml = reinterpret_cast<float2*>(smem + C::kSmemMl);
  long long* const s_pre = reinterpret_cast<long long*>(smem + C::kSmemPre);
  const uint32_t bar0 = sbase + C::kSmemBar;
#define BAR(i) (bar0 + 8u * (uint32_t)(i))
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = (tid >> 5) - 1;  // of the consumers; the producer comes first
  const WaitCtl wc{a.err, a.wait_ns, &s_abort};

  if (tid < kStages) {
    mbar_init(BAR(BAR_FULL + tid), 1);
    mbar_init(BAR(BAR_EMPTY + tid), 1);
    fence_mbarrier_init();
  } else if (tid < kStages + 2) {
    mbar_init(BAR(BAR_Q + tid - kStages), 1);
    mbar_init(BAR(BAR_Q_FREE + tid - kStages), kConsumers);
    fence_mbarrier_init();
  }
  if (tid == 0) s_abort = 0;
  // rows of the query tile that no copy fills read as zero
  for (int i = tid; i < (int)(2 * kQ / 16); i += kThreads)
    reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_shared();
  griddep_wait();

  tiles_before_each<C>(a, s_pre, s_scan);
  const Share share =
      share_of(s_pre[a.batch] * a.Hkv, C::kWhole ? 1 : a.part.min_tiles, gridDim.x, blockIdx.x);

  if (warp < 0) {
    // ---------------- producer ----------------
    const int box_shift = min(a.shift, 6), box = 1 << box_shift;  // rows a copy, at most
    const bool tiled = a.shift >= kTiledShift;
    // eight lanes look after a tile of a group, a box each; ring, slot and turn: the
    // next tile's warp, its place in the warp's ring, the parity of the phase before
    const int tile = lane >> 3, in_tile = (lane & 7) << box_shift;
    int ring = 0, slot = 0, turn = 1;
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
      ok = !(nq >= 2) || mbar_nap_warp(BAR(BAR_Q_FREE + qbuf), ((nq >> 1) - 1) & 1, wc);
      if (!ok) break;
      if (lane == 0) {
        s_item[qbuf] = Item{r, sg.kv, sg.t0, t1, C::kWhole || (sg.t0 == 0 && t1 == sg.nt)};
        mbar_arrive_expect_tx(BAR(BAR_Q + qbuf), a.split * a.G * 128);
        tma_load_4d(sbase + qbuf * kQ, &tm_q, BAR(BAR_Q + qbuf), 0, 0, sg.kv, r.q0);
      }
      ++nq;
      const uint8_t* const kp = static_cast<const uint8_t*>(kc.p) + sg.kv * kc.h;
      const uint8_t* const vp = static_cast<const uint8_t*>(vc.p) + sg.kv * vc.h;
      for (int t = sg.t0; t < t1; t += kGroup) {
        const int n = min(kGroup, t1 - t);
        const bool has = tile < n;
        int to_ring = ring + tile, to_slot = slot, to_turn = turn;
        if (to_ring >= kConsumers) {
          to_ring -= kConsumers;
          if (++to_slot == kRing) to_slot = 0, to_turn ^= 1;
        }
        const int s = to_ring * kRing + to_slot;
        ok = !has || mbar_try_wait(BAR(BAR_EMPTY + s), to_turn) ||
             mbar_nap(BAR(BAR_EMPTY + s), to_turn, wc);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if ((ring += n) >= kConsumers) {
          ring -= kConsumers;
          if (++slot == kRing) slot = 0, turn ^= 1;
        }
        it += n;
        const int k0 = (t + tile) * kTileKeys, at = k0 + in_tile;  // the lane's first key
        if (((t * kTileKeys) >> a.shift) - base >= 32) {
          base += 32;
          ids = next;
          next = base + 32 + lane < n_pages ? row[base + 32 + lane] : a.pages;
        }
        const int which = (at >> a.shift) - base;  // below 64 where there are keys
        const int id0 = __shfl_sync(0xffffffffu, ids, which & 31);
        const int id1 = __shfl_sync(0xffffffffu, next, which & 31);
        // boxes, and units of eight, that hold keys below n_keys; the rest of the
        // stage is masked
        const int keys = has ? min(max(r.n_keys - k0, 0), kTileKeys) : 0;
        const uint32_t full = BAR(BAR_FULL + s);
        if (has && (lane & 7) == 0)
          mbar_arrive_expect_tx(
              full, 2 * kUnitBytes *
                        (tiled ? ((keys + box - 1) & -box) / 8 : (keys + 7) / 8));
        __syncwarp();
        if (in_tile < keys) {
          int id = which < 32 ? id0 : id1;
          const bool fine = page_ok(id, a.pages);
          bad |= !fine;
          if (!fine) id = 0;  // the first page takes the place of one that does not exist
          const uint32_t to = sbase + C::kSmemStage + s * kStage + in_tile / 8 * kUnitBytes;
          const int unit = (at & ((1 << a.shift) - 1)) / 8;
          if (tiled) {
            tma_load_4d(to, &tm_k, full, 0, unit, sg.kv, id);
            tma_load_4d(to + kHalf, &tm_v, full, 0, unit, sg.kv, id);
          } else {
            const uint32_t bytes = (min(box, keys - in_tile) + 7) / 8 * kUnitBytes;
            bulk_load(to, kp + id * kc.pg + unit * kUnitBytes, bytes, full);
            bulk_load(to + kHalf, vp + id * vc.pg + unit * kUnitBytes, bytes, full);
          }
        }
      }
      if (!ok) break;
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
      for (int w = 0; w < kConsumers; ++w) {
        const int uses = (it + kConsumers - 1 - w) / kConsumers;  // tiles of warp w
        for (int k = max(uses - kRing, 0); k < uses; ++k)
          drain_wait(BAR(BAR_FULL + w * kRing + k % kRing), k / kRing & 1);
      }
    }
  } else {
    // ---------------- consumers ----------------
    const int g = lane >> 2, tq = lane & 3;
    const int mi = lane >> 3, mr = lane & 7;
    // the warp's scales of K, then of V, [key] {low, low, high, high}
    float4* const s_scale = reinterpret_cast<float4*>(smem + C::kSmemJoin + warp * C::kJoin);
    using AllCols = std::integral_constant<int, kCols>;
    using OneCol = std::integral_constant<int, 1>;
    int it = 0, nq = 0, slot = 0, turn = 0;
    for (long long pos = share.begin; pos < share.end;) {
      const int qbuf = nq & 1;
      // Q's fragments: products 0 and 1 take the low channels (words 0 and 1 of a
      // lane's codes), 2 and 3 the high ones
      uint32_t q[kCols][4][2];
      float z_lo[kCols][4], z_hi[kCols][4];  // where scores start
      float2 unit[kCols];                    // of the scores of rows 2 tq, 2 tq + 1
      bool far = false;                      // they have none: the edge's walk
      Item sg{};
      bool ok = mbar_wait_warp(BAR(BAR_Q + qbuf), (nq >> 1) & 1, wc);
      if (ok) {
        sg = s_item[qbuf];
        float x[kCols][2][8], top[kCols][2];  // a row's largest element of either group
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // channels 32 h + 8 tq .. + 7 of row 8 n + g
            const uint4 w = *reinterpret_cast<const uint4*>(
                smem + qbuf * kQ + sw128_offset(8 * n + g, 4 * h + tq));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[n][h][2 * i] = half_to_f32<BF16>((uint16_t)u[i]);
              x[n][h][2 * i + 1] = half_to_f32<BF16>((uint16_t)(u[i] >> 16));
              t = fmaxf(t, fmaxf(fabsf(x[n][h][2 * i]), fabsf(x[n][h][2 * i + 1])));
            }
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
            top[n][h] = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
          }
          // a row that counts, is finite and not zero
          const float most = fmaxf(top[n][0], top[n][1]), least = fminf(top[n][0], top[n][1]);
          if (8 * n + g < sg.r.n_new * a.G && most < INFINITY && most > 0.f) {
            const float at = a.c * fminf(most, kFar);
            far |= !(fmaxf(most, at) <= kFar && fminf(most, at) >= 1.f / kFar);
            far |= least > 0.f && least < most * kQApart;
          }
        }
        far = __any_sync(0xffffffffu, far);
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
          // q times 2^sh: the row's, or a group's, largest element counts 2^9 or 2^13
          const float both = fmaxf(top[n][0], top[n][1]);
          const int sh[2] = {
              min(max(13 - order(far ? top[n][0] : both), -103 - a.drop), 127),
              min(max(9 - order(far ? top[n][1] : both), -107 - a.drop), 123)};
          float sum[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float f = exp2i(sh[h]);
            sum[h] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t w = pack_f16x2(x[n][h][4 * i + j] * f, x[n][h][4 * i + j + 2] * f);
                q[n][2 * h + i][j] = w;
                sum[h] += f16_bits_to_f32((uint16_t)w) + f16_bits_to_f32((uint16_t)(w >> 16));
              }
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
          }
          // what a product counts: with c and for both groups together (far: not used),
          // and a group at a time, 2^drop too little
          const float back = a.c * exp2i(min(20 - sh[1], 127));
          if (tq == 0)
            s_ml[warp * kRows + 8 * n + g] =
                make_float2(exp2i(24 - a.drop - sh[0]), exp2i(20 - a.drop - sh[1]));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            z_lo[n][e] = z_lo[n][2 + e] =
                -kLoZero * __shfl_sync(0xffffffffu, sum[0], 8 * tq + 4 * e);
            z_hi[n][e] = z_hi[n][2 + e] =
                -kHiZero * __shfl_sync(0xffffffffu, sum[1], 8 * tq + 4 * e);
          }
          unit[n].x = __shfl_sync(0xffffffffu, back, 8 * tq);
          unit[n].y = __shfl_sync(0xffffffffu, back, 8 * tq + 4);
        }
        __syncwarp();
      }
      ++nq;
      const int t1 = sg.t1, n_keys = sg.r.n_keys;
      pos += C::kWhole ? 1 : t1 - sg.t0;
      const int first_lim = row_limit(n_keys, sg.r.n_new, 0);  // keys that every row sees
      // neg_m: kBias - m in base 2; most: what a lane's weights of a row in a step may
      // add up to.  V's scales count in units of their own, low and high channels, which
      // only rise; v_inv are their inverses
      float2 neg_m[kCols], most[kCols], l[kCols];
      float2 v_inv = make_float2(kVNone, kVNone);
      float o[kCols][4][4];
#pragma unroll
      for (int n = 0; n < kCols; ++n) {
        most[n] = make_float2(-1.f, -1.f);  // no m yet
        neg_m[n] = l[n] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
      }

      // The warp's keys of a tile for the first `cols` column tiles.  The answer is false
      // where a scale of V lies outside the units' range.  EDGE: whatever the keys are; else
      // every row sees all of them, and a tile that gives false has not been done.
      const auto walk = [&](auto edge_tag, auto cols_tag, uint32_t ks, int k0) -> bool {
        constexpr bool EDGE = decltype(edge_tag)::value;
        constexpr int cols = decltype(cols_tag)::value;
        const uint32_t vs = ks + kHalf;
        // scales, each twice, to where the lanes of a key find them: keys `lane` and 32 on
        const int in_unit = (lane >> 3) * kUnitBytes + kUnitScales + (lane & 7) * 4;
        uint32_t vw[2];  // V's: low and high channels
        float2 v[2];     // in their units
        const auto in_units = [&] {
#pragma unroll
          for (int x = 0; x < 2; ++x)
            v[x] = make_float2(half_to_f32<BF16>((uint16_t)vw[x]) * v_inv.x,
                               half_to_f32<BF16>((uint16_t)(vw[x] >> 16)) * v_inv.y);
        };
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          vw[x] = lds32(vs + in_unit + 4 * x * kUnitBytes);
          // keys that no row sees count as zero whatever stands there
          if (EDGE && k0 + lane + 32 * x >= n_keys) vw[x] = 0;
        }
        in_units();
        const bool first = !EDGE && v_inv.x == kVNone && v_inv.y == kVNone;
        if (first) {  // units at the tile's largest scales, if the others fit
          float t[2] = {0.f, 0.f};
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 m = magnitudes<BF16>(vw[x]);
            t[0] = fmaxf(t[0], m.x), t[1] = fmaxf(t[1], m.y);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)  // as bits, which rise with them
            t[h] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(t[h])));
          if (t[0] > 0.f && t[0] < INFINITY) v_inv.x = inverse_unit(t[0]);
          if (t[1] > 0.f && t[1] < INFINITY) v_inv.y = inverse_unit(t[1]);
          in_units();
        }
        // a scale that the units do not hold, a zero among them (a NaN may stay: it gives
        // NaN to the rows that see it, which in a full tile are all)
        float2 size[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          size[x] = make_float2(fabsf(v[x].x), fabsf(v[x].y));
          if (EDGE && k0 + lane + 32 * x >= n_keys) size[x] = make_float2(1.f, 1.f);
        }
        bool out =
            !(fmaxf(fmax3(size[0].x, size[0].y, size[1].x), size[1].y) <= kVMost &&
              fminf(fminf(size[0].x, size[0].y), fminf(size[1].x, size[1].y)) >= kVLeast);
        if (EDGE) out |= odd_scale<BF16>(vw[0]) || odd_scale<BF16>(vw[1]);
        bool odd = false;   // EDGE: a scale that some row must not meet
        bool wide = false;  // EDGE: weights as two bfloat16 numbers
        const bool even = !EDGE || !__any_sync(0xffffffffu, out);
        const auto apart = [&](uint32_t w) {  // of a key that some row misses: not a product
          const float2 m = magnitudes<BF16>(w);
          return odd_scale<BF16>(w) || m.x * v_inv.x > kVTop || m.y * v_inv.y > kVTop;
        };
        if (!even) {
          // the largest finite scale and the least above zero: of keys that every row
          // sees, and of all where there is neither such a scale nor a unit
          float t[2], u[2], inv[2] = {v_inv.x, v_inv.y};
#pragma unroll 1
          for (int lim = first_lim;; lim = n_keys) {
            t[0] = t[1] = 0.f, u[0] = u[1] = INFINITY;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float2 m = magnitudes<BF16>(vw[x]);
              const bool in = k0 + lane + 32 * x < lim;
              if (in && m.x < INFINITY && m.x > 0.f)
                t[0] = fmaxf(t[0], m.x), u[0] = fminf(u[0], m.x);
              if (in && m.y < INFINITY && m.y > 0.f)
                t[1] = fmaxf(t[1], m.y), u[1] = fminf(u[1], m.y);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // as bits, which rise with them
              t[h] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(t[h])));
              u[h] = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(u[h])));
              // up to the largest where binary16 holds the others beside it; else, where
              // it must be, low
              const bool none = inv[h] == kVNone;
              if (t[h] > 0.f && (none || (lim == first_lim && t[h] * inv[h] > kVMost))) {
                const float to = inverse_unit(t[h]);
                if (u[h] * to >= kVLeast)
                  inv[h] = to;
                else if (none || t[h] * inv[h] > kVTop)
                  inv[h] = inverse_unit(fmaxf(u[h], t[h] * kVFar));
              }
            }
            if (lim == n_keys || (inv[0] != kVNone && inv[1] != kVNone)) break;
          }
          const float2 f = make_float2(inv[0] * inverse2(v_inv.x), inv[1] * inverse2(v_inv.y));
#pragma unroll
          for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[n][j][e] *= (j & 1) ? f.y : f.x;
          v_inv = make_float2(inv[0], inv[1]);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (k0 + lane + 32 * x >= first_lim && apart(vw[x])) vw[x] = 0, odd = true;
          in_units();
          out = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float lo = fabsf(v[x].x), hi = fabsf(v[x].y);
            out |= lo > kVMost || (lo < kVLeast && lo > 0.f);
            out |= hi > kVMost || (hi < kVLeast && hi > 0.f);
          }
          wide = __any_sync(0xffffffffu, out);
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t kw = lds32(ks + in_unit + 4 * x * kUnitBytes);
          const float lo = half_to_f32<BF16>((uint16_t)kw),
                      hi = half_to_f32<BF16>((uint16_t)(kw >> 16));
          s_scale[lane + 32 * x] = make_float4(lo, lo, hi, hi);
          s_scale[kTileKeys + lane + 32 * x] = make_float4(v[x].x, v[x].x, v[x].y, v[x].y);
        }
        __syncwarp();
        // EDGE: what products of rows 2 tq and 2 tq + 1 count, low and high channels
        float2 r_lo[cols], r_hi[cols];
#pragma unroll
        for (int n = 0; EDGE && n < cols; ++n) {
          const float4 r = *reinterpret_cast<const float4*>(s_ml + warp * kRows + 8 * n + 2 * tq);
          r_lo[n] = make_float2(r.x, r.z), r_hi[n] = make_float2(r.y, r.w);
        }
        // scores: [.][step][key g, key g + 8 of the step], rows 2 tq and 2 tq + 1
        float2 sc[cols][kSteps][2];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          uint32_t x[4][4];  // product, fragment register
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint2 w = lds64(ks + (2 * i + u) * kUnitBytes + lane * 8);  // key g, g + 8
            raw_codes(w.x, x[0][u], x[2][u], x[0][2 + u], x[2][2 + u]);
            raw_codes(w.y, x[1][u], x[3][u], x[1][2 + u], x[3][2 + u]);
          }
          const float4 s4[2] = {s_scale[16 * i + g], s_scale[16 * i + 8 + g]};  // K's
#pragma unroll
          for (int n = 0; n < cols; ++n) {
            float lo[4], hi[4];
            mma_f16(lo, x[0], q[n][0], z_lo[n]);
            mma_f16(hi, x[2], q[n][2], z_hi[n]);
            mma_f16(lo, x[1], q[n][1], lo);
            mma_f16(hi, x[3], q[n][3], hi);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float2 a2 = make_float2(lo[2 * u], lo[2 * u + 1]),
                     b2 = make_float2(hi[2 * u], hi[2 * u + 1]);
              if (EDGE) a2 = __fmul2_rn(a2, r_lo[n]), b2 = __fmul2_rn(b2, r_hi[n]);
              sc[n][i][u] = __ffma2_rn(a2, make_float2(s4[u].x, s4[u].y),
                                       __fmul2_rn(b2, make_float2(s4[u].z, s4[u].w)));
            }
          }
        }
        if (EDGE) {
          const int n_new = s_item[qbuf].r.n_new;
#pragma unroll
          for (int n = 0; n < cols; ++n) {
            const int lim0 = row_limit(n_keys, n_new, (8 * n + 2 * tq) / a.G),
                      lim1 = row_limit(n_keys, n_new, (8 * n + 2 * tq + 1) / a.G);
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int key = k0 + 16 * i + 8 * u + g;
                if (key >= lim0) sc[n][i][u].x = -INFINITY;
                if (key >= lim1) sc[n][i][u].y = -INFINITY;
              }
          }
        }
        const auto unit_of = [&](int n) {
          return EDGE ? make_float2(a.c_drop, a.c_drop) : unit[n];
        };
        float2 p[cols][kSteps][2], sum[cols];
        const auto weigh = [&] {
          bool big = false;
#pragma unroll
          for (int n = 0; n < cols; ++n) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const float2 x = __ffma2_rn(sc[n][i][u], unit_of(n), neg_m[n]);
                p[n][i][u] = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                sum[n] = i + u ? __fadd2_rn(sum[n], p[n][i][u]) : p[n][i][u];
              }
            big |= sum[n].x > most[n].x || sum[n].y > most[n].y;
          }
          return big;
        };
        const bool big = weigh();
        if (__any_sync(0xffffffffu, big || (!EDGE && out))) {
          if (!EDGE && __any_sync(0xffffffffu, out)) {
            if (first) v_inv = make_float2(kVNone, kVNone);
            return false;
          }
#pragma unroll
          for (int n = 0; n < cols; ++n) {
            float2 x = make_float2(-INFINITY, -INFINITY), f = make_float2(1.f, 1.f);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
              x.x = fmax3(x.x, sc[n][i][0].x, sc[n][i][1].x);
              x.y = fmax3(x.y, sc[n][i][0].y, sc[n][i][1].y);
            }
#pragma unroll
            for (int by = 4; by < 32; by <<= 1) {
              x.x = fmaxf(x.x, __shfl_xor_sync(0xffffffffu, x.x, by));
              x.y = fmaxf(x.y, __shfl_xor_sync(0xffffffffu, x.y, by));
            }
            follow(x.x, unit_of(n).x, &neg_m[n].x, &most[n].x, &l[n].x, &f.x);
            follow(x.y, unit_of(n).y, &neg_m[n].y, &most[n].y, &l[n].y, &f.y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              o[n][j][0] *= f.x, o[n][j][2] *= f.x;
              o[n][j][1] *= f.y, o[n][j][3] *= f.y;
            }
          }
          __syncwarp();
          weigh();
        }
#pragma unroll
        for (int n = 0; n < cols; ++n) l[n] = __fadd2_rn(l[n], sum[n]);
        // O += V^T P^T.  WIDE: weights times scales in two terms
        const auto product = [&](auto wide_tag) {
          constexpr bool WIDE = decltype(wide_tag)::value;
          constexpr int kTerms = WIDE ? 2 : 1;
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            uint32_t pf[kTerms][cols][2][2];  // [.][.][low, high channels][keys]
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float4 s4 = s_scale[kTileKeys + 16 * i + 8 * u + g];
#pragma unroll
              for (int n = 0; n < cols; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float2 w = __fmul2_rn(p[n][i][u], h ? make_float2(s4.z, s4.w)
                                                            : make_float2(s4.x, s4.y));
                  const uint32_t term = pack2<WIDE>(w.x, w.y);
                  pf[0][n][h][u] = transpose8(term);
                  if (WIDE)
                    pf[kTerms - 1][n][h][u] = transpose8(
                        pack2<WIDE>(w.x - half_to_f32<WIDE>((uint16_t)term),
                                    w.y - half_to_f32<WIDE>((uint16_t)(term >> 16))));
                }
            }
            uint32_t w[4];
            ldmatrix_x4_trans(vs + (2 * i + (mi & 1)) * kUnitBytes + mr * 32 + (mi >> 1) * 16, w);
            // channel tiles 2 g, 32 + 2 g, 2 g + 1, 33 + 2 g (rows g; + 16 in rows g + 8)
            uint32_t x[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint32_t word = w[r == 1 ? 2 : (r == 2 ? 1 : r)];
              if (WIDE)
                scaled_codes<true>(word, kLoUnit, kHiUnit, x[0][r], x[1][r], x[2][r], x[3][r]);
              else
                signed_codes(word, x[0][r], x[1][r], x[2][r], x[3][r]);
            }
#pragma unroll
            for (int n = 0; n < cols; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < kTerms; ++k)
                  mma_16816<WIDE>(o[n][j], x[j], pf[k][n][j & 1][0], pf[k][n][j & 1][1]);
          }
        };
        if (EDGE && wide)
          product(std::true_type{});
        else
          product(std::false_type{});
        if (EDGE && __any_sync(0xffffffffu, odd)) {
          // what those keys give the rows that see them, in binary32
          const int n_new = s_item[qbuf].r.n_new;
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll 1
              for (int k = 0; k < 8; ++k) {
                const int key = k0 + 16 * i + 8 * u + k;
                const uint32_t at = vs + (2 * i + u) * kUnitBytes;
                const uint32_t sw = lds32(at + kUnitScales + 4 * k);
                if (key < first_lim || key >= n_keys || !apart(sw)) continue;
#pragma unroll
                for (int n = 0; n < cols; ++n)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const float wt = __shfl_sync(0xffffffffu, e ? p[n][i][u].y : p[n][i][u].x,
                                                 4 * k + tq);
                    const int lim = row_limit(n_keys, n_new, (8 * n + 2 * tq + e) / a.G);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                      for (int h = 0; h < 2; ++h) {  // row g + 8 h of channel tile j
                        const int byte = 16 * h + 2 * g + (j >> 1);
                        const uint32_t b = smem[at - sbase + k * 32 + byte] >> (4 * (j & 1));
                        const float v = (float)((int)(b & 15) - 8) *
                                        half_to_f32<BF16>((uint16_t)(sw >> (16 * (j & 1))));
                        // both of the key's groups were dropped
                        const float f =
                            (j & 1) ? v * v_inv.y * 0x1p-20f : v * v_inv.x * 0x1p-24f;
                        if (key < lim) o[n][j][2 * h + e] = fmaf(wt, f, o[n][j][2 * h + e]);
                      }
                  }
              }
        }
        return even;
      };
      // A tile behind one with scales out of range goes to the edge's walk at once: 64
      // requests of 2048..8192 keys, 32 / 8 heads, 48 us, with V times 2^0..2^20 by key 83
      // (93 where each tile tries the other walk first), with an eighth of V zero 64 (75).
      bool uneven = far;
      for (int t = sg.t0 + (warp + kConsumers - it % kConsumers) % kConsumers; t < t1;
           t += kConsumers) {
        const int s = warp * kRing + slot;
        ok = mbar_nap_warp(BAR(BAR_FULL + s), turn, wc);
        if (!ok) break;
        if (++slot == kRing) slot = 0, turn ^= 1;
        const uint32_t ks = sbase + C::kSmemStage + s * kStage;
        // One column tile where the item fills no more: 64 one-token requests of a call that
        // may have four tokens each take 60 us so, 70 with both.
        bool edge = uneven || past_limit(t * kTileKeys, kTileKeys, first_lim);
        if (!edge) {
          if (kCols > 1 && sg.r.n_new * a.G <= 8)
            edge = !walk(std::false_type{}, OneCol{}, ks, t * kTileKeys);
          else
            edge = !walk(std::false_type{}, AllCols{}, ks, t * kTileKeys);
        }
        if (__builtin_expect(edge, 0))
          uneven = !walk(std::true_type{}, AllCols{}, ks, t * kTileKeys) || far;
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(BAR_EMPTY + s));
      }
      it += t1 - sg.t0;
      const Request r = sg.r;
      const int rows = r.n_new * a.G;

      // ---------------- the consumer warps meet ----------------
      constexpr int kWarpLd = C::kJoin / 4;
      __syncwarp();  // the scales have been read
#pragma unroll
      for (int n = 0; n < kCols; ++n) {
#pragma unroll
        for (int by = 4; by < 32; by <<= 1) {
          l[n].x += __shfl_xor_sync(0xffffffffu, l[n].x, by);
          l[n].y += __shfl_xor_sync(0xffffffffu, l[n].y, by);
        }
        const int row = 8 * n + 2 * tq;
        constexpr float kOne = 0x1p-10f;  // of a weight that counts 2^kBias
        static_assert(kBias == 10.f, "kOne");
        if (g == 0) {
          s_ml[warp * kRows + row] = make_float2(
              most[n].x < 0.f ? -INFINITY : kBias - neg_m[n].x, l[n].x * kOne);
          s_ml[warp * kRows + row + 1] = make_float2(
              most[n].y < 0.f ? -INFINITY : kBias - neg_m[n].y, l[n].y * kOne);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // low and high channels, back to units of one
          const float raw = (x ? 0x1p20f : 0x1p24f) * kOne,
                      v_unit = inverse2(x ? v_inv.y : v_inv.x);
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<float2*>(s_join + warp * kWarpLd + (row + e) * kLd + 32 * x +
                                         16 * h + 2 * g) =
                  make_float2(o[n][x][2 * h + e] * raw * v_unit,
                              o[n][2 + x][2 * h + e] * raw * v_unit);
        }
      }
      // where a wait gave up, all leave together
      if (named_barrier_any(1, kConsumers * 32, !ok)) break;
      const int c0 = (tid & 7) * 8;
      for (int row = (tid - 32) >> 3; row < min(rows, kRows); row += kConsumers * 4) {
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) mm = fmaxf(mm, s_ml[w * kRows + row].x);
        // a NaN anywhere in the row's scores stays one
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, ll = 0.f;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) {
          const float2 ml = s_ml[w * kRows + row];
          if (ml.x == -INFINITY && ml.y == 0.f) continue;
          const float f = ex2_approx(ml.x - mm);
          ll = fmaf(ml.y, f, ll);
          const float* const d = s_join + w * kWarpLd + row * kLd + c0;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = fmaf(d[e], f, acc[e]);
        }
        const int tok = r.q0 + row / a.G, h = sg.kv * a.G + row % a.G;
        if (sg.whole)
          write_row<BF16>(a.o, a.lse, a.tokens, tok, h, c0, acc, mm, ll);
        else
          store_part(a.part, blockIdx.x, sg.t0 == 0, row, c0, acc, mm, ll);
      }
      named_barrier_sync(1, kConsumers * 32);
      if (lane == 0) mbar_arrive(BAR(BAR_Q_FREE + qbuf));
    }
  }
#undef BAR
}

template <class C>
int launch(const PagedDims& d, const DevCtx& ctx, const RowsArg& q, const PoolArg& kc,
           const PoolArg& vc, const DecodeArgs& args, int blocks, int which, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  const uint32_t units = (1u << d.shift) / 8;
  const uint32_t box = units < kTileKeys / 8 ? units : kTileKeys / 8;
  if (!encode_tmap_4d(&tq, d.bf16, q.p, d.G, d.Hkv, d.tokens, q.h, q.h * d.G, q.t, d.G, 1,
                      args.split))
    return ATTN_ERR_CUDA;
  tk = tv = tq;  // small pages: not used
  if (d.shift >= kTiledShift &&
      (!encode_tmap_units(&tk, kc.p, units, d.Hkv, d.pages, kc.h, kc.pg, box) ||
       !encode_tmap_units(&tv, vc.p, units, d.Hkv, d.pages, vc.h, vc.pg, box)))
    return ATTN_ERR_CUDA;
  const size_t smem = C::kSmemPre + 8 * (size_t)(d.batch + 1) + 1024;
  auto* kernel = d.bf16 ? paged_decode4_kernel<true, C> : paged_decode4_kernel<false, C>;
  const int rc = allow_smem(which + d.bf16, reinterpret_cast<const void*>(kernel),
                            C::kSmemPre + 8 * (kMaxPagedBatch + 1) + 1024);
  if (rc != ATTN_OK) return rc;
  return cuda_status(launch_dependent(kernel, dim3(blocks), dim3(C::kThreads), smem, stream, tq,
                                      tk, tv, args, kc, vc));
}

}  // namespace

constexpr int kWholeKeys = 1024;

namespace {
// The most new tokens of a request that a call has for this kernel.
int tokens4(const PagedDims& d) {
  return d.max_new < decode_tokens(d.G) ? d.max_new : decode_tokens(d.G);
}

// Beside chunks, requests of nine to sixteen rows are rare and go as items of up to
// eight, which read K and V again (from L2 for the most part): 32 requests over
// 2048..8192 keys, 32 / 8 heads, and a chunk of 300 tokens, us with two column tiles for
// all / with items of eight: one token each 91 / 82, four 95 / 106.
bool splits(const PagedDims& d) { return d.G <= 8 && d.max_new > decode_tokens(d.G); }

template <int COLS>
int launch_cols(const PagedDims& d, const DevCtx& ctx, const RowsArg& q, const PoolArg& kc,
                const PoolArg& vc, const DecodeArgs& args, int blocks, int which,
                cudaStream_t stream) {
  if (decode4_whole(d, ctx.sm_count))
    return launch<Config<COLS, true>>(d, ctx, q, kc, vc, args, d.batch * d.Hkv, which + 2, stream);
  return launch<Config<COLS, false>>(d, ctx, q, kc, vc, args, blocks, which, stream);
}
}  // namespace

// Whole items where each finds a block at once and the table leaves room for no more
// than kWholeKeys keys a request: the parts and the second launch fall away.  Split /
// whole, us (8 K/V heads): one request of 100 keys 7.3 / 5.9, of 777 10.8 / 9.2, of 1500
// 10.2 / 13.0; eight of 250 10.4 / 6.9, of 777 12.2 / 9.8, of 1500 11.0 / 13.7; fifty of
// 500 17.9 / 9.6.  The width stands for the lengths, which the host does not see: a wide
// table over short caches (the default of a server's is every page) takes the split form.
bool decode4_whole(const PagedDims& d, int sm_count) {
  return !splits(d) && (long long)d.batch * d.Hkv <= decode4_blocks(d) * sm_count &&
         ((long long)d.width << d.shift) <= kWholeKeys;
}

// One column tile serves a token step of up to eight heads a group.
int decode4_rows(const PagedDims& d) {
  return splits(d) || tokens4(d) * d.G <= 8 ? Config<1, false>::kRows : Config<2, false>::kRows;
}
int decode4_blocks(const PagedDims& d) {
  return decode4_rows(d) <= 8 ? Config<1, false>::kBlocks : Config<2, false>::kBlocks;
}
static_assert(Config<1, false>::kBlocks == 3 && Config<1, false>::kRows == 8 &&
                  Config<2, false>::kBlocks == 2 && Config<2, false>::kRows == kDecodeRows,
              "the workspace holds their parts");

int launch_paged_decode4(const PagedDims& d, const DevCtx& ctx, const RowsArg& q,
                         const PoolArg& kc, const PoolArg& vc, const int32_t* table,
                         const int32_t* cu, const int32_t* lens, const PartArgs& part, int blocks,
                         const RowsArg& o, float* lse, cudaStream_t stream) {
  const int ntok = tokens4(d);
  const DecodeArgs args{d.batch, d.tokens, d.H, d.Hkv, d.G, ntok, d.max_new, d.pages, d.width,
                        d.shift, d.c, cu, lens, table, o, lse, part, ctx.err, ctx.wait_ns,
                        splits(d) ? 8 / d.G : ntok, d.c < kFar ? kDrop : 0,
                        d.c < kFar ? ldexpf(d.c, kDrop) : d.c};
  if (splits(d))
    return launch<Config<1, false, true>>(d, ctx, q, kc, vc, args, blocks, kSmemDecode4SplitF16,
                                          stream);
  if (ntok * d.G <= 8)
    return launch_cols<1>(d, ctx, q, kc, vc, args, blocks, kSmemDecode4F16, stream);
  return launch_cols<2>(d, ctx, q, kc, vc, args, blocks, kSmemDecode4WideF16, stream);
}

}  // namespace css
