// serve_tiles.cu - attention of many rows on the tensor cores: whole packed
// prompts, and chunks of new tokens over a paged cache.
//
// Method: for every key tile that a row tile sees, S = Q K^T; t = S c in base
// 2; P = 2^(t - m); l += sum P (binary32, P unrounded); O += P V with P
// rounded to the operands' type, which the matrix product takes (error against
// 64 bits 2.2e-4 to 2.9e-4 in binary16 and 2.1e-3 to 2.3e-3 in bfloat16, where
// rounding O alone gives 2.0e-4 and 1.7e-3); O / l and L = m + log2 l.  m follows the
// running maximum only when that has grown by more than kSlack: P may then
// reach 2^kSlack, which changes no relative rounding (binary16 holds it, sums
// are binary32), and O is rescaled a few times a row instead of at nearly
// every tile.
//
// Rows: a row tile of 128 holds tpt = 128 / G tokens times the G query heads
// of one K/V head (row = token * G + head), so that a group's heads share
// every K and V tile and a short chunk still fills the rows.  A work item is
// three such tiles, one behind the other, that share K/V tiles of 64 keys.
// Packed prompts cut the token axis into windows of 3 tpt tokens whatever
// sequences lie in them, each row with its own interval of keys [lo, hi): many
// short sequences share a tile, and no table of blocks is needed.  Paged
// chunks cut each request's new tokens, and the list of their key tiles is
// shared out over the blocks in equal runs (serve_parts.cuh).
//
// Warps (16, 128 registers a thread):
//   0-3, 4-7, 8-11  softmax of row tile 0, 1, 2: one thread per row (= tensor-
//       memory lane)
//   12-14  products of a row tile each: S of the next key tile as soon as the
//       softmax has read this one's, then O += P V
//   15  allocates, finds the work items and issues the TMA loads (Q, K, V
//       rows; a copy per page, lanes in parallel).  Packed: a block takes over
//       the next window that no block has started (cluster launch control),
//       whose description and first loads then overlap the window before
// Tensor memory (480 of 512 columns): S 64 columns a row tile, P 32, O 64.
// A row's thread holds a tile's whole S (64 values) in registers, so S is free
// for the next product at once; P waits in registers for the product before.
//
// Why three tiles of 64 keys: one tile step of a softmax warp is a chain of
// waits and tensor-memory round trips that its arithmetic does not fill, so
// the work in flight sets the rate.  With two row tiles of 128 keys (two
// softmax warps a scheduler) a pair of steps took 2650 clocks where the
// exponential, conversion and add pipes need 1311, however the two were
// phased and however many warps issued the products (1.25 ms for a prompt of
// 16384 tokens, 32 / 4 heads); three tiles of 64 keys take 0.95 ms.
//
// Measured (GB300): that prompt 951 to 959 us in a captured graph and 977 to 992
// call by call = 1108 to 1156 TFLOP/s, 59 to 62% of the measured dense rate; 16
// prompts of 256..4096 tokens, 32 / 8 heads, 508 us = 854 TFLOP/s, of which five
// to six tile steps a window are its border: the last products, the epilogue and
// the next window's first steps, one behind the other.
// The matrix pipe is busy 46% of the time and the issue slots 59%:
// what bounds is the latency of a tile step (wait for S, load, maximum,
// exponentials, store of P, wait of the products) times the three in flight.
// Slower were: a warp for S and one for O += P V (1.38 ms, the second's own
// latency), six issuing warps of 20 with registers moved between the warps
// (1.13 ms, the waiting warps' polls), P tested against the last maximum
// first and the maximum taken only where it grew (1.06 ms).
//
// A 4-bit cache (pool4.cuh): packed rows land in raw stages, and the softmax of row
// tile n mod 3 turns those of key tile n into the 16-bit rows of a K/V stage, exactly,
// two steps before their use.  Four chunks of 301..1024 tokens over 2048..8192 keys, 32 / 8
// heads, take 128 us where the 16-bit cache takes 108, a prompt of 16384 tokens 1.40 ms
// against 1.07: the counters have 300 instructions more a thread and key tile, waits
// included, on the chain of every third step (82 million for the 16 bits, 108 for the 4).
// Slower were: two row tiles and four warps that unpack beside them (134 us, 1.56 ms),
// warp 15 for all tiles (163, 1.98) or every fourth (154, 1.69), warps 12 to 15 for a
// quarter of each (159, 1.73: products come late).  Four warps more beside three row
// tiles leave 96 registers a thread, too few for the softmax also where registers are
// moved to it.
//
// What a mask excludes cannot reach a row, infinities and NaN included: S is
// replaced by -inf, and on tiles where some row misses a key the rows of V
// are looked at.  Rows of V past the last key of the item are set to zero;
// where another row of V holds a value that is not finite, the tile's product
// is formed by the row's own thread over the keys that it sees.
#include <math.h>

#include "pool4.cuh"
#include "serve_index.h"
#include "serve_internal.h"
#include "serve_parts.cuh"
#include "sm103.cuh"
#include "warp_mma.cuh"

namespace css {
namespace {

// What a kernel reads: packed prompts, a paged cache, a paged cache of 4 bits.
enum Mode { kPacked, kPaged, kPaged4 };
constexpr int kNT = 3;   // row tiles of a work item
constexpr int kBN = 64;  // keys a tile
constexpr int kMaxStages = 6;
constexpr int kThreads = 512;
constexpr float kSlack = 8.f;
constexpr uint32_t kTileBytes = 128 * 128;
constexpr uint32_t kHalfBytes = kBN * 128;         // K (or V) of a stage
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr uint32_t kSmemStage0 = 2 * kNT * kTileBytes;  // behind two Q buffers
// 4 bits: one stage less, packed rows in its place
constexpr int kStages4 = kMaxStages - 1, kRaw = kNT;
constexpr int kAhead = 2;  // steps between unpacking a tile and its use
constexpr uint32_t kRawHalf = kBN / 8 * kUnitBytes;  // K (or V) of a raw stage
constexpr uint32_t kSmemRaw = kSmemStage0 + kStages4 * kStageBytes;
static_assert(kRaw * 2 * kRawHalf <= kStageBytes, "raw stages");
constexpr uint32_t kSmemBar = kSmemStage0 + kMaxStages * kStageBytes;
constexpr uint32_t kSmemPre = kSmemBar + 512;  // paged: prefix of tiles

constexpr uint32_t kColS = 0;                // + 64 t
constexpr uint32_t kColP = kColS + 64 * kNT;  // + 32 t
constexpr uint32_t kColO = kColP + 32 * kNT;  // + 64 t
constexpr uint32_t kTmemCols = 512;
static_assert(kColO + 64 * kNT <= kTmemCols, "tensor memory");

enum {
  BAR_Q = 0,                             // [Q buffer] the item's Q tiles landed
  BAR_Q_FREE = BAR_Q + 2,                // [Q buffer] every row tile's products done
  BAR_KV_FULL = BAR_Q_FREE + 2,          // [stage] (4 bits: unpacked by four warps)
  BAR_KV_EMPTY = BAR_KV_FULL + kMaxStages,  // [stage] every row tile's products done
  BAR_S_FULL = BAR_KV_EMPTY + kMaxStages,   // [t]
  BAR_S_FREE = BAR_S_FULL + kNT,         // [t] read by the softmax (128 threads)
  BAR_P_FULL = BAR_S_FREE + kNT,         // [t] P stored, O rescaled (128 threads)
  BAR_P_FREE = BAR_P_FULL + kNT,         // [t] O += P V done
  BAR_O_FREE = BAR_P_FREE + kNT,         // [t] the epilogue has read O (128 threads)
  BAR_V_OK = BAR_O_FREE + kNT,           // [t] rows of V looked at (128 threads)
  BAR_UNIT = BAR_V_OK + kNT,             // [item buffer] description written
  BAR_UNIT_FREE = BAR_UNIT + 2,          // [item buffer] read by 5 kNT warps
  BAR_MMA_DONE = BAR_UNIT_FREE + 2,      // every product of the block done (kNT commits)
  BAR_TAKE = BAR_MMA_DONE + 1,           // an answer of take_block
  BAR_RAW_FULL = BAR_TAKE + 1,           // [raw stage] 4-bit rows landed
  BAR_RAW_EMPTY = BAR_RAW_FULL + kRaw,   // [raw stage] read (4 warps)
  BAR_COUNT = BAR_RAW_EMPTY + kRaw
};
static_assert(BAR_COUNT * 8 <= 512, "barrier area");

// A work item as warp 15 describes it.  Keys count from the item's first key.
struct Unit {
  int more;      // 0: no further item
  int q0;        // token row of the first row tile's first row
  int q_end;     // token rows from here on are not the item's
  int kv;
  int kbeg;      // packed: row of key 0
  int j0, nj;    // key tiles j0 .. j0 + nj - 1
  int t0[kNT], t1[kNT];          // those of row tile t: [t0, t1), counted from j0
  int lo_max[kNT], hi_min[kNT];  // keys that every row of tile t sees: [lo_max, hi_min)
  int kend;      // no row sees a key from here on
  int s0, s1;    // packed: first and last sequence in the window
  int lim;       // paged: keys that the first token of the item sees
  int whole;     // O is finished here; else a part
  int tail;      // the part starts the item
};

struct TileArgs {
  int tokens, batch, H, Hkv, G, tpt, causal, windows;
  float c;
  const int32_t *cu, *lens, *table;
  int pages, width, shift, skip, max_new;
  RowsArg o;
  float* lse;
  PartArgs part;
  uint32_t* err;
  uint64_t wait_ns;
  PoolArg kc, vc;  // 4 bits
};

__device__ __forceinline__ float as_f(uint32_t u) { return __uint_as_float(u); }

template <bool BF16>
constexpr uint32_t idesc(int N, int b_mn) {
  return idesc_f16_f32(128, N, 0, b_mn) | (BF16 ? (1u << 7) | (1u << 10) : 0u);
}

// ---------------------------------------------------------------- paged items
struct PagedReq {
  int q0, n_new, n_keys;  // n_new 0: not for this kernel
};

__device__ __forceinline__ PagedReq paged_req(const TileArgs& a, int i, bool* bad) {
  const RowRange r = row_range(a.cu[i], a.cu[i + 1], a.tokens);
  bool b;
  PagedReq q{r.begin, r.end - r.begin, key_count(a.lens[i], a.width, a.shift, &b)};
  *bad = r.bad || b || q.n_new > a.max_new;
  if (q.n_new <= a.skip || q.n_new > a.max_new) q.n_new = 0;
  return q;
}

// A place in the list of tiles: tile t0 of a row block of a request and head.
struct Place {
  PagedReq r;
  int req, kv, blk, t0;
};

// The place at position pos of the list; pre[i] counts the tiles of one head
// of the requests before i.  Called by a whole warp.
__device__ __forceinline__ Place place_at(const TileArgs& a, const long long* pre, long long pos) {
  int lo = 0, hi = a.batch;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] * a.Hkv <= pos)
      lo = mid + 1;
    else
      hi = mid;
  }
  Place p;
  p.req = lo - 1;
  bool b;
  p.r = paged_req(a, p.req, &b);
  const int w = kNT * a.tpt;
  const long long per = pre[lo] - pre[p.req], off = pos - pre[p.req] * a.Hkv;
  p.kv = (int)quot(off, per);
  const long long at = off - (long long)p.kv * per;
  // the last block with tiles_before <= at: the warp's lanes try 32 at a time
  const int lane = threadIdx.x & 31;
  int x = 0, n = (p.r.n_new + w - 1) / w;  // the block is in [x, x + n)
  long long before = 0;
  while (n > 1) {
    const int step = (n + 31) / 32, mine = x + min(lane * step, n - 1);
    const long long v = tiles_before(p.r.n_keys, p.r.n_new, w, kBN, mine);
    const int hit = __popc(__ballot_sync(0xffffffffu, lane * step < n && v <= at)) - 1;
    before = __shfl_sync(0xffffffffu, v, hit);
    x += hit * step;
    n = min(step, n - hit * step);
  }
  p.blk = x;
  p.t0 = (int)(at - before);
  return p;
}

// The place behind a block: the next block, head or request with rows.  Called
// only where the list goes on; never past the last request, also where lens
// changed meanwhile.
__device__ __forceinline__ void next_block(const TileArgs& a, Place* p) {
  p->t0 = 0;
  if (++p->blk * kNT * a.tpt < p->r.n_new) return;
  p->blk = 0;
  if (++p->kv < a.Hkv) return;
  p->kv = 0;
  do {
    bool b;
    p->req = min(p->req + 1, a.batch - 1);
    p->r = paged_req(a, p->req, &b);
  } while (p->r.n_new == 0 && p->req + 1 < a.batch);
}

// Describes the item at a place, tiles [t0, t1) of nt; lane t looks after row
// tile t.
__device__ __forceinline__ void paged_unit(const TileArgs& a, const Place& p, int t1, int nt,
                                           Unit* u) {
  const int w = kNT * a.tpt, lane = threadIdx.x & 31, t = lane;
  const int q0 = p.r.q0 + p.blk * w, q_end = min(p.r.q0 + p.r.n_new, q0 + w);
  const int lim = row_limit(p.r.n_keys, p.r.n_new, p.blk * w);
  const int first = q0 + t * a.tpt, past = min(q_end, first + a.tpt);
  const bool some = t < kNT && first < past;
  const int keys = some ? lim + (past - 1 - q0) : 0;  // the last row's
  const int n = keys <= 0 ? 0 : (keys - 1) / kBN + 1;
  const int mine = some ? max(0, min(n, t1) - p.t0) : 0;
  const int nj = __reduce_max_sync(0xffffffffu, mine);
  const int kend = __reduce_max_sync(0xffffffffu, max(keys, 0));
  if (t < kNT) {
    u->t0[t] = 0;
    u->t1[t] = mine;
    u->lo_max[t] = 0;
    u->hi_min[t] = some ? lim + (first - q0) : 0;
  }
  if (lane == 0) {
    u->more = 1;
    u->q0 = q0;
    u->q_end = q_end;
    u->kv = p.kv;
    u->kbeg = 0;
    u->j0 = p.t0;
    u->nj = nj;
    u->kend = kend;
    u->s0 = u->s1 = 0;
    u->lim = lim;
    u->whole = p.t0 == 0 && t1 == nt;
    u->tail = p.t0 == 0;
  }
}

// --------------------------------------------------------------- packed items
// Lanes 2 t and 2 t + 1 look after the first and the last row of row tile t.
// Kept short: a block runs it once or a few times, and code that has to be
// fetched first takes some ten clocks an instruction.
__device__ __forceinline__ void packed_unit(const TileArgs& a, int block, Unit* u) {
  const int w = kNT * a.tpt, win_rev = block / a.Hkv;
  const int lane = threadIdx.x & 31, t = lane >> 1;
  const int q0 = (a.windows - 1 - win_rev) * w, q_end = min(a.tokens, q0 + w);
  // the first and last row of the tile that lie in a sequence
  const int first = max(q0 + t * a.tpt, a.cu[0]);
  const int past = min(min(q_end, q0 + (t + 1) * a.tpt), a.cu[a.batch]);
  const bool some = t < kNT && first < past;
  // the last sequence that starts at or before this lane's row: the warp looks
  // at 32 offsets at once, the lane bisects what lies between two of them
  const int row = lane & 1 ? past - 1 : first;
  const int step = (a.batch + 31) / 32;
  const int v = a.cu[min(lane * step, a.batch - 1)];
  int lo = 0;
#pragma unroll 1
  for (int i = 0; i < 2 * kNT; ++i) {
    const int x = __shfl_sync(0xffffffffu, row, i);
    const int c = __popc(__ballot_sync(0xffffffffu, lane * step < a.batch && v <= x));
    if (lane == i) lo = max(c - 1, 0) * step;
  }
  int hi = min(lo + step, a.batch);
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= row)
      lo = mid;
    else
      hi = mid;
  }
  __syncwarp();
  const RowRange r = row_range(a.cu[lo], a.cu[lo + 1], a.tokens);
  // key 0 of the window is the first key of its first row
  const unsigned live = __ballot_sync(0xffffffffu, some);
  const int lead = live ? __ffs(live) - 1 : 0, tail = live ? 31 - __clz(live) : 0;
  const int kbeg = live ? __shfl_sync(0xffffffffu, r.begin, lead) : 0;
  const int s0 = __shfl_sync(0xffffffffu, lo, lead), s1 = __shfl_sync(0xffffffffu, lo, tail);
  const int begin = r.begin - kbeg, end = (a.causal ? row + 1 : r.end) - kbeg;
  // even lanes hold the first row's, odd lanes the last row's
  const int begin_last = __shfl_down_sync(0xffffffffu, begin, 1);
  const int end_last = __shfl_down_sync(0xffffffffu, end, 1);
  const int t0 = some ? max(begin, 0) / kBN : 0;
  const int t1 = some ? max(t0, (max(end_last, 0) + kBN - 1) / kBN) : 0;
  const bool mine = !(lane & 1) && t < kNT;
  const int nj = __reduce_max_sync(0xffffffffu, mine ? t1 : 0);
  const int kend = __reduce_max_sync(0xffffffffu, mine && some ? end_last : 0);
  if (mine) {
    u->t0[t] = t0;
    u->t1[t] = t1;
    u->lo_max[t] = some ? begin_last : 0;
    u->hi_min[t] = some ? end : 0;
  }
  if (lane == 0) {
    u->more = 1;
    u->q0 = q0;
    u->q_end = q_end;
    u->kv = block - win_rev * a.Hkv;
    u->kbeg = kbeg;
    u->j0 = 0;
    u->nj = nj;
    u->kend = kend;
    u->s0 = s0;
    u->s1 = live ? s1 : -1;
    u->lim = 0;
    u->whole = 1;
    u->tail = 0;
  }
}

// ------------------------------------------------------------------- softmax
// Sets the columns of a 32-column chunk outside [lo, hi) to -inf.
__device__ __forceinline__ void mask32(uint32_t (&v)[32], int lo, int hi) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (e < lo || e >= hi) v[e] = 0xff800000u;
}

__device__ __forceinline__ float max64(const uint32_t (&v)[32], const uint32_t (&w)[32]) {
  float a = -INFINITY, b = a, c = a, d = a;
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    a = fmax3(a, as_f(v[e]), as_f(v[e + 1]));
    b = fmax3(b, as_f(v[e + 2]), as_f(v[e + 3]));
    c = fmax3(c, as_f(w[e]), as_f(w[e + 1]));
    d = fmax3(d, as_f(w[e + 2]), as_f(w[e + 3]));
  }
  return fmaxf(fmax3(a, b, c), d);
}

// P = 2^(S c - m) of 32 columns as 16 packed words, and the sum of the
// unrounded values.
template <bool BF16>
__device__ __forceinline__ void exp32(const uint32_t (&v)[32], float c, float neg_m, uint32_t* pk,
                                      float2& s0, float2& s1) {
  const float2 c2 = make_float2(c, c), nm2 = make_float2(neg_m, neg_m);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float2 t = __ffma2_rn(make_float2(as_f(v[e]), as_f(v[e + 1])), c2, nm2);
    const float2 x = make_float2(ex2_approx(t.x), ex2_approx(t.y));
    if (e & 2)
      s0 = __fadd2_rn(s0, x);
    else
      s1 = __fadd2_rn(s1, x);
    pk[e >> 1] = pack2<BF16>(x.x, x.y);
  }
}

// O *= alpha for the rows of a warp.
__device__ __noinline__ void rescale(uint32_t t_o, float alpha) {
  const float2 al = make_float2(alpha, alpha);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t o[32];
    tmem_ld32_wait(t_o + 32 * h, o);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float2 x = __fmul2_rn(make_float2(as_f(o[e]), as_f(o[e + 1])), al);
      o[e] = __float_as_uint(x.x), o[e + 1] = __float_as_uint(x.y);
    }
    tmem_st32(t_o + 32 * h, o);
  }
}

template <bool BF16>
__device__ __forceinline__ bool any_nonfinite(const uint4& w) {
  constexpr uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  bool r = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= (x[i] & e) == e || (x[i] & (e << 16)) == (e << 16);
  return r;
}

// O += P V of one row over the keys [lo, hi) of the tile, by the row's own
// thread: P from its tensor-memory columns, V from the stage.  Rare.
template <bool BF16>
__device__ __noinline__ void row_product(uint32_t t_p, uint32_t t_o, const uint8_t* v, int lo,
                                         int hi, bool first) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {  // 16 columns at a time
    uint32_t o[16];
    float acc[16];
    tmem_ld16_wait(t_o + 16 * c, o);
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = first ? 0.f : as_f(o[e]);
#pragma unroll 1
    for (int i = 0; i < kBN / 32; ++i) {  // 32 keys at a time
      uint32_t p[16];
      __syncwarp();
      tmem_ld16_wait(t_p + 16 * i, p);
#pragma unroll 2
      for (int k = 0; k < 32; ++k) {
        const int key = 32 * i + k;
        if (key >= lo && key < hi) {
          const float w = half_to_f32<BF16>((uint16_t)(p[k >> 1] >> (16 * (k & 1))));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 x =
                *reinterpret_cast<const uint4*>(v + key * 128 + (((2 * c + h) ^ (key & 7)) << 4));
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[8 * h + 2 * e] =
                  fmaf(w, half_to_f32<BF16>((uint16_t)y[e]), acc[8 * h + 2 * e]);
              acc[8 * h + 2 * e + 1] =
                  fmaf(w, half_to_f32<BF16>((uint16_t)(y[e] >> 16)), acc[8 * h + 2 * e + 1]);
            }
          }
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(acc[e]);
    tmem_st16(t_o + 16 * c, o);
  }
  tmem_st_wait();
}

// 4 bits: key tile n's packed rows to the 16-bit rows of its K/V stage, as TMA would
// have written them, by the 128 threads of a row tile's softmax: a row of K or of V a
// thread.  Parities tell two uses of a stage apart, not three: a raw stage always
// belongs to the same row tile, and who unpacks tile n has waited for the end of tile
// n - 3 - kStages4, stages coming free in order, also for a row tile that sees no key of
// them.
template <bool BF16>
__device__ __forceinline__ bool unpack_tile(uint8_t* smem, uint32_t bar0, int n,
                                            const WaitCtl& wc) {
  const int row = threadIdx.x & (kBN - 1), from = n % kRaw, s = n % kStages4;
  const bool is_v = (threadIdx.x & 127) >= kBN;
  if (!mbar_wait_inline(bar0 + 8u * (BAR_RAW_FULL + from), (n / kRaw) & 1, wc)) return false;
  const uint8_t* const unit = smem + kSmemRaw + from * 2 * kRawHalf + (is_v ? kRawHalf : 0) +
                              (row >> 3) * kUnitBytes;
  const uint4 c0 = *reinterpret_cast<const uint4*>(unit + (row & 7) * 32);
  const uint4 c1 = *reinterpret_cast<const uint4*>(unit + (row & 7) * 32 + 16);
  const uint32_t sw = *reinterpret_cast<const uint32_t*>(unit + kUnitScales + (row & 7) * 4);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar0 + 8u * (BAR_RAW_EMPTY + from));
  if (n >= kStages4 &&
      !mbar_wait_inline(bar0 + 8u * (BAR_KV_EMPTY + s), (n / kStages4 - 1) & 1, wc))
    return false;
  const uint32_t s_lo = __byte_perm(sw, sw, 0x1010), s_hi = __byte_perm(sw, sw, 0x3232);
  uint8_t* const to = smem + kSmemStage0 + s * kStageBytes + (is_v ? kHalfBytes : 0) + row * 128;
  const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
  for (int c = 0; c < 4; ++c) {  // channels 8 c .. and 32 + 8 c ..
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t l0, h0, l1, h1;
      scaled_codes<BF16>(w[2 * c + i], s_lo, s_hi, l0, h0, l1, h1);
      lo[2 * i] = __byte_perm(l0, l1, 0x5410);
      lo[2 * i + 1] = __byte_perm(l0, l1, 0x7632);
      hi[2 * i] = __byte_perm(h0, h1, 0x5410);
      hi[2 * i + 1] = __byte_perm(h0, h1, 0x7632);
    }
    *reinterpret_cast<uint4*>(to + ((c ^ (row & 7)) << 4)) =
        make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(to + (((c + 4) ^ (row & 7)) << 4)) =
        make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
  fence_proxy_async_shared();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar0 + 8u * (BAR_KV_FULL + s));
  return true;
}

template <int MODE, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const TileArgs a) {
  constexpr bool PAGED = MODE != kPacked, FOUR = MODE == kPaged4;
  constexpr int kStages = FOUR ? kStages4 : kMaxStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ Unit s_unit[2];
  __shared__ __align__(16) uint4 s_answer;
  __shared__ int s_odd[kNT][2];  // [t][use & 1]: number of the use whose V is not all finite
  __shared__ volatile int s_turn[kNT];  // [t] key tiles whose product is issued
  __shared__ long long s_scan[kThreads / 32];
  griddep_launch_dependents();
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (sbase - smem_u32(smem_raw));
  const uint32_t bar0 = sbase + kSmemBar;
  long long* const s_pre = reinterpret_cast<long long*>(smem + kSmemPre);
#define BAR(i) (bar0 + 8u * (uint32_t)(i))
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const WaitCtl wc{a.err, a.wait_ns, &s_abort};

  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(BAR_Q + i), 1);
      mbar_init(BAR(BAR_Q_FREE + i), kNT);
      mbar_init(BAR(BAR_UNIT + i), 1);
      mbar_init(BAR(BAR_UNIT_FREE + i), 5 * kNT);
    }
    for (int i = 0; i < kNT; ++i) {
      s_turn[i] = 0;
      s_odd[i][0] = s_odd[i][1] = 0;
      mbar_init(BAR(BAR_S_FULL + i), 1);
      mbar_init(BAR(BAR_S_FREE + i), 128);
      mbar_init(BAR(BAR_P_FULL + i), 128);
      mbar_init(BAR(BAR_P_FREE + i), 1);
      mbar_init(BAR(BAR_O_FREE + i), 128);
      mbar_init(BAR(BAR_V_OK + i), 128);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(BAR(BAR_KV_FULL + s), FOUR ? 4 : 1);
      mbar_init(BAR(BAR_KV_EMPTY + s), kNT);
    }
    mbar_init(BAR(BAR_MMA_DONE), kNT);
    mbar_init(BAR(BAR_TAKE), 1);
    for (int s = 0; FOUR && s < kRaw; ++s) {
      mbar_init(BAR(BAR_RAW_FULL + s), 1);
      mbar_init(BAR(BAR_RAW_EMPTY + s), 4);
    }
    fence_mbarrier_init();
  }
  if (warp == 15) tmem_alloc(smem_u32(&s_tmem), kTmemCols);
  if (a.tpt * a.G < 128) {  // rows that no copy fills read as zero
    for (int i = tid; i < (int)(2 * kNT * kTileBytes / 16); i += kThreads)
      reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_shared();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  griddep_wait();

  Share share{0, 0, 0, 0};
  if (PAGED) {
    // tiles of one head before each request, every block for itself
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int i0 = min(a.batch, tid * per), i1 = min(a.batch, i0 + per);
    const int w = kNT * a.tpt;
    long long sum = 0;
    bool bad = false;
    for (int i = i0; i < i1; ++i) {
      bool b;
      const PagedReq r = paged_req(a, i, &b);
      bad |= b;
      if (r.n_new > 0) sum += tiles_before(r.n_keys, r.n_new, w, kBN, (r.n_new + w - 1) / w);
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
    for (int x = 0; x < warp; ++x) before += s_scan[x];
    for (int i = i0; i < i1; ++i) s_pre[i + 1] += before;
    if (tid == 0) s_pre[0] = 0;
    __syncthreads();
    share = share_of(s_pre[a.batch] * a.Hkv, a.part.min_tiles, gridDim.x, blockIdx.x);
  }

  Place place{};
  if (PAGED && warp == 15 && share.begin < share.end) place = place_at(a, s_pre, share.begin);

  if (warp < 4 * kNT) {
    // ---------------- softmax: thread = row of tile t ----------------
    const int t = warp >> 2, row = tid & 127;
    const int rt = row / a.G, rh = row - rt * a.G;  // token and head of the row
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + kColS + 64 * t;
    const uint32_t t_p = tmem + lane_base + kColP + 32 * t;
    const uint32_t t_o = tmem + lane_base + kColO + 64 * t;
    const float c = a.c;
    int kt = 0, ns = 0, nv = 0;  // tiles walked, S tiles read, V tiles looked at
    bool ok = true;
    for (int nu = 0; ok; ++nu) {
      if (!mbar_wait_inline(BAR(BAR_UNIT + (nu & 1)), (nu >> 1) & 1, wc)) break;
      const Unit& su = s_unit[nu & 1];
      if (!su.more) break;
      const int j0 = su.t0[t], j1 = su.t1[t];
      // keys that this row sees: [lo, hi) from the item's first key
      int lo = 0, hi = 0;
      bool valid;
      {
        const int tok = su.q0 + t * a.tpt + rt;
        valid = rt < a.tpt && tok < su.q_end;
        if (PAGED) {
          if (valid) hi = su.lim + (tok - su.q0);
        } else if (valid) {
          int s = su.s0;
          if (su.s1 > s) s += last_at_or_below(a.cu + s, su.s1 - s + 1, tok);
          const RowRange r = row_range(a.cu[max(s, 0)], a.cu[max(s, 0) + 1], a.tokens);
          valid = s >= su.s0 && s <= su.s1 && tok >= r.begin && tok < r.end;
          lo = r.begin - su.kbeg;
          hi = valid ? (a.causal ? tok + 1 : r.end) - su.kbeg : 0;
        }
        lo -= su.j0 * kBN;  // from here on, keys count from the first tile walked
        hi -= su.j0 * kBN;
      }
      const int lo_max = su.lo_max[t] - su.j0 * kBN, hi_min = su.hi_min[t] - su.j0 * kBN;
      float m = -INFINITY, l = 0.f;
      if (FOUR)  // the item's first tiles; the others kAhead steps before their use
        for (int j = 0; ok && j < min(kAhead, su.nj); ++j)
          if ((kt + j) % kNT == t) ok = unpack_tile<BF16>(smem, bar0, kt + j, wc);
      for (int j = FOUR ? 0 : j0; ok && j < (FOUR ? su.nj : j1); ++j) {
        if (FOUR) {
          if (j + kAhead < su.nj && (kt + j + kAhead) % kNT == t &&
              !unpack_tile<BF16>(smem, bar0, kt + j + kAhead, wc)) {
            ok = false;
            break;
          }
          if (j >= j1) continue;  // j0 is 0
        }
        const int k0 = j * kBN;
        const bool edge =
            k0 < lo_max || past_limit(k0, kBN, hi_min);  // the same for the whole tile
        const int lo_l = lo - k0, hi_l = hi - k0;
        if (!mbar_wait_inline(BAR(BAR_S_FULL + t), ns & 1, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t x0[32], x1[32];
        tmem_ld32x2_wait(t_s, t_s + 32, x0, x1);
        tc_fence_before();
        mbar_arrive(BAR(BAR_S_FREE + t));
        if (__builtin_expect(edge, 0)) {
          mask32(x0, lo_l, hi_l);
          mask32(x1, lo_l - 32, hi_l - 32);
        }
        const float mx = max64(x0, x1);
        // c > 0, so max(S) c is the maximum of the scaled scores
        const float top = mx * c;
        float alpha = 1.f;
        const bool moved = __any_sync(0xffffffffu, top > m + kSlack);
        if (__builtin_expect(moved, 0)) {
          if (top > m + kSlack) {  // m = -inf: any key that is seen
            const float m_new = fmaxf(m, top);
            alpha = ex2_approx(m - m_new);
            m = m_new;
          }
          __syncwarp();
        }
        const float neg_m = m == -INFINITY ? 0.f : -m;
        uint32_t pk[32];
        float2 a0 = make_float2(0.f, 0.f), a1 = a0;
        exp32<BF16>(x0, c, neg_m, pk, a0, a1);
        exp32<BF16>(x1, c, neg_m, pk + 16, a0, a1);
        const float2 s01 = __fadd2_rn(a0, a1);
        l = l * alpha + (s01.x + s01.y);
        // P of the previous tile has been read by its product, and O is final
        // for a rescale
        if (ns > 0 && !mbar_wait_inline(BAR(BAR_P_FREE + t), (ns - 1) & 1, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        bool by_rows = false;
        if (__builtin_expect(edge, 0)) {
          // look at row `row` of the V tile
          const int s = (kt + j) % kStages;
          if (!mbar_wait_inline(BAR(BAR_KV_FULL + s), ((kt + j) / kStages) & 1, wc)) {
            ok = false;
            break;
          }
          if (row < kBN) {
            uint4* const vr = reinterpret_cast<uint4*>(smem + kSmemStage0 + s * kStageBytes +
                                                       kHalfBytes + row * 128);
            if (k0 + row >= su.kend - su.j0 * kBN) {
#pragma unroll
              for (int i = 0; i < 8; ++i) vr[i] = make_uint4(0, 0, 0, 0);
              fence_proxy_async_shared();
            } else {
              bool odd = false;
#pragma unroll
              for (int i = 0; i < 8; ++i) odd |= any_nonfinite<BF16>(vr[i]);
              if (odd) *(volatile int*)&s_odd[t][ns & 1] = ns + 1;
            }
          }
          mbar_arrive(BAR(BAR_V_OK + t));
          if (!mbar_wait_inline(BAR(BAR_V_OK + t), nv & 1, wc)) {
            ok = false;
            break;
          }
          ++nv;
          by_rows = *(volatile int*)&s_odd[t][ns & 1] == ns + 1;
        }
        if (j > j0 && moved && __any_sync(0xffffffffu, alpha != 1.f)) rescale(t_o, alpha);
        tmem_st32(t_p, pk);
        if (__builtin_expect(by_rows, 0)) {
          tmem_st_wait();
          row_product<BF16>(
              t_p, t_o, smem + kSmemStage0 + ((kt + j) % kStages) * kStageBytes + kHalfBytes,
              max(lo_l, 0), min(hi_l, kBN), j == j0);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(BAR(BAR_P_FULL + t));
        ++ns;
      }
      if (!ok) break;
      kt += su.nj;

      // ---------------- epilogue ----------------
      uint32_t o0[32], o1[32];
      if (j1 > j0) {
        // the last product of the item is the one that frees its P
        if (!mbar_wait_inline(BAR(BAR_P_FREE + t), (ns - 1) & 1, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        tmem_ld32x2_wait(t_o, t_o + 32, o0, o1);
        tc_fence_before();
        mbar_arrive(BAR(BAR_O_FREE + t));
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o0[e] = o1[e] = 0;
      }
      if (valid) {
        const int tok = su.q0 + t * a.tpt + rt, h = su.kv * a.G + rh;
        if (!PAGED || su.whole) {
          const bool some = l > 0.f || l != l;
          const float inv = some ? 1.0f / l : 0.f;
          uint4* const dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o.p) +
                                                      (long long)tok * a.o.t + (long long)h * a.o.h);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = 8 * (i & 3) + 2 * e;
              const float p = as_f(i < 4 ? o0[at] : o1[at]), q = as_f(i < 4 ? o0[at + 1] : o1[at + 1]);
              w[e] = some ? pack2<BF16>(p * inv, q * inv) : 0u;
            }
            dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (a.lse) a.lse[(long long)h * a.tokens + tok] = some ? m + lg2_approx(l) : -INFINITY;
        } else {
          const long long at = part_row(a.part, blockIdx.x, su.tail, t * a.tpt * a.G + row);
          // rows without a key so far have no sums: O may hold anything then
          const bool some = l > 0.f || l != l;
          float4* const d = reinterpret_cast<float4*>(a.part.o + at * 64);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            d[i] = some ? make_float4(as_f(o0[4 * i]), as_f(o0[4 * i + 1]), as_f(o0[4 * i + 2]),
                                      as_f(o0[4 * i + 3]))
                        : make_float4(0.f, 0.f, 0.f, 0.f);
            d[8 + i] = some ? make_float4(as_f(o1[4 * i]), as_f(o1[4 * i + 1]),
                                          as_f(o1[4 * i + 2]), as_f(o1[4 * i + 3]))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
          }
          a.part.ml[at] = make_float2(some ? m : -INFINITY, l);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(BAR_UNIT_FREE + (nu & 1)));
    }
  } else {
    if (warp == 15) {
      // ---------------- work items and loads ----------------
      int kt = 0, nu = 0, nq = 0;
      bool ok = true, bad = false, tail = false, checks = false;
      const int q_rows = a.tpt * a.G;
      // the stages that the copies land in
      constexpr int kLand = FOUR ? kRaw : kStages, BAR_FULL = FOUR ? BAR_RAW_FULL : BAR_KV_FULL,
                    BAR_EMPTY = FOUR ? BAR_RAW_EMPTY : BAR_KV_EMPTY;
      long long pos = share.begin;
      int block = blockIdx.x, taken = 0;  // packed: the window and head in hand
      for (;; ++nu) {
        const int ub = nu & 1;
        if (!PAGED && nu > 0) {
          // asked for once this window's loads are under way: no earlier, so
          // that the last windows go to the blocks that get there first
          if (lane == 0) {
            fence_proxy_async_shared();
            mbar_arrive_expect_tx(BAR(BAR_TAKE), 16);
            take_block(smem_u32(&s_answer), BAR(BAR_TAKE));
          }
          __syncwarp();
          ++taken;
          if (!mbar_wait_warp(BAR(BAR_TAKE), (nu - 1) & 1, wc)) {
            ok = false;
            break;
          }
          block = taken_block(smem_u32(&s_answer));
          __syncwarp();
        }
        if (nu >= 2 && !mbar_wait_warp(BAR(BAR_UNIT_FREE + ub), ((nu >> 1) - 1) & 1, wc)) {
          ok = false;
          break;
        }
        Unit& u = s_unit[ub];
        const bool more = PAGED ? pos < share.end : block >= 0;
        int steps = 0, nt = 0;
        if (!more) {
          if (lane == 0) u.more = 0;
        } else if (PAGED) {
          nt = tiles_of_block(place.r.n_keys, place.r.n_new, kNT * a.tpt, kBN, place.blk);
          place.t0 = min(place.t0, nt - 1);  // it is less, unless lens changed meanwhile
          steps = (int)min((long long)(nt - place.t0), share.end - pos);
          paged_unit(a, place, place.t0 + steps, nt, &u);
        } else {
          packed_unit(a, block, &u);
          checks |= block == 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(BAR_UNIT + ub));
        if (!more) break;
        const int req = place.req, n_keys = place.r.n_keys;
        if (PAGED) {
          if (!u.whole && u.tail) {
            tail = true;
            if (lane == 0)
              a.part.desc[blockIdx.x] = PartDesc{u.q0, u.kv, (u.q_end - u.q0) * a.G,
                                                 last_block(share, pos + nt - 1)};
          }
          pos += steps;
          if (pos < share.end) next_block(a, &place);
        }
        if (u.nj == 0) continue;
        const int qbuf = nq & 1;
        if (nq >= 2 && !mbar_wait_warp(BAR(BAR_Q_FREE + qbuf), ((nq >> 1) - 1) & 1, wc)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const uint32_t q_s = sbase + qbuf * kNT * kTileBytes;
          int n = 0;
#pragma unroll
          for (int t = 0; t < kNT; ++t) n += u.t1[t] > u.t0[t];
          mbar_arrive_expect_tx(BAR(BAR_Q + qbuf), n * q_rows * 128);
#pragma unroll
          for (int t = 0; t < kNT; ++t)
            if (u.t1[t] > u.t0[t])
              tma_load_4d(q_s + t * kTileBytes, &tm_q, BAR(BAR_Q + qbuf), 0, 0, u.kv,
                          u.q0 + t * a.tpt);
        }
        __syncwarp();
        ++nq;
        // paged: page ids 32 at a time, one group ahead
        const int32_t* const row = PAGED ? a.table + (long long)req * a.width : nullptr;
        const int n_pages = PAGED ? (int)pages_for(n_keys, a.shift) : 0;
        const int box = PAGED ? min(1 << a.shift, kBN) : kBN;
        const int boxes = kBN / box;
        int base = PAGED ? (int)(((long long)u.j0 * kBN) >> a.shift) : 0;
        int ids = 0, next = 0;
        if (PAGED) {
          ids = base + lane < n_pages ? row[base + lane] : a.pages;
          next = base + 32 + lane < n_pages ? row[base + 32 + lane] : a.pages;
        }
        for (int j = 0; j < u.nj; ++j, ++kt) {
          const int s = kt % kLand;
          if (kt >= kLand && !mbar_wait_warp(BAR(BAR_EMPTY + s), (kt / kLand - 1) & 1, wc)) {
            ok = false;
            break;
          }
          const uint32_t st = FOUR ? sbase + kSmemRaw + s * 2 * kRawHalf
                                   : sbase + kSmemStage0 + s * kStageBytes;
          const int k0 = (u.j0 + j) * kBN;
          if (PAGED) {
            const int page = k0 >> a.shift;
            if (page - base >= 32) {
              base += 32;
              ids = next;
              next = base + 32 + lane < n_pages ? row[base + 32 + lane] : a.pages;
            }
            const int live = n_keys <= k0 ? 0 : min(boxes, (n_keys - k0 - 1) / box + 1);
            const int bx = lane & 15;
            const int id = __shfl_sync(0xffffffffu, ids, (page - base + (boxes > 1 ? bx : 0)) & 31);
            const bool fine = page_ok(id, a.pages);
            if (FOUR) {
              // units that hold keys below n_keys; the rest of the stage is masked
              const int units = n_keys <= k0 ? 0 : min(kBN / 8, (n_keys - k0 - 1) / 8 + 1);
              if (lane == 0) mbar_arrive_expect_tx(BAR(BAR_RAW_FULL + s), 2 * units * kUnitBytes);
              __syncwarp();
              if (bx < live) {
                bad |= !fine;
                // of a page that does not exist the first one takes the place
                const PoolArg& pool = lane < 16 ? a.kc : a.vc;
                const int u0 = bx * (box / 8),
                          off = boxes > 1 ? 0 : (k0 & ((1 << a.shift) - 1)) / 8 * kUnitBytes;
                bulk_load(st + (lane >> 4) * kRawHalf + u0 * kUnitBytes,
                          static_cast<const uint8_t*>(pool.p) + (fine ? id : 0) * pool.pg +
                              u.kv * pool.h + off,
                          min(box / 8, units - u0) * kUnitBytes, BAR(BAR_RAW_FULL + s));
              }
              __syncwarp();
              continue;
            }
            if (lane == 0) mbar_arrive_expect_tx(BAR(BAR_KV_FULL + s), 2 * live * box * 128);
            __syncwarp();
            if (bx < live) {
              bad |= !fine;
              tma_load_4d(st + (lane >> 4) * kHalfBytes + bx * box * 128, lane < 16 ? &tm_k : &tm_v,
                          BAR(BAR_KV_FULL + s), 0, boxes > 1 ? 0 : k0 & ((1 << a.shift) - 1), u.kv,
                          fine ? id : a.pages);  // past the pool: reads as zero
            }
          } else if (lane == 0) {
            mbar_arrive_expect_tx(BAR(BAR_KV_FULL + s), kStageBytes);
            tma_load_4d(st, &tm_k, BAR(BAR_KV_FULL + s), 0, u.kbeg + k0, u.kv, 0);
            tma_load_4d(st + kHalfBytes, &tm_v, BAR(BAR_KV_FULL + s), 0, u.kbeg + k0, u.kv, 0);
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      if (checks) {
        // every pair of offsets is looked at once, whichever rows it spans
        for (int i = lane; i < a.batch; i += 32)
          bad |= row_range(a.cu[i], a.cu[i + 1], a.tokens).bad;
      }
      if (bad) atomicOr(a.err, kErrIndex);
      if (PAGED) {
        if (!tail && lane == 0) a.part.desc[blockIdx.x] = PartDesc{0, 0, 0, 0};
      }
      // no copy may still be landing when the block exits (matters only when a
      // wait gave up)
      if (lane == 0) {
        if (taken > 0) drain_wait(BAR(BAR_TAKE), (taken - 1) & 1);
        for (int q = 0; q < 2 && q < nq; ++q) drain_wait(BAR(BAR_Q + q), ((nq - q + 1) / 2 - 1) & 1);
        for (int k = kt > kLand ? kt - kLand : 0; k < kt; ++k)
          drain_wait(BAR(BAR_FULL + k % kLand), (k / kLand) & 1);
      }
    } else {
      // ---------------- products of row tile t ----------------
      const int t = warp - 12;
      const uint32_t d_s = tmem + kColS + 64 * t, d_p = tmem + kColP + 32 * t,
                     d_o = tmem + kColO + 64 * t;
      int kt = 0, nq = 0, ns = 0, np = 0, no = 0;
      bool ok = true;
      for (int nu = 0; ok; ++nu) {
        if (!mbar_wait_inline(BAR(BAR_UNIT + (nu & 1)), (nu >> 1) & 1, wc)) break;
        const Unit& su = s_unit[nu & 1];
        const int more = su.more, nj = su.nj, j0 = su.t0[t], j1 = su.t1[t];
        // keys that every row of the tile sees, from the first tile walked
        const int lo_max = su.lo_max[t] - su.j0 * kBN, hi_min = su.hi_min[t] - su.j0 * kBN;
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(BAR_UNIT_FREE + (nu & 1)));
        if (!more) break;
        if (nj == 0) continue;
        const int qbuf = nq & 1;
        if (!mbar_wait_inline(BAR(BAR_Q + qbuf), (nq >> 1) & 1, wc)) break;
        const uint32_t q_lo = sdesc_lo(sbase + (qbuf * kNT + t) * kTileBytes, 16);
        // step j forms S of key tile j, then O += P V of tile j - 1.  Every
        // stage is waited for and released, whether the row tile uses it or
        // not: a barrier's parity tells two uses of a stage apart, not three
        for (int j = 0; ok && j <= nj; ++j) {
          if (j < nj) {
            const int s = (kt + j) % kStages;
            ok = mbar_wait_inline(BAR(BAR_KV_FULL + s), ((kt + j) / kStages) & 1, wc);
            if (ok && j >= j0 && j < j1) {
              ok = ns == 0 || mbar_wait_inline(BAR(BAR_S_FREE + t), (ns - 1) & 1, wc);
              if (!ok) break;
              tc_fence_after();
              const uint32_t k_lo = sdesc_lo(sbase + kSmemStage0 + s * kStageBytes, 16);
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_ss(d_s, sdesc_of(q_lo + 2 * kk), sdesc_of(k_lo + 2 * kk), idesc<BF16>(64, 0),
                         kk > 0);
                mma_commit(BAR(BAR_S_FULL + t));
              }
              __syncwarp();
              ++ns;
            }
            if (!ok) break;
          }
          if (j > 0) {
            const int i = j - 1, s = (kt + i) % kStages;
            if (i >= j0 && i < j1) {
              ok = mbar_wait_inline(BAR(BAR_P_FULL + t), np & 1, wc);
              // the item's first product overwrites O: the epilogue before must
              // have read it
              if (ok && i == j0 && no > 0)
                ok = mbar_wait_inline(BAR(BAR_O_FREE + t), (no - 1) & 1, wc);
              if (!ok) break;
              // A hint, bounded and without consequence for results: the row
              // tiles' products go one behind the other.  Issued together they
              // interleave on the pipe, end together and pull the three
              // softmaxes into step, where they queue for the same units
              // (prompt of 16384 tokens, 32 / 4 heads: 1108 -> 1074 us).
              if (t > 0 && s_turn[t - 1] <= kt + i)
                for (int spin = 0; spin < 8 && s_turn[t - 1] <= kt + i; ++spin) {}
              tc_fence_after();
              const uint32_t v_lo =
                  sdesc_lo(sbase + kSmemStage0 + s * kStageBytes + kHalfBytes, 8192);
              // on a masked tile the rows' threads may have formed the product
              const bool by_rows =
                  (i * kBN < lo_max || past_limit(i * kBN, kBN, hi_min)) &&
                  s_odd[t][np & 1] == np + 1;
              if (elect_one()) {
                if (!by_rows) {
#pragma unroll
                  for (int kk = 0; kk < kBN / 16; ++kk)
                    mma_ts(d_o, d_p + kk * 8, sdesc_of(v_lo + 128 * kk), idesc<BF16>(64, 1),
                           (i > j0 || kk > 0) ? 1u : 0u);
                }
                mma_commit(BAR(BAR_P_FREE + t));
                mma_commit(BAR(BAR_KV_EMPTY + s));
              }
              __syncwarp();
              ++np;
            } else if (FOUR) {
              // behind the products before, so that stages come free in their order
              if (elect_one()) mma_commit(BAR(BAR_KV_EMPTY + s));
              __syncwarp();
            } else if (lane == 0) {
              mbar_arrive(BAR(BAR_KV_EMPTY + s));
            }
            s_turn[t] = kt + i + 1;
          }
        }
        if (!ok) break;
        if (elect_one()) mma_commit(BAR(BAR_Q_FREE + qbuf));
        __syncwarp();
        kt += nj;
        ++nq;
        if (j1 > j0) ++no;
      }
      if (elect_one()) mma_commit(BAR(BAR_MMA_DONE));
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 15) {
    tc_fence_after();
    // every product of this block has completed before its tensor memory goes
    drain_wait(BAR(BAR_MMA_DONE), 0);
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
#undef BAR
}

}  // namespace

int launch_packed_fwd(const PackedDims& d, const DevCtx& ctx, const RowsArg& q, const RowsArg& k,
                      const RowsArg& v, const int32_t* cu, const RowsArg& o, float* lse,
                      cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  TileArgs a{};
  a.tokens = d.tokens;
  a.batch = d.batch;
  a.H = d.H;
  a.Hkv = d.Hkv;
  a.G = d.G;
  a.tpt = 128 / d.G;
  a.causal = d.causal;
  a.c = d.c;
  a.cu = cu;
  a.o = o;
  a.lse = lse;
  a.err = ctx.err;
  a.wait_ns = ctx.wait_ns;
  if (!encode_tmap_4d(&tq, d.bf16, q.p, d.G, d.Hkv, d.tokens, q.h, q.h * d.G, q.t, d.G, 1, a.tpt) ||
      !encode_tmap_4d(&tk, d.bf16, k.p, d.tokens, d.Hkv, 1, k.t, k.h, 64, kBN, 1, 1) ||
      !encode_tmap_4d(&tv, d.bf16, v.p, d.tokens, d.Hkv, 1, v.t, v.h, 64, kBN, 1, 1))
    return ATTN_ERR_CUDA;
  const int window = kNT * a.tpt;
  a.windows = (d.tokens + window - 1) / window;
  const long long units = (long long)d.Hkv * a.windows;
  if (units > 0x7fffffffLL) return ATTN_ERR_SHAPE;
  auto* kernel = d.bf16 ? tiles_kernel<kPacked, true> : tiles_kernel<kPacked, false>;
  const size_t smem = kSmemPre + 1024;
  const int rc = allow_smem(d.bf16 ? kSmemPackedBf16 : kSmemPackedF16,
                            reinterpret_cast<const void*>(kernel), smem);
  if (rc != ATTN_OK) return rc;
  return cuda_status(launch_dependent(kernel, dim3((unsigned)units), dim3(kThreads), smem, stream,
                                      tq, tk, tv, a));
}

int launch_paged_rows(const PagedDims& d, const DevCtx& ctx, const RowsArg& q, const PoolArg& kc,
                      const PoolArg& vc, const int32_t* table, const int32_t* cu,
                      const int32_t* lens, const PartArgs& part, int blocks, int skip,
                      bool four, const RowsArg& o, float* lse, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  TileArgs a{};
  a.tokens = d.tokens;
  a.batch = d.batch;
  a.H = d.H;
  a.Hkv = d.Hkv;
  a.G = d.G;
  a.tpt = 128 / d.G;
  a.causal = 1;
  a.c = d.c;
  a.cu = cu;
  a.lens = lens;
  a.table = table;
  a.pages = d.pages;
  a.width = d.width;
  a.shift = d.shift;
  a.skip = skip;
  a.max_new = d.max_new;
  a.o = o;
  a.lse = lse;
  a.part = part;
  a.err = ctx.err;
  a.wait_ns = ctx.wait_ns;
  a.kc = kc;
  a.vc = vc;
  const uint32_t box = (1u << d.shift) < kBN ? (1u << d.shift) : kBN;
  const uint64_t P = 1ull << d.shift;
  if (!encode_tmap_4d(&tq, d.bf16, q.p, d.G, d.Hkv, d.tokens, q.h, q.h * d.G, q.t, d.G, 1, a.tpt))
    return ATTN_ERR_CUDA;
  tk = tv = tq;  // 4 bits: not used
  if (!four &&
      (!encode_tmap_4d(&tk, d.bf16, kc.p, P, d.Hkv, d.pages, kc.r, kc.h, kc.pg, box, 1, 1) ||
       !encode_tmap_4d(&tv, d.bf16, vc.p, P, d.Hkv, d.pages, vc.r, vc.h, vc.pg, box, 1, 1)))
    return ATTN_ERR_CUDA;
  auto* kernel = d.bf16 ? tiles_kernel<kPaged, true> : tiles_kernel<kPaged, false>;
  if (four) kernel = d.bf16 ? tiles_kernel<kPaged4, true> : tiles_kernel<kPaged4, false>;
  const size_t smem = kSmemPre + 8 * (size_t)(d.batch + 1) + 1024;
  const int rc =
      allow_smem((four ? kSmemRows4F16 : kSmemRowsF16) + (d.bf16 ? 1 : 0),
                 reinterpret_cast<const void*>(kernel),
                 kSmemPre + 8 * (size_t)(4096 + 1) + 1024);
  if (rc != ATTN_OK) return rc;
  return cuda_status(launch_dependent(kernel, dim3(blocks), dim3(kThreads), smem, stream, tq, tk,
                                      tv, a));
}

}  // namespace css
