// serve_tiles.cu - attention of many rows on the tensor cores: whole packed
// prompts, and chunks of new tokens over a paged cache.
//
// Method: for every key tile that a row tile sees, S = Q K^T; t = S c in base
// 2; P = 2^(t - m); l += sum P (binary32, P unrounded); O += P V with P
// rounded to the operands' type; O / l and L = m + log2 l.  m follows the
// running maximum only when that has grown by more than kSlack: P may then
// reach 2^kSlack, which changes no relative rounding (binary16 holds it, sums
// are binary32), and O is rescaled a few times a row instead of at nearly
// every tile.
//
// Rows: a row tile of 128 holds tpt = 128 / G tokens times the G query heads
// of one K/V head (row = token * G + head), so that a group's heads share
// every K and V tile and a short chunk still fills the rows.  A work item is
// two such tiles, A and B, one behind the other, that share K/V tiles of 128
// keys.  Packed prompts cut the token axis into windows of 2 tpt tokens
// whatever sequences lie in them, each row with its own interval of keys
// [lo, hi): many short sequences share a tile, and no table of blocks is
// needed.  Paged chunks cut each request's new tokens, and the list of their
// key tiles is shared out over the blocks in equal runs (serve_parts.cuh).
//
// Warps (12, 168 registers a thread):
//   0-3 softmax of tile A, one thread per row (= tensor-memory lane); 4-7 of B
//   8   finds the work items and issues the TMA loads (Q, K, V rows; a copy
//       per page, lanes in parallel)
//   9, 10 products of tile A and of tile B: S of the next key tile, then
//       O += P V of this one, in the order in which their inputs get ready
//   11  only allocates
// Tensor memory: S_A, S_B 128 columns each, P_A, P_B 64, O_A, O_B 64.  S is
// computed in halves of 64 keys with barriers of their own: a row's thread
// keeps the first half in registers from the maximum to the exponential, so
// that the next tile's first half is computed during the exponentials of this
// one, and the second half while the last of them finish; the round trip
// softmax -> product -> softmax no longer sits in every tile's path.
//
// What a mask excludes cannot reach a row, infinities and NaN included: S is
// replaced by -inf, and on tiles where some row misses a key the rows of V
// are looked at.  Rows of V past the last key of the item are set to zero;
// where another row of V holds a value that is not finite, the tile's product
// is formed by the row's own thread over the keys that it sees.
#include <math.h>

#include "serve_index.h"
#include "serve_internal.h"
#include "serve_parts.cuh"
#include "sm103.cuh"
#include "warp_mma.cuh"

namespace css {
namespace {

constexpr int kBN = 128;  // keys a tile
constexpr int kStages = 4;
constexpr int kThreads = 384;
constexpr float kSlack = 8.f;
constexpr uint32_t kTileBytes = 128 * 128;
constexpr uint32_t kStageBytes = 2 * kTileBytes;  // K tile, V tile
constexpr uint32_t kSmemStage0 = 4 * kTileBytes;  // behind two Q buffers of two tiles
constexpr uint32_t kSmemBar = kSmemStage0 + kStages * kStageBytes;
constexpr uint32_t kSmemPre = kSmemBar + 512;  // paged: prefix of tiles

constexpr uint32_t kColS = 0;    // + 128 t
constexpr uint32_t kColP = 256;  // + 64 t
constexpr uint32_t kColO = 384;  // + 64 t
constexpr uint32_t kTmemCols = 512;

enum {
  BAR_Q = 0,                             // [Q buffer] the item's Q tiles landed
  BAR_Q_FREE = BAR_Q + 2,                // [Q buffer] both chains are done with it
  BAR_KV_FULL = BAR_Q_FREE + 2,          // [stage]
  BAR_KV_EMPTY = BAR_KV_FULL + kStages,  // [stage] both chains are done with it
  BAR_S_FULL = BAR_KV_EMPTY + kStages,   // [2 t + half]
  BAR_S_FREE = BAR_S_FULL + 4,           // [2 t + half] read by the softmax (128 threads)
  BAR_P_FULL = BAR_S_FREE + 4,           // [t] P stored, O rescaled (128 threads)
  BAR_P_FREE = BAR_P_FULL + 2,           // [t] O += P V done
  BAR_O_FREE = BAR_P_FREE + 2,           // [t] the epilogue has read O (128 threads)
  BAR_V_OK = BAR_O_FREE + 2,             // [t] rows of V looked at (128 threads)
  BAR_UNIT = BAR_V_OK + 2,               // [item buffer] description written
  BAR_UNIT_FREE = BAR_UNIT + 2,          // [item buffer] read by 8 + 2 warps
  BAR_MMA_DONE = BAR_UNIT_FREE + 2,      // every product of the block done (2 commits)
  BAR_COUNT
};
static_assert(BAR_COUNT * 8 <= 512, "barrier area");

// A work item as warp 8 describes it.  Keys count from the item's first key.
struct Unit {
  int more;      // 0: no further item
  int q0;        // token row of tile A's first row
  int q_end;     // token rows from here on are not the item's
  int kv;
  int kbeg;      // packed: row of key 0
  int j0, nj;    // key tiles j0 .. j0 + nj - 1
  int t0[2], t1[2];          // those of row tile t: [t0, t1), counted from j0
  int lo_max[2], hi_min[2];  // keys that every row of tile t sees: [lo_max, hi_min)
  int kend;      // no row sees a key from here on
  int s0, s1;    // packed: first and last sequence in the window
  int lim;       // paged: keys that the first token of the item sees
  int whole;     // O is finished here; else a part
  int tail;      // the part starts the item
};

struct TileArgs {
  int tokens, batch, H, Hkv, G, tpt, causal;
  float c;
  const int32_t *cu, *lens, *table;
  int pages, width, shift, skip, max_new;
  RowsArg o;
  float* lse;
  PartArgs part;
  uint32_t* err;
  uint64_t wait_ns;
};

__device__ __forceinline__ float as_f(uint32_t u) { return __uint_as_float(u); }

template <bool BF16>
constexpr uint32_t idesc(int N, int b_mn) {
  return idesc_f16_f32(128, N, 0, b_mn) | (BF16 ? (1u << 7) | (1u << 10) : 0u);
}

// sum over i < n of floor((a i + b) / m), all non-negative, m > 0
__host__ __device__ inline long long floor_sum(long long n, long long m, long long a, long long b) {
  long long s = 0;
  while (n > 0) {
    s += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const long long x = a;
    a = m;
    m = x;
  }
  return s;
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
  if (q.n_new <= a.skip) q.n_new = 0;
  return q;
}

// Key tiles of the first nb row blocks (w tokens each) of a request, one head.
// Block b's last row sees base + min(n_new, (b + 1) w) keys, base = n_keys -
// n_new; a block has at least one tile.
__device__ __forceinline__ long long tiles_before(const PagedReq& r, int w, int nb) {
  const long long base = (long long)r.n_keys - r.n_new;
  long long full = nb;  // blocks whose last row is a full block's
  long long s = 0;
  if ((long long)nb * w > r.n_new) {
    full = nb - 1;
    s += max(1ll, ((long long)r.n_keys + kBN - 1) / kBN);
  }
  // blocks that end at or before key 0 count one tile
  long long lead = 0;
  if (base < 0) lead = min(full, (-base) / w);
  const long long b0 = base + lead * w;  // > -w
  return s + lead + floor_sum(full - lead, kBN, w, b0 + w + kBN - 1);
}

__device__ __forceinline__ int tiles_of_block(const PagedReq& r, int w, int b) {
  const long long end = (long long)r.n_keys - r.n_new + min((long long)r.n_new, (b + 1ll) * w);
  return end <= 0 ? 1 : (int)((end + kBN - 1) / kBN);
}

__device__ __forceinline__ void paged_unit(const TileArgs& a, const long long* pre, long long pos,
                                           long long end, Unit* u, int* req, int* n_keys,
                                           int* steps) {
  int lo = 0, hi = a.batch;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] * a.Hkv <= pos)
      lo = mid + 1;
    else
      hi = mid;
  }
  const int i = lo - 1;
  bool b;
  const PagedReq r = paged_req(a, i, &b);
  const int w = 2 * a.tpt;
  const int nblk = (r.n_new + w - 1) / w;
  const long long per = pre[i + 1] - pre[i], off = pos - pre[i] * a.Hkv;
  const int kv = (int)(off / per);
  const long long at = off - (long long)kv * per;
  int x = 0, y = nblk;  // the last block with tiles_before <= at
  while (x < y) {
    const int mid = (x + y) >> 1;
    if (tiles_before(r, w, mid) <= at)
      x = mid + 1;
    else
      y = mid;
  }
  const int blk = x - 1;
  const int nt = tiles_of_block(r, w, blk);
  const int t0 = (int)(at - tiles_before(r, w, blk));
  const long long left = end - pos;
  const int t1 = left < nt - t0 ? t0 + (int)left : nt;
  *req = i;
  *n_keys = r.n_keys;
  *steps = t1 - t0;
  u->more = 1;
  u->q0 = r.q0 + blk * w;
  u->q_end = min(r.q0 + r.n_new, u->q0 + w);
  u->kv = kv;
  u->kbeg = 0;
  u->j0 = t0;
  u->lim = r.n_keys - r.n_new + 1 + blk * w;
  u->nj = 0;
  u->kend = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = u->q0 + t * a.tpt, past = min(u->q_end, first + a.tpt);
    u->t0[t] = u->t1[t] = 0;
    u->lo_max[t] = u->hi_min[t] = 0;
    if (first < past) {
      const int keys = u->lim + (past - 1 - u->q0);  // the last row's
      u->hi_min[t] = u->lim + (first - u->q0);
      const int n = keys <= 0 ? 0 : (keys + kBN - 1) / kBN;
      u->t1[t] = max(0, min(n, t1) - t0);
      u->kend = max(u->kend, keys);
    }
    u->nj = max(u->nj, u->t1[t]);
  }
  u->whole = t0 == 0 && t1 == nt;
  u->tail = t0 == 0;
  u->s0 = u->s1 = 0;
}

// --------------------------------------------------------------- packed items
__device__ __forceinline__ void packed_unit(const TileArgs& a, int block, Unit* u) {
  const int nwin = (a.tokens + 2 * a.tpt - 1) / (2 * a.tpt);
  const int kv = block % a.Hkv, win = nwin - 1 - block / a.Hkv;
  u->more = 1;
  u->kv = kv;
  u->q0 = win * 2 * a.tpt;
  u->q_end = min(a.tokens, u->q0 + 2 * a.tpt);
  u->j0 = u->nj = 0;
  u->lim = 0;
  u->whole = 1;
  u->tail = 0;
  u->kend = 0;
  u->kbeg = 0;
  u->s0 = 0;
  u->s1 = -1;
  // first and last row that belong to a sequence, of both tiles; lane l of the
  // first four searches one of them
  const int front = a.cu[0], back = a.cu[a.batch];
  const int lane = threadIdx.x & 31;
  int f[2], e[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    f[t] = max(u->q0 + t * a.tpt, front);
    e[t] = min(min(u->q_end, u->q0 + (t + 1) * a.tpt), back) - 1;
  }
  const int want = lane == 0 ? f[0] : lane == 1 ? e[0] : lane == 2 ? f[1] : e[1];
  int s = last_at_or_below(a.cu, a.batch, want);
  s = s < 0 ? 0 : s;
  const RowRange r = row_range(a.cu[s], a.cu[s + 1], a.tokens);
  bool seen = false;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int sf = __shfl_sync(0xffffffffu, s, 2 * t), se = __shfl_sync(0xffffffffu, s, 2 * t + 1);
    const int bf = __shfl_sync(0xffffffffu, r.begin, 2 * t);
    const int ef = __shfl_sync(0xffffffffu, r.end, 2 * t);
    const int be = __shfl_sync(0xffffffffu, r.begin, 2 * t + 1);
    const int ee = __shfl_sync(0xffffffffu, r.end, 2 * t + 1);
    u->t0[t] = u->t1[t] = u->lo_max[t] = u->hi_min[t] = 0;
    if (f[t] > e[t]) continue;
    if (!seen) {
      seen = true;
      u->kbeg = bf;
      u->s0 = sf;
    }
    u->s1 = se;
    u->hi_min[t] = (a.causal ? f[t] + 1 : ef) - u->kbeg;
    u->lo_max[t] = be - u->kbeg;
    const int keys = (a.causal ? e[t] + 1 : ee) - u->kbeg;
    u->t0[t] = max(0, bf - u->kbeg) / kBN;
    u->t1[t] = max(u->t0[t], (max(keys, 0) + kBN - 1) / kBN);
    u->kend = max(u->kend, keys);
    u->nj = max(u->nj, u->t1[t]);
  }
}

// ------------------------------------------------------------------- softmax
// Sets the columns of a 32-column chunk outside [lo, hi) to -inf.
__device__ __forceinline__ void mask32(uint32_t (&v)[32], int lo, int hi) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (e < lo || e >= hi) v[e] = 0xff800000u;
}

__device__ __forceinline__ float max32(const uint32_t (&v)[32], float m) {
  float a = m, b = -INFINITY;
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    a = fmax3(a, as_f(v[e]), as_f(v[e + 1]));
    b = fmax3(b, as_f(v[e + 2]), as_f(v[e + 3]));
  }
  return fmaxf(a, b);
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
__device__ __forceinline__ void row_product(uint32_t t_p, uint32_t t_o, const uint8_t* v, int lo,
                                            int hi, float alpha, bool first) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {  // 16 columns at a time
    uint32_t o[16];
    float acc[16];
    tmem_ld16_wait(t_o + 16 * c, o);
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = first ? 0.f : as_f(o[e]) * alpha;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {  // 32 keys at a time
      uint32_t p[16];
      __syncwarp();
      tmem_ld16_wait(t_p + 16 * i, p);
#pragma unroll
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

template <bool PAGED, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const TileArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ Unit s_unit[2];
  __shared__ int s_odd[2][2];  // [t][use & 1]: number of the use whose V is not all finite
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
    s_odd[0][0] = s_odd[0][1] = s_odd[1][0] = s_odd[1][1] = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(BAR_Q + i), 1);
      mbar_init(BAR(BAR_Q_FREE + i), 2);
      mbar_init(BAR(BAR_P_FULL + i), 128);
      mbar_init(BAR(BAR_P_FREE + i), 1);
      mbar_init(BAR(BAR_O_FREE + i), 128);
      mbar_init(BAR(BAR_V_OK + i), 128);
      mbar_init(BAR(BAR_UNIT + i), 1);
      mbar_init(BAR(BAR_UNIT_FREE + i), 10);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(BAR(BAR_S_FULL + i), 1);
      mbar_init(BAR(BAR_S_FREE + i), 128);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(BAR(BAR_KV_FULL + s), 1);
      mbar_init(BAR(BAR_KV_EMPTY + s), 2);
    }
    mbar_init(BAR(BAR_MMA_DONE), 2);
    fence_mbarrier_init();
  }
  if (warp == 11) tmem_alloc(smem_u32(&s_tmem), kTmemCols);
  if (a.tpt * a.G < 128) {  // rows that no copy fills read as zero
    for (int i = tid; i < (int)(4 * kTileBytes / 16); i += kThreads)
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
    const int w = 2 * a.tpt;
    long long sum = 0;
    bool bad = false;
    for (int i = i0; i < i1; ++i) {
      bool b;
      const PagedReq r = paged_req(a, i, &b);
      bad |= b;
      s_pre[i + 1] = sum += r.n_new > 0 ? tiles_before(r, w, (r.n_new + w - 1) / w) : 0;
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
  } else if (blockIdx.x == 0) {
    // every pair of offsets is looked at once, whichever rows it spans
    bool bad = false;
    for (int i = tid; i < a.batch; i += kThreads)
      bad |= row_range(a.cu[i], a.cu[i + 1], a.tokens).bad;
    if (bad) atomicOr(a.err, kErrIndex);
  }

  if (warp == 8) {
    // ---------------- work items and loads ----------------
    int kt = 0, nu = 0, nq = 0;
    bool ok = true, bad = false, tail = false;
    const int q_rows = a.tpt * a.G;
    long long pos = share.begin;
    for (bool more = true; more; ++nu) {
      Unit u;
      int req = 0, n_keys = 0, steps = 0;
      u.more = 0;
      if (PAGED) {
        if (pos < share.end) paged_unit(a, s_pre, pos, share.end, &u, &req, &n_keys, &steps);
      } else {
        if (nu == 0) packed_unit(a, blockIdx.x, &u);
      }
      more = u.more != 0;
      const int ub = nu & 1;
      if (nu >= 2 && !mbar_wait_warp(BAR(BAR_UNIT_FREE + ub), ((nu >> 1) - 1) & 1, wc)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        s_unit[ub] = u;
        mbar_arrive(BAR(BAR_UNIT + ub));
      }
      if (!more) break;
      if (PAGED) {
        if (!u.whole && u.tail) {
          tail = true;
          if (lane == 0) {
            const int left = tiles_of_block(PagedReq{0, u.q_end - u.q0, u.lim - 1 + (u.q_end - u.q0)},
                                            2 * a.tpt, 0);
            a.part.desc[blockIdx.x] = PartDesc{u.q0, u.kv, (u.q_end - u.q0) * a.G,
                                               last_block(share, pos + left - 1)};
          }
        }
        pos += steps;
      }
      if (u.nj == 0) continue;
      const int qbuf = nq & 1;
      if (nq >= 2 && !mbar_wait_warp(BAR(BAR_Q_FREE + qbuf), ((nq >> 1) - 1) & 1, wc)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        const uint32_t q_s = sbase + qbuf * 2 * kTileBytes;
        const int na = u.t1[0] > u.t0[0], nb = u.t1[1] > u.t0[1];
        mbar_arrive_expect_tx(BAR(BAR_Q + qbuf), (na + nb) * q_rows * 128);
        if (na) tma_load_4d(q_s, &tm_q, BAR(BAR_Q + qbuf), 0, 0, u.kv, u.q0);
        if (nb) tma_load_4d(q_s + kTileBytes, &tm_q, BAR(BAR_Q + qbuf), 0, 0, u.kv, u.q0 + a.tpt);
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
        const int s = kt % kStages;
        if (kt >= kStages && !mbar_wait_warp(BAR(BAR_KV_EMPTY + s), (kt / kStages - 1) & 1, wc)) {
          ok = false;
          break;
        }
        const uint32_t st = sbase + kSmemStage0 + s * kStageBytes;
        const int k0 = (u.j0 + j) * kBN;
        if (PAGED) {
          const int page = k0 >> a.shift;
          if (page - base >= 32) {
            base += 32;
            ids = next;
            next = base + 32 + lane < n_pages ? row[base + 32 + lane] : a.pages;
          }
          const int live = n_keys <= k0 ? 0 : min(boxes, (n_keys - k0 + box - 1) / box);
          const int bx = lane & 15;
          const int id = __shfl_sync(0xffffffffu, ids, (page - base + (boxes > 1 ? bx : 0)) & 31);
          const bool fine = page_ok(id, a.pages);
          if (lane == 0) mbar_arrive_expect_tx(BAR(BAR_KV_FULL + s), 2 * live * box * 128);
          __syncwarp();
          if (bx < live) {
            bad |= !fine;
            tma_load_4d(st + (lane >> 4) * kTileBytes + bx * box * 128, lane < 16 ? &tm_k : &tm_v,
                        BAR(BAR_KV_FULL + s), 0, boxes > 1 ? 0 : k0 & ((1 << a.shift) - 1), u.kv,
                        fine ? id : a.pages);  // past the pool: reads as zero
          }
        } else if (lane == 0) {
          mbar_arrive_expect_tx(BAR(BAR_KV_FULL + s), kStageBytes);
          tma_load_4d(st, &tm_k, BAR(BAR_KV_FULL + s), 0, u.kbeg + k0, u.kv, 0);
          tma_load_4d(st + kTileBytes, &tm_v, BAR(BAR_KV_FULL + s), 0, u.kbeg + k0, u.kv, 0);
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    if (PAGED) {
      if (bad) atomicOr(a.err, kErrIndex);
      if (!tail && lane == 0) a.part.desc[blockIdx.x] = PartDesc{0, 0, 0, 0};
    }
    // no copy may still be landing when the block exits (matters only when a
    // wait gave up)
    if (lane == 0) {
      for (int q = 0; q < 2 && q < nq; ++q) drain_wait(BAR(BAR_Q + q), ((nq - q + 1) / 2 - 1) & 1);
      for (int k = kt > kStages ? kt - kStages : 0; k < kt; ++k)
        drain_wait(BAR(BAR_KV_FULL + k % kStages), (k / kStages) & 1);
    }
  } else if (warp == 9 || warp == 10) {
    // ---------------- products of row tile t ----------------
    const int t = warp - 9;
    const uint32_t d_s = tmem + kColS + 128 * t, d_p = tmem + kColP + 64 * t,
                   d_o = tmem + kColO + 64 * t;
    int kt = 0, nq = 0, ns = 0, np = 0, no = 0;
    bool ok = true;
    for (int nu = 0; ok; ++nu) {
      if (!mbar_wait_warp(BAR(BAR_UNIT + (nu & 1)), (nu >> 1) & 1, wc)) break;
      const Unit& su = s_unit[nu & 1];
      const int more = su.more, nj = su.nj, j0 = su.t0[t], j1 = su.t1[t];
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(BAR_UNIT_FREE + (nu & 1)));
      if (!more) break;
      if (nj == 0) continue;
      const int qbuf = nq & 1;
      if (!mbar_wait_warp(BAR(BAR_Q + qbuf), (nq >> 1) & 1, wc)) break;
      const uint32_t q_s = sbase + (qbuf * 2 + t) * kTileBytes;
      // step j forms S of key tile j, then O += P V of tile j - 1
      for (int j = 0; ok && j <= nj; ++j) {
        if (j < nj) {
          const int s = (kt + j) % kStages;
          ok = mbar_wait_warp(BAR(BAR_KV_FULL + s), ((kt + j) / kStages) & 1, wc);
          if (!ok) break;
          if (j >= j0 && j < j1) {
            const uint32_t k_s = sbase + kSmemStage0 + s * kStageBytes;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              if (ns > 0 && !mbar_wait_warp(BAR(BAR_S_FREE + 2 * t + h), (ns - 1) & 1, wc)) {
                ok = false;
                break;
              }
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_ss(d_s + 64 * h, sdesc_sw128(q_s + kk * 32, 16, 1024),
                         sdesc_sw128(k_s + h * 8192 + kk * 32, 16, 1024), idesc<BF16>(64, 0),
                         kk > 0);
                mma_commit(BAR(BAR_S_FULL + 2 * t + h));
              }
              __syncwarp();
            }
            if (!ok) break;
            ++ns;
          }
        }
        if (j > 0) {
          const int i = j - 1, s = (kt + i) % kStages;
          if (i >= j0 && i < j1) {
            if (!mbar_wait_warp(BAR(BAR_P_FULL + t), np & 1, wc)) {
              ok = false;
              break;
            }
            // the item's first product overwrites O: the epilogue before must
            // have read it
            if (i == j0 && no > 0 && !mbar_wait_warp(BAR(BAR_O_FREE + t), (no - 1) & 1, wc)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t v_s = sbase + kSmemStage0 + s * kStageBytes + kTileBytes;
            const bool by_rows = s_odd[t][np & 1] == np + 1;  // the rows' threads did it
            if (elect_one()) {
              if (!by_rows) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                  mma_ts(d_o, d_p + kk * 8, sdesc_sw128(v_s + kk * 2048, 8192, 1024),
                         idesc<BF16>(64, 1), (i > j0 || kk > 0) ? 1u : 0u);
              }
              mma_commit(BAR(BAR_P_FREE + t));
            }
            __syncwarp();
            ++np;
          }
          if (elect_one()) mma_commit(BAR(BAR_KV_EMPTY + s));
          __syncwarp();
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
  } else if (warp < 8) {
    // ---------------- softmax: thread = row of tile t ----------------
    const int t = warp >> 2, row = tid & 127;
    const int rt = row / a.G, rh = row - rt * a.G;  // token and head of the row
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + kColS + 128 * t;
    const uint32_t t_p = tmem + lane_base + kColP + 64 * t;
    const uint32_t t_o = tmem + lane_base + kColO + 64 * t;
    const float c = a.c;
    int kt = 0, ns = 0, nv = 0;  // tiles walked, S tiles read, V tiles looked at
    bool ok = true;
    for (int nu = 0; ok; ++nu) {
      if (!mbar_wait_warp(BAR(BAR_UNIT + (nu & 1)), (nu >> 1) & 1, wc)) break;
      const Unit& su = s_unit[nu & 1];
      const int more = su.more, nj = su.nj, j0 = su.t0[t], j1 = su.t1[t], kbase = su.j0 * kBN;
      const int lo_max = su.lo_max[t], hi_min = su.hi_min[t], kend = su.kend;
      const int tok = su.q0 + t * a.tpt + rt, kv = su.kv;
      const int whole = su.whole, tail = su.tail, lrow = t * a.tpt * a.G + row;
      const int kbeg = su.kbeg, s0 = su.s0, s1 = su.s1, lim = su.lim + (tok - su.q0);
      bool valid = more && rt < a.tpt && tok < su.q_end;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(BAR_UNIT_FREE + (nu & 1)));
      if (!more) break;
      // keys that this row sees: [lo, hi) from the item's first key
      int lo = 0, hi = 0;
      if (PAGED) {
        if (valid) hi = lim;
      } else if (valid) {
        int s = s0;
        if (s1 > s0) s += last_at_or_below(a.cu + s0, s1 - s0 + 1, tok);
        const RowRange r = row_range(a.cu[s], a.cu[s + 1], a.tokens);
        valid = s >= s0 && s <= s1 && tok >= r.begin && tok < r.end;
        lo = r.begin - kbeg;
        hi = valid ? (a.causal ? tok + 1 : r.end) - kbeg : 0;
      }
      float m = -INFINITY, l = 0.f;
      for (int j = j0; j < j1; ++j) {
        const int k0 = kbase + j * kBN;
        const bool edge = k0 < lo_max || k0 + kBN > hi_min;  // the same for the whole tile
        const int lo_l = lo - k0, hi_l = hi - k0;
        if (!mbar_wait_warp(BAR(BAR_S_FULL + 2 * t), ns & 1, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t x0[32], x1[32];  // the first half, kept until the exponentials
        tmem_ld32x2_wait(t_s, t_s + 32, x0, x1);
        tc_fence_before();
        mbar_arrive(BAR(BAR_S_FREE + 2 * t));
        if (edge) {
          mask32(x0, lo_l, hi_l);
          mask32(x1, lo_l - 32, hi_l - 32);
        }
        float mx = max32(x1, max32(x0, -INFINITY));
        if (!mbar_wait_warp(BAR(BAR_S_FULL + 2 * t + 1), ns & 1, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t y[32];
        tmem_ld32_wait(t_s + 64, y);
        if (edge) mask32(y, lo_l - 64, hi_l - 64);
        mx = max32(y, mx);
        tmem_ld32_wait(t_s + 96, y);
        if (edge) mask32(y, lo_l - 96, hi_l - 96);
        mx = max32(y, mx);
        // c > 0, so max(S) c is the maximum of the scaled scores
        const float top = mx * c;
        float alpha = 1.f;
        if (top > m + kSlack || m == -INFINITY) {
          const float m_new = fmaxf(m, top);
          alpha = ex2_approx(m - (m_new == -INFINITY ? 0.f : m_new));
          m = m_new;
        }
        const float neg_m = m == -INFINITY ? 0.f : -m;
        uint32_t pk[64];
        float2 a0 = make_float2(0.f, 0.f), a1 = a0;
        exp32<BF16>(x0, c, neg_m, pk, a0, a1);
        exp32<BF16>(x1, c, neg_m, pk + 16, a0, a1);
        exp32<BF16>(y, c, neg_m, pk + 48, a0, a1);
        tmem_ld32_wait(t_s + 64, y);
        tc_fence_before();
        mbar_arrive(BAR(BAR_S_FREE + 2 * t + 1));
        if (edge) mask32(y, lo_l - 64, hi_l - 64);
        exp32<BF16>(y, c, neg_m, pk + 32, a0, a1);
        const float2 s01 = __fadd2_rn(a0, a1);
        l = l * alpha + (s01.x + s01.y);

        bool by_rows = false;
        const uint8_t* v_s = smem;
        if (edge) {
          // look at row `row` of the V tile
          const int s = (kt + j) % kStages;
          if (!mbar_wait_warp(BAR(BAR_KV_FULL + s), ((kt + j) / kStages) & 1, wc)) {
            ok = false;
            break;
          }
          uint8_t* const v = smem + kSmemStage0 + s * kStageBytes + kTileBytes;
          v_s = v;
          uint4* const vr = reinterpret_cast<uint4*>(v + row * 128);
          if (k0 + row >= kend) {
#pragma unroll
            for (int i = 0; i < 8; ++i) vr[i] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_shared();
          } else {
            bool odd = false;
#pragma unroll
            for (int i = 0; i < 8; ++i) odd |= any_nonfinite<BF16>(vr[i]);
            if (odd) *(volatile int*)&s_odd[t][ns & 1] = ns + 1;
          }
          mbar_arrive(BAR(BAR_V_OK + t));
          if (!mbar_wait_warp(BAR(BAR_V_OK + t), nv & 1, wc)) {
            ok = false;
            break;
          }
          ++nv;
          by_rows = *(volatile int*)&s_odd[t][ns & 1] == ns + 1;
        }
        // P of the previous tile has been read by its product, and O is final
        // for a rescale
        if (ns > 0 && !mbar_wait_warp(BAR(BAR_P_FREE + t), (ns - 1) & 1, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        {
          const uint32_t(&w0)[32] = *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]);
          const uint32_t(&w1)[32] = *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]);
          tmem_st32(t_p, w0);
          tmem_st32(t_p + 32, w1);
        }
        if (by_rows) {
          tmem_st_wait();
          row_product<BF16>(t_p, t_o, v_s, max(lo_l, 0), min(hi_l, kBN), alpha, j == j0);
        } else if (j > j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          uint32_t o0[32], o1[32];
          tmem_ld32x2_wait(t_o, t_o + 32, o0, o1);
          const float2 al = make_float2(alpha, alpha);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = __fmul2_rn(make_float2(as_f(o0[e]), as_f(o0[e + 1])), al);
            const float2 z = __fmul2_rn(make_float2(as_f(o1[e]), as_f(o1[e + 1])), al);
            o0[e] = __float_as_uint(x.x), o0[e + 1] = __float_as_uint(x.y);
            o1[e] = __float_as_uint(z.x), o1[e + 1] = __float_as_uint(z.y);
          }
          tmem_st32(t_o, o0);
          tmem_st32(t_o + 32, o1);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(BAR(BAR_P_FULL + t));
        ++ns;
      }
      if (!ok) break;
      kt += nj;

      // ---------------- epilogue ----------------
      uint32_t o0[32], o1[32];
      if (j1 > j0) {
        // the last product of the item is the one that frees its P
        if (!mbar_wait_warp(BAR(BAR_P_FREE + t), (ns - 1) & 1, wc)) {
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
        const int h = kv * a.G + rh;
        if (!PAGED || whole) {
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
          const long long at = part_row(a.part, blockIdx.x, tail, lrow);
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
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 11) {
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
  const long long units = (long long)d.Hkv * ((d.tokens + 2 * a.tpt - 1) / (2 * a.tpt));
  if (units > 0x7fffffffLL) return ATTN_ERR_SHAPE;
  auto* kernel = d.bf16 ? tiles_kernel<false, true> : tiles_kernel<false, false>;
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
                      const RowsArg& o, float* lse, cudaStream_t stream) {
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
  const uint32_t box = (1u << d.shift) < kBN ? (1u << d.shift) : kBN;
  const uint64_t P = 1ull << d.shift;
  if (!encode_tmap_4d(&tq, d.bf16, q.p, d.G, d.Hkv, d.tokens, q.h, q.h * d.G, q.t, d.G, 1, a.tpt) ||
      !encode_tmap_4d(&tk, d.bf16, kc.p, P, d.Hkv, d.pages, kc.r, kc.h, kc.pg, box, 1, 1) ||
      !encode_tmap_4d(&tv, d.bf16, vc.p, P, d.Hkv, d.pages, vc.r, vc.h, vc.pg, box, 1, 1))
    return ATTN_ERR_CUDA;
  auto* kernel = d.bf16 ? tiles_kernel<true, true> : tiles_kernel<true, false>;
  const size_t smem = kSmemPre + 8 * (size_t)(d.batch + 1) + 1024;
  const int rc =
      allow_smem(d.bf16 ? kSmemRowsBf16 : kSmemRowsF16, reinterpret_cast<const void*>(kernel),
                 kSmemPre + 8 * (size_t)(4096 + 1) + 1024);
  if (rc != ATTN_OK) return rc;
  return cuda_status(launch_dependent(kernel, dim3(blocks), dim3(kThreads), smem, stream, tq, tk,
                                      tv, a));
}

}  // namespace css
