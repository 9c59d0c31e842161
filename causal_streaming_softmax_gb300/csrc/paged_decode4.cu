// paged_decode4.cu - attention of a request's few new rows (new tokens x heads of
// a group <= 16) over the pages of a 4-bit cache: the token step of a server.
//
// The arithmetic is that of the 16-bit kernel (S = Q K^T, P = 2^(S c - m), running
// maximum m and sum l in binary32, O += P V with P rounded to the operands' type)
// over values code * scale, which are exact in 16 bits (pool4.cuh).
//
// 72 bytes a key and K/V head come from memory where the 16-bit cache has 256, so
// the same arithmetic has less than a third of the time, and the number of
// instructions a key decides.  Hence:
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
//  * K's codes go into the product unscaled and unsigned and the scale of a key is
//    applied to its scores: binary16 as subnormals, code * 2^-24 (or 2^-20) being
//    the bits of the code themselves, bfloat16 as 16 + code; the offset times the
//    sum of q is where the accumulators start;
//  * V's codes become code * scale (the scale varies along the sum): exact;
//  * the maximum is followed only when a score passes it by kSlack, so that a step
//    has one vote instead of a reduction over the keys' lanes.
// The list of key tiles, the producer warp and the joining of parts are those of
// the 16-bit kernel (serve_decode.cuh, serve_parts.cuh).
#include <math.h>

#include "pool4.cuh"
#include "serve_decode.cuh"
#include "serve_index.h"
#include "serve_internal.h"
#include "serve_parts.cuh"
#include "sm103.cuh"
#include "warp_mma.cuh"

namespace css {
namespace {

constexpr float kSlack = 8.f;
constexpr int kLd = 68;  // floats a row of the joining buffer (bank spread)

// A block's shape.  COLS: column tiles of eight query rows.
template <int COLS>
struct Config {
  static constexpr bool kWhole = false;
  static constexpr int kCols = COLS, kRows = 8 * COLS;
  static constexpr int kBlocks = COLS == 1 ? 2 : 1;  // a SM
  static constexpr int kConsumers = 8, kStages = COLS == 1 ? 4 : 3;
  static constexpr int kThreads = 32 * (kConsumers + 1);
  static constexpr int kWarpKeys = 32, kTileKeys = kWarpKeys * kConsumers;
  static constexpr uint32_t kHalf = kTileKeys / 8 * kUnitBytes;  // K (or V) of a stage
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr uint32_t kQ = kDecodeRows * 128;
  static constexpr uint32_t kSmemStage = 2 * kQ;  // behind two Q buffers
  static constexpr uint32_t kSmemJoin = kSmemStage + kStages * kStage;
  static constexpr uint32_t kSmemMl = kSmemJoin + kConsumers * kRows * kLd * 4;
  static constexpr uint32_t kSmemBar = kSmemMl + kConsumers * kRows * 8;
  static constexpr uint32_t kSmemPre = kSmemBar + 128;  // + 8 (batch + 1), + alignment slack
  // barriers
  static constexpr int kFull = 0, kEmpty = kStages, kQFull = 2 * kStages, kQFree = kQFull + 2;
  static_assert((kQFree + 2) * 8 <= 128, "barrier area");
  static_assert(kHalf % 16 == 0 && kSmemMl % 16 == 0 && kSmemBar % 16 == 0, "alignment");
  static_assert(kSmemPre + 8 * (kMaxPagedBatch + 1) + 1024 <= 227 * 1024 - 2048,
                "shared memory of a block");
};
constexpr int kTileKeys = Config<1>::kTileKeys;

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

// Whether one of the two scales of a row is an infinity or NaN.
template <bool BF16>
__device__ __forceinline__ bool odd_scale(uint32_t s) {
  constexpr uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
  return (s & e) == e || (s & (e << 16)) == (e << 16);
}

template <bool BF16, class C>
__global__ void __launch_bounds__(C::kThreads, C::kBlocks)
    paged_decode4_kernel(const __grid_constant__ CUtensorMap tm_q, const DecodeArgs a,
                         const PoolArg kc, const PoolArg vc) {
  constexpr int kConsumers = C::kConsumers, kStages = C::kStages, kThreads = C::kThreads,
                kTileKeys = C::kTileKeys, kCols = C::kCols, kRows = C::kRows,
                kWarpKeys = C::kWarpKeys, kSteps = kWarpKeys / 16;
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
    reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_shared();
  griddep_wait();

  tiles_before_each<C>(a, s_pre, s_scan);
  const Share share = share_of(s_pre[a.batch] * a.Hkv, a.part.min_tiles, gridDim.x, blockIdx.x);

  if (warp == kConsumers) {
    // ---------------- producer ----------------
    const int box = min(1 << a.shift, kTileKeys);  // rows a copy, at most
    const int boxes = kTileKeys / box;             // copies a tile of K (and of V)
    const bool small = boxes > 1;                  // a copy a page
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
      const int t1 = (int)min((long long)sg.nt, sg.t0 + (share.end - pos));
      const int32_t* const row = a.table + (long long)sg.req * a.width;
      const int n_pages = (int)pages_for(r.n_keys, a.shift);
      int base = (int)(((long long)sg.t0 * kTileKeys) >> a.shift);
      int ids = nx_ids, next = nx_next;
      const long long last = pos - sg.t0 + sg.nt - 1;  // the item's last position
      pos += t1 - sg.t0;
      if (pos < share.end) {
        next_place<C>(a, s_pre, &nx);
        read_ids();
      }
      const int qbuf = nq & 1;
      ok = !(nq >= 2) || mbar_wait_warp(BAR(BAR_Q_FREE + qbuf), ((nq >> 1) - 1) & 1, wc);
      if (!ok) break;
      if (lane == 0) {
        s_item[qbuf] = Item{r, sg.kv, sg.t0, t1, sg.t0 == 0 && t1 == sg.nt};
        mbar_arrive_expect_tx(BAR(BAR_Q + qbuf), a.ntok * a.G * 128);
        tma_load_4d(sbase + qbuf * kQ, &tm_q, BAR(BAR_Q + qbuf), 0, 0, sg.kv, r.q0);
      }
      ++nq;
      const uint8_t* const kp = static_cast<const uint8_t*>(kc.p) + sg.kv * kc.h;
      const uint8_t* const vp = static_cast<const uint8_t*>(vc.p) + sg.kv * vc.h;
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
        // units that hold keys below n_keys; the rest of the stage is masked
        const int live = r.n_keys <= k0 ? 0 : min(kTileKeys / 8, (r.n_keys - k0 - 1) / 8 + 1);
        const uint32_t st = sbase + C::kSmemStage + s * kStage;
        if (lane == 0) mbar_arrive_expect_tx(BAR(BAR_FULL + s), 2 * live * kUnitBytes);
        __syncwarp();
#pragma unroll 1
        for (int b0 = 0; b0 < boxes; b0 += 32) {
          const int bx = b0 + lane;
          // a tile of the smallest pages needs all 32 ids of a group
          const int id = __shfl_sync(0xffffffffu, ids, (page - base + (small ? bx : 0)) & 31);
          const bool fine = page_ok(id, a.pages);
          const int u0 = bx * (box / 8), units = min(box / 8, live - u0);
          if (bx < boxes && units > 0) {
            bad |= !fine;
            // of a page that does not exist the first one takes the place
            const long long p = fine ? id : 0;
            const int off = small ? 0 : (k0 & ((1 << a.shift) - 1)) / 8 * kUnitBytes;
            bulk_load(st + u0 * kUnitBytes, kp + p * kc.pg + off, units * kUnitBytes,
                      BAR(BAR_FULL + s));
            bulk_load(st + kHalf + u0 * kUnitBytes, vp + p * vc.pg + off, units * kUnitBytes,
                      BAR(BAR_FULL + s));
          }
        }
      }
      if (sg.t0 == 0 && t1 < sg.nt) {
        tail = true;
        if (lane == 0)
          a.part.desc[blockIdx.x] = PartDesc{r.q0, sg.kv, r.n_new * a.G, last_block(share, last)};
      }
    }
    if (lane == 0 && !tail) a.part.desc[blockIdx.x] = PartDesc{0, 0, 0, 0};
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
      // Q's fragments: products 0 and 1 take the low channels (words 0 and 1 of a
      // lane's codes), 2 and 3 the high ones
      uint32_t q[kCols][4][2];
      float z_lo[kCols][2], z_hi[kCols][2];  // where the scores of rows 2 tq, 2 tq + 1 start
      Item sg{};
      bool ok = mbar_wait_warp(BAR(BAR_Q + qbuf), (nq >> 1) & 1, wc);
      if (ok) {
        sg = s_item[qbuf];
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
          float sum[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // channels 32 h + 8 tq .. + 7 of row 8 n + g
            const uint4 w = *reinterpret_cast<const uint4*>(
                smem + qbuf * kQ + sw128_offset(8 * n + g, 4 * h + tq));
            q[n][2 * h][0] = __byte_perm(w.x, w.y, 0x5410);
            q[n][2 * h][1] = __byte_perm(w.x, w.y, 0x7632);
            q[n][2 * h + 1][0] = __byte_perm(w.z, w.w, 0x5410);
            q[n][2 * h + 1][1] = __byte_perm(w.z, w.w, 0x7632);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            sum[h] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sum[h] += half_to_f32<BF16>((uint16_t)u[i]) + half_to_f32<BF16>((uint16_t)(u[i] >> 16));
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            z_lo[n][e] = -Raw<BF16>::kLoZero * __shfl_sync(0xffffffffu, sum[0], 8 * tq + 4 * e);
            z_hi[n][e] = -Raw<BF16>::kHiZero * __shfl_sync(0xffffffffu, sum[1], 8 * tq + 4 * e);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(BAR_Q_FREE + qbuf));
      }
      ++nq;
      const Request r = sg.r;
      const int t1 = sg.t1, rows = r.n_new * a.G;
      pos += t1 - sg.t0;
      // keys that this lane's rows see
      const int first_lim = row_limit(r.n_keys, r.n_new, 0);
      int lim[kCols][2];
      float m[kCols][2], l[kCols][2];
      float o[kCols][4][4];
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          lim[n][e] = row_limit(r.n_keys, r.n_new, (8 * n + 2 * tq + e) / a.G);
          m[n][e] = -INFINITY;
          l[n][e] = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) o[n][j][e] = o[n][j][2 + e] = 0.f;
        }

      for (int t = sg.t0; t < t1; ++t, ++it) {
        const int s = it % kStages;
        ok = mbar_wait_warp(BAR(BAR_FULL + s), (it / kStages) & 1, wc);
        if (!ok) break;
        const uint32_t ks =
            sbase + C::kSmemStage + s * kStage + warp * (kWarpKeys / 8) * kUnitBytes;
        const uint32_t vs = ks + kHalf;
        const int k0 = t * kTileKeys + warp * kWarpKeys;
        const bool edge = past_limit(k0, kWarpKeys, first_lim);  // some row misses a key

        // scores in base 2: [.][step][key g, key g + 8 of the step][row 2 tq, 2 tq + 1]
        float p[kCols][kSteps][2][2];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          uint32_t x[4][4];  // product, fragment register
#pragma unroll
          for (int u = 0; u < 2; ++u) {  // keys g and g + 8
            const uint2 w = lds64(ks + (2 * i + u) * kUnitBytes + lane * 8);
            raw_codes<BF16>(w.x, x[0][u], x[2][u], x[0][2 + u], x[2][2 + u]);
            raw_codes<BF16>(w.y, x[1][u], x[3][u], x[1][2 + u], x[3][2 + u]);
          }
          float s_lo[2], s_hi[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t w = lds32(ks + (2 * i + u) * kUnitBytes + kUnitScales + g * 4);
            s_lo[u] = half_to_f32<BF16>((uint16_t)w) * (a.c * Raw<BF16>::kLoUnit);
            s_hi[u] = half_to_f32<BF16>((uint16_t)(w >> 16)) * (a.c * Raw<BF16>::kHiUnit);
          }
#pragma unroll
          for (int n = 0; n < kCols; ++n) {
            float lo[4] = {z_lo[n][0], z_lo[n][1], z_lo[n][0], z_lo[n][1]};
            float hi[4] = {z_hi[n][0], z_hi[n][1], z_hi[n][0], z_hi[n][1]};
            mma_16816<BF16>(lo, x[0], q[n][0][0], q[n][0][1]);
            mma_16816<BF16>(hi, x[2], q[n][2][0], q[n][2][1]);
            mma_16816<BF16>(lo, x[1], q[n][1][0], q[n][1][1]);
            mma_16816<BF16>(hi, x[3], q[n][3][0], q[n][3][1]);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                p[n][i][u][e] = fmaf(lo[2 * u + e], s_lo[u], hi[2 * u + e] * s_hi[u]);
          }
        }
        if (edge) {
#pragma unroll
          for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (k0 + 16 * i + 8 * u + g >= lim[n][e]) p[n][i][u][e] = -INFINITY;
        }
        float top[kCols][2];
        bool grew = false;
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[n][e] = fmaxf(p[n][0][0][e], p[n][0][1][e]);
#pragma unroll
            for (int i = 1; i < kSteps; ++i)
              top[n][e] = fmax3(top[n][e], p[n][i][0][e], p[n][i][1][e]);
            grew |= top[n][e] > m[n][e] + kSlack;
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = top[n][e];
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
              if (x > m[n][e]) {
                const float f = ex2_approx(m[n][e] - x);
                m[n][e] = x;
                l[n][e] *= f;
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][j][e] *= f, o[n][j][2 + e] *= f;
              }
            }
          __syncwarp();
        }
        uint32_t pf[kCols][kSteps][2];
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
          const float u0 = m[n][0] == -INFINITY ? 0.f : m[n][0];
          const float u1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              p[n][i][u][0] = ex2_approx(p[n][i][u][0] - u0);
              p[n][i][u][1] = ex2_approx(p[n][i][u][1] - u1);
              l[n][0] += p[n][i][u][0];
              l[n][1] += p[n][i][u][1];
              pf[n][i][u] = transpose8(pack2<BF16>(p[n][i][u][0], p[n][i][u][1]));
            }
        }
        bool odd = false;  // a scale of the edge that some row must not meet
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          uint32_t w[4];
          ldmatrix_x4_trans(vs + (2 * i + (mi & 1)) * kUnitBytes + mr * 32 + (mi >> 1) * 16, w);
          uint32_t s_lo[2], s_hi[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {  // keys 2 tq and the next of either unit
            uint2 sw = lds64(vs + (2 * i + u) * kUnitBytes + kUnitScales + tq * 8);
            if (edge) {
              // keys that no row sees count as zero whatever stands there, and so, for
              // now, does one that some row misses and that is not finite
              const int key = k0 + 16 * i + 8 * u + 2 * tq;
              if (key >= r.n_keys) sw.x = 0;
              if (key + 1 >= r.n_keys) sw.y = 0;
              if (key >= first_lim && odd_scale<BF16>(sw.x)) sw.x = 0, odd = true;
              if (key + 1 >= first_lim && odd_scale<BF16>(sw.y)) sw.y = 0, odd = true;
            }
            s_lo[u] = __byte_perm(sw.x, sw.y, 0x5410);
            s_hi[u] = __byte_perm(sw.x, sw.y, 0x7632);
          }
          // channel tiles 2 g, 32 + 2 g, 2 g + 1, 33 + 2 g (rows g; + 16 in rows g + 8)
          uint32_t x[4][4];
          scaled_codes<BF16>(w[0], s_lo[0], s_hi[0], x[0][0], x[1][0], x[2][0], x[3][0]);
          scaled_codes<BF16>(w[2], s_lo[0], s_hi[0], x[0][1], x[1][1], x[2][1], x[3][1]);
          scaled_codes<BF16>(w[1], s_lo[1], s_hi[1], x[0][2], x[1][2], x[2][2], x[3][2]);
          scaled_codes<BF16>(w[3], s_lo[1], s_hi[1], x[0][3], x[1][3], x[2][3], x[3][3]);
#pragma unroll
          for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_16816<BF16>(o[n][j], x[j], pf[n][i][0], pf[n][i][1]);
        }
        if (edge && __any_sync(0xffffffffu, odd)) {
          // what those keys give the rows that see them
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll 1
              for (int k = 0; k < 8; ++k) {
                const int key = k0 + 16 * i + 8 * u + k;
                const uint32_t unit = vs + (2 * i + u) * kUnitBytes;
                const uint32_t sw = lds32(unit + kUnitScales + 4 * k);
                float wt[kCols][2];
#pragma unroll
                for (int n = 0; n < kCols; ++n)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    wt[n][e] = __shfl_sync(0xffffffffu, p[n][i][u][e], 4 * k + tq);
                if (key < first_lim || key >= r.n_keys || !odd_scale<BF16>(sw)) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {  // row g + 8 h of channel tile j
                    const int byte = 16 * h + 2 * g + (j >> 1);
                    const uint32_t b = smem[unit - sbase + k * 32 + byte] >> (4 * (j & 1));
                    const float v = (float)((int)(b & 15) - 8) *
                                    half_to_f32<BF16>((uint16_t)(sw >> (16 * (j & 1))));
#pragma unroll
                    for (int n = 0; n < kCols; ++n)
#pragma unroll
                      for (int e = 0; e < 2; ++e)
                        if (key < lim[n][e])
                          o[n][j][2 * h + e] = fmaf(wt[n][e], v, o[n][j][2 * h + e]);
                  }
              }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(BAR_EMPTY + s));
      }

      // ---------------- the consumer warps meet ----------------
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
          l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
          l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
          const int row = warp * kRows + 8 * n + 2 * tq + e;
          if (g == 0) s_ml[row] = make_float2(m[n][e], l[n][e]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < 2; ++x)  // low and high channels
              *reinterpret_cast<float2*>(s_join + row * kLd + 32 * x + 16 * h + 2 * g) =
                  make_float2(o[n][x][2 * h + e], o[n][2 + x][2 * h + e]);
        }
      // where a wait gave up, all leave together
      if (named_barrier_any(1, kConsumers * 32, !ok)) break;
      const int row = tid >> 3, c0 = (tid & 7) * 8;
      if (row < rows && row < kRows) {
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
          const float* const d = s_join + (w * kRows + row) * kLd + c0;
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
    }
  }
#undef BAR
}

template <class C>
int launch(const PagedDims& d, const DevCtx& ctx, const RowsArg& q, const PoolArg& kc,
           const PoolArg& vc, const DecodeArgs& args, int blocks, int which, cudaStream_t stream) {
  CUtensorMap tq;
  if (!encode_tmap_4d(&tq, d.bf16, q.p, d.G, d.Hkv, d.tokens, q.h, q.h * d.G, q.t, d.G, 1,
                      args.ntok))
    return ATTN_ERR_CUDA;
  const size_t smem = C::kSmemPre + 8 * (size_t)(d.batch + 1) + 1024;
  auto* kernel = d.bf16 ? paged_decode4_kernel<true, C> : paged_decode4_kernel<false, C>;
  const int rc = allow_smem(which + d.bf16, reinterpret_cast<const void*>(kernel),
                            C::kSmemPre + 8 * (kMaxPagedBatch + 1) + 1024);
  if (rc != ATTN_OK) return rc;
  return cuda_status(launch_dependent(kernel, dim3(blocks), dim3(C::kThreads), smem, stream, tq,
                                      args, kc, vc));
}

}  // namespace

// A table that leaves a request one tile gives every item to one block.
bool decode4_whole(const PagedDims& d) { return ((long long)d.width << d.shift) <= kTileKeys; }

int launch_paged_decode4(const PagedDims& d, const DevCtx& ctx, const RowsArg& q,
                         const PoolArg& kc, const PoolArg& vc, const int32_t* table,
                         const int32_t* cu, const int32_t* lens, const PartArgs& part, int blocks,
                         const RowsArg& o, float* lse, cudaStream_t stream) {
  // as many tokens as a call has at most: a token step of up to eight heads a group
  // needs one column tile
  const int ntok = d.max_new < decode_tokens(d.G) ? d.max_new : decode_tokens(d.G);
  const DecodeArgs args{d.batch, d.tokens, d.H, d.Hkv, d.G, ntok, d.max_new, d.pages, d.width,
                        d.shift, d.c, cu, lens, table, o, lse, part, ctx.err, ctx.wait_ns};
  if (ntok * d.G <= 8)
    return launch<Config<1>>(d, ctx, q, kc, vc, args, blocks, kSmemDecode4F16, stream);
  return launch<Config<2>>(d, ctx, q, kc, vc, args, blocks, kSmemDecode4WideF16, stream);
}

}  // namespace css
