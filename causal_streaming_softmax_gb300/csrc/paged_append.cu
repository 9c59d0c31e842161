// paged_append.cu - new tokens into the paged cache with the position rotation
// applied on the way (16-bit or 4-bit pools), and rows of a 4-bit pool read back.
//
// Half-split rotation of a row x at position p, c < 32:
//   y[c]      = x[c] cos[p][c] - x[c + 32] sin[p][c]
//   y[c + 32] = x[c + 32] cos[p][c] + x[c] sin[p][c]
// both products rounded to binary32 and then added (no fused multiply-add, so
// that any program which does the same gets the same codes and the same 16-bit
// rows bit for bit).  q goes to q_out and k to its slot, v to its slot unturned.
// Into a 4-bit pool the turned binary32 values are quantised (pool4.cuh), without
// a rounding to 16 bits in between.
//
// Four threads have a row, each eight channels of its low half and the eight that
// belong to them of its high half: the rotation, the byte that holds a channel of
// either half, and both groups' extrema (two shuffles) need no other thread.  A
// warp has eight or sixteen rows (q, k, v heads) of one token, whose position it finds
// by trying 32 offsets at a time while its rows are under way.
//
// Bound by memory: 128 bytes read and written a row of q, k and v, 36 written into 4
// bits.  36,000 tokens of 32 / 8 heads in bfloat16 take 68 us = 6.5 TB/s, 96% of the
// measured copy rate (one set of eight rows a warp 90 us, three 71, six 74; blocks for
// all the work instead of a full SM's 75).  22,900 tokens into 4 bits 53 us, 69% of it:
// the arithmetic of a K or V row, some 200 instructions a thread, takes as long as its
// bytes (1700 instructions a token, issue slots 67% busy; three blocks a SM 52.8 us,
// four 53.3, two 62).  64 tokens 2.4 us, one 1.9: launch and the chain offsets ->
// length -> angles.  Rows read back: 150,000 random slots, 4 heads, 39 us = 4.6 TB/s (a
// row's 36 bytes lie in two sectors, so that 64 come from memory for each); a whole
// pool in order 14 us of a floor of 11.6.
#include "pool4.cuh"
#include "serve_index.h"
#include "serve_internal.h"
#include "sm103.cuh"

namespace css {
namespace {

constexpr int kThreads = 256;

// The request that token t belongs to and the token's position, or -1.  Called by
// a whole warp.
__device__ __forceinline__ int position_of(const AppendArgs& a, int t) {
  const int lane = threadIdx.x & 31;
  int at = 0, n = a.batch;  // the request is in [at, at + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int v = a.cu[at + min(lane * step, n - 1)];
    const int hit = max(__popc(__ballot_sync(0xffffffffu, lane * step < n && v <= t)) - 1, 0);
    at += hit * step;
    n = min(step, n - hit * step);
  }
  const RowRange r = row_range(a.cu[at], a.cu[at + 1], a.tokens);
  const long long pos = (long long)a.lens[at] - (r.end - r.begin) + (t - r.begin);
  return r.bad || t < r.begin || t >= r.end || pos < 0 || pos >= a.angles ? -1 : (int)pos;
}

template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& w, float2 (&x)[4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = make_float2(half_to_f32<BF16>((uint16_t)u[i]),
                       half_to_f32<BF16>((uint16_t)(u[i] >> 16)));
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float2 (&x)[4]) {
  return make_uint4(pack2<BF16>(x[0].x, x[0].y), pack2<BF16>(x[1].x, x[1].y),
                    pack2<BF16>(x[2].x, x[2].y), pack2<BF16>(x[3].x, x[3].y));
}

// The four lanes of a row: extrema over the row's group.
__device__ __forceinline__ void extrema(const float2 (&x)[4], float* mx, float* mn) {
  *mx = *mn = x[0].x;
  *mx = max3_nan(*mx, x[0].y, x[1].x), *mn = min3_nan(*mn, x[0].y, x[1].x);
  *mx = max3_nan(*mx, x[1].y, x[2].x), *mn = min3_nan(*mn, x[1].y, x[2].x);
  *mx = max3_nan(*mx, x[2].y, x[3].x), *mn = min3_nan(*mn, x[2].y, x[3].x);
  // the last value and two lanes beside
  const float a = max3_nan(*mx, x[3].y, x[3].y), b = min3_nan(*mn, x[3].y, x[3].y);
  *mx = max3_nan(a, __shfl_xor_sync(0xffffffffu, a, 1), a);
  *mn = min3_nan(b, __shfl_xor_sync(0xffffffffu, b, 1), b);
  *mx = max3_nan(*mx, __shfl_xor_sync(0xffffffffu, *mx, 2), *mx);
  *mn = min3_nan(*mn, __shfl_xor_sync(0xffffffffu, *mn, 2), *mn);
}

// kSets: sets of eight rows that a warp takes of a token, their loads under way
// before the position is known.
template <bool BF16, bool ROTATE, bool FOUR, int kSets>
__global__ void __launch_bounds__(kThreads, FOUR ? 3 : 4) append_kernel(const AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, c0 = (lane & 3) * 8;
  const int rows = a.H + 2 * a.Hkv;  // without rotation q stays, and H is 0
  const int warps = gridDim.x * (kThreads / 32);
  const int first = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  bool bad = false;
  for (long long i = first; i < (long long)a.tokens * a.parts; i += warps) {
    const int t = (int)quot(i, a.parts), part = (int)(i - (long long)t * a.parts);
    const int slot = a.slots[t];
    uint4 w_lo[kSets], w_hi[kSets];
    const int set0 = part * kSets;
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
      const int row = (set0 + j) * 8 + (lane >> 2);
      w_lo[j] = w_hi[j] = make_uint4(0, 0, 0, 0);
      if (row < rows) {
        const bool is_q = row < a.H, is_v = row >= a.H + a.Hkv;
        const int h = row - (is_q ? 0 : (is_v ? a.H + a.Hkv : a.H));
        const RowsArg& src = is_q ? a.q : (is_v ? a.v : a.k);
        const uint16_t* const p = static_cast<const uint16_t*>(src.p) + t * src.t + h * src.h + c0;
        w_lo[j] = *reinterpret_cast<const uint4*>(p);
        w_hi[j] = *reinterpret_cast<const uint4*>(p + 32);
      }
    }
    if (slot < 0) continue;
    const int page = slot >> a.shift, r = slot & ((1 << a.shift) - 1);
    const int pos = ROTATE ? position_of(a, t) : 0;
    if (!page_ok(page, a.pages) || pos < 0) {
      bad = true;
      continue;
    }
    float2 co[4], si[4];
    if (ROTATE) {
      const float4* const c = reinterpret_cast<const float4*>(a.cos_tab + pos * 32ll + c0);
      const float4* const s = reinterpret_cast<const float4*>(a.sin_tab + pos * 32ll + c0);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 cw = c[e], sw = s[e];
        co[2 * e] = make_float2(cw.x, cw.y), co[2 * e + 1] = make_float2(cw.z, cw.w);
        si[2 * e] = make_float2(sw.x, sw.y), si[2 * e + 1] = make_float2(sw.z, sw.w);
      }
    }
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
      const int row0 = (set0 + j) * 8, row = row0 + (lane >> 2);
      if (row0 >= rows) break;  // the same for the whole warp
      const bool live = row < rows, is_q = row < a.H, is_v = row >= a.H + a.Hkv;
      const int h = row - (is_q ? 0 : (is_v ? a.H + a.Hkv : a.H));
      float2 x[4], y[4];
      widen8<BF16>(w_lo[j], x);
      widen8<BF16>(w_hi[j], y);
      if (ROTATE && !is_v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // one by one: pairs of products and sums are fused
          const float2 u =
              make_float2(__fsub_rn(__fmul_rn(x[e].x, co[e].x), __fmul_rn(y[e].x, si[e].x)),
                          __fsub_rn(__fmul_rn(x[e].y, co[e].y), __fmul_rn(y[e].y, si[e].y)));
          y[e] = make_float2(__fadd_rn(__fmul_rn(y[e].x, co[e].x), __fmul_rn(x[e].x, si[e].x)),
                             __fadd_rn(__fmul_rn(y[e].y, co[e].y), __fmul_rn(x[e].y, si[e].y)));
          x[e] = u;
        }
        w_lo[j] = narrow8<BF16>(x);
        w_hi[j] = narrow8<BF16>(y);
      }
      const PoolArg& pool = is_v ? a.vc : a.kc;
      if (live && (is_q || !FOUR)) {
        uint16_t* const p = (is_q ? static_cast<uint16_t*>(a.q_out.p) + t * a.q_out.t +
                                        h * a.q_out.h
                                  : static_cast<uint16_t*>(pool.p) + page * pool.pg + h * pool.h +
                                        r * pool.r) +
                            c0;
        *reinterpret_cast<uint4*>(p) = w_lo[j];
        *reinterpret_cast<uint4*>(p + 32) = w_hi[j];
      }
      if (FOUR && row0 + 8 > a.H) {  // the same for the whole warp
        float mx0, mn0, mx1, mn1;
        extrema(x, &mx0, &mn0);
        extrema(y, &mx1, &mn1);
        const uint32_t h0 = group_scale<BF16>(mx0, mn0), h1 = group_scale<BF16>(mx1, mn1);
        const Quotient lo = quotient(half_to_f32<BF16>((uint16_t)h0)),
                       hi = quotient(half_to_f32<BF16>((uint16_t)h1));
        const uint2 w = make_uint2(lo.codes(x[0], x[1]) | hi.codes(y[0], y[1]) << 4,
                                   lo.codes(x[2], x[3]) | hi.codes(y[2], y[3]) << 4);
        if (live && !is_q) {
          uint8_t* const p = static_cast<uint8_t*>(pool.p) + page * pool.pg + h * pool.h;
          *reinterpret_cast<uint2*>(p + code_at(r) + c0) = w;
          if (c0 == 0) *reinterpret_cast<uint32_t*>(p + scale_at(r)) = h0 | h1 << 16;
        }
      }
    }
  }
  if (bad) atomicOr(a.err, kErrIndex);
}

struct LoadArgs {
  int tokens, Hkv, pages, shift;
  PoolArg kc, vc;
  const int32_t* slots;
  RowsArg k, v;
  uint32_t* err;
};

// Four threads have a row of K and of V, as above; kMoves such rows of a thread are
// under way together (150,000 random slots: one 44 us, two 40, four 39).
template <bool BF16, int kMoves>
__global__ void __launch_bounds__(kThreads) load4_kernel(const LoadArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const long long n = (long long)a.tokens * a.Hkv * 4;
  const long long step = (long long)gridDim.x * kThreads * kMoves;
  bool bad = false;
  for (long long i0 = (long long)blockIdx.x * kThreads * kMoves + threadIdx.x; i0 < n; i0 += step) {
    uint2 code[kMoves][2];
    uint32_t scale[kMoves][2];
    long long k_at[kMoves], v_at[kMoves];
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      const long long i = i0 + u * kThreads;
      k_at[u] = -1;
      if (i >= n) continue;
      const int c0 = (int)(i & 3) * 8;
      const int t = (int)quot(i >> 2, a.Hkv), h = (int)((i >> 2) - (long long)t * a.Hkv);
      const int slot = a.slots[t];
      if (slot < 0) continue;
      const int page = slot >> a.shift, r = slot & ((1 << a.shift) - 1);
      if (!page_ok(page, a.pages)) {
        bad = true;
        continue;
      }
      const uint8_t* const kp = static_cast<const uint8_t*>(a.kc.p) + page * a.kc.pg + h * a.kc.h;
      const uint8_t* const vp = static_cast<const uint8_t*>(a.vc.p) + page * a.vc.pg + h * a.vc.h;
      code[u][0] = *reinterpret_cast<const uint2*>(kp + code_at(r) + c0);
      code[u][1] = *reinterpret_cast<const uint2*>(vp + code_at(r) + c0);
      scale[u][0] = *reinterpret_cast<const uint32_t*>(kp + scale_at(r));
      scale[u][1] = *reinterpret_cast<const uint32_t*>(vp + scale_at(r));
      k_at[u] = t * a.k.t + h * a.k.h + c0;
      v_at[u] = t * a.v.t + h * a.v.h + c0;
    }
#pragma unroll
    for (int u = 0; u < kMoves; ++u) {
      if (k_at[u] < 0) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float s0 = half_to_f32<BF16>((uint16_t)scale[u][j]),
                    s1 = half_to_f32<BF16>((uint16_t)(scale[u][j] >> 16));
        float2 x[4], y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t b = ((e & 2) ? code[u][j].y : code[u][j].x) >> (16 * (e & 1));
          x[e] = make_float2((float)((int)(b & 15) - 8) * s0, (float)((int)(b >> 8 & 15) - 8) * s0);
          y[e] = make_float2((float)((int)(b >> 4 & 15) - 8) * s1,
                             (float)((int)(b >> 12 & 15) - 8) * s1);
        }
        uint16_t* const p =
            static_cast<uint16_t*>(j ? a.v.p : a.k.p) + (j ? v_at[u] : k_at[u]);
        *reinterpret_cast<uint4*>(p) = narrow8<BF16>(x);
        *reinterpret_cast<uint4*>(p + 32) = narrow8<BF16>(y);
      }
    }
  }
  if (bad) atomicOr(a.err, kErrIndex);
}

template <int kSets>
void (*append_of(bool bf16, bool rotate, bool four))(AppendArgs) {
  if (!four)
    return bf16 ? append_kernel<true, true, false, kSets>
                : append_kernel<false, true, false, kSets>;
  if (rotate)
    return bf16 ? append_kernel<true, true, true, kSets> : append_kernel<false, true, true, kSets>;
  return bf16 ? append_kernel<true, false, true, kSets> : append_kernel<false, false, true, kSets>;
}

constexpr int kManySets = 2, kManyMoves = 4;
// A thread takes several pieces where there is more than so many blocks a SM of work.
// Of 16 bits (32 / 8 heads; one set, two): 800 tokens 3.1, 3.3 us; 1200 4.5, 3.9; 1600
// 5.0, 4.1; 6400 17.5, 15.8: once not all warps of one set are resident.  Into 4 bits
// a set's arithmetic is longer.  With rotation (32 / 8 heads): 1600 5.6, 6.1; 3200 8.7,
// 8.7; 6400 15.5, 14.1; 12800 33.2, 30.7; 50000 120, 104.  Without (16 heads): 800 3.3,
// 3.7; 1600 4.4, 4.1 (but 9.1, 9.4 with 2070 rows read back behind it); 12800 20.9, 19.7.
// Rows read back (4 heads, random slots; one, four): 80,000 22.2, 23.0; 150,000 44, 39.
constexpr int kMany = 4, kMany4 = 16, kManyLoad = 48;
constexpr int kBlocks = 8;  // a full SM

}  // namespace

int launch_paged_append(const PagedDims& d, const DevCtx& ctx, AppendArgs a, bool rotate,
                        bool four, cudaStream_t stream) {
  a.tokens = d.tokens, a.batch = d.batch, a.H = d.H, a.Hkv = d.Hkv;
  a.pages = d.pages, a.shift = d.shift;
  a.err = ctx.err;
  const int sets = (d.H + 2 * d.Hkv + 7) / 8;  // of eight rows, a token
  const long long warps = (long long)(four ? kMany4 : kMany) * (kThreads / 32) * ctx.sm_count;
  const bool many = sets > 1 && (long long)d.tokens * sets > warps;
  a.parts = many ? (sets + kManySets - 1) / kManySets : sets;
  auto* kernel =
      many ? append_of<kManySets>(d.bf16, rotate, four) : append_of<1>(d.bf16, rotate, four);
  const long long per = kThreads / 32, most = (long long)kBlocks * ctx.sm_count;
  const long long blocks = ((long long)d.tokens * a.parts + per - 1) / per;
  return cuda_status(launch_dependent(kernel, dim3((unsigned)(blocks > most ? most : blocks)),
                                      dim3(kThreads), 0, stream, a));
}

int launch_paged_load4(const PagedDims& d, const DevCtx& ctx, const PoolArg& kc, const PoolArg& vc,
                       const int32_t* slots, const RowsArg& k, const RowsArg& v,
                       cudaStream_t stream) {
  const LoadArgs args{d.tokens, d.Hkv, d.pages, d.shift, kc, vc, slots, k, v, ctx.err};
  const long long threads = (long long)d.tokens * d.Hkv * 4;
  const bool many = threads > (long long)kManyLoad * kThreads * ctx.sm_count;
  const long long per = (many ? kManyMoves : 1) * kThreads;
  const long long most = (long long)kBlocks * ctx.sm_count;
  const long long blocks = (threads + per - 1) / per;
  void (*kernel)(LoadArgs);
  if (many)
    kernel = d.bf16 ? load4_kernel<true, kManyMoves> : load4_kernel<false, kManyMoves>;
  else
    kernel = d.bf16 ? load4_kernel<true, 1> : load4_kernel<false, 1>;
  return cuda_status(launch_dependent(kernel, dim3((unsigned)(blocks > most ? most : blocks)),
                                      dim3(kThreads), 0, stream, args));
}

}  // namespace css
