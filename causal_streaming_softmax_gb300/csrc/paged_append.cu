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
// warp has one token, whose position it finds by trying 32 offsets at a time, and
// walks through its rows (q, k, v heads) eight by eight with the angles in
// registers.
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
__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = half_to_f32<BF16>((uint16_t)u[i]);
    x[2 * i + 1] = half_to_f32<BF16>((uint16_t)(u[i] >> 16));
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
  return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]),
                    pack2<BF16>(x[6], x[7]));
}

// The four lanes of a row: extrema over the row's group.
__device__ __forceinline__ void extrema(const float (&x)[8], float* mx, float* mn) {
  *mx = *mn = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) *mx = max_nan(*mx, x[i]), *mn = min_nan(*mn, x[i]);
#pragma unroll
  for (int by = 1; by < 4; by <<= 1) {
    *mx = max_nan(*mx, __shfl_xor_sync(0xffffffffu, *mx, by));
    *mn = min_nan(*mn, __shfl_xor_sync(0xffffffffu, *mn, by));
  }
}

template <bool BF16, bool ROTATE, bool FOUR>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, c0 = (lane & 3) * 8;
  const int first = ROTATE ? 0 : a.H, rows = a.H + 2 * a.Hkv;  // without rotation q stays
  const long long warps = (long long)gridDim.x * (kThreads / 32);
  const long long n = (long long)a.tokens * a.parts;
  bool bad = false;
  for (long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < n;
       i += warps) {
    const int t = (int)quot(i, a.parts), part = (int)(i - (long long)t * a.parts);
    const int slot = a.slots[t];
    if (slot < 0) continue;
    const int page = slot >> a.shift, r = slot & ((1 << a.shift) - 1);
    const int pos = ROTATE ? position_of(a, t) : 0;
    if (!page_ok(page, a.pages) || pos < 0) {
      bad = true;
      continue;
    }
    float co[8], si[8];
    if (ROTATE) {
      const float4* const c = reinterpret_cast<const float4*>(a.cos_tab + pos * 32ll + c0);
      const float4* const s = reinterpret_cast<const float4*>(a.sin_tab + pos * 32ll + c0);
      const float4 c_lo = c[0], c_hi = c[1], s_lo = s[0], s_hi = s[1];
      co[0] = c_lo.x, co[1] = c_lo.y, co[2] = c_lo.z, co[3] = c_lo.w;
      co[4] = c_hi.x, co[5] = c_hi.y, co[6] = c_hi.z, co[7] = c_hi.w;
      si[0] = s_lo.x, si[1] = s_lo.y, si[2] = s_lo.z, si[3] = s_lo.w;
      si[4] = s_hi.x, si[5] = s_hi.y, si[6] = s_hi.z, si[7] = s_hi.w;
    }
    for (int row0 = first + part * a.per; row0 < min(rows, first + (part + 1) * a.per);
         row0 += 8) {
      const int row = row0 + (lane >> 2);
      const bool live = row < rows, is_q = row < a.H, is_v = row >= a.H + a.Hkv;
      const int h = live ? row - (is_q ? 0 : (is_v ? a.H + a.Hkv : a.H)) : 0;
      const RowsArg& src = is_q ? a.q : (is_v ? a.v : a.k);
      uint4 w_lo = make_uint4(0, 0, 0, 0), w_hi = w_lo;
      if (live) {
        const uint16_t* const p =
            static_cast<const uint16_t*>(src.p) + t * src.t + h * src.h + c0;
        w_lo = *reinterpret_cast<const uint4*>(p);
        w_hi = *reinterpret_cast<const uint4*>(p + 32);
      }
      float x[8], y[8];
      widen8<BF16>(w_lo, x);
      widen8<BF16>(w_hi, y);
      if (ROTATE && !is_v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = __fsub_rn(__fmul_rn(x[e], co[e]), __fmul_rn(y[e], si[e]));
          y[e] = __fadd_rn(__fmul_rn(y[e], co[e]), __fmul_rn(x[e], si[e]));
          x[e] = u;
        }
        w_lo = narrow8<BF16>(x);
        w_hi = narrow8<BF16>(y);
      }
      const PoolArg& pool = is_v ? a.vc : a.kc;
      if (is_q || !FOUR) {
        uint16_t* const p = is_q ? static_cast<uint16_t*>(a.q_out.p) + t * a.q_out.t + h * a.q_out.h
                                 : static_cast<uint16_t*>(pool.p) + page * pool.pg + h * pool.h +
                                       r * pool.r;
        if (live) {
          *reinterpret_cast<uint4*>(p + c0) = w_lo;
          *reinterpret_cast<uint4*>(p + c0 + 32) = w_hi;
        }
      }
      if (FOUR && row0 + 8 > a.H) {  // the same for the whole warp
        float mx0, mn0, mx1, mn1;
        extrema(x, &mx0, &mn0);
        extrema(y, &mx1, &mn1);
        const uint32_t h0 = group_scale<BF16>(mx0, mn0), h1 = group_scale<BF16>(mx1, mn1);
        const float s0 = half_to_f32<BF16>((uint16_t)h0), s1 = half_to_f32<BF16>((uint16_t)h1);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e >> 2] |= (code_of(x[e], s0) | code_of(y[e], s1) << 4) << (8 * (e & 3));
        if (live && !is_q) {
          uint8_t* const p = static_cast<uint8_t*>(pool.p) + page * pool.pg + h * pool.h;
          *reinterpret_cast<uint2*>(p + code_at(r) + c0) = make_uint2(w[0], w[1]);
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

// Four threads have a row of K and of V, as above.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) load4_kernel(const LoadArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const long long n = (long long)a.tokens * a.Hkv * 4;
  bool bad = false;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kThreads) {
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
    const uint2 code[2] = {*reinterpret_cast<const uint2*>(kp + code_at(r) + c0),
                           *reinterpret_cast<const uint2*>(vp + code_at(r) + c0)};
    const uint32_t scale[2] = {*reinterpret_cast<const uint32_t*>(kp + scale_at(r)),
                               *reinterpret_cast<const uint32_t*>(vp + scale_at(r))};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float s0 = half_to_f32<BF16>((uint16_t)scale[j]),
                  s1 = half_to_f32<BF16>((uint16_t)(scale[j] >> 16));
      float x[8], y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = ((e & 4) ? code[j].y : code[j].x) >> (8 * (e & 3));
        x[e] = (float)((int)(b & 15) - 8) * s0;
        y[e] = (float)((int)(b >> 4 & 15) - 8) * s1;
      }
      const RowsArg& to = j ? a.v : a.k;
      uint16_t* const p = static_cast<uint16_t*>(to.p) + t * to.t + h * to.h + c0;
      *reinterpret_cast<uint4*>(p) = narrow8<BF16>(x);
      *reinterpret_cast<uint4*>(p + 32) = narrow8<BF16>(y);
    }
  }
  if (bad) atomicOr(a.err, kErrIndex);
}

}  // namespace

int launch_paged_append(const PagedDims& d, const DevCtx& ctx, AppendArgs a, bool rotate,
                        bool four, cudaStream_t stream) {
  const int rows = (rotate ? d.H : 0) + 2 * d.Hkv;
  a.tokens = d.tokens, a.batch = d.batch, a.H = d.H, a.Hkv = d.Hkv;
  a.pages = d.pages, a.shift = d.shift;
  a.err = ctx.err;
  a.per = 8;
  a.parts = (rows + a.per - 1) / a.per;
  void (*kernel)(AppendArgs);
  if (!four)
    kernel = d.bf16 ? append_kernel<true, true, false> : append_kernel<false, true, false>;
  else if (rotate)
    kernel = d.bf16 ? append_kernel<true, true, true> : append_kernel<false, true, true>;
  else
    kernel = d.bf16 ? append_kernel<true, false, true> : append_kernel<false, false, true>;
  const long long per = kThreads / 32, most = 8LL * ctx.sm_count;
  const long long blocks = ((long long)d.tokens * a.parts + per - 1) / per;
  return cuda_status(launch_dependent(kernel, dim3((unsigned)(blocks > most ? most : blocks)),
                                      dim3(kThreads), 0, stream, a));
}

int launch_paged_load4(const PagedDims& d, const DevCtx& ctx, const PoolArg& kc, const PoolArg& vc,
                       const int32_t* slots, const RowsArg& k, const RowsArg& v,
                       cudaStream_t stream) {
  const LoadArgs args{d.tokens, d.Hkv, d.pages, d.shift, kc, vc, slots, k, v, ctx.err};
  const long long blocks = ((long long)d.tokens * d.Hkv * 4 + kThreads - 1) / kThreads;
  const long long most = 8LL * ctx.sm_count;
  return cuda_status(launch_dependent(d.bf16 ? load4_kernel<true> : load4_kernel<false>,
                                      dim3((unsigned)(blocks > most ? most : blocks)),
                                      dim3(kThreads), 0, stream, args));
}

}  // namespace css
