// serve_attend.cu - attention of packed and paged rows, plain form: one warp a
// (token, query head).
//
// t_j = (q . k_j) c in base 2 over the keys j that the row sees, 32 keys at a
// time, one key a lane: m' = max(m, max t), P = 2^(t - m'), l = l 2^(m - m')
// + sum P, O = O 2^(m - m') + P V with two columns a lane; O / l and
// L = m + log2 l.  Everything in binary32; masked keys are not read.
#include "serve_index.h"
#include "serve_internal.h"
#include "sm103.cuh"

namespace css {
namespace {

constexpr int kThreads = 256;

struct AttendArgs {
  int tokens, batch, H, G, causal, paged, max_new;
  int pages, width, shift;
  float c;
  RowsArg q, o;
  PoolArg k, v;  // packed: one page of all tokens
  const int32_t *cu, *lens, *table;
  float* lse;
  uint32_t* err;
  int skip;
};

template <bool BF16>
__device__ __forceinline__ float2 widen(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return make_float2(f16_bits_to_f32((uint16_t)w), f16_bits_to_f32((uint16_t)(w >> 16)));
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) attend_kernel(const AttendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long gid = (long long)blockIdx.x * kThreads + threadIdx.x, wid = gid >> 5;
  // every pair of offsets is looked at once, whichever rows it spans
  for (long long x = gid; x < a.batch; x += (long long)gridDim.x * kThreads) {
    const RowRange r = row_range(a.cu[x], a.cu[x + 1], a.tokens);
    if (r.bad || r.end - r.begin > a.max_new) atomicOr(a.err, kErrIndex);
  }
  if (wid >= (long long)a.tokens * a.H) return;
  const int t = (int)(wid / a.H), h = (int)(wid - (long long)t * a.H), kv = h / a.G;
  const int i = last_at_or_below(a.cu, a.batch + 1, t);
  if (i < 0 || i >= a.batch) return;  // outside every sequence
  const RowRange rr = row_range(a.cu[i], a.cu[i + 1], a.tokens);
  bool bad = rr.bad;
  int n = 0;  // visible keys
  if (t >= rr.begin && t < rr.end) {
    if (a.paged) {
      if (rr.end - rr.begin <= a.skip) return;
      bool b;
      const int len = key_count(a.lens[i], a.width, a.shift, &b);
      bad |= b;
      n = max(0, len - (rr.end - 1 - t));
    } else {
      n = a.causal ? t + 1 - rr.begin : rr.end - rr.begin;
    }
  } else {
    if (bad && lane == 0) atomicOr(a.err, kErrIndex);
    return;
  }
  float q[64];
  const uint16_t* qp = static_cast<const uint16_t*>(a.q.p) + t * a.q.t + h * a.q.h;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const uint4 w = reinterpret_cast<const uint4*>(qp)[x];
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const float2 f = widen<BF16>(ws[y]);
      q[x * 8 + y * 2] = f.x;
      q[x * 8 + y * 2 + 1] = f.y;
    }
  }
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
  for (int k0 = 0; k0 < n; k0 += 32) {
    const int j = k0 + lane;
    long long kat = -1, vat = -1;
    if (j < n) {
      long long page = 0, row = rr.begin + j;
      if (a.paged) {
        const int id = a.table[(long long)i * a.width + (j >> a.shift)];
        page = id;
        row = j & ((1 << a.shift) - 1);
        if (!page_ok(id, a.pages)) bad = true, page = -1;
      }
      if (page >= 0) {
        kat = page * a.k.pg + kv * a.k.h + row * a.k.r;
        vat = page * a.v.pg + kv * a.v.h + row * a.v.r;
      }
    }
    float s = -INFINITY;
    if (kat >= 0) {
      const uint16_t* kp = static_cast<const uint16_t*>(a.k.p) + kat;
      s = 0.f;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint4 w = reinterpret_cast<const uint4*>(kp)[x];
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float2 f = widen<BF16>(ws[y]);
          s = fmaf(q[x * 8 + y * 2], f.x, s);
          s = fmaf(q[x * 8 + y * 2 + 1], f.y, s);
        }
      }
      s *= a.c;
    }
    float mx = s;
#pragma unroll
    for (int by = 16; by; by >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, by));
    const float m2 = fmaxf(m, mx), mu = m2 == -INFINITY ? 0.f : m2;
    const float alpha = exp2f(m - mu), p = exp2f(s - mu);
    m = m2;
    float ps = p;
#pragma unroll
    for (int by = 16; by; by >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, by);
    l = l * alpha + ps;
    o0 *= alpha;
    o1 *= alpha;
    const int cnt = min(32, n - k0);
    for (int x = 0; x < cnt; ++x) {
      const float px = __shfl_sync(0xffffffffu, p, x);
      const long long at = __shfl_sync(0xffffffffu, vat, x);
      if (at >= 0) {
        const float2 f = widen<BF16>(
            reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.v.p) + at)[lane]);
        o0 = fmaf(px, f.x, o0);
        o1 = fmaf(px, f.y, o1);
      }
    }
  }
  const bool any = l > 0.f || l != l;
  const float inv = any ? 1.f / l : 0.f;
  o0 *= inv;
  o1 *= inv;
  uint32_t* op = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o.p) + t * a.o.t +
                                             h * a.o.h);
  op[lane] = BF16 ? pack_bf16x2(o0, o1) : pack_f16x2(o0, o1);
  if (a.lse && lane == 0) a.lse[(long long)h * a.tokens + t] = any ? m + log2f(l) : -INFINITY;
  if (bad) atomicOr(a.err, kErrIndex);
}

int launch(const AttendArgs& a, bool bf16, cudaStream_t stream) {
  const long long blocks = ((long long)a.tokens * a.H * 32 + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return ATTN_ERR_SHAPE;
  return cuda_status(launch_dependent(bf16 ? attend_kernel<true> : attend_kernel<false>,
                                      dim3((unsigned)blocks), dim3(kThreads), 0, stream, a));
}

}  // namespace

int launch_packed_fwd(const PackedDims& d, const DevCtx& ctx, const RowsArg& q, const RowsArg& k,
                      const RowsArg& v, const int32_t* cu, const RowsArg& o, float* lse,
                      cudaStream_t stream) {
  const AttendArgs a{d.tokens, d.batch, d.H, d.G, d.causal, 0, d.tokens, 1, 0, 0, d.c, q, o,
                     PoolArg{k.p, 0, k.h, k.t}, PoolArg{v.p, 0, v.h, v.t}, cu, nullptr, nullptr,
                     lse, ctx.err, 0};
  return launch(a, d.bf16, stream);
}

int launch_paged_rows(const PagedDims& d, const DevCtx& ctx, const RowsArg& q, const PoolArg& kc,
                     const PoolArg& vc, const int32_t* table, const int32_t* cu,
                     const int32_t* lens, const RowsArg& o, float* lse, int skip,
                     cudaStream_t stream) {
  const AttendArgs a{d.tokens, d.batch, d.H, d.G, 1, 1, d.max_new, d.pages, d.width, d.shift, d.c, q, o, kc,
                     vc, cu, lens, table, lse, ctx.err, skip};
  return launch(a, d.bf16, stream);
}

}  // namespace css
