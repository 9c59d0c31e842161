// paged_plan.cu - block tables, slot map and offsets of one serving step from
// the requests' lengths, with pages handed out and taken back.
//
// With c_i cached and n_i new tokens of request i, P tokens a page:
//   need_i = ceil((c_i + n_i) / P) - ceil(c_i / P), a = exclusive scan of need,
//   table[i][ceil(c_i / P) + j] = ring[(head + a_i + j) mod N],
//   cu = scan of n, slot(t) = table[i][p / P] P + p mod P, p = c_i + t - cu_i,
// and a finished request's pages go behind the ring's tail.
//
// Latency bound: a few numbers a request and one a token.  One launch: every
// block scans all requests itself (4 at most a thread, three sums at once),
// which is cheaper than a second launch or a wait between blocks, and then
// takes its share of the tokens and pages, finding the request of each by
// bisection of the scanned offsets in shared memory.  The pages read are at
// the ring's head and the table's old entries, those written behind its tail
// and in the table's new entries, so no block reads what another writes.
// cached is read again where a token or page is placed; should another stream
// write it meanwhile, the place is checked, not trusted.
// Measured (GB300): 64 requests of one token 3.4 us, 512 requests with 110,000
// slots 6.1 us, of which about 2 are the launch.
#include "serve_index.h"
#include "serve_internal.h"
#include "sm103.cuh"

namespace css {
namespace {

constexpr int kPer = 4;  // requests a thread scans

struct PlanArgs {
  int batch, tokens, pages, width, shift;
  const int32_t *cached, *fresh, *state;
  int32_t *ring, *table, *cu, *lens, *slots, *next;
  uint32_t* err;
};

struct Sums {
  long long add, need, back;
};

__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return Sums{a.add + b.add, a.need + b.need, a.back + b.back};
}

__device__ __forceinline__ Sums shfl_up(const Sums& a, int by) {
  return Sums{__shfl_up_sync(0xffffffffu, a.add, by), __shfl_up_sync(0xffffffffu, a.need, by),
              __shfl_up_sync(0xffffffffu, a.back, by)};
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const PlanArgs a) {
  constexpr int kMaxBatch = kThreads * kPer;
  __shared__ int s_cu[kMaxBatch + 1], s_need[kMaxBatch + 1], s_back[kMaxBatch + 1];
  __shared__ Sums s_warp[kThreads / 32];
  __shared__ int s_status[kThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = a.state[0], free = a.state[1];

  PlanRow row[kPer];
  Sums mine{0, 0, 0};
  int status = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = tid * kPer + j;
    if (i < a.batch) {
      row[j] = plan_row(a.cached[i], a.fresh[i], a.width, a.shift);
      mine = mine + Sums{row[j].add, row[j].need, row[j].back};
      status |= row[j].status;
    }
  }
  Sums upto = mine;  // inclusive over the warp
#pragma unroll
  for (int by = 1; by < 32; by <<= 1) {
    const Sums o = shfl_up(upto, by);
    if (lane >= by) upto = upto + o;
  }
  status = (int)__reduce_or_sync(0xffffffffu, (unsigned)status);
  if (lane == 31) {
    s_warp[warp] = upto;
    s_status[warp] = status;
  }
  __syncthreads();
  Sums before{0, 0, 0}, total{0, 0, 0};
  const int used = (a.batch + 32 * kPer - 1) / (32 * kPer);  // warps that hold requests
#pragma unroll 4
  for (int w = 0; w < used; ++w) {
    if (w == warp) before = total;
    total = total + s_warp[w];
    status |= s_status[w];
  }
  status = plan_status(status, total.add, total.need, total.back, head, free, a.pages, a.tokens);

  const int first = blockIdx.x * kThreads + tid, step = gridDim.x * kThreads;
  if (status != 0) {
    for (int t = first; t < a.tokens; t += step) a.slots[t] = -1;
    if (blockIdx.x == 0) {
      for (int i = tid; i <= a.batch; i += kThreads) a.cu[i] = 0;
      for (int i = tid; i < a.batch; i += kThreads) a.lens[i] = a.cached[i];
      if (tid == 0) {
        a.next[0] = head;
        a.next[1] = free;
        a.next[2] = 0;
        a.next[3] = status;
      }
    }
    return;
  }

  // the sums fit 32 bits from here on: add <= tokens, need and back <= pages
  Sums at = before + Sums{upto.add - mine.add, upto.need - mine.need, upto.back - mine.back};
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = tid * kPer + j;
    if (i < a.batch) {
      s_cu[i] = (int)at.add;
      s_need[i] = (int)at.need;
      s_back[i] = (int)at.back;
      if (blockIdx.x == 0) {
        a.cu[i] = (int)at.add;
        a.lens[i] = a.fresh[i] < 0 ? 0 : a.cached[i] + a.fresh[i];
      }
      at = at + Sums{row[j].add, row[j].need, row[j].back};
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.cu[a.batch] = (int)total.add;
    a.next[0] = ring_at(head, total.need, a.pages);
    a.next[1] = (int)(free - total.need + total.back);
    a.next[2] = (int)total.need;
    a.next[3] = 0;
  }
  __syncthreads();

  bool bad = false;
  for (int t = first; t < a.tokens; t += step) {
    int slot = -1;
    if (t < total.add) {
      const int i = last_at_or_below(s_cu, a.batch, t);
      const long long c = a.cached[i], pos = c + (t - s_cu[i]);
      const long long have = pages_for(c, a.shift), pg = pos >> a.shift;
      const long long x = s_need[i] + (pg - have);  // handed out: place behind the head
      int id = -1;
      if (pg < have) {
        if (pg >= 0 && pg < a.width) id = a.table[(long long)i * a.width + pg];
      } else if (x < total.need) {
        id = a.ring[ring_at(head, x, a.pages)];
      }
      if (page_ok(id, a.pages))
        slot = (id << a.shift) + ((int)pos & ((1 << a.shift) - 1));
      else
        bad = true;
    }
    a.slots[t] = slot;
  }
  for (int x = first; x < total.need; x += step) {
    const int i = last_at_or_below(s_need, a.batch, x);
    const long long at = pages_for(a.cached[i], a.shift) + (x - s_need[i]);
    if (at >= 0 && at < a.width)
      a.table[(long long)i * a.width + at] = a.ring[ring_at(head, x, a.pages)];
    else
      bad = true;
  }
  for (int y = first; y < total.back; y += step) {
    const int i = last_at_or_below(s_back, a.batch, y);
    const int id = a.table[(long long)i * a.width + (y - s_back[i])];
    bad |= !page_ok(id, a.pages);  // told now, not by whom it is handed to later
    a.ring[ring_at(head, (long long)free + y, a.pages)] = id;
  }
  if (bad) atomicOr(a.err, kErrIndex);
}

}  // namespace

int launch_paged_plan(const PagedDims& d, const DevCtx& ctx, const int32_t* cached,
                      const int32_t* fresh, int32_t* ring, const int32_t* state, int32_t* table,
                      int32_t* cu, int32_t* lens, int32_t* slots, int32_t* next,
                      cudaStream_t stream) {
  const PlanArgs args{d.batch, d.tokens, d.pages, d.width, d.shift, cached, fresh, state,
                      ring,    table,    cu,      lens,    slots,   next,   ctx.err};
  // 256 threads scan up to 1024 requests, 1024 threads 4096: the smaller block
  // starts and meets faster (64 requests 3.7 us against 4.2, 512 requests with
  // 110,000 slots 5.8 against 6.7; 128 threads measured the same as 256).
  const auto blocks = [&](int threads) {
    const int n = (d.tokens + 2 * threads - 1) / (2 * threads);
    const int most = ctx.sm_count * (1024 / threads);
    return dim3(n < 1 ? 1 : (n > most ? most : n));
  };
  if (d.batch <= 256 * kPer)
    return cuda_status(
        launch_dependent(paged_plan_kernel<256>, blocks(256), dim3(256), 0, stream, args));
  static_assert(1024 * kPer >= 4096, "admitted batch");
  return cuda_status(
      launch_dependent(paged_plan_kernel<1024>, blocks(1024), dim3(1024), 0, stream, args));
}

}  // namespace css
