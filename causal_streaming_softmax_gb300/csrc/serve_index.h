// serve_index.h - index arithmetic of the packed and paged calls, host and
// device: what keeps every access inside the tensors whatever the device
// arrays of offsets, lengths, slots and page ids hold.  Plain C++ so that it
// is tested on the host.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define CSS_HD __host__ __device__ __forceinline__
#else
#define CSS_HD inline
#endif

namespace css {

// Rows [begin, end) of one sequence, and whether its offsets were in order
// and inside [0, tokens].  A sequence with bad offsets is cut to what lies
// inside (empty when they run backwards).
struct RowRange {
  int begin, end;
  bool bad;
};

CSS_HD RowRange row_range(int32_t c0, int32_t c1, int32_t tokens) {
  RowRange r;
  r.bad = c0 < 0 || c1 < c0 || c1 > tokens;
  r.begin = c0 < 0 ? 0 : (c0 > tokens ? tokens : c0);
  r.end = c1 > tokens ? tokens : c1;
  if (r.end < r.begin) r.end = r.begin;
  return r;
}

// Largest i in [0, n) with cu[i] <= x, or -1.  With ascending offsets that is
// the last sequence that starts at or before row x; empty sequences that start
// at x too come before it.  Bounded for any contents.
CSS_HD int last_at_or_below(const int32_t* cu, int n, int32_t x) {
  int lo = 0, hi = n;  // cu[lo - 1] <= x < cu[hi] in ascending order
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= x)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo - 1;
}

// Keys of a request that lie in its table: lens cut to [0, width * page].
CSS_HD int key_count(int32_t len, int32_t table_width, int32_t page_shift, bool* bad) {
  const long long cap = (long long)table_width << page_shift;
  *bad = len < 0 || (long long)len > cap;
  return len < 0 ? 0 : ((long long)len > cap ? (int)cap : len);
}

// Pages that hold n tokens.
CSS_HD long long pages_for(long long n, int page_shift) {
  return (n + ((1ll << page_shift) - 1)) >> page_shift;
}

CSS_HD bool page_ok(int32_t id, int32_t num_pages) { return id >= 0 && id < num_pages; }

// Position x behind the ring's head (0 <= head < n, 0 <= x <= n).
CSS_HD int ring_at(int head, long long x, int n) {
  const long long p = (long long)head + x;
  return (int)(p >= n ? p - n : p);
}

// What one request asks of a plan.
struct PlanRow {
  long long add;   // new tokens
  long long have;  // pages it holds
  long long need;  // pages it is handed
  long long back;  // pages it gives back
  int status;      // ATTN_PLAN_ bits of this row alone (width, state)
};

CSS_HD PlanRow plan_row(int32_t cached, int32_t fresh, int32_t table_width, int page_shift) {
  PlanRow r;
  r.status = 0;
  long long c = cached;
  if (c < 0) {
    r.status |= 8;  // ATTN_PLAN_STATE
    c = 0;
  }
  r.have = pages_for(c, page_shift);
  r.add = fresh < 0 ? 0 : fresh;
  const long long total = pages_for(c + r.add, page_shift);
  if (total > table_width) r.status |= 2;  // ATTN_PLAN_WIDTH
  r.need = fresh < 0 ? 0 : total - r.have;
  r.back = fresh < 0 ? r.have : 0;
  return r;
}

// The status of a whole plan from its sums.
CSS_HD int plan_status(int rows, long long add, long long need, long long back, int head, int free,
                       int num_pages, int tokens) {
  int st = rows;
  if (head < 0 || head >= num_pages || free < 0 || free > num_pages ||
      (long long)free + back > num_pages)
    st |= 8;
  if (need > free) st |= 1;
  if (add > tokens) st |= 4;
  return st;
}

}  // namespace css
