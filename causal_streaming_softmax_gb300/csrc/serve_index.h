// serve_index.h - index arithmetic of the packed and paged calls, host and
// device: what keeps every access inside the tensors whatever the device
// arrays of offsets, lengths, slots and page ids hold.  Plain C++ so that it
// is tested on the host.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define CSS_HD __host__ __device__ __forceinline__
#define CSS_RARE static __host__ __device__ __noinline__
#else
#define CSS_HD inline
#define CSS_RARE static inline
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

// Keys that the row of new token tok of n_new sees, the last token's is n_keys;
// a row past the last token counts as the last.  May be negative.
CSS_HD int row_limit(int n_keys, int n_new, int tok) {
  const int behind = n_new - 1 - tok;
  return n_keys - (behind > 0 ? behind : 0);
}

// Whether the keys [k0, k0 + n) pass lim, without forming k0 + n.
CSS_HD bool past_limit(int k0, int n, int lim) { return lim - k0 < n; }

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

// a / b of non-negative numbers: the 32-bit division where both fit (a 64-bit
// one is some four hundred clocks, and several stand before a block's first
// load).
CSS_HD long long quot(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

struct Share {
  long long begin, end;
  long long each;  // positions of a block; the first `more` blocks take one more
  int more, blocks;
};

CSS_HD Share share_of(long long total, int min_tiles, int grid, int block) {
  Share s;
  const long long most = quot(total, min_tiles);
  s.blocks = most < 1 ? 1 : (most < grid ? (int)most : grid);
  s.each = quot(total, s.blocks);
  s.more = (int)(total - s.each * s.blocks);
  if (block >= s.blocks) {
    s.begin = s.end = total;
  } else {
    s.begin = block * s.each + (block < s.more ? block : s.more);
    s.end = s.begin + s.each + (block < s.more ? 1 : 0);
  }
  return s;
}

// The block whose share holds position x.
CSS_HD int last_block(const Share& s, long long x) {
  const long long big = s.more * (s.each + 1);  // positions of the longer shares
  return x < big ? (int)quot(x, s.each + 1) : s.more + (int)quot(x - big, s.each);
}

// sum over i < n of floor((a i + b) / m), all non-negative, m > 0
CSS_RARE long long floor_sum(long long n, long long m, long long a, long long b) {
  long long s = 0;
  while (n > 0) {
    const long long qa = quot(a, m), qb = quot(b, m);
    s += n * (n - 1) / 2 * qa + n * qb;
    a -= qa * m;
    b -= qb * m;
    const long long y = a * n + b;
    if (y < m) break;
    n = quot(y, m);
    b = y - n * m;
    const long long x = a;
    a = m;
    m = x;
  }
  return s;
}

// Key tiles (bn keys) of the first nb row blocks (w tokens each) of a request
// with n_keys keys, its n_new new tokens the last of them.  Block b's last row
// sees n_keys - n_new + min(n_new, (b + 1) w) keys; a block has at least one
// tile.  nb is at most the request's blocks.
CSS_HD long long tiles_before(int n_keys, int n_new, int w, int bn, int nb) {
  const long long base = (long long)n_keys - n_new;
  long long full = nb;  // blocks whose last row is a full block's
  long long s = 0;
  if ((long long)nb * w > n_new) {
    full = nb - 1;
    s = n_keys <= 0 ? 1 : (n_keys - 1) / bn + 1;
  }
  // blocks that end at or before key 0 count one tile
  long long lead = 0;
  if (base < 0) {
    lead = quot(-base, w);
    if (lead > full) lead = full;
  }
  s += lead;
  const long long n = full - lead, first = base + (lead + 1) * w + bn - 1;  // first > 0 where n > 0
  if (n > 32 || first + n * w > 0x7fffffffLL) return n > 0 ? s + floor_sum(n, bn, w, first) : s;
  // a few blocks: the sum itself is faster than the divisions
  uint32_t sum = 0, at = (uint32_t)first;
  for (int b = 0; b < (int)n; ++b, at += (uint32_t)w) sum += at / (uint32_t)bn;
  return s + sum;
}

// Whether the description of a part, as block c of `blocks` left it in the
// workspace, names rows of the output and parts that exist (room: rows a part
// has room for).  It does unless something else wrote the workspace meanwhile.
CSS_HD bool part_ok(int q0, int kv, int rows, int last, int c, int blocks, int room, int tokens,
                    int Hkv, int G) {
  return q0 >= 0 && q0 <= tokens && kv >= 0 && kv < Hkv && rows >= 0 && rows <= room &&
         rows <= (long long)(tokens - q0) * G && last >= c && last < blocks;
}

CSS_HD int tiles_of_block(int n_keys, int n_new, int w, int bn, int b) {
  const long long past = (b + 1ll) * w;
  const long long end = (long long)n_keys - n_new + (past < n_new ? past : n_new);
  return end <= 0 ? 1 : (int)((end - 1) / bn) + 1;
}

}  // namespace css
