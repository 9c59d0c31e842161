"""The packed and paged calls without a GPU: refusals on the host before any
launch, and the index arithmetic that keeps device accesses inside the tensors
whatever the device arrays hold."""
import ctypes
import itertools
import os
import random
import subprocess
import sys

import pytest
import torch

import serve_util
from causal_streaming_softmax_gb300 import api, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def packed(**kw):
    base = dict(tokens=100, batch=3, heads=4, kv_heads=2, head_dim=64, causal=1, dtype=0,
                scale=0.125, q_token=256, q_head=64, k_token=128, k_head=64, v_token=128,
                v_head=64, o_token=256, o_head=64)
    base.update(kw)
    return api.AttnPackedShape(**base)


def paged(**kw):
    base = dict(batch=3, tokens=10, heads=4, kv_heads=2, head_dim=64, page_size=16, num_pages=50,
                table_width=8, max_new=4, dtype=1, scale=0.125, q_token=256, q_head=64,
                o_token=256, o_head=64, k_token=128, k_head=64, v_token=128, v_head=64,
                kc_page=2048, kc_head=1024, kc_row=64, vc_page=2048, vc_head=1024, vc_row=64)
    base.update(kw)
    return api.AttnPagedShape(**base)


def fwd(lib, s, q=P, k=P, v=P, cu=P, o=P, lse=None):
    return lib.attn_packed_fwd(None if s is None else ctypes.byref(s), q, k, v, cu, o, lse, None)


def pfwd(lib, s, q=P, k=P, v=P, table=P, cu=P, lens=P, ws=P, n=1 << 40, o=P, lse=None):
    return lib.attn_paged_fwd(None if s is None else ctypes.byref(s), q, k, v, table, cu, lens,
                              ws, n, o, lse, None)


BAD_PACKED = [
    dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(batch=0), dict(batch=65536), dict(heads=3),
    dict(heads=0), dict(kv_heads=0), dict(heads=258, kv_heads=2), dict(head_dim=128),
    dict(causal=2), dict(dtype=2), dict(dtype=-1), dict(scale=0.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(scale=-1.0), dict(q_token=0), dict(k_head=0), dict(v_token=60),
    dict(q_head=68), dict(k_token=-256), dict(o_head=1 << 38),
    dict(o_token=64), dict(o_token=192), dict(o_token=64, o_head=99 * 64),
]


@pytest.mark.parametrize("kw", BAD_PACKED)
def test_packed_shape_refused(lib, kw):
    assert fwd(lib, packed(**kw)) == api.ATTN_ERR_SHAPE


def test_packed_pointers_refused(lib):
    assert fwd(lib, None) == api.ATTN_ERR_NULL
    s = packed()
    for name in ("q", "k", "v", "cu", "o"):
        assert fwd(lib, s, **{name: None}) == api.ATTN_ERR_NULL, name
        assert fwd(lib, s, **{name: P + 2}) == api.ATTN_ERR_ALIGN, name
    assert fwd(lib, s, lse=P + 4) == api.ATTN_ERR_ALIGN
    # nothing to do: no pointer is looked at
    assert fwd(lib, packed(tokens=0), None, None, None, None, None) == api.ATTN_OK
    # the stride of a dimension of one is not read
    assert fwd(lib, packed(tokens=1, q_token=3, o_token=0), cu=None) == api.ATTN_ERR_NULL


BAD_PAGED = [
    dict(batch=0), dict(batch=4097), dict(tokens=-1), dict(page_size=4), dict(page_size=2048),
    dict(page_size=24), dict(page_size=0), dict(num_pages=0), dict(num_pages=1 << 27),
    dict(table_width=0), dict(table_width=1 << 27),
]
BAD_ATTEND = BAD_PAGED + [
    dict(heads=5), dict(kv_heads=0), dict(head_dim=32), dict(dtype=7), dict(scale=0.0),
    dict(max_new=0), dict(heads=129, kv_heads=1), dict(q_token=8), dict(o_token=64),
    dict(kc_page=0), dict(kc_row=65), dict(vc_head=-1024), dict(vc_row=32),
]


@pytest.mark.parametrize("kw", BAD_ATTEND)
def test_paged_shape_refused(lib, kw):
    assert pfwd(lib, paged(**kw)) == api.ATTN_ERR_SHAPE
    if not set(kw) & {"q_token", "o_token", "kc_page", "kc_row", "vc_head", "vc_row"}:
        s = paged(**kw)
        assert lib.attn_paged_workspace_bytes(ctypes.byref(s)) == 0


def test_paged_pointers_refused(lib):
    assert pfwd(lib, None) == api.ATTN_ERR_NULL
    s = paged()
    for name in ("q", "k", "v", "table", "cu", "lens", "ws", "o"):
        assert pfwd(lib, s, **{name: None}) == api.ATTN_ERR_NULL, name
        assert pfwd(lib, s, **{name: P + 2}) == api.ATTN_ERR_ALIGN, name
    need = lib.attn_paged_workspace_bytes(ctypes.byref(s))
    assert need > 0
    assert pfwd(lib, s, n=need - 1) == api.ATTN_ERR_WORKSPACE
    assert pfwd(lib, paged(tokens=0), *[None] * 7, 0, None) == api.ATTN_OK


def plan_args():
    return [P + 4096 * i for i in range(9)]


def plan(lib, s, args):
    return lib.attn_paged_plan(None if s is None else ctypes.byref(s), *args, None)


@pytest.mark.parametrize("kw", BAD_PAGED)
def test_plan_shape_refused(lib, kw):
    assert plan(lib, paged(**kw), plan_args()) == api.ATTN_ERR_SHAPE


def test_plan_pointers_refused(lib):
    assert plan(lib, None, plan_args()) == api.ATTN_ERR_NULL
    for i in range(9):
        a = plan_args()
        a[i] = None
        assert plan(lib, paged(), a) == api.ATTN_ERR_NULL, i
        a[i] = P + 1 + 4096 * i
        assert plan(lib, paged(), a) == api.ATTN_ERR_ALIGN, i
    # partly on top of one another: the last entry of cached, the first of lens
    a = plan_args()
    a[6] = a[0] + 8
    assert plan(lib, paged(), a) == api.ATTN_ERR_SHAPE
    # cached, fresh, ring, state, table, cu, lens, slots, next: an output given twice
    read_only = {0, 1, 3}
    for i, j in itertools.combinations(range(9), 2):
        if i in read_only and j in read_only:
            continue
        a = plan_args()
        a[j] = a[i]
        assert plan(lib, paged(), a) == api.ATTN_ERR_SHAPE, (i, j)


def test_store_refused(lib):
    def store(s, k=P, v=P, slots=P, kc=P, vc=P):
        return lib.attn_paged_store(None if s is None else ctypes.byref(s), k, v, slots, kc, vc,
                                    None)
    assert store(None) == api.ATTN_ERR_NULL
    for kw in BAD_PAGED + [dict(kv_heads=0), dict(dtype=3), dict(head_dim=32), dict(k_token=8),
                           dict(v_head=0), dict(kc_row=0), dict(vc_page=100)]:
        assert store(paged(**kw)) == api.ATTN_ERR_SHAPE, kw
    for name in ("k", "v", "slots", "kc", "vc"):
        assert store(paged(), **{name: None}) == api.ATTN_ERR_NULL, name
        assert store(paged(), **{name: P + 2}) == api.ATTN_ERR_ALIGN, name
    assert store(paged(tokens=0), None, None, None, None, None) == api.ATTN_OK
    # rows of a pool on top of one another
    for kw in (dict(kc_row=64, kc_head=64), dict(vc_head=512), dict(vc_page=1024),
               dict(kc_row=128, kc_head=1024, kc_page=2048)):
        assert store(paged(**kw)) == api.ATTN_ERR_SHAPE, kw
    # any order of strides that keeps them apart
    for kw in (dict(kc_row=128, kc_head=64, kc_page=2048), dict(kc_page=64, kc_head=3200, kc_row=6400),
               dict(vc_row=72, vc_head=1160, vc_page=2400)):
        assert store(paged(**kw), slots=None) == api.ATTN_ERR_NULL, kw


def test_error_string(lib):
    assert "outside its range" in api.error_string(api.ATTN_ERR_DEVICE_INDEX)


def test_python_binding_refuses_cpu_tensors_and_types():
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    s = api.PackedShape(4, 1, 2, 1)
    with pytest.raises(ValueError):
        api.attn_packed_fwd(s, h(4, 2, 64), h(4, 1, 64), h(4, 1, 64), i(2), h(4, 2, 64))
    with pytest.raises(TypeError):
        api.attn_packed_fwd(s, h(4, 2, 64).float(), h(4, 1, 64), h(4, 1, 64), i(2), h(4, 2, 64))
    with pytest.raises(TypeError):
        api.attn_packed_fwd(s, None, h(4, 1, 64), h(4, 1, 64), i(2), h(4, 2, 64))
    with pytest.raises(TypeError):
        api.PagedShape(1, 1, 1, 1, 16, 4, 4, dtype=torch.float32).c_bytes()
    with pytest.raises(api.AttnError):
        api.paged_workspace_bytes(api.PagedShape(1, 1, 3, 2, 16, 4, 4))
    p = api.PagedShape(2, 4, 2, 1, 16, 4, 4)
    with pytest.raises(ValueError):
        api.attn_paged_plan(p, i(2), i(2), i(4), i(4), i(2, 4), i(3), i(2), i(4), i(4))


# ------------------------------------------------------------ index arithmetic
HARNESS = r"""
#include <stdio.h>
#include "serve_index.h"
using namespace css;
int main() {
  int what;
  while (scanf("%d", &what) == 1) {
    if (what == 0) {
      int a, b, t; scanf("%d %d %d", &a, &b, &t);
      RowRange r = row_range(a, b, t);
      printf("%d %d %d\n", r.begin, r.end, (int)r.bad);
    } else if (what == 1) {
      int n, x; static int32_t cu[1000]; scanf("%d %d", &n, &x);
      for (int i = 0; i < n; ++i) scanf("%d", &cu[i]);
      printf("%d\n", last_at_or_below(cu, n, x));
    } else if (what == 2) {
      int len, w, s; bool bad; scanf("%d %d %d", &len, &w, &s);
      int k = key_count(len, w, s, &bad);
      printf("%d %d\n", k, (int)bad);
    } else if (what == 3) {
      int h, n; long long x; scanf("%d %lld %d", &h, &x, &n);
      printf("%d\n", ring_at(h, x, n));
    } else if (what == 4) {
      int c, f, w, s; scanf("%d %d %d %d", &c, &f, &w, &s);
      PlanRow r = plan_row(c, f, w, s);
      printf("%lld %lld %lld %lld %d\n", r.add, r.have, r.need, r.back, r.status);
    } else if (what == 6) {
      long long t; int m, g, b; scanf("%lld %d %d %d", &t, &m, &g, &b);
      Share s = share_of(t, m, g, b);
      printf("%lld %lld %d\n", s.begin, s.end, s.blocks);
    } else if (what == 7) {
      long long t, x; int m, g; scanf("%lld %d %d %lld", &t, &m, &g, &x);
      Share s = share_of(t, m, g, 0);
      printf("%d\n", last_block(s, x));
    } else if (what == 8) {
      int k, n, w, bn, nb; scanf("%d %d %d %d %d", &k, &n, &w, &bn, &nb);
      printf("%lld %d\n", tiles_before(k, n, w, bn, nb), tiles_of_block(k, n, w, bn, nb));
    } else {
      int rows, head, fr, np, tok; long long add, need, back;
      scanf("%d %lld %lld %lld %d %d %d %d", &rows, &add, &need, &back, &head, &fr, &np, &tok);
      printf("%d\n", plan_status(rows, add, need, back, head, fr, np, tok));
    }
  }
  return 0;
}
"""

EXTREMES = [-2 ** 31, -2 ** 31 + 1, -7, -1, 0, 1, 5, 99, 100, 101, 2 ** 30, 2 ** 31 - 1]


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    d = tmp_path_factory.mktemp("serve_index")
    (d / "h.cpp").write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-I", build.CSRC, "-o", str(d / "h"),
                    str(d / "h.cpp")], check=True)

    def ask(lines):
        r = subprocess.run([str(d / "h")], input="\n".join(lines), capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return [[int(x) for x in ln.split()] for ln in r.stdout.splitlines()]
    return ask


def test_row_range_stays_inside(harness):
    asks = [(a, b, t) for a in EXTREMES for b in EXTREMES for t in (0, 1, 100)]
    for (a, b, t), (begin, end, bad) in zip(asks, harness("0 %d %d %d" % x for x in asks)):
        assert 0 <= begin <= end <= t
        assert bad == (not 0 <= a <= b <= t)
        if not bad:
            assert (begin, end) == (a, b)


def test_bisection(harness):
    r = random.Random(1)
    asks = []
    for _ in range(300):
        n = r.randint(1, 40)
        cu = sorted(r.randint(0, 50) for _ in range(n))
        asks.append((cu, r.randint(-1, 60)))
    for _ in range(200):  # any contents: the answer stays in range
        asks.append(([r.choice(EXTREMES) for _ in range(r.randint(1, 40))], r.choice(EXTREMES)))
    got = harness("1 %d %d %s" % (len(c), x, " ".join(map(str, c))) for c, x in asks)
    for k, ((cu, x), (i,)) in enumerate(zip(asks, got)):
        assert -1 <= i < len(cu)
        if k < 300:
            assert i == max((j for j, c in enumerate(cu) if c <= x), default=-1)


def test_key_count_stays_in_the_table(harness):
    asks = [(n, w, s) for n in EXTREMES for w, s in ((1, 3), (7, 4), ((1 << 27) - 1, 4),
                                                     ((1 << 21) - 1, 10))]
    for (n, w, s), (k, bad) in zip(asks, harness("2 %d %d %d" % x for x in asks)):
        assert 0 <= k <= w << s
        assert bad == (not 0 <= n <= w << s)
        if not bad:
            assert k == n


def test_ring_positions(harness):
    asks = [(h, x, n) for n in (1, 2, 7) for h in range(n) for x in range(n + 1)]
    asks += [(2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31 - 1)]
    for (h, x, n), (p,) in zip(asks, harness("3 %d %d %d" % a for a in asks)):
        assert p == (h + x) % n


def test_plan_rows_and_status(harness):
    asks = [(c, f, w, s) for c in EXTREMES for f in EXTREMES for w, s in ((1, 3), (50, 4),
                                                                          ((1 << 27) - 1, 4))]
    up = lambda x, s: (x + (1 << s) - 1) >> s
    for (c, f, w, s), (add, have, need, back, st) in zip(
            asks, harness("4 %d %d %d %d" % a for a in asks)):
        cc = max(c, 0)
        assert add == max(f, 0) and have == up(cc, s)
        assert need == (up(cc + f, s) - have if f >= 0 else 0) and need >= 0
        assert back == (have if f < 0 else 0)
        assert st == (8 if c < 0 else 0) + (2 if up(cc + max(f, 0), s) > w else 0)
    big = 4096 * (2 ** 31 - 1)
    cases = [((0, 5, 2, 0, 0, 2, 10, 5), 0), ((0, 5, 3, 0, 0, 2, 10, 5), 1),
             ((0, 6, 2, 0, 0, 2, 10, 5), 4), ((2, 5, 2, 0, 0, 2, 10, 5), 2),
             ((0, 5, 2, 0, -1, 2, 10, 5), 8), ((0, 5, 2, 0, 10, 2, 10, 5), 8),
             ((0, 5, 2, 0, 0, 11, 10, 5), 8), ((0, 5, 0, 9, 0, 2, 10, 5), 8),
             ((0, 5, 2, 8, 0, 2, 10, 5), 0), ((8, big, big, big, 5, 2, 10, 5), 13)]
    got = harness("5 %s" % " ".join(map(str, a)) for a, _ in cases)
    assert [g[0] for g in got] == [w for _, w in cases]


def test_shares_partition_the_list(harness):
    r = random.Random(5)
    for total in (0, 1, 3, 4, 5, 1000, 12345, 2 ** 31 - 1, 2 ** 33 + 7, 2 ** 52 + 12345):
        for least, grid in ((1, 1), (4, 304), (2, 152), (8, 3)):
            got = harness("6 %d %d %d %d" % (total, least, grid, b) for b in range(grid))
            at = 0
            for b, (begin, end, blocks) in enumerate(got):
                assert 1 <= blocks <= grid and (blocks == 1 or blocks * least <= total)
                if b < blocks:
                    assert begin == at and end >= begin
                    assert end - begin - total // blocks in (0, 1)
                    at = end
                else:
                    assert begin == end == total
            assert at == total
            if total:
                xs = [0, total - 1] + [r.randrange(total) for _ in range(20)]
                xs += [g[0] for g in got if g[0] < total] + [g[1] - 1 for g in got if g[1] > g[0]]
                ans = harness("7 %d %d %d %d" % (total, least, grid, x) for x in xs)
                for x, (b,) in zip(xs, ans):
                    assert got[b][0] <= x < got[b][1], (total, least, grid, x, b)


def test_tiles_of_row_blocks(harness):
    r = random.Random(6)
    asks, want = [], []
    for _ in range(3000):
        n = r.randint(1, 900)
        k = r.choice([r.randint(0, 3000), r.randint(0, n), n, 0, 2 ** 31 - 1])
        w, bn = 3 * (128 // r.randint(1, 128)), r.choice([64, 128])
        blocks = -(-n // w)
        ends = [k - n + min(n, (b + 1) * w) for b in range(blocks)]
        tiles = [1 if e <= 0 else -(-e // bn) for e in ends]
        nb = r.choice([0, 1, blocks // 2, blocks - 1])
        if nb >= blocks:
            continue
        asks.append("8 %d %d %d %d %d" % (k, n, w, bn, nb))
        want.append([sum(tiles[:nb]), tiles[nb]])
        asks.append("8 %d %d %d %d %d" % (k, n, w, bn, blocks))
        want.append([sum(tiles), None])
    for a, g, x in zip(asks, harness(asks), want):
        assert g[0] == x[0] and x[1] in (None, g[1]), a


def test_host_form_of_the_plan():
    """The plan's plain form: pages are handed out once, come back, and every
    slot is the place its table names."""
    r = random.Random(3)
    page, width, N, B = 8, 6, 40, 7
    ring, state = list(range(N)), [0, N, 0, 0]
    table, lens = [[-1] * width for _ in range(B)], [0] * B
    for _ in range(200):
        fresh = [r.choice([-1, 0, 1, 1, 1, r.randint(0, 12)]) for _ in range(B)]
        cu, new, slots, ring, table, nxt = serve_util.plan_host(lens, fresh, ring, state, table,
                                                                60, page, width)
        if nxt[3]:
            assert new == lens and set(slots) == {-1}
            fresh = [-1] * B
            cu, new, slots, ring, table, nxt = serve_util.plan_host(lens, fresh, ring, state,
                                                                    table, 60, page, width)
            assert nxt[3] == 0
        lens, state = new, nxt
        held = [table[i][x] for i in range(B) for x in range(-(-lens[i] // page))]
        free = [ring[(state[0] + x) % N] for x in range(state[1])]
        assert sorted(held + free) == list(range(N))
        live = [s for s in slots if s >= 0]
        assert len(set(live)) == len(live) == cu[-1]


def test_step_rows_are_checked_ahead():
    """A cache step looks at strides, alignment and overlap before its first launch."""
    f16 = torch.float16
    room = torch.empty(10 * 4 * 72 + 8, dtype=f16)

    def look(shape, strides, at=0, written=False):
        api._step_rows(room.as_strided(shape, strides, at), "x", f16, shape, -1, written)

    look((10, 4, 64), (256, 64, 1))
    look((10, 4, 64), (64, 640, 1), written=True)          # head-major
    look((10, 4, 64), (64, 72, 1))                         # rows that overlap may be read
    look((1, 1, 64), (3, 5, 1), written=True)              # strides of ones are not read
    look((10, 1, 64), (64, 0, 1), 8, written=True)
    look((0, 4, 64), (256, 64, 1), written=True)
    for bad in (((10, 4, 64), (0, 64, 1)), ((10, 4, 64), (256, 0, 1)), ((10, 4, 64), (256, 66, 1)),
                ((10, 4, 64), (256, 56, 1)), ((10, 4, 64), (256, 64, 1), 4),
                ((10, 4, 64), (64, 72, 1), 0, True)):
        with pytest.raises(ValueError):
            look(*bad)


LIMITS = r"""
#include <stdio.h>
#include "serve_index.h"
using namespace css;
int main() {
  int what;
  while (scanf("%d", &what) == 1) {
    if (what == 0) {
      int k, n, tok; scanf("%d %d %d", &k, &n, &tok);
      printf("%d\n", row_limit(k, n, tok));
    } else {
      int k0, n, lim; scanf("%d %d %d", &k0, &n, &lim);
      printf("%d\n", (int)past_limit(k0, n, lim));
    }
  }
  return 0;
}
"""


def test_row_limits_at_the_longest_lengths(tmp_path):
    """Which keys a row sees, and whether a run of keys passes that, without
    leaving 32 bits at the most keys a table may hold (2^28 - 1 pages of 8)."""
    (tmp_path / "h.cpp").write_text(LIMITS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-I", build.CSRC, "-o", str(tmp_path / "h"),
                    str(tmp_path / "h.cpp")], check=True)
    most = 8 * (2 ** 28 - 1)
    lens = [0, 1, 2, 15, 16, 63, 64, 65, 1000, most - 70, most - 17, most - 16, most - 1, most]
    asks, want = [], []
    for k in lens:
        for n in (1, 2, 16, 2 ** 30):
            for tok in {0, 1, 15, min(n - 1, 383)}:  # rows past the last one too
                asks.append("0 %d %d %d" % (k, n, tok))
                want.append(min(k, k - n + 1 + tok))
        for k0 in {0, 16, max(0, k - 1) // 16 * 16, max(0, k - 1) // 64 * 64, max(0, k - 1) // 64 * 64 + 48}:
            if k0 < 2 ** 31:
                for n in (16, 64):
                    for lim in (k, k - 15, k - 383):
                        asks.append("1 %d %d %d" % (k0, n, lim))
                        want.append(int(k0 + n > lim))
    r = subprocess.run([str(tmp_path / "h")], input="\n".join(asks), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert [int(x) for x in r.stdout.split()] == want


PARTS = r"""
#include <stdio.h>
#include "serve_index.h"
using namespace css;
int main() {
  int a[10];
  for (;;) {
    for (int i = 0; i < 10; ++i)
      if (scanf("%d", &a[i]) != 1) return 0;
    printf("%d\n", (int)part_ok(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9]));
  }
}
"""


def test_descriptions_of_parts_are_checked(tmp_path):
    """Whatever a workspace holds, a part that passes names rows of the output
    and parts of the workspace."""
    (tmp_path / "h.cpp").write_text(PARTS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-I", build.CSRC, "-o", str(tmp_path / "h"),
                    str(tmp_path / "h.cpp")], check=True)
    r = random.Random(7)
    asks, want = [], []
    for _ in range(4000):
        blocks, room, hkv, g = r.choice([1, 152, 304]), r.choice([16, 384]), r.randint(1, 9), \
            r.choice([1, 3, 4, 17, 128])
        c, tokens = r.randrange(blocks), r.choice([1, 5, 100, 2 ** 30])
        near = lambda *x: r.choice(EXTREMES + [y + z for y in x for z in (-1, 0, 1)])
        q0, kv, rows, last = near(0, tokens), near(0, hkv), near(0, room, g), near(c, blocks)
        if r.random() < 0.5:
            kv, last = r.randrange(hkv), r.randrange(c, blocks)
        asks.append((q0, kv, rows, last, c, blocks, room, tokens, hkv, g))
        ok = 0 <= kv < hkv and 0 <= rows <= room and c <= last < blocks and q0 >= 0
        ok = ok and all(q0 + x // g < tokens for x in range(rows)) and q0 <= tokens
        want.append(int(ok))
    got = subprocess.run([str(tmp_path / "h")], input="\n".join(
        " ".join(map(str, a)) for a in asks), capture_output=True, text=True)
    assert got.returncode == 0, got.stderr
    assert [int(x) for x in got.stdout.split()] == want
    assert 100 < sum(want) < 3900


def test_step_refuses_a_stream_of_another_device():
    """It would run on the current stream of the cache's own device instead."""
    class Stream:
        device_index = 3

    cache = api.PagedCache.__new__(api.PagedCache)  # a cache without a GPU: its device is -1
    cache.k = torch.zeros(1)
    with pytest.raises(ValueError, match="another device"):
        cache.step(None, None, None, None, None, stream=Stream())


def test_the_marshaller_is_built_for_one_pytorch(lib, monkeypatch):
    """One made for another PyTorch or Python is made again, whatever the
    files' times say, and is not bound."""
    assert build.marshal_up_to_date()
    key = build.marshal_key()
    assert api._native.built_for == key
    for part in (torch.__version__, str(torch.version.cuda), torch.version.git_version):
        assert part in key
    with monkeypatch.context() as m:
        m.setattr(build, "marshal_key", lambda *a: key.replace("torch ", "torch 1"))
        assert not build.marshal_up_to_date()
        m.setattr(api, "_native", None)
        with pytest.raises(ImportError, match="built for"):
            api._bind_native(lib)
        assert api._native is None
    assert build.marshal_up_to_date()


def test_the_library_does_not_need_the_marshaller(lib, monkeypatch):
    """Without it, or with one of another PyTorch, the library loads, says so
    once, and every call goes through api's own checks."""
    name = api.__package__ + "._marshal"
    for how in (lambda m: m.setitem(sys.modules, name, None),
                lambda m: m.setattr(build, "marshal_key", lambda *a: "another")):
        with monkeypatch.context() as m:
            m.setattr(api, "_lib", None)
            m.setattr(api, "_native", None)
            how(m)
            with pytest.warns(RuntimeWarning, match="_marshal.so"):
                assert api.load_library() is not None
            assert api._native is None and api.load_library() is api._lib
            assert api.paged_workspace_bytes(api.PagedShape(1, 1, 4, 2, 16, 4, 4)) > 0
            i = lambda *s: torch.zeros(*s, dtype=torch.int32)
            with pytest.raises(ValueError, match="CUDA tensors"):
                api.attn_paged_plan(api.PagedShape(2, 4, 2, 1, 16, 4, 4), i(2), i(2), i(4), i(4),
                                    i(2, 4), i(3), i(2), i(4), i(4))


def test_build_leaves_out_a_marshaller_that_cannot_be_built(lib, monkeypatch, tmp_path):
    """A PyTorch without CUDA, or none, does not stop the library's build."""
    assert build.marshal_missing() is None
    with monkeypatch.context() as m:
        m.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
        m.setattr(build, "MARSHAL_KEY", str(tmp_path / "marshal.key"))
        m.setattr(build, "_torch", lambda: str(tmp_path))
        assert build.marshal_missing() == "a PyTorch with CUDA"
        assert build.build() == build.LIB and not os.path.exists(build.MARSHAL)
        m.setattr(build.importlib.util, "find_spec", lambda n: None)
        assert build.marshal_missing() == "PyTorch"
        assert build.build() == build.LIB and not os.path.exists(build.MARSHAL)
