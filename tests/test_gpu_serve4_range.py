"""Attention over a 4-bit cache whose magnitudes differ: by channel group, by key, and
behind the mask.  A row's bound knows the keys that the row sees and no others."""
import random

import pytest

from serve4_range_util import own64, problem
from serve4_util import put
from serve_util import check

pytestmark = pytest.mark.gpu

SENTINEL = 7.0


@pytest.fixture(scope="module")
def torch(cuda_device):
    import torch
    from causal_streaming_softmax_gb300 import build
    build.build()
    return torch


@pytest.fixture(autouse=True)
def no_device_error(cuda_device):
    from causal_streaming_softmax_gb300 import api
    yield
    assert api.last_device_error() == 0


def run(torch, p, max_new=None, scale=0.125):
    from causal_streaming_softmax_gb300 import api
    q, kc, vc, table, cu, lens = p
    t, H, _ = q.shape
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    s = api.PagedShape(len(lens), t, H, kc.shape[1], kc.shape[2] * 8, kc.shape[0], len(table[0]),
                       max_new=max_new or max(b - a for a, b in zip(cu, cu[1:])), dtype=q.dtype,
                       scale=scale)
    ws = api.alloc_paged_workspace(s)
    ws.fill_(255)
    o = torch.full_like(q, SENTINEL)
    lse = torch.full((H, t), SENTINEL, device="cuda")
    api.attn_paged_fwd4(s, q, kc, vc, i32(table), i32(cu), i32(lens), ws, o, lse)
    return o, lse


def run_and_check(torch, p, max_new=None, scale=0.125):
    o, lse = run(torch, p, max_new, scale)
    for rows, eo, el, to, tl in own64(*p, scale):
        check(o[rows], eo, to, "O of rows %s" % rows)
        check(lse[:, rows], el, tl, "L of rows %s" % rows)
    return o, lse


# The launches of the call: requests (keys, new tokens), heads, page, max_new.
FORMS = {
    "whole": ([(777, 1), (130, 1)], (8, 2), 16, None),
    "whole_wide": ([(700, 2), (90, 1)], (8, 1), 16, None),
    "split": ([(3000, 1), (1500, 1)], (8, 2), 64, None),
    "split_wide": ([(2600, 4), (64, 1), (1029, 3)], (8, 2), 32, None),
    "sub_items": ([(2600, 4), (900, 1), (300, 40)], (8, 2), 16, None),
    "one_head": ([(5000, 1)], (2, 2), 128, None),
    "tiles": ([(500, 70), (64, 64)], (8, 2), 16, None),
}


def shapes(kind, span):
    """What V's magnitudes are: 2^-span/2 .. 2^span/2 by channel, key or block."""
    import torch
    half = span // 2

    def scatter(n, seed, values):
        r = random.Random(seed)
        return torch.tensor([2.0 ** r.choice(values) for _ in range(n)], device="cuda",
                            dtype=torch.float64)[:, None, None]

    def by_key(f):
        def shape(i, x):
            n = x.shape[0]
            x *= f(i, n)
        return shape

    pos = lambda n: torch.arange(n, device="cuda", dtype=torch.float64) / max(1, n - 1)
    up = lambda i, n: (2.0 ** (span * pos(n) - half))[:, None, None]
    down = lambda i, n: (2.0 ** (half - span * pos(n)))[:, None, None]

    def low_channels(i, x):
        x[..., :32] *= 2.0 ** -half
        x[..., 32:] *= 2.0 ** half

    def high_channels(i, x):
        x[..., :32] *= 2.0 ** half
        x[..., 32:] *= 2.0 ** -half

    def one_channel(i, x):  # an outlier of one channel in every sixth key
        x *= 2.0 ** -half
        x[::6, :, 5] = 2.0 ** half

    def zeros(i, x):
        x[1::2] = 0
        x[::5, :, 32:] = 0
        x *= 2.0 ** -half

    return {
        "low_channels": low_channels, "high_channels": high_channels, "one_channel": one_channel,
        "rising": by_key(up), "falling": by_key(down), "zeros": zeros,
        "steps": by_key(lambda i, n: (2.0 ** ((torch.arange(n, device="cuda") // 70 % 5) *
                                              (span / 4.0) - half))[:, None, None]),
        "scatter": by_key(lambda i, n: scatter(n, i, range(-half, half + 1))),
        "few_large": by_key(lambda i, n: scatter(n, i, [-half] * 40 + [half])),
        "few_small": by_key(lambda i, n: scatter(n, i, [half] * 40 + [-half])),
    }[kind]


KINDS = ["low_channels", "high_channels", "one_channel", "rising", "falling", "zeros", "steps",
         "scatter", "few_large", "few_small"]
SPANS = {"float16": (6, 26), "bfloat16": (8, 40, 90)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,span", [(d, s) for d in SPANS for s in SPANS[d]])
def test_values_of_mixed_magnitudes(torch, form, kind, dtype, span):
    reqs, heads, page, max_new = FORMS[form]
    p = problem(reqs, *heads, page, getattr(torch, dtype), 7 + span, shape_v=shapes(kind, span))
    o, _ = run_and_check(torch, p, max_new)
    o2, _ = run(torch, p, max_new)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,span", [("float16", 26), ("bfloat16", 40), ("bfloat16", 90)])
def test_large_values_of_keys_that_hardly_count(torch, form, dtype, span):
    """Keys with weights of some 2^-58 and V far above the others': neither do the others
    disappear, nor does what such a key adds where it is comparable."""
    reqs, heads, page, max_new = FORMS[form]

    def away(i, x):
        x[3::29] = 0
        x[3::29, :, 0] = -40

    def large(i, x):
        x *= 2.0 ** -(span // 2)
        x[3::29] *= 2.0 ** span

    def ask(q):
        q[..., 0] = 8

    run_and_check(torch, problem(reqs, *heads, page, getattr(torch, dtype), 3, away, large, ask),
                  max_new)


@pytest.mark.parametrize("dtype,span", [("float16", 13), ("float16", 26), ("bfloat16", 14),
                                        ("bfloat16", 40), ("bfloat16", 90), ("bfloat16", 160)])
@pytest.mark.parametrize("heads,new,keys,other", [
    ((8, 2), 4, 700, 1), ((8, 2), 2, 64 * 9 + 1, 1), ((8, 1), 2, 3000, 1), ((2, 2), 16, 400, 1),
    ((8, 2), 4, 4, 1), ((2, 2), 16, 16, 1), ((8, 2), 4, 2000, 40), ((8, 2), 40, 300, 1)])
def test_values_behind_the_mask(torch, dtype, span, heads, new, keys, other):
    """The later tokens' V is far larger: earlier rows are what they are without it."""
    dt, half = getattr(torch, dtype), span // 2
    reqs = [(keys, new), (other + 50, other)]

    def values(later):
        def shape(i, x):
            x *= 2.0 ** -half
            if i == 0 and later:
                x[keys - new // 2:] *= 2.0 ** span
        return shape

    p = problem(reqs, *heads, 16, dt, 11, shape_v=values(True))
    o, L = run(torch, p)
    before = new - new // 2
    for rows, eo, el, to, tl in own64(*p):
        a, b = rows.start, rows.start + before if rows.start == 0 else rows.stop
        check(o[a:b], eo[:b - a], to[:b - a], "O")
        if span < 100:
            check(o[rows], eo, to, "O of all rows")
        check(L[:, rows], el, tl, "L")
    plain, L2 = run(torch, problem(reqs, *heads, 16, dt, 11, shape_v=values(False)))
    off = (o[:before].double() - plain[:before].double()).abs()
    assert bool((off <= 2 * own64(*p)[0][3][:before]).all())


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("at", [1, 64, 65, 255, 256, 600, 2000])
def test_one_large_value_anywhere(torch, dtype, at):
    """One key of one request, in either group, among ordinary ones; V's unit moves while
    the sums of the keys before it are there, and not back."""
    e = 12 if dtype == "float16" else 40

    def shape(i, x):
        x[max(0, x.shape[0] - at - i), 0, 32 * (i % 2) + 3] = 2.0 ** e * (-1) ** i

    reqs = [(2100, 1), (2100, 2), (2164, 1), (2000 + at, 1)]
    run_and_check(torch, problem(reqs, 8, 2, 16, getattr(torch, dtype), at, shape_v=shape))


# dtype, binary orders between q's channel groups (K has them the other way round)
APART = [("float16", 8), ("float16", 13), ("float16", 22), ("bfloat16", 12), ("bfloat16", 14),
         ("bfloat16", 36), ("bfloat16", 80), ("bfloat16", 160)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,span", APART)
def test_queries_whose_groups_lie_apart(torch, form, dtype, span):
    """Either group of q is far below the other where K's is far above: both count.
    Every third row is small as a whole."""
    reqs, heads, page, max_new = FORMS[form]
    low = span // 2 if heads[0] != 2 else -(span // 2)

    def keys(i, x):
        x[..., :32] *= 2.0 ** low
        x[..., 32:] *= 2.0 ** -low

    def ask(q):
        q[..., :32] *= 2.0 ** -low
        q[..., 32:] *= 2.0 ** low
        q[::3] *= 2.0 ** -9

    run_and_check(torch, problem(reqs, *heads, page, getattr(torch, dtype), span, keys, None, ask),
                  max_new)


# dtype, log2 of q, of K and of the scale: of scores of ordinary size
FAR = [("float16", 12, -10, -5), ("float16", -12, 10, -1), ("bfloat16", 60, -117, 54),
       ("bfloat16", 110, -110, -3), ("bfloat16", 120, -120, -3), ("bfloat16", 126, -124, -3),
       ("bfloat16", -110, 110, -3), ("bfloat16", -125, 120, 2), ("bfloat16", 3, 100, -106),
       ("bfloat16", 20, 100, -123), ("bfloat16", -60, -60, 117), ("bfloat16", 100, 20, -123),
       ("bfloat16", -100, 20, 77), ("bfloat16", 0, -120, 117)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,qe,ke,se", FAR)
def test_queries_and_scales_far_from_one(torch, form, dtype, qe, ke, se):
    reqs, heads, page, max_new = FORMS[form]

    def keys(i, x):
        x *= 2.0 ** ke

    def ask(q):
        q *= 2.0 ** (qe - 1)
        q[::2, 1::2] = 0  # beside rows of zeros

    run_and_check(torch, problem(reqs, *heads, page, getattr(torch, dtype), 50 + se, keys, None,
                                 ask), max_new, 2.0 ** se)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("scale", [1e-15, 1e-20, 1e-30, 1.2e-38, 1e-42])
@pytest.mark.parametrize("form", ["whole", "whole_wide", "split_wide", "sub_items", "tiles"])
def test_rows_of_zeros_under_small_scales(torch, dtype, scale, form):
    """Such a row is the mean of the values that it sees, the masked ones left out."""
    reqs, heads, page, max_new = FORMS[form]

    def ask(q):
        q[:, ::2] = 0

    import struct
    scale = struct.unpack("f", struct.pack("f", scale))[0]
    run_and_check(torch, problem(reqs, *heads, page, getattr(torch, dtype), 9, shape_q=ask),
                  max_new, scale)


@pytest.mark.parametrize("form", ["whole_wide", "split_wide", "sub_items"])
def test_rows_that_are_not_finite_beside_rows_far_apart(torch, form):
    """An infinity or a NaN in q spoils its own row alone, whatever the others ask for."""
    reqs, heads, page, max_new = FORMS[form]

    def ask(q):
        q[0, 1, :32] *= 2.0 ** -70

    p = problem(reqs, *heads, page, torch.bfloat16, 4, shape_q=ask)
    q = p[0]
    good, _ = run(torch, p, max_new)
    q[0, 0, 3], q[1, 2, 40], q[1, 3, 63] = float("inf"), float("nan"), -float("inf")
    o, L = run(torch, p, max_new)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[1, 2] = bad[1, 3] = True
    assert torch.isnan(o[bad]).all()
    assert torch.equal(o[~bad].view(torch.int16), good[~bad].view(torch.int16))
    q[bad] = 1.0
    for rows, eo, el, to, tl in own64(*p):
        fine = ~bad[rows]
        check(o[rows][fine], eo[fine], to[fine], "O")
        check(L[:, rows].T[fine], el.T[fine], tl.T[fine], "L")


@pytest.mark.parametrize("heads,max_new", [((8, 2), None), ((2, 2), None), ((8, 1), None),
                                           ((8, 2), 40)])
@pytest.mark.parametrize("scale", [0.125, 1e-30])
def test_rows_that_see_nothing_beside_extremes(torch, heads, max_new, scale):
    """Fewer keys than new tokens: the first rows are zero and -infinity whatever the
    others' q, K and V ask for."""
    reqs = [(0, 1), (1, 2), (1, 1), (2, 2), (700, 2), (0, 2), (65, 2)]
    dt = torch.bfloat16

    def ask(q):
        q[::2, :, :32] *= 2.0 ** -60
        q[1::2, ::2] = 0

    p = problem(reqs, *heads, 8, dt, 23, None, shapes("scatter", 80), ask)
    o, L = run_and_check(torch, p, max_new, scale)
    assert (o[0] == 0).all() and torch.isneginf(L[:, 0]).all()
    assert (o[1] == 0).all() and torch.isneginf(L[:, 1]).all()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("form,new", [("whole_wide", 2), ("split_wide", 4), ("tiles", 70)])
def test_any_bytes_behind_the_mask(torch, dtype, form, new):
    """The last new token's rows of K and V hold any bytes: infinite, NaN, largest and
    smallest scales among them.  The rows before it are what they were."""
    reqs, heads, page, max_new = FORMS[form]
    q, kc, vc, table, cu, lens = problem(reqs, *heads, page, getattr(torch, dtype), 6)
    want = own64(q, kc, vc, table, cu, lens)[0]
    at = lens[0] - 1
    where = [torch.tensor([x]) for x in (table[0][at // page], at % page)]
    g = torch.Generator().manual_seed(2)
    for rep in range(12):
        for pool in (kc, vc):
            rows = torch.randint(0, 256, (1, heads[1], 36), generator=g, dtype=torch.uint8)
            if rep < 6:  # scales of every exponent: infinities, NaN, the largest, the smallest
                rows[..., 33::2] = [0x7c, 0xfc, 0x7f, 0x7b, 0x00, 0x80][rep]
            put(pool, *where, rows.cuda())
        o, L = run(torch, (q, kc, vc, table, cu, lens), max_new)
        check(o[:new - 1], want[1][:-1], want[3][:-1], "O, %d" % rep)
        check(L[:, :new - 1], want[2][:, :-1], want[4][:, :-1], "L, %d" % rep)
