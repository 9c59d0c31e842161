"""The rotated append, the 4-bit cache and attention over it on the GPU: rows bit
for bit, attention against 64 bits."""
import math
import random

import pytest

from serve4_util import (attend4, gather, pack, paged4_64, pool_of, put, quantise, rotate,
                         row_bytes, values)
from serve_util import attend64, check

pytestmark = pytest.mark.gpu

NAN = float("nan")
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


def scan(xs):
    out = [0]
    for x in xs:
        out.append(out[-1] + x)
    return out


def i32(torch, xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def rnd(torch, shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def angles(torch, n):
    x = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32)
    return x.cos().float(), x.sin().float()


def same(a, b, what=""):
    """Bit for bit, of 16-bit or byte tensors."""
    import torch
    if a.dtype != torch.uint8:
        a, b = a.contiguous().view(torch.int16), b.contiguous().view(torch.int16)
    assert a.shape == b.shape and torch.equal(a, b), \
        "%s: %d differ, first at %s" % (what, int((a != b).sum()),
                                        (a != b).nonzero()[:3].tolist())


def bytes_pool(torch, pages, heads, page, seed):
    """A pool of any bytes, to see that the others stay as they are."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 256, (pages, heads, page // 8, 288), generator=g, device="cuda",
                         dtype=torch.uint8)


# ---------------------------------------------------------------------- append
def append_problem(torch, reqs, H, Hkv, page, dtype, seed, pad=0, layout="fused"):
    """reqs: (tokens in the cache before, new ones; -1 new: finished)."""
    r = random.Random(seed)
    new = [max(0, n) for _, n in reqs]
    cu, t = scan(new), sum(new) + pad
    pages = -(-t // page) + 4
    order = r.sample(range(pages * page), t)
    slots = order[:sum(new)] + [-1] * pad
    for i in range(0, sum(new), 11):
        if i % 2:
            slots[i] = -1
    lens = [c + n if n >= 0 else 0 for c, n in reqs]
    if layout == "fused":
        x = rnd(torch, (t, H + 2 * Hkv, 64), dtype, seed)
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    else:
        q, k, v = (rnd(torch, (h, t, 64), dtype, seed + i).permute(1, 0, 2)
                   for i, h in enumerate((H, Hkv, Hkv)))
    return q, k, v, slots, cu, lens, pages


def positions(cu, lens):
    return [m - (b - a) + i for (a, b), m in zip(zip(cu, cu[1:]), lens) for i in range(b - a)]


APPENDS = [[(0, 1)], [(776, 1)], [(3, 0), (0, 1), (9, -1), (0, 3)], [(5, 40), (0, 1), (100, 7)],
           [(i, 1 + i % 3) for i in range(40)], [(7, 1)] * 33, [(2 * i, i % 4) for i in range(300)],
           [(0, 700)], [(50, -1), (60, 0), (1000, 65)]]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads", [(2, 1), (4, 4), (15, 5), (32, 8), (128, 1)])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(torch, dtype, heads, case):
    from causal_streaming_softmax_gb300 import api
    (H, Hkv), dt = heads, getattr(torch, dtype)
    page = [8, 16, 64, 1024][(case + H) % 4]
    q, k, v, slots, cu, lens, pages = append_problem(
        torch, APPENDS[case], H, Hkv, page, dt, 10 * case + H, case % 3 * 2,
        ["fused", "planes"][case % 2])
    t = q.shape[0]
    cos, sin = angles(torch, max(max(lens), 1))
    kc, vc = (rnd(torch, (pages, Hkv, page, 64), dt, 5 + i) for i in range(2))
    if case % 2:  # [page][row][head]
        kc, vc = (x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (kc, vc))
    want_k, want_v, want_q = kc.clone(), vc.clone(), torch.full((t, H, 64), SENTINEL,
                                                               dtype=dt, device="cuda")
    rows = torch.tensor([i for i in range(cu[-1]) if slots[i] >= 0], device="cuda",
                        dtype=torch.int64)
    pos = torch.tensor(positions(cu, lens), device="cuda", dtype=torch.int64)[rows]
    at = torch.tensor(slots, device="cuda")[rows]
    want_q[rows] = rotate(q[rows], cos[pos], sin[pos]).to(dt)
    want_k[at // page, :, at % page] = rotate(k[rows], cos[pos], sin[pos]).to(dt)
    want_v[at // page, :, at % page] = v[rows]
    out = torch.full((H, t, 64), SENTINEL, dtype=dt, device="cuda").permute(1, 0, 2) \
        if case % 2 else torch.full((t, H + 1, 72), SENTINEL, dtype=dt, device="cuda")[:, :H, :64]
    s = api.PagedShape(len(lens), t, H, Hkv, page, pages, 1, dtype=dt)
    api.attn_paged_append(s, q, k, v, cos, sin, i32(torch, slots), i32(torch, cu),
                          i32(torch, lens), out, kc, vc)
    same(out, want_q, "q")
    same(kc, want_k, "K")
    same(vc, want_v, "V")
    # in place: q's own rows
    kc.zero_()
    q0, mine = q.clone(), q.clone(memory_format=torch.preserve_format)
    api.attn_paged_append(s, mine, k, v, cos, sin, i32(torch, slots), i32(torch, cu),
                          i32(torch, lens), mine, kc, vc)
    q0[rows] = want_q[rows]
    same(mine, q0, "q in place")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads", [(2, 1), (15, 5), (32, 8), (16, 16)])
@pytest.mark.parametrize("turn", [True, False])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append4(torch, dtype, heads, turn, case):
    from causal_streaming_softmax_gb300 import api
    (H, Hkv), dt = heads, getattr(torch, dtype)
    page = [8, 16, 64, 1024][(case + H) % 4]
    q, k, v, slots, cu, lens, pages = append_problem(
        torch, APPENDS[case], H, Hkv, page, dt, 10 * case + H, case % 3 * 2,
        ["fused", "planes"][case % 2])
    t = q.shape[0]
    cos, sin = angles(torch, max(max(lens), 1))
    kc, vc = (bytes_pool(torch, pages, Hkv, page, 9 + i) for i in range(2))
    if case % 2:  # K and V of a page side by side
        both = torch.stack([kc, vc], 1)
        kc, vc = both[:, 0], both[:, 1]
    want_k, want_v = row_bytes(kc), row_bytes(vc)
    rows = torch.tensor([i for i in range(cu[-1]) if slots[i] >= 0], device="cuda",
                        dtype=torch.int64)
    pos = torch.tensor(positions(cu, lens), device="cuda", dtype=torch.int64)[rows]
    at = torch.tensor(slots, device="cuda")[rows]
    turned = rotate(k[rows], cos[pos], sin[pos]) if turn else k[rows].float()
    want_k[at // page, :, at % page] = pack(*quantise(turned, dt))
    want_v[at // page, :, at % page] = pack(*quantise(v[rows].float(), dt))
    s = api.PagedShape(len(lens), t, H, Hkv, page, pages, 1, dtype=dt)
    if turn:
        out = torch.full((t, H, 64), SENTINEL, dtype=dt, device="cuda")
        api.attn_paged_append4(s, q, k, v, cos, sin, i32(torch, slots), i32(torch, cu),
                               i32(torch, lens), out, kc, vc)
        want_q = torch.full_like(out, SENTINEL)
        want_q[rows] = rotate(q[rows], cos[pos], sin[pos]).to(dt)
        same(out, want_q, "q")
    else:
        api.attn_paged_append4(s, None, k, v, None, None, i32(torch, slots), None, None, None, kc,
                               vc)
    same(row_bytes(kc), want_k, "K")
    same(row_bytes(vc), want_v, "V")
    # and back
    if t == 0:
        return
    ko, vo = (torch.full((t, Hkv, 64), SENTINEL, dtype=dt, device="cuda") for _ in range(2))
    api.attn_paged_load4(s, i32(torch, slots), kc, vc, ko, vo)
    for got, pool in ((ko, kc), (vo, vc)):
        want = torch.full_like(got, SENTINEL)
        want[rows] = values(pool, dt)[0][at // page, :, at % page].to(dt)
        same(got, want, "read back")


@pytest.mark.parametrize("bits,turn", [(16, True), (4, True), (4, False)])
def test_append_and_load_of_many_tokens(torch, bits, turn):
    """So many that a thread takes several rows; an odd number of eights of rows."""
    from causal_streaming_softmax_gb300 import api
    H = Hkv = 17
    dt, page = torch.bfloat16, 64
    q, k, v, slots, cu, lens, pages = append_problem(torch, [(7, 11000), (0, 8000), (50, 1001)],
                                                     H, Hkv, page, dt, 77, pad=5)
    t = q.shape[0]
    cos, sin = angles(torch, max(lens))
    rows = torch.tensor([i for i in range(cu[-1]) if slots[i] >= 0], device="cuda")
    pos = torch.tensor(positions(cu, lens), device="cuda")[rows]
    at = torch.tensor(slots, device="cuda")[rows]
    s = api.PagedShape(len(lens), t, H, Hkv, page, pages, 1, dtype=dt)
    out = torch.full((t, H, 64), SENTINEL, dtype=dt, device="cuda")
    args = (i32(torch, slots), i32(torch, cu), i32(torch, lens), out)
    turned = rotate(k[rows], cos[pos], sin[pos]) if turn else k[rows].float()
    if turn:
        want_q = torch.full_like(out, SENTINEL)
        want_q[rows] = rotate(q[rows], cos[pos], sin[pos]).to(dt)
    if bits == 16:
        kc, vc = (rnd(torch, (pages, Hkv, page, 64), dt, 5 + i) for i in range(2))
        want_k, want_v = kc.clone(), vc.clone()
        want_k[at // page, :, at % page] = turned.to(dt)
        want_v[at // page, :, at % page] = v[rows]
        api.attn_paged_append(s, q, k, v, cos, sin, *args, kc, vc)
        same(kc, want_k, "K")
        same(vc, want_v, "V")
        same(out, want_q, "q")
        return
    kc, vc = (bytes_pool(torch, pages, Hkv, page, 9 + i) for i in range(2))
    want_k, want_v = row_bytes(kc), row_bytes(vc)
    want_k[at // page, :, at % page] = pack(*quantise(turned, dt))
    want_v[at // page, :, at % page] = pack(*quantise(v[rows].float(), dt))
    if turn:
        api.attn_paged_append4(s, q, k, v, cos, sin, *args, kc, vc)
        same(out, want_q, "q")
    else:
        api.attn_paged_append4(s, None, k, v, None, None, args[0], None, None, None, kc, vc)
    same(row_bytes(kc), want_k, "K")
    same(row_bytes(vc), want_v, "V")
    # and back, every slot twice
    twice = torch.cat([args[0], args[0].flip(0)])
    both = torch.cat([rows, 2 * t - 1 - rows])
    s = api.PagedShape(1, 2 * t, H, Hkv, page, pages, 1, dtype=dt)
    ko, vo = (torch.full((2 * t, Hkv, 64), SENTINEL, dtype=dt, device="cuda") for _ in range(2))
    api.attn_paged_load4(s, twice, kc, vc, ko, vo)
    for got, pool in ((ko, kc), (vo, vc)):
        want = torch.full_like(got, SENTINEL)
        want[both] = values(pool, dt)[0][at // page, :, at % page].to(dt).repeat(2, 1, 1)
        same(got, want, "read back")


@pytest.mark.parametrize("n", [1, 31, 32, 33, 1023, 1024, 1025, 4096])
def test_append_finds_every_request(torch, n):
    """As many requests as the search for a token's request takes steps."""
    from causal_streaming_softmax_gb300 import api
    r = random.Random(n)
    reqs = [(r.randint(0, 50), r.choice([0, 1, 2])) for _ in range(n)]
    reqs[0], reqs[-1] = (3, 1), (5, 2)
    q, k, v, slots, cu, lens, pages = append_problem(torch, reqs, 2, 1, 16, torch.float16, n)
    cos, sin = angles(torch, 60)
    kc, vc = (torch.zeros((pages, 1, 16, 64), dtype=torch.float16, device="cuda")
              for _ in range(2))
    out = torch.full_like(q.contiguous(), SENTINEL)
    s = api.PagedShape(n, q.shape[0], 2, 1, 16, pages, 1)
    api.attn_paged_append(s, q, k, v, cos, sin, i32(torch, slots), i32(torch, cu),
                          i32(torch, lens), out, kc, vc)
    pos = torch.tensor(positions(cu, lens), device="cuda")
    want = rotate(q, cos[pos], sin[pos]).to(torch.float16)
    want[torch.tensor(slots, device="cuda") < 0] = SENTINEL
    same(out, want, "q")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_quantised_values_at_the_ends(torch, dtype):
    """Zeros, the smallest and largest numbers, ties between codes and between
    scales, extrema of either sign, infinities and NaN."""
    from causal_streaming_softmax_gb300 import api
    dt = getattr(torch, dtype)
    fi = torch.finfo(dt)
    rows = [torch.zeros(64), torch.full((64,), fi.tiny), torch.full((64,), fi.max),
            torch.full((64,), -fi.max), torch.linspace(-fi.max, fi.max, 64, dtype=torch.float64),
            torch.arange(64) * fi.smallest_normal / 64, torch.arange(64) - 32.0,
            32.0 - torch.arange(64), torch.arange(64) * 0.5, (torch.arange(64) % 16 - 8) * 0.25,
            (torch.arange(64) % 32) * 0.0625 - 1, torch.tensor([1.0, -1.0] * 32),
            torch.tensor([-3.0, 3.0] * 32), torch.tensor([0.0] * 63 + [1e-3])]
    smallest = float(torch.ldexp(torch.tensor(1.0, dtype=torch.float64),
                                 torch.tensor(-24 if dt == torch.float16 else -133)))
    rows += [torch.arange(64, dtype=torch.float64) * smallest * m for m in (1, 2, 5, 17)]
    for bad in (NAN, math.inf, -math.inf):
        x = torch.linspace(-2, 2, 64)
        x[40] = bad
        rows.append(x)
    g = torch.Generator().manual_seed(3)
    for e in range(-18, 12):
        rows.append(torch.randn(64, generator=g) * 2.0 ** e)
    x = torch.stack([r.double() for r in rows]).to(dt).cuda()[:, None].contiguous()
    n = x.shape[0]
    pages = -(-n // 16)
    kc, vc = (bytes_pool(torch, pages, 1, 16, 4) for _ in range(2))
    s = api.PagedShape(1, n, 1, 1, 16, pages, 1, dtype=dt)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    api.attn_paged_append4(s, None, x, x, None, None, slots, None, None, None, kc, vc)
    want = pack(*quantise(x.float(), dt))
    for pool in (kc, vc):
        got = row_bytes(pool).transpose(1, 2).reshape(pages * 16, 1, 36)[:n]
        same(got, want, "rows")
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    api.attn_paged_load4(s, slots, kc, vc, ko, vo)
    same(ko, vo, "K and V")
    for i in range(n):
        for part in (slice(0, 32), slice(32, 64)):
            a, b = x[i, 0, part].double(), ko[i, 0, part].double()
            if not torch.isfinite(a).all():
                assert torch.isnan(b).all()
                continue
            assert torch.isfinite(b).all()
            # what the largest scale stands for; values beyond come back as that
            most = 65280.0 if dt == torch.float16 else 2.0 ** 126
            a = a.clamp(-most, most)
            step = float(a.abs().max()) / 8 * (1 + 2.0 ** -(8 if dt == torch.float16 else 5))
            # the far end from the extremum loses up to a step.  The smallest scales are
            # multiples of 2^-24 (binary16) and 2^-130 (bfloat16: five bits of binary32's
            # smallest exponent), so a scale is off by up to half of that and a value by
            # eight times as much
            off = float((a - b).abs().max())
            unit = 2.0 ** (-24 if dt == torch.float16 else -130)
            assert off <= step + 4 * unit, (i, off, step)


def test_append_reports_positions_and_slots(torch):
    """A position past the tables, a negative one, a token outside every request
    and a slot past the pool are left out and reported, the others done."""
    from causal_streaming_softmax_gb300 import api
    dt = torch.float16
    for four in (False, True):
        for trouble in ("late", "early", "outside", "slot", "offsets"):
            q, k, v = (rnd(torch, (6, h, 64), dt, 1 + h) for h in (4, 2, 2))
            cos, sin = angles(torch, 20)
            cu, lens, slots = [0, 2, 6], [20, 9], [3, 4, 5, 6, 7, 8]
            left = {"late": [0, 1], "early": [2, 3], "outside": [4, 5], "slot": [2],
                    "offsets": [2, 3, 4, 5]}[trouble]
            if trouble == "late":
                lens[0] = 22
            if trouble == "early":
                lens[1] = 2
            if trouble == "outside":
                cu[2] = 4
            if trouble == "slot":
                slots[2] = 64
            if trouble == "offsets":
                cu[2] = 7
            out = torch.full((6, 4, 64), SENTINEL, dtype=dt, device="cuda")
            if four:
                kc, vc = (bytes_pool(torch, 4, 2, 16, 3) for _ in range(2))
            else:
                kc, vc = (torch.zeros((4, 2, 16, 64), dtype=dt, device="cuda") for _ in range(2))
            before = kc.clone()
            s = api.PagedShape(2, 6, 4, 2, 16, 4, 2, dtype=dt)
            f = api.attn_paged_append4 if four else api.attn_paged_append
            f(s, q, k, v, cos, sin, i32(torch, slots), i32(torch, cu), i32(torch, lens), out, kc,
              vc)
            assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX, trouble
            for t in range(6):
                assert bool((out[t] == SENTINEL).all()) == (t in left), (trouble, t)
            if four:
                kc, before = row_bytes(kc), row_bytes(before)
            for t in range(6):
                if t in left and slots[t] < 64:
                    assert torch.equal(kc[0, :, slots[t]], before[0, :, slots[t]]), (trouble, t)


def test_load4_reports_a_slot_past_the_pool(torch):
    from causal_streaming_softmax_gb300 import api
    kc, vc = (pool_of(rnd(torch, (3, 2, 8, 64), torch.float16, i), torch.float16) for i in (1, 2))
    k, v = (torch.full((4, 2, 64), SENTINEL, dtype=torch.float16, device="cuda") for _ in range(2))
    s = api.PagedShape(1, 4, 2, 2, 8, 3, 1)
    api.attn_paged_load4(s, i32(torch, [5, 24, 5, 2 ** 31 - 1]), kc, vc, k, v)
    assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX
    assert (k[1] == SENTINEL).all() and (v[3] == SENTINEL).all()
    same(k[0], values(kc, torch.float16)[0][0, :, 5].half())
    same(k[2], k[0])


# ------------------------------------------------------------------- attention
def paged4_problem(torch, reqs, H, Hkv, page, dtype, seed, layout="pages", pad=0, std=1.0):
    """reqs: (keys in the cache, new tokens).  Places that no request holds read as
    NaN; unused table entries name pages that do not exist."""
    r = random.Random(seed)
    up = [-(-max(n, 0) // page) for n, _ in reqs]
    width, pages = max(1, max(up)) + 1, sum(up) + 3
    order = list(range(pages))
    r.shuffle(order)
    table, used = [], torch.zeros((pages, page), dtype=torch.bool)
    for (n, _), u in zip(reqs, up):
        ids = [order.pop() for _ in range(u)]
        for x in range(max(n, 0)):
            used[ids[x // page], x % page] = True
        table.append(ids + [r.choice([-1, pages, 2 ** 31 - 1, -2 ** 31])] * (width - u))
    used = used.cuda()
    pools = []
    for i in range(2):
        x = rnd(torch, (pages, Hkv, page, 64), dtype, seed + 50 + i, std if i == 0 else 1.0)
        x.masked_fill_(~used[:, None, :, None], NAN)
        x = pool_of(x, dtype)
        if layout == "heads":  # [head][page]
            x = x.transpose(0, 1).contiguous().transpose(0, 1)
        elif layout == "both":
            x = torch.stack([x, x], 1)[:, i]
        pools.append(x)
    new = [n for _, n in reqs]
    cu = scan(new)
    q = rnd(torch, (cu[-1] + pad, H, 64), dtype, seed + 60, 2.0)
    return q, pools[0], pools[1], table, cu, [n for n, _ in reqs], width


def run_paged4(torch, q, kc, vc, table, cu, lens, max_new=None, lse=True, o=None, stream=None,
               scale=0.125):
    from causal_streaming_softmax_gb300 import api
    t, H, _ = q.shape
    s = api.PagedShape(len(lens), t, H, kc.shape[1], kc.shape[2] * 8, kc.shape[0], len(table[0]),
                       max_new=max_new or max(1, max(b - a for a, b in zip(cu, cu[1:]))),
                       dtype=q.dtype, scale=scale)
    ws = api.alloc_paged_workspace(s)
    ws.fill_(255)  # its contents mean nothing
    if o is None:
        o = torch.full((t, H, 64), SENTINEL, dtype=q.dtype, device="cuda")
    L = torch.full((H, t), SENTINEL, device="cuda") if lse else None
    api.attn_paged_fwd4(s, q, kc, vc, i32(torch, table), i32(torch, cu), i32(torch, lens), ws, o,
                        L, stream=stream)
    return o, L


def check_paged4(torch, q, kc, vc, table, cu, lens, o, L, scale=0.125):
    inside = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    tt = torch.tensor(table, dtype=torch.int64, device="cuda")
    for rows, eo, el, to, tl in paged4_64(q, kc, vc, tt, cu, lens, scale):
        check(o[rows], eo, to, "O of rows %s" % rows)
        if L is not None:
            check(L[:, rows], el, tl, "L of rows %s" % rows)
        inside[rows] = True
    assert (o[~inside] == SENTINEL).all(), "a row outside the requests was written"
    if L is not None:
        assert (L[:, ~inside] == SENTINEL).all()


REQS = [
    [(1, 1)],
    [(0, 0)],
    [(777, 1)],
    [(16, 1), (17, 1), (15, 1), (1, 1), (0, 0), (64, 1), (65, 1), (2000, 1)],
    [(255, 1), (256, 1), (257, 1), (31, 1), (33, 1), (511, 1), (513, 1), (8, 1)],
    [(5000, 1), (3, 1)],
    [(100, 2), (7, 2), (2, 2), (129, 1), (1, 2)],           # a few new tokens each
    [(50, 50), (1, 1), (300, 33), (128, 128)],              # prompts and tokens
    [(0, 1), (1, 3), (2, 5), (700, 1)],                     # rows that see nothing
    [(3000, 700), (64, 64), (9, 1), (4097, 129)],
    [(1 + 37 * i % 400, 1) for i in range(150)],
    [(40 + i, 1 + i % 5) for i in range(90)],
    [(20000, 3), (11, 2)],
]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads", [(2, 1), (4, 4), (8, 2), (15, 5), (16, 1), (9, 1)])
@pytest.mark.parametrize("reqs", range(len(REQS)))
def test_paged4(torch, dtype, heads, reqs):
    H, Hkv = heads
    page = [16, 8, 64, 256, 32, 128, 1024][(reqs + H) % 7]
    p = paged4_problem(torch, REQS[reqs], H, Hkv, page, getattr(torch, dtype), 100 * reqs + H,
                       ["pages", "heads", "both"][(reqs + H) % 3], pad=(reqs % 3) * 2)
    q, kc, vc, table, cu, lens, _ = p
    if q.shape[0] == 0:
        q = rnd(torch, (3, H, 64), q.dtype, 1)
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens, lse=reqs % 2 == 0)
    check_paged4(torch, q, kc, vc, table, cu, lens, o, L)


@pytest.mark.parametrize("heads", [(128, 1), (100, 1), (40, 2), (17, 1), (33, 1)])
@pytest.mark.parametrize("new", [1, 2, 9])
def test_paged4_wide_groups(torch, heads, new):
    p = paged4_problem(torch, [(500, new), (13, new), (1, 1)], heads[0], heads[1], 16,
                       torch.float16, 3)
    q, kc, vc, table, cu, lens, _ = p
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens)
    check_paged4(torch, q, kc, vc, table, cu, lens, o, L)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("scale,std", [(1.0, 1.0), (0.01, 1.0), (3.0, 0.1), (0.125, 30.0)])
@pytest.mark.parametrize("reqs", [[(900, 1), (33, 2)], [(500, 90)]])
def test_paged4_scales_and_large_scores(torch, dtype, scale, std, reqs):
    p = paged4_problem(torch, reqs, 8, 2, 16, getattr(torch, dtype), 8, std=std)
    q, kc, vc, table, cu, lens, _ = p
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens, scale=scale)
    check_paged4(torch, q, kc, vc, table, cu, lens, o, L, scale)


# the type, and the binary orders of K and V
MAGNITUDES = [("float16", -8, -14), ("float16", 3, 8), ("float16", 0, 12), ("bfloat16", -60, -100),
              ("bfloat16", 20, 100), ("bfloat16", 0, -120), ("bfloat16", 0, 120)]


@pytest.mark.parametrize("dtype,ke,ve", MAGNITUDES)
@pytest.mark.parametrize("reqs", [[(700, 1), (33, 2)], [(300, 40)]])
def test_paged4_small_and_large_magnitudes(torch, dtype, ke, ve, reqs):
    """K and V far from one; the scale of the scores takes K's back."""
    dt = getattr(torch, dtype)
    q, _, _, table, cu, lens, _ = paged4_problem(torch, reqs, 8, 2, 16, dt, 13)
    pages = max(p for row in table for p in row if 0 <= p < 10 ** 6) + 1
    kc, vc = (pool_of((rnd(torch, (pages, 2, 16, 64), torch.float32, 80 + e % 7) * 2.0 ** e).to(dt),
                      dt) for e in (ke, ve))
    scale = 0.125 * 2.0 ** -ke
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens, scale=scale)
    check_paged4(torch, q, kc, vc, table, cu, lens, o, L, scale)


@pytest.mark.parametrize("B", [1, 57, 58])
@pytest.mark.parametrize("keys", [1007, 1008, 1009, 1030])
def test_paged4_around_whole_items(torch, B, keys):
    """Tables that hold just 1024 keys and just more, with as many items as blocks."""
    reqs = [(keys - 13 * i % 500, 1) for i in range(B)]
    q, kc, vc, table, cu, lens, _ = paged4_problem(torch, reqs, 8, 8, 16, torch.float16, keys + B)
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens)
    check_paged4(torch, q, kc, vc, table, cu, lens, o, L)


@pytest.mark.parametrize("bound", [1, 2, 4, 40, 1000])
def test_paged4_whatever_the_bound_on_new_tokens(torch, bound):
    p = paged4_problem(torch, [(900, 1), (33, 1), (1, 1)], 8, 2, 32, torch.bfloat16, 4)
    q, kc, vc, table, cu, lens, _ = p
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens, max_new=bound)
    check_paged4(torch, q, kc, vc, table, cu, lens, o, L)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("page", [8, 16, 256])
@pytest.mark.parametrize("new", [1, 2, 4, 5, 64, 150])
def test_paged4_bad_values_stay_where_they_are_seen(torch, dtype, page, new):
    """A NaN or infinite scale among the new tokens' keys does not reach the rows
    before it, nor the other group's channels (V)."""
    dt = getattr(torch, dtype)
    bits = {"nan": (0x7e00, 0x7fc0), "inf": (0x7c00, 0x7f80), "-inf": (0xfc00, 0xff80)}
    word = {n: b[dt == torch.bfloat16] for n, b in bits.items()}
    p = paged4_problem(torch, [(300, new), (new, new), (260, 1)], 8, 2, page, dt, 5)
    q, kc, vc, table, cu, lens, _ = p

    def spoil(pool, req, pos, head, group, what):
        r = pos % page
        b = 256 + r % 8 * 4 + 2 * group
        w = word[what]
        pool[table[req][pos // page], head, r // 8, b] = w & 255
        pool[table[req][pos // page], head, r // 8, b + 1] = w >> 8

    for req, back in ((0, 1), (1, new // 2)):
        pos = lens[req] - max(1, back)
        spoil(vc, req, pos, 0, 0, "nan")
        spoil(vc, req, pos, 1, 1, "inf")
        spoil(vc, req, max(0, pos - 2), 1, 0, "-inf")
    spoil(kc, 0, lens[0] - new // 2 - 1, 1, 0, "nan")
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens)
    # A pool's scales are finite or NaN (the append writes no others).  An infinite one
    # gives the rows that see it infinities or NaN where its values are infinities or
    # NaN: which of them is not promised.
    tt = torch.tensor(table, dtype=torch.int64, device="cuda")
    for rows, eo, el, to, tl in paged4_64(q, kc, vc, tt, cu, lens):
        fine = torch.isfinite(eo)
        assert not torch.isfinite(o[rows][~fine]).any()
        check(o[rows][fine], eo[fine], to[fine], "O of rows %s" % rows)
        check(L[:, rows], el, tl, "L of rows %s" % rows)


def test_paged4_queries_that_are_not_finite(torch):
    """A row of q with an infinity or a NaN gives NaN, and no other row does."""
    q, kc, vc, table, cu, lens, _ = paged4_problem(torch, [(300, 2), (70, 40)], 8, 2, 16,
                                                   torch.float16, 5)
    q[0, 3, 5], q[1, 7, 40], q[9, 0, 63] = math.inf, NAN, -math.inf
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[1, 7] = bad[9, 0] = True
    assert torch.isnan(o[0, 3]).all() and torch.isnan(o[1, 7]).all()
    assert torch.isfinite(o[~bad]).all() and torch.isfinite(L.T[~bad]).all()
    q[0, 3, 5], q[1, 7, 40], q[9, 0, 63] = 0, 0, 0
    o2, _ = run_paged4(torch, q, kc, vc, table, cu, lens)
    same(o[~bad], o2[~bad])


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,first", [((16, 1), 2), ((8, 2), 5), ((33, 1), 1), ((24, 3), 3)])
def test_paged4_chunks_of_unequal_row_tiles(torch, dtype, heads, first):
    """Many chunks whose last row tiles are short or empty, over short and long caches:
    items of one key tile and of many follow one another in a block."""
    r = random.Random(first)
    reqs = []
    for i in range(120):
        n = r.choice([first, first + 1, 8, 9, 17, 25, 33, 65, 70])
        reqs.append((max(n, r.choice([1, 30, 64, 65, 129, 400, 1500])), n))
    reqs[60] = (9000, 100)
    page = [8, 16, 64, 32][first % 4]
    p = paged4_problem(torch, reqs, heads[0], heads[1], page, getattr(torch, dtype), 21 + first)
    q, kc, vc, table, cu, lens, _ = p
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens)
    check_paged4(torch, q, kc, vc, table, cu, lens, o, L)
    for _ in range(4):
        o2, L2 = run_paged4(torch, q, kc, vc, table, cu, lens)
        assert torch.equal(o, o2) and torch.equal(L, L2)


@pytest.mark.parametrize("heads", [(2, 2), (4, 2), (15, 5), (8, 2), (5, 1), (12, 2), (7, 1),
                                   (8, 1)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_paged4_several_tokens_beside_a_chunk(torch, heads, dtype):
    """Requests of nine to sixteen rows are several items there; some see no key."""
    most = 16 // (heads[0] // heads[1])
    reqs = [(900, 40)]
    for n in range(1, most + 1):
        reqs += [(4000 - 7 * n, n), (n, n), (max(0, n - 3), n), (0, n), (64 + n - 1, n), (321, n)]
    q, kc, vc, table, cu, lens, _ = paged4_problem(torch, reqs, heads[0], heads[1], 16,
                                                   getattr(torch, dtype), 41)
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens)
    check_paged4(torch, q, kc, vc, table, cu, lens, o, L)
    o2, L2 = run_paged4(torch, q, kc, vc, table, cu, lens)
    assert torch.equal(o, o2) and torch.equal(L, L2)


@pytest.mark.parametrize("heads", [(8, 1), (12, 4), (5, 1)])
def test_paged4_one_and_several_tokens_in_a_call(torch, heads):
    """Items of up to eight rows, and of up to sixteen, in one call."""
    n = 16 // (heads[0] // heads[1])
    reqs = [(5000, 1), (4000, n), (700, 1), (n, n), (65, 1), (64, n), (300, 1)] * 5
    q, kc, vc, table, cu, lens, _ = paged4_problem(torch, reqs, heads[0], heads[1], 16,
                                                   torch.bfloat16, 31)
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens)
    check_paged4(torch, q, kc, vc, table, cu, lens, o, L)


def test_paged4_is_deterministic(torch):
    reqs = [(random.Random(i).randint(1, 3000), 1 + (i % 7 == 0) * 40) for i in range(60)]
    q, kc, vc, table, cu, lens, _ = paged4_problem(torch, reqs, 8, 2, 16, torch.float16, 6)
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens)
    for _ in range(3):
        o2, L2 = run_paged4(torch, q, kc, vc, table, cu, lens)
        assert torch.equal(o, o2) and torch.equal(L, L2)


def test_paged4_strided_output_and_queries(torch):
    q, kc, vc, table, cu, lens, _ = paged4_problem(torch, [(90, 3), (700, 20), (5, 1)], 8, 2, 16,
                                                   torch.bfloat16, 7)
    t = q.shape[0]
    wide = torch.zeros((t, 12, 64), dtype=q.dtype, device="cuda")
    wide[:, 2:10] = q
    o = torch.full((8, t, 64), SENTINEL, dtype=q.dtype, device="cuda").permute(1, 0, 2)
    o, L = run_paged4(torch, wide[:, 2:10], kc, vc, table, cu, lens, o=o)
    check_paged4(torch, q, kc, vc, table, cu, lens, o, L)


@pytest.mark.parametrize("new", [1, 3, 30])
def test_paged4_bad_pages_and_lengths_are_reported(torch, new):
    """The other requests are as they were."""
    from causal_streaming_softmax_gb300 import api
    reqs = [(900, new), (40, new), (300, new)]
    q, kc, vc, table, cu, lens, width = paged4_problem(torch, reqs, 8, 2, 16, torch.float16, 9)
    good, _ = run_paged4(torch, q, kc, vc, table, cu, lens)
    page, table[0][30] = table[0][30], 2 ** 31 - 1
    o, _ = run_paged4(torch, q, kc, vc, table, cu, lens)
    assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX
    same(o[cu[1]:], good[cu[1]:])
    table[0][30] = page
    for bad in (-1, width * 16 + 1, 2 ** 31 - 1):
        o, _ = run_paged4(torch, q, kc, vc, table, cu, [900, bad, 300])
        assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX
        same(o[cu[2]:], good[cu[2]:])
        same(o[:cu[1]], good[:cu[1]])


@pytest.mark.parametrize("heads", [(8, 2), (4, 4), (17, 1)])
@pytest.mark.parametrize("bound", [1, 3, 5, 20, 39])
def test_paged4_more_new_tokens_than_the_bound(torch, heads, bound):
    from causal_streaming_softmax_gb300 import api
    H, Hkv = heads
    reqs = [(100, 1), (200, 40), (50, 1)]
    q, kc, vc, table, cu, lens, _ = paged4_problem(torch, reqs, H, Hkv, 16, torch.float16, 12)
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens, max_new=bound)
    assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX
    assert (o[1:41] == SENTINEL).all() and (L[:, 1:41] == SENTINEL).all()
    tt = torch.tensor(table, dtype=torch.int64, device="cuda")
    for rows, eo, el, to, tl in paged4_64(q, kc, vc, tt, cu, lens)[::2]:
        check(o[rows], eo, to, "O")
        check(L[:, rows], el, tl, "L")


@pytest.mark.parametrize("heads", [(2, 1), (17, 1)])
def test_paged4_the_largest_batch(torch, heads):
    H, Hkv = heads
    reqs = [(1 + i % 60, 1) for i in range(4096)]
    q, kc, vc, table, cu, lens, _ = paged4_problem(torch, reqs, H, Hkv, 16, torch.float16, 2)
    o, L = run_paged4(torch, q, kc, vc, table, cu, lens)
    pick = [0, 1, 59, 60, 2047, 3333, 4095]
    pools = values(kc, q.dtype) + values(vc, q.dtype)
    tt = torch.tensor(table, dtype=torch.int64, device="cuda")
    for i in pick:
        eo, el, to, tl = attend4(q[i:i + 1], *(gather(x, tt[i], lens[i]) for x in pools),
                                 torch.tensor([lens[i]], device="cuda"))
        check(o[i:i + 1], eo, to, "O of %d" % i)
        check(L[:, i:i + 1], el, tl, "L of %d" % i)
    assert torch.isfinite(L).all()


def test_pools_beyond_32_bits(torch):
    """Pages whose bytes lie past 2^32, read, written and attended."""
    from causal_streaming_softmax_gb300 import api
    pages, page, Hkv = 1 << 21, 16, 4
    kc, vc = (torch.zeros((pages, Hkv, 2, 288), dtype=torch.uint8, device="cuda")
              for _ in range(2))
    dt, n = torch.float16, 40
    ids = [pages - 1, 5, pages - 2]
    slots = [ids[i // page] * page + i % page for i in range(n)]
    k, v = rnd(torch, (n, Hkv, 64), dt, 1), rnd(torch, (n, Hkv, 64), dt, 2)
    s = api.PagedShape(1, n, 8, Hkv, page, pages, 3, max_new=n, dtype=dt)
    api.attn_paged_append4(s, None, k, v, None, None, i32(torch, slots), None, None, None, kc, vc)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    api.attn_paged_load4(s, i32(torch, slots), kc, vc, ko, vo)
    for x, y in ((k, ko), (v, vo)):
        codes, scales = quantise(x.float(), dt)
        want = codes.double() * scales.double().repeat_interleave(32, -1)
        same(y, want.to(dt))
    for new in (1, n):
        q = rnd(torch, (new, 8, 64), dt, 3, 2.0)
        o, L = run_paged4(torch, q, kc, vc, [ids], [0, new], [n])
        kd, vd = ko.double(), vo.double()
        sk, sv = (quantise(x.float(), dt)[1].double().abs().repeat_interleave(32, -1)
                  for x in (k, v))
        eo, el, to, tl = attend4(q, kd, sk, vd, sv,
                                 torch.arange(n - new + 1, n + 1, device="cuda"))
        check(o, eo, to, "O")
        check(L, el, tl, "L")


# -------------------------------------------------------------------- together
def serve(torch, bits, turn, dtype, steps=14):
    """A small server: requests come, grow by chunks and tokens, and finish."""
    from causal_streaming_softmax_gb300 import api
    H, Hkv, B, page, dt = 8, 2, 5, 16, getattr(torch, dtype)
    cache = api.PagedCache(B, H, Hkv, num_pages=90, page_size=page, table_width=40, dtype=dt,
                           bits=bits)
    cos, sin = angles(torch, 640)
    r = random.Random(11)
    hist = [[] for _ in range(B)]  # of each token: K, V, their scales
    for step in range(steps):
        fresh = [r.choice([1, 1, 1, r.randint(0, 70), -1 if len(hist[i]) > 150 else 1])
                 for i in range(B)]
        n = sum(max(0, f) for f in fresh)
        x = rnd(torch, (n, H + 2 * Hkv, 64), dt, 1000 + step)
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        before = x.clone()
        o = torch.empty((n, H, 64), dtype=dt, device="cuda")
        L = torch.empty((H, n), device="cuda")
        more = dict(cos=cos, sin=sin) if turn else {}
        cache.step(i32(torch, fresh), q, k, v, o, L, max_new=max(max(fresh), 1), **more)
        same(x, before, "q, k and v")
        assert cache.status() == 0 and api.last_device_error() == 0
        at = 0
        for i, f in enumerate(fresh):
            if f < 0:
                hist[i] = []
                continue
            if f:
                pos = torch.arange(len(hist[i]), len(hist[i]) + f, device="cuda")
                rows = slice(at, at + f)
                kf, qr = k[rows].float(), q[rows]
                if turn:
                    kf, qr = rotate(k[rows], cos[pos], sin[pos]), \
                        rotate(qr, cos[pos], sin[pos]).to(dt)
                if bits == 4:
                    (kq, ks), (vq, vs) = quantise(kf, dt), quantise(v[rows].float(), dt)
                    ks, vs = (y.double().repeat_interleave(32, -1) for y in (ks, vs))
                    hist[i] += list(zip(kq * ks, vq * vs, ks.abs(), vs.abs()))
                else:
                    hist[i] += list(zip(kf.to(dt), v[rows], kf, kf))
                kk, vv, ss, vss = (torch.stack([h[j] for h in hist[i]]) for j in range(4))
                m = len(hist[i])
                seen = torch.arange(m - f + 1, m + 1, device="cuda")
                eo, el, to, tl = attend4(qr, kk, ss, vv, vss, seen) if bits == 4 else \
                    attend64(qr, kk, vv, seen)
                check(o[rows], eo, to, "step %d request %d" % (step, i))
                check(L[:, rows], el, tl, "L of step %d request %d" % (step, i))
            at += f
        assert cache.lens.tolist() == [len(h) for h in hist]
    return cache, hist


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("bits,turn", [(4, True), (4, False), (16, True)])
def test_a_server_of_several_steps(torch, dtype, bits, turn):
    cache, hist = serve(torch, bits, turn, dtype)
    if bits == 16:
        with pytest.raises(ValueError, match="16-bit"):
            cache.load(None, None, None)
        return
    for i, h in enumerate(hist):  # what the cache holds
        m = len(h)
        j = torch.arange(m, device="cuda")
        slots = (cache.table[i][j // 16] * 16 + j % 16).to(torch.int32)
        k, v = (torch.empty((m, 2, 64), dtype=cache.dtype, device="cuda") for _ in range(2))
        cache.load(slots, k, v)
        if m:
            same(k, torch.stack([x[0] for x in h]).to(cache.dtype), "K of %d" % i)
            same(v, torch.stack([x[1] for x in h]).to(cache.dtype), "V of %d" % i)


@pytest.mark.parametrize("bits", [4, 16])
def test_captured_steps_replay(torch, bits):
    """Token steps captured into a graph on a stream of their own and replayed
    between eager ones give what eager steps give."""
    from causal_streaming_softmax_gb300 import api
    H, Hkv, B, dt = 8, 2, 3, torch.bfloat16
    cos, sin = angles(torch, 400)
    caches = [api.PagedCache(B, H, Hkv, num_pages=60, dtype=dt, bits=bits) for _ in range(2)]
    plen = [37, 5, 130]
    x = rnd(torch, (sum(plen), H + 2 * Hkv, 64), dt, 20)
    parts = lambda y: (y[:, :H], y[:, H:H + Hkv], y[:, H + Hkv:])
    for c in caches:
        o = torch.empty((sum(plen), H, 64), dtype=dt, device="cuda")
        c.step(i32(torch, plen), *parts(x), o, max_new=130, cos=cos, sin=sin)
    one = i32(torch, [1] * B)
    buf = [(rnd(torch, (B, H + 2 * Hkv, 64), dt, 30 + i),
            torch.empty((B, H, 64), dtype=dt, device="cuda")) for i in range(2)]
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        for y, o in buf:
            caches[0].step(one, *parts(y), o, max_new=1, cos=cos, sin=sin)
    for rep in range(12):
        for i, (y, o) in enumerate(buf):
            y.copy_(rnd(torch, y.shape, dt, 100 + 2 * rep + i))
        want = []
        for y, _ in buf:
            want.append(torch.empty((B, H, 64), dtype=dt, device="cuda"))
            caches[1].step(one, *parts(y), want[-1], max_new=1, cos=cos, sin=sin)
        if rep % 4 == 3:
            for y, o in buf:
                caches[0].step(one, *parts(y), o, max_new=1, cos=cos, sin=sin)
        else:
            g.replay()
        torch.cuda.synchronize()
        for (_, o), w in zip(buf, want):
            same(o, w, "replay %d" % rep)
    assert caches[0].lens.tolist() == caches[1].lens.tolist() == [n + 24 for n in plen]
    same(caches[0].k.view(torch.uint8), caches[1].k.view(torch.uint8))


def test_a_position_past_the_tables_in_a_step(torch):
    from causal_streaming_softmax_gb300 import api
    cache = api.PagedCache(2, 4, 2, num_pages=8, bits=4)
    cos, sin = angles(torch, 10)
    x = rnd(torch, (14, 8, 64), torch.float16, 3)
    o = torch.empty((14, 4, 64), dtype=torch.float16, device="cuda")
    cache.step(i32(torch, [11, 3]), x[:, :4], x[:, 4:6], x[:, 6:], o, cos=cos, sin=sin)
    assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX
    kq, ks = quantise(rotate(x[11:, 4:6], cos[:3], sin[:3]), torch.float16)
    vq, vs = quantise(x[11:, 6:].float(), torch.float16)
    ks, vs = (y.double().repeat_interleave(32, -1) for y in (ks, vs))
    eo, _, to, _ = attend4(rotate(x[11:, :4], cos[:3], sin[:3]).half(), kq * ks, ks.abs(), vq * vs,
                           vs.abs(), torch.arange(1, 4, device="cuda"))
    check(o[11:], eo, to, "the other request")


def test_calls_on_a_stream_and_both_marshalling_paths(torch, monkeypatch):
    """The call on another stream, and through api's own checks, gives the same."""
    from causal_streaming_softmax_gb300 import api
    assert api._native is not None or api.load_library() and api._native is not None
    q, kc, vc, table, cu, lens, _ = paged4_problem(torch, [(900, 1), (300, 2)], 8, 2, 16,
                                                   torch.float16, 9)
    want, wl = run_paged4(torch, q, kc, vc, table, cu, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, gl = run_paged4(torch, q, kc, vc, table, cu, lens, stream=side)
    torch.cuda.synchronize()
    same(got, want)
    assert torch.equal(gl, wl)
    cos, sin = angles(torch, 1000)
    k, v = rnd(torch, (3, 2, 64), torch.float16, 1), rnd(torch, (3, 2, 64), torch.float16, 2)
    k16 = torch.zeros((4, 2, 16, 64), dtype=torch.float16, device="cuda")
    outs = []
    for native in (api._native, None):
        monkeypatch.setattr(api, "_native", native)
        s = api.PagedShape(2, 3, 8, 2, 16, kc.shape[0], len(table[0]))
        s16 = api.PagedShape(2, 3, 8, 2, 16, 4, 1)
        args = (cos, sin, i32(torch, [1, 2, 40]), i32(torch, cu), i32(torch, lens))
        k4, v4, ka, va = kc.clone(), vc.clone(), k16.clone(), k16.clone()
        q1, q2 = torch.zeros_like(q), torch.zeros_like(q)
        api.attn_paged_append4(s, q, k, v, *args, q1, k4, v4)
        api.attn_paged_append(s16, q, k, v, *args, q2, ka, va)
        ko, vo = torch.zeros_like(k), torch.zeros_like(v)
        api.attn_paged_load4(s, args[2], k4, v4, ko, vo)
        api.attn_paged_append4(s, None, v, k, None, None, args[2], None, None, None, k4, v4)
        o, L = run_paged4(torch, q, kc, vc, table, cu, lens)
        outs.append([k4, v4, ka, va, q1, q2, ko, vo, o])
    for a, b in zip(*outs):
        same(a, b)
    same(outs[0][-1], want)


def test_python_names_what_is_wrong(torch):
    from causal_streaming_softmax_gb300 import api
    dt = torch.float16
    s = api.PagedShape(1, 2, 4, 2, 16, 3, 1, dtype=dt)
    q, k, v = (rnd(torch, (2, h, 64), dt, h) for h in (4, 2, 2))
    cos, sin = angles(torch, 8)
    slots, cu, lens = i32(torch, [0, 1]), i32(torch, [0, 2]), i32(torch, [2])
    pool, pool16 = api.alloc_paged_pool4(s), torch.zeros((3, 2, 16, 64), dtype=dt, device="cuda")
    a4 = lambda **kw: api.attn_paged_append4(*(dict(s=s, q=q, k=k, v=v, cos=cos, sin=sin,
                                                    slots=slots, cu=cu, lens=lens, q_out=q,
                                                    kc=pool, vc=pool.clone()) | kw).values())
    a4()
    for kw, name in ((dict(cos=cos[:, :16]), "cos"), (dict(sin=sin[:4]), "sin"),
                     (dict(cos=cos.half()), "cos"), (dict(sin=None), "sin"),
                     (dict(cos=None), "cos"), (dict(cos=cos[:0], sin=sin[:0]), "cos and sin"),
                     (dict(q=None), "q"), (dict(q_out=q[:1]), "q_out"),
                     (dict(lens=lens.cpu()), "lens"), (dict(kc=pool[..., :256]), "k_cache"),
                     (dict(vc=pool16), "v_cache"), (dict(slots=slots.long()), "slots"),
                     (dict(kc=torch.zeros((3, 2, 2, 300), dtype=torch.uint8,
                                          device="cuda")[..., :288]), "k_cache")):
        with pytest.raises((TypeError, ValueError), match=name):
            a4(**kw)
    with pytest.raises(api.AttnError):  # pools on an odd byte
        a4(kc=torch.zeros(pool.numel() + 8, dtype=torch.uint8, device="cuda")[8:].view(pool.shape))
    with pytest.raises((TypeError, ValueError), match="k_cache"):
        api.attn_paged_append(s, q, k, v, cos, sin, slots, cu, lens, q, pool, pool16)
    with pytest.raises((TypeError, ValueError), match="k_cache"):
        api.attn_paged_load4(s, slots, pool16, pool, k, v)
    with pytest.raises((TypeError, ValueError), match="v_cache"):
        api.attn_paged_fwd4(s, q, pool, pool16, i32(torch, [[0]]), cu, lens,
                            api.alloc_paged_workspace(s), q.clone())
    cache = api.PagedCache(1, 4, 2, num_pages=3, bits=4)
    o = torch.full_like(q, SENTINEL)
    for kw in (dict(cos=cos), dict(sin=sin), dict(cos=cos, sin=sin[:3]),
               dict(cos=cos.double(), sin=sin), dict(cos=cos[:0], sin=sin[:0])):
        with pytest.raises((TypeError, ValueError)):
            cache.step(i32(torch, [2]), q, k, v, o, **kw)
    assert cache.lens.tolist() == [0] and (o == SENTINEL).all()
    with pytest.raises(ValueError, match="bits"):
        api.PagedCache(1, 4, 2, num_pages=3, bits=8)


def test_arrays_that_something_else_writes(torch):
    """Lengths, offsets, slots and pages that change under the calls: wrong rows, but
    every call ends and nothing outside the tensors is touched."""
    from causal_streaming_softmax_gb300 import api
    reqs = [(700, 1), (300, 3), (500, 40), (64, 1)]
    q, kc, vc, table, cu, lens, _ = paged4_problem(torch, reqs, 8, 2, 16, torch.float16, 9)
    t, H, B = q.shape[0], 8, len(reqs)
    s = api.PagedShape(B, t, H, 2, 16, kc.shape[0], len(table[0]), max_new=40)
    ws = api.alloc_paged_workspace(s)
    guard = torch.full((t + 64, H, 64), SENTINEL, dtype=q.dtype, device="cuda")
    o = guard[32:32 + t]
    arrays = [i32(torch, x) for x in (table, cu, lens)]
    slots = torch.randint(0, kc.shape[0] * 16, (t,), dtype=torch.int32, device="cuda")
    good = [x.clone() for x in arrays] + [slots.clone()]
    cos, sin = angles(torch, 800)
    k, v = rnd(torch, (t, 2, 64), q.dtype, 1), rnd(torch, (t, 2, 64), q.dtype, 2)
    k4, v4 = kc.clone(), vc.clone()
    side = torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(1)
    torch.cuda.synchronize()
    for rep in range(60):
        with torch.cuda.stream(side):
            for _ in range(6):
                for x, y in zip(arrays + [slots], good):
                    x.copy_(torch.randint(-5, 900, x.shape, generator=g, device="cuda",
                                          dtype=torch.int32))
                    x.copy_(y)
        for _ in range(4):
            api.attn_paged_fwd4(s, q, kc, vc, *arrays, ws, o)
            api.attn_paged_append4(s, q, k, v, cos, sin, slots, *arrays[1:], o, k4, v4)
            api.attn_paged_load4(s, slots, k4, v4, k, v)
    torch.cuda.synchronize()
    assert (guard[:32] == SENTINEL).all() and (guard[32 + t:] == SENTINEL).all()
    assert api.last_device_error() in (api.ATTN_OK, api.ATTN_ERR_DEVICE_INDEX)
    o.fill_(SENTINEL)
    api.attn_paged_fwd4(s, q, kc, vc, *arrays, ws, o)
    check_paged4(torch, q, kc, vc, table, cu, lens, o, None)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("heads,reqs,bound", [
    ((8, 8), [(30000, 1)] * 9, 1), ((8, 2), [(9000, 1)] * 70, 1), ((8, 2), [(5000, 4)] * 40, 4),
    ((16, 1), [(20000, 1)] * 20, 1), ((8, 2), [(4000, 3)] * 50 + [(3000, 200)], 200)])
def test_paged_stays_inside_its_workspace(torch, bits, heads, reqs, bound):
    """Every block leaves parts, in a workspace of just the size asked for."""
    from causal_streaming_softmax_gb300 import api
    q, kc, vc, table, cu, lens, width = paged4_problem(torch, reqs, *heads, 64, torch.float16, 17)
    if bits == 16:
        kc, vc = (values(x, q.dtype)[0].half() for x in (kc, vc))
    s = api.PagedShape(len(lens), q.shape[0], *heads, 64, kc.shape[0], width, max_new=bound)
    need = api.paged_workspace_bytes(s)
    room = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    o = torch.full_like(q, SENTINEL)
    call = api.attn_paged_fwd4 if bits == 4 else api.attn_paged_fwd
    call(s, q, kc, vc, i32(torch, table), i32(torch, cu), i32(torch, lens), room[:need], o)
    assert (room[need:] == 171).all()
    if bits == 4:
        check_paged4(torch, q, kc, vc, table, cu, lens, o, None)
    else:
        assert torch.isfinite(o).all()
