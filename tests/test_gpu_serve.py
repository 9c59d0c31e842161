"""The packed and paged calls on the GPU against plain 64-bit forms."""
import math
import random

import pytest

from serve_util import attend64, check, gather, packed64, paged64, plan_host

pytestmark = pytest.mark.gpu

NAN = float("nan")


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


def packed_inputs(torch, t, H, Hkv, dtype, seed, layout="fused"):
    if layout == "fused":  # column blocks of one projection
        x = rnd(torch, (t, H + 2 * Hkv, 64), dtype, seed)
        x[:, :H] *= 2
        return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    if layout == "planes":  # [heads][tokens][64]
        return tuple(rnd(torch, (h, t, 64), dtype, seed + i, s).permute(1, 0, 2)
                     for i, (h, s) in enumerate(((H, 2.0), (Hkv, 1.0), (Hkv, 1.0))))
    return (rnd(torch, (t, H, 64), dtype, seed, 2.0), rnd(torch, (t, Hkv, 64), dtype, seed + 1),
            rnd(torch, (t, Hkv, 64), dtype, seed + 2))


SENTINEL = 7.0


def run_packed(torch, q, k, v, cu, causal=True, scale=0.125, lse=True, o_layout="dense",
               stream=None):
    from causal_streaming_softmax_gb300 import api
    t, H, _ = q.shape
    dt = q.dtype
    if o_layout == "planes":
        o = torch.full((H, t, 64), SENTINEL, dtype=dt, device="cuda").permute(1, 0, 2)
    elif o_layout == "wide":
        o = torch.full((t, H + 3, 72), SENTINEL, dtype=dt, device="cuda")[:, 1:H + 1, :64]
    else:
        o = torch.full((t, H, 64), SENTINEL, dtype=dt, device="cuda")
    L = torch.full((H, t), SENTINEL, device="cuda") if lse else None
    s = api.PackedShape(t, len(cu) - 1, H, k.shape[1], causal=causal, scale=scale, dtype=dt)
    api.attn_packed_fwd(s, q, k, v, i32(torch, cu), o, L, stream=stream)
    return o, L


def check_packed(torch, q, k, v, cu, causal, o, L, scale=0.125):
    inside = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for rows, eo, el, to, tl in packed64(q, k, v, cu, causal, scale):
        check(o[rows], eo, to, "O of rows %s" % rows)
        if L is not None:
            check(L[:, rows], el, tl, "L of rows %s" % rows)
        inside[rows] = True
    assert (o[~inside] == SENTINEL).all(), "a row outside the sequences was written"
    if L is not None:
        assert (L[:, ~inside] == SENTINEL).all()


PACKS = [[1], [0], [2], [0, 3, 0, 0, 5, 0], [63, 64, 65], [127, 128, 129], [1] * 300,
         [300, 1, 517, 32, 33, 31], [1025], [5, 900, 4, 3], list(range(0, 60, 3))]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads", [(2, 1), (4, 4), (8, 2), (15, 5), (8, 1), (7, 1)])
@pytest.mark.parametrize("pack", range(len(PACKS)))
def test_packed(torch, dtype, heads, pack):
    H, Hkv = heads
    lens = PACKS[pack]
    cu = scan(lens)
    if pack % 2:  # rows before the first sequence and behind the last
        cu = [c + 3 for c in cu]
    t = cu[-1] + (5 if pack % 2 else 0)
    if t == 0:
        t = 2
    dt = getattr(torch, dtype)
    q, k, v = packed_inputs(torch, t, H, Hkv, dt, 10 * pack + H,
                            ["fused", "planes", "dense"][(pack + H) % 3])
    for causal in (True, False):
        o, L = run_packed(torch, q, k, v, cu, causal,
                          o_layout=["dense", "wide", "planes"][pack % 3], lse=pack % 4 != 3)
        check_packed(torch, q, k, v, cu, causal, o, L)


@pytest.mark.parametrize("heads", [(128, 1), (100, 1), (65, 1), (34, 2), (33, 1)])
def test_packed_wide_groups(torch, heads):
    H, Hkv = heads
    cu = scan([3, 130, 1, 40])
    q, k, v = packed_inputs(torch, cu[-1], H, Hkv, torch.bfloat16, 5)
    o, L = run_packed(torch, q, k, v, cu)
    check_packed(torch, q, k, v, cu, True, o, L)


@pytest.mark.parametrize("scale", [1.0, 0.01, 3.0])
def test_packed_scales_and_large_scores(torch, scale):
    cu = scan([200, 77])
    q, k, v = packed_inputs(torch, cu[-1], 4, 2, torch.float16, 8)
    q, k = q * 4, k * 4
    o, L = run_packed(torch, q, k, v, cu, scale=scale)
    check_packed(torch, q, k, v, cu, True, o, L, scale)


@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_bad_values_stay_where_they_are_seen(torch, H, Hkv, causal):
    """NaN and infinities in one sequence's keys reach the rows that see them
    and no other: not earlier rows, not the neighbours, not the padding."""
    lens = [40, 200, 3, 129, 260]
    cu = [c + 2 for c in scan(lens)]
    t = cu[-1] + 9
    q, k, v = (x.clone() for x in packed_inputs(torch, t, H, Hkv, torch.float16, 4, "dense"))
    for x in (q, k, v):
        x[:2] = NAN
        x[cu[-1]:] = math.inf
    v[cu[1] + 150, 0, 5] = NAN
    v[cu[1] + 170, 1, 9] = math.inf
    v[cu[3] + 128] = -math.inf
    k[cu[4] + 100, 0] = NAN
    v[cu[4] + 131, 1, 3] = math.inf
    q[cu[2] + 1, 0] = NAN
    o, L = run_packed(torch, q, k, v, cu, causal)
    check_packed(torch, q, k, v, cu, causal, o, L)


def test_packed_long_prompt(torch):
    """Sampled rows of a long prompt."""
    n, H, Hkv = 9001, 4, 2
    q, k, v = packed_inputs(torch, n, H, Hkv, torch.bfloat16, 6)
    o, L = run_packed(torch, q, k, v, [0, n])
    rows = torch.tensor([0, 1, 127, 128, 255, 256, 4095, 4096, 8999, 9000], device="cuda")
    eo, el, to, tl = attend64(q[rows], k, v, rows + 1)
    check(o[rows], eo, to, "O")
    check(L[:, rows], el, tl, "L")


def test_packed_many_units_are_deterministic(torch):
    cu = scan([random.Random(1).randint(1, 700) for _ in range(40)])
    q, k, v = packed_inputs(torch, cu[-1], 8, 2, torch.float16, 7)
    o, L = run_packed(torch, q, k, v, cu)
    for _ in range(3):
        o2, L2 = run_packed(torch, q, k, v, cu)
        assert torch.equal(o, o2) and torch.equal(L, L2)


def test_packed_agrees_with_the_padded_forward(torch):
    """The same rows as attn_fwd computes from padded planes."""
    from causal_streaming_softmax_gb300 import api
    lens, T, H, Hkv = [256, 192, 64], 256, 4, 2
    cu = scan(lens)
    q, k, v = packed_inputs(torch, cu[-1], H, Hkv, torch.float16, 9)
    o, L = run_packed(torch, q, k, v, cu)
    pad = lambda x: torch.stack([torch.nn.functional.pad(
        x[a:b], (0, 0, 0, 0, 0, T - (b - a))).permute(1, 0, 2) for a, b in zip(cu, cu[1:])])
    s = api.Shape(3, T, H, Hkv, seq_lens=i32(torch, lens), v_rows=True)
    bufs = api.Buffers(s, workspace=False)
    api.attn_fwd(s, pad(q).contiguous(), pad(k).contiguous(), pad(v).contiguous(), bufs.o, bufs.lse)
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        _, _, to, tl = attend64(q[a:b], k[a:b], v[a:b],
                                torch.arange(1, b - a + 1, device="cuda"))
        check(bufs.o[i, :b - a].view(b - a, H, 64), o[a:b].double(), 2 * to, "padded O")
        check(bufs.lse[i, :, :b - a], L[:, a:b].double(), 2 * tl, "padded L")


# ---------------------------------------------------------------- paged cache
def paged_problem(torch, reqs, H, Hkv, page, dtype, seed, layout="pages", stale=NAN, pad=0):
    """reqs: (keys in the cache, new tokens).  Places that no request holds are
    ``stale``; unused table entries name pages that do not exist."""
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
        x = rnd(torch, (pages, Hkv, page, 64), dtype, seed + 50 + i)
        x.masked_fill_(~used[:, None, :, None], stale)
        if layout == "rows":  # [page][row][head]
            x = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        elif layout == "both":  # K and V of a page side by side
            x = torch.stack([x, x], 1)[:, i]
        pools.append(x)
    new = [n for _, n in reqs]
    cu = scan(new)
    q = rnd(torch, (cu[-1] + pad, H, 64), dtype, seed + 60, 2.0)
    return q, pools[0], pools[1], table, cu, [n for n, _ in reqs], width


def run_paged(torch, q, kc, vc, table, cu, lens, max_new=None, lse=True, o=None, stream=None):
    from causal_streaming_softmax_gb300 import api
    t, H, _ = q.shape
    B = len(lens)
    s = api.PagedShape(B, t, H, kc.shape[1], kc.shape[2], kc.shape[0], len(table[0]),
                       max_new=max_new or max(1, max(b - a for a, b in zip(cu, cu[1:]))),
                       dtype=q.dtype)
    ws = api.alloc_paged_workspace(s)
    ws.fill_(255)  # its contents mean nothing
    if o is None:
        o = torch.full((t, H, 64), SENTINEL, dtype=q.dtype, device="cuda")
    L = torch.full((H, t), SENTINEL, device="cuda") if lse else None
    api.attn_paged_fwd(s, q, kc, vc, i32(torch, table), i32(torch, cu), i32(torch, lens), ws, o, L,
                       stream=stream)
    return o, L


def check_paged(torch, q, kc, vc, table, cu, lens, o, L):
    inside = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    tt = torch.tensor(table, dtype=torch.int64, device="cuda")
    for rows, eo, el, to, tl in paged64(q, kc, vc, tt, cu, lens):
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
@pytest.mark.parametrize("heads", [(2, 1), (4, 4), (8, 2), (15, 5), (16, 1)])
@pytest.mark.parametrize("reqs", range(len(REQS)))
def test_paged(torch, dtype, heads, reqs):
    H, Hkv = heads
    page = [16, 8, 64, 256, 32, 128, 1024][(reqs + H) % 7]
    p = paged_problem(torch, REQS[reqs], H, Hkv, page, getattr(torch, dtype), 100 * reqs + H,
                      ["pages", "rows", "both"][(reqs + H) % 3], pad=(reqs % 3) * 2)
    q, kc, vc, table, cu, lens, _ = p
    if q.shape[0] == 0:
        q = rnd(torch, (3, H, 64), q.dtype, 1)
    o, L = run_paged(torch, q, kc, vc, table, cu, lens, lse=reqs % 2 == 0)
    check_paged(torch, q, kc, vc, table, cu, lens, o, L)


@pytest.mark.parametrize("heads", [(128, 1), (100, 1), (40, 2), (17, 1), (33, 1)])
@pytest.mark.parametrize("new", [1, 2, 9])
def test_paged_wide_groups(torch, heads, new):
    p = paged_problem(torch, [(500, new), (13, new), (1, 1)], heads[0], heads[1], 16,
                      torch.float16, 3)
    q, kc, vc, table, cu, lens, _ = p
    o, L = run_paged(torch, q, kc, vc, table, cu, lens)
    check_paged(torch, q, kc, vc, table, cu, lens, o, L)


@pytest.mark.parametrize("bound", [1, 4, 40, 1000])
def test_paged_whatever_the_bound_on_new_tokens(torch, bound):
    """max_new is a bound: any value at or above the truth gives the answer."""
    p = paged_problem(torch, [(900, 1), (33, 1), (1, 1)], 8, 2, 32, torch.bfloat16, 4)
    q, kc, vc, table, cu, lens, _ = p
    o, L = run_paged(torch, q, kc, vc, table, cu, lens, max_new=bound)
    check_paged(torch, q, kc, vc, table, cu, lens, o, L)


@pytest.mark.parametrize("new", [2, 5, 64, 150])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2)])
def test_paged_bad_values_stay_where_they_are_seen(torch, new, H, Hkv):
    """A NaN among the new tokens' keys does not reach the rows before it."""
    p = paged_problem(torch, [(300, new), (new, new), (260, 1)], H, Hkv, 16, torch.float16, 5,
                      stale=math.inf)
    q, kc, vc, table, cu, lens, _ = p
    for req, back in ((0, 1), (1, new // 2)):
        pos = lens[req] - max(1, back)
        pg = table[req][pos // 16]
        vc[pg, 0, pos % 16, 7] = NAN
        vc[pg, 1, pos % 16, 9] = math.inf
    pos = lens[0] - new // 2 - 1
    kc[table[0][pos // 16], 1, pos % 16, 3] = NAN
    o, L = run_paged(torch, q, kc, vc, table, cu, lens)
    check_paged(torch, q, kc, vc, table, cu, lens, o, L)


def test_paged_is_deterministic(torch):
    reqs = [(random.Random(i).randint(1, 3000), 1 + (i % 7 == 0) * 40) for i in range(60)]
    q, kc, vc, table, cu, lens, _ = paged_problem(torch, reqs, 8, 2, 16, torch.float16, 6)
    o, L = run_paged(torch, q, kc, vc, table, cu, lens)
    for _ in range(3):
        o2, L2 = run_paged(torch, q, kc, vc, table, cu, lens)
        assert torch.equal(o, o2) and torch.equal(L, L2)


def test_paged_strided_output_and_queries(torch):
    q, kc, vc, table, cu, lens, _ = paged_problem(torch, [(90, 3), (700, 20), (5, 1)], 8, 2, 16,
                                                  torch.bfloat16, 7)
    t = q.shape[0]
    wide = torch.zeros((t, 12, 64), dtype=q.dtype, device="cuda")
    wide[:, 2:10] = q
    o = torch.full((8, t, 64), SENTINEL, dtype=q.dtype, device="cuda").permute(1, 0, 2)
    o, L = run_paged(torch, wide[:, 2:10], kc, vc, table, cu, lens, o=o)
    check_paged(torch, q, kc, vc, table, cu, lens, o, L)


# ------------------------------------------------------------- plan and store
def run_plan(torch, cached, fresh, ring, state, table, tokens, page, width):
    from causal_streaming_softmax_gb300 import api
    B, N = len(cached), len(ring)
    s = api.PagedShape(B, tokens, 1, 1, page, N, width)
    out = {n: torch.full((k,), -99, dtype=torch.int32, device="cuda")
           for n, k in (("cu", B + 1), ("lens", B), ("slots", tokens), ("next", 4))}
    ring, table = i32(torch, ring), i32(torch, table)
    api.attn_paged_plan(s, i32(torch, cached), i32(torch, fresh), ring, i32(torch, state), table,
                        out["cu"], out["lens"], out["slots"], out["next"])
    return [out["cu"].tolist(), out["lens"].tolist(), out["slots"].tolist(), ring.tolist(),
            table.tolist(), out["next"].tolist()]


@pytest.mark.parametrize("B,page,hi,new", [(1, 16, 100, 1), (1, 8, 0, 5000), (7, 16, 300, 90),
                                           (64, 16, 900, 1), (513, 32, 200, 30),
                                           (4096, 8, 40, 9), (33, 1024, 3000, 2000)])
@pytest.mark.parametrize("trouble", ["", "pages", "width", "tokens", "state", "negative", "full"])
def test_plan(torch, B, page, hi, new, trouble):
    r = random.Random(B + page)
    cached = [r.randint(0, hi) for _ in range(B)]
    fresh = [r.choice([-1, 0, 1, r.randint(0, new)]) for _ in range(B)]
    up = lambda x: -(-x // page)
    width = max(1, max(up(c + max(0, f)) for c, f in zip(cached, fresh)))
    held = sum(up(c) for c in cached)
    need = sum(up(c + f) - up(c) for c, f in zip(cached, fresh) if f > 0)
    total = sum(max(0, f) for f in fresh)
    if trouble in ("", "pages", "full"):
        spare = {"": 3, "pages": -1, "full": 0}[trouble]
    else:
        spare = 3
    if trouble == "pages" and need == 0:
        pytest.skip("needs no page")
    N = max(1, held + need + max(0, spare) if trouble != "pages" else held + need)
    order = list(range(N))
    r.shuffle(order)
    table = []
    for c in cached:
        table.append([order.pop() for _ in range(up(c))] + [-1] * (width - up(c)))
    free = need - 1 if trouble == "pages" else len(order)
    head = r.randrange(N)
    ring = [-5] * N
    for x, p in enumerate(order[:free]):
        ring[(head + x) % N] = p
    tokens = total + r.choice([0, 5])
    if trouble == "width":
        cached[B // 2], fresh[B // 2] = width * page, 1
    if trouble == "tokens":
        fresh[-1], tokens = max(1, fresh[-1]), 0
    if trouble == "state":
        head = N
    if trouble == "negative":
        cached[0] = -3
    want = plan_host(cached, fresh, ring, [head, free], table, tokens, page, width)
    assert (want[5][3] != 0) == (trouble not in ("", "full"))
    got = run_plan(torch, cached, fresh, ring, [head, free, 0, 0], table, tokens, page, width)
    for name, g, w in zip(("cu", "lens", "slots", "ring", "table", "next"), got, want):
        assert g == list(w), name


def test_plan_reports_a_page_that_does_not_exist(torch):
    from causal_streaming_softmax_gb300 import api
    got = run_plan(torch, [0, 3], [5, 1], [99, -4, 2, 3], [0, 4, 0, 0], [[-1] * 4, [7, 0, 0, 0]],
                   6, 8, 4)
    assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX
    assert got[2] == [-1] * 6


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("Hkv,page,n", [(1, 16, 1), (8, 16, 64), (5, 32, 999), (3, 8, 5000),
                                        (16, 256, 300)])
@pytest.mark.parametrize("layout", ["pages", "rows"])
def test_store(torch, dtype, Hkv, page, n, layout):
    from causal_streaming_softmax_gb300 import api
    dt = getattr(torch, dtype)
    pages = -(-n // page) + 4
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(pages * page, generator=g)[:n].to(torch.int32)
    slots[::7] = -1
    slots = slots.cuda()
    kv = rnd(torch, (n, 2 * Hkv, 64), dt, n)
    kv[0] = NAN
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    pools = []
    for i in range(2):
        x = rnd(torch, (pages, Hkv, page, 64), dt, 70 + i)
        if layout == "rows":
            x = x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        pools.append(x)
    want = [x.clone() for x in pools]
    live = slots >= 0
    at = slots[live].long()
    for w, x in zip(want, (k, v)):
        w[at // page, :, at % page] = x[live]
    s = api.PagedShape(1, n, Hkv, Hkv, page, pages, 1, dtype=dt)
    api.attn_paged_store(s, k, v, slots, *pools)
    for w, x in zip(want, pools):
        assert torch.equal(w.view(torch.int16), x.contiguous().view(torch.int16).view(w.shape))


def test_store_skips_and_reports_a_slot_past_the_pool(torch):
    from causal_streaming_softmax_gb300 import api
    k = rnd(torch, (3, 1, 64), torch.float16, 1)
    kc = torch.zeros((2, 1, 8, 64), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    s = api.PagedShape(1, 3, 1, 1, 8, 2, 1)
    api.attn_paged_store(s, k, k, i32(torch, [16, 2 ** 31 - 1, 9]), kc, vc)
    assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX
    assert torch.equal(kc[1, 0, 1], k[2, 0]) and int((kc != 0).any(-1).sum()) == 1


# --------------------------------------------------- device arrays that lie
def test_bad_offsets_are_reported(torch):
    from causal_streaming_softmax_gb300 import api
    q, k, v = packed_inputs(torch, 50, 4, 2, torch.float16, 1)
    for cu in ([0, 60], [0, 2 ** 31 - 1], [-5, 50], [0, 30, 20, 50]):
        run_packed(torch, q, k, v, cu)
        assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX, cu


def test_bad_pages_are_reported(torch):
    """A page id outside the pool, a length past the table, offsets past the
    rows: reported, the other requests right."""
    from causal_streaming_softmax_gb300 import api
    for new in (1, 40):
        q, kc, vc, table, cu, lens, width = paged_problem(
            torch, [(200, new), (500, new), (100, new)], 8, 2, 16, torch.float16, 2)
        for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
            tab = [list(r) for r in table]
            tab[1][3] = bad
            o, L = run_paged(torch, q, kc, vc, tab, cu, lens)
            assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX
            tt = torch.tensor(table, device="cuda")
            for i in (0, 2):
                r = paged64(q, kc, vc, tt, cu, lens)[i]
                check(o[r[0]], r[1], r[3], "request %d" % i)
        for bad in (16 * width + 1, 2 ** 31 - 1, -1):
            run_paged(torch, q, kc, vc, [[0] * width] * 3, cu, [200, bad, 100])
            assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX
        run_paged(torch, q, kc, vc, table, [0, new, 2 * new, 3 * new + 1], lens, max_new=new + 1)
        assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX


def test_more_new_tokens_than_the_bound_are_reported(torch):
    from causal_streaming_softmax_gb300 import api
    q, kc, vc, table, cu, lens, _ = paged_problem(torch, [(200, 40), (500, 1)], 8, 2, 16,
                                                  torch.float16, 2)
    run_paged(torch, q, kc, vc, table, cu, lens, max_new=1)
    assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX


# ------------------------------------------------------------------- together
def serve(torch, steps, graph=None):
    """A small server: requests come, grow by chunks and tokens, and finish.
    Returns every row's output beside the row's request and position."""
    from causal_streaming_softmax_gb300 import api
    H, Hkv, B, page = 8, 2, 5, 16
    cache = api.PagedCache(B, H, Hkv, num_pages=90, page_size=page, table_width=40)
    r = random.Random(11)
    hist = [[] for _ in range(B)]
    for step in range(steps):
        fresh = [r.choice([1, 1, 1, r.randint(0, 70), -1 if len(hist[i]) > 150 else 1])
                 for i in range(B)]
        n = sum(max(0, f) for f in fresh)
        q, k, v = packed_inputs(torch, n, H, Hkv, torch.float16, 1000 + step)
        o = torch.empty((n, H, 64), dtype=torch.float16, device="cuda")
        L = torch.empty((H, n), device="cuda")
        cache.step(i32(torch, fresh), q, k, v, o, L, max_new=max(max(fresh), 1))
        at = 0
        for i, f in enumerate(fresh):
            if f < 0:
                hist[i] = []
                continue
            hist[i] += [(k[at + x], v[at + x]) for x in range(f)]
            m = len(hist[i])
            if f:
                ks = torch.stack([x[0] for x in hist[i]])
                vs = torch.stack([x[1] for x in hist[i]])
                seen = torch.arange(m - f + 1, m + 1, device="cuda")
                eo, el, to, tl = attend64(q[at:at + f], ks, vs, seen)
                check(o[at:at + f], eo, to, "step %d request %d" % (step, i))
                check(L[:, at:at + f], el, tl, "L of step %d request %d" % (step, i))
            at += f
        assert cache.status() == 0
        assert cache.lens.tolist() == [len(h) for h in hist]
        assert cache.free_pages() == 90 - sum(-(-len(h) // page) for h in hist)


def test_a_server_of_several_steps(torch):
    serve(torch, 25)


def test_prompt_through_the_cache_equals_the_packed_prompt(torch):
    """A prompt in chunks over the cache gives what attn_packed_fwd gives."""
    from causal_streaming_softmax_gb300 import api
    H, Hkv, n = 8, 2, 700
    q, k, v = packed_inputs(torch, n, H, Hkv, torch.bfloat16, 12)
    o, L = run_packed(torch, q, k, v, [0, n])
    _, _, to, tl = attend64(q, k, v, torch.arange(1, n + 1, device="cuda"))
    cache = api.PagedCache(1, H, Hkv, num_pages=50, dtype=torch.bfloat16)
    at = 0
    for c in (1, 3, 200, 1, 129, 366):
        o2 = torch.empty((c, H, 64), dtype=q.dtype, device="cuda")
        L2 = torch.empty((H, c), device="cuda")
        cache.step(i32(torch, [c]), q[at:at + c], k[at:at + c], v[at:at + c], o2, L2, max_new=c)
        check(o2, o[at:at + c].double(), 2 * to[at:at + c], "chunk at %d" % at)
        check(L2, L[:, at:at + c].double(), 2 * tl[:, at:at + c], "L of chunk at %d" % at)
        at += c


def test_a_refused_step_leaves_everything(torch):
    from causal_streaming_softmax_gb300 import api
    cache = api.PagedCache(2, 4, 2, num_pages=4)
    q, k, v = packed_inputs(torch, 70, 4, 2, torch.float16, 1)
    o = torch.full((70, 4, 64), SENTINEL, dtype=torch.float16, device="cuda")
    cache.step(i32(torch, [60, 10]), q, k, v, o)
    assert cache.status() == api.PLAN_PAGES and cache.free_pages() == 4
    assert (o == SENTINEL).all() and (cache.k == 0).all() and cache.lens.tolist() == [0, 0]
    cache.step(i32(torch, [40, 10]), q[:50], k[:50], v[:50], o[:50])
    assert cache.status() == 0 and cache.free_pages() == 0


def test_captured_steps_replay(torch):
    """Two token steps captured into a graph and replayed, on a stream of
    their own: the tokens go on, the plan, store and attention follow."""
    from causal_streaming_softmax_gb300 import api
    H, Hkv, B = 8, 2, 3
    cache = api.PagedCache(B, H, Hkv, num_pages=60)
    plen = [37, 5, 130]
    q, k, v = packed_inputs(torch, sum(plen), H, Hkv, torch.float16, 20)
    o = torch.empty((sum(plen), H, 64), dtype=torch.float16, device="cuda")
    cache.step(i32(torch, plen), q, k, v, o, max_new=130)
    cu = scan(plen)
    hist = [[(k[j], v[j]) for j in range(a, b)] for a, b in zip(cu, cu[1:])]
    one = i32(torch, [1] * B)
    buf = [[x.clone() for x in packed_inputs(torch, B, H, Hkv, torch.float16, 21)]
           + [torch.empty((B, H, 64), dtype=torch.float16, device="cuda")] for _ in range(2)]
    # a warm-up pair of steps outside the graph
    for qs, ks, vs, out in buf:
        cache.step(one, qs, ks, vs, out, max_new=1)
        for i in range(B):
            hist[i].append((ks[i].clone(), vs[i].clone()))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        for qs, ks, vs, out in buf:
            cache.step(one, qs, ks, vs, out, max_new=1)
    for rep in range(40):
        for s, b in enumerate(buf):
            for x, y in zip(b, packed_inputs(torch, B, H, Hkv, torch.float16, 100 + 2 * rep + s)):
                x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        for qs, ks, vs, out in buf:
            for i in range(B):
                hist[i].append((ks[i].clone(), vs[i].clone()))
        if rep % 13 == 0:
            qs, ks, vs, out = buf[1]
            for i in range(B):
                kk, vv = (torch.stack([h[j] for h in hist[i]]) for j in (0, 1))
                seen = torch.tensor([len(hist[i])], device="cuda")
                eo, _, to, _ = attend64(qs[i:i + 1], kk, vv, seen)
                check(out[i:i + 1], eo, to, "replay %d request %d" % (rep, i))
    assert cache.lens.tolist() == [len(h) for h in hist] and cache.status() == 0


def test_calls_on_two_streams(torch):
    """The same problem on two streams at once, each with its own workspace."""
    q, kc, vc, table, cu, lens, _ = paged_problem(torch, [(3000, 1), (40, 1)] * 8, 8, 2, 16,
                                                  torch.float16, 9)
    o, L = run_paged(torch, q, kc, vc, table, cu, lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([run_paged(torch, q, kc, vc, table, cu, lens) for _ in range(5)])
    torch.cuda.synchronize()
    for per in got:
        for o2, L2 in per:
            assert torch.equal(o, o2) and torch.equal(L, L2)


def test_pool_beyond_32_bits(torch):
    """Element offsets past 2^32 in the pools."""
    from causal_streaming_softmax_gb300 import api
    H, Hkv, page = 8, 4, 1024
    pages = (1 << 32) // (Hkv * page * 64) + 3  # 8.6 GB a pool
    kc = torch.zeros((pages, Hkv, page, 64), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    table = [[pages - 1, 0, pages - 2]]
    n = 2500
    k, v = (rnd(torch, (n, Hkv, 64), torch.float16, i) for i in (1, 2))
    slots = torch.tensor([table[0][p // page] * page + p % page for p in range(n)],
                         dtype=torch.int32, device="cuda")
    s = api.PagedShape(1, n, H, Hkv, page, pages, 3)
    api.attn_paged_store(s, k, v, slots, kc, vc)
    assert torch.equal(gather(kc, torch.tensor(table[0], device="cuda"), n), k)
    for new in (1, 100):
        q = rnd(torch, (new, H, 64), torch.float16, 3, 2.0)
        o, L = run_paged(torch, q, kc, vc, table, [0, new], [n])
        check_paged(torch, q, kc, vc, table, [0, new], [n], o, L)


def test_requests_that_share_pages(torch):
    """Two requests over the same pages (a prompt's common beginning) read
    them alike, each to its own length."""
    for new in (1, 30):
        q, kc, vc, table, cu, lens, _ = paged_problem(torch, [(400, new), (400, new), (90, new)],
                                                      8, 2, 16, torch.float16, 13)
        table[1], lens = list(table[0]), [400, 333, 90]
        o, L = run_paged(torch, q, kc, vc, table, cu, lens)
        check_paged(torch, q, kc, vc, table, cu, lens, o, L)


@pytest.mark.parametrize("heads", [(2, 1), (17, 1)])
def test_the_largest_batch(torch, heads):
    reqs = [(i % 50, min(1, i % 50)) for i in range(4096)]
    q, kc, vc, table, cu, lens, _ = paged_problem(torch, reqs, heads[0], heads[1], 8,
                                                  torch.bfloat16, 14)
    o, L = run_paged(torch, q, kc, vc, table, cu, lens)
    pick = [0, 1, 2, 49, 50, 99, 2047, 4001, 4095]
    tt = torch.tensor([table[i] for i in pick], device="cuda")
    for i, row in zip(pick, tt):
        a, b, m = cu[i], cu[i + 1], lens[i]
        seen = torch.full((b - a,), m, device="cuda")
        eo, el, to, tl = attend64(q[a:b], gather(kc, row, m), gather(vc, row, m), seen)
        check(o[a:b], eo, to, "request %d" % i)
        check(L[:, a:b], el, tl, "L of request %d" % i)
    assert torch.isfinite(o).all()


def test_many_empty_sequences(torch):
    r = random.Random(2)
    lens = [0] * 65535
    for i in r.sample(range(65535), 700):
        lens[i] = r.randint(1, 3)
    cu = scan(lens)
    q, k, v = packed_inputs(torch, cu[-1], 4, 2, torch.float16, 15)
    o, L = run_packed(torch, q, k, v, cu)
    live = [0] + [c for c, n in zip(cu[1:], lens) if n]  # the same without the empty ones
    check_packed(torch, q, k, v, live, True, o, L)


def test_step_on_a_stream_of_its_own(torch):
    from causal_streaming_softmax_gb300 import api
    n = 90
    q, k, v = packed_inputs(torch, n, 8, 2, torch.float16, 16)
    cache = api.PagedCache(1, 8, 2, num_pages=20)
    o = torch.empty((n, 8, 64), dtype=torch.float16, device="cuda")
    fresh = [i32(torch, [50]), i32(torch, [40])]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    cache.step(fresh[0], q[:50], k[:50], v[:50], o[:50], stream=s)
    cache.step(fresh[1], q[50:], k[50:], v[50:], o[50:], stream=s)
    s.synchronize()
    check_packed(torch, q, k, v, [0, n], True, o, None)


def test_step_refuses_before_it_plans(torch):
    from causal_streaming_softmax_gb300 import api
    q, k, v = packed_inputs(torch, 10, 4, 2, torch.float16, 17)
    cache = api.PagedCache(1, 4, 2, num_pages=5)
    o = torch.empty((10, 4, 64), dtype=torch.float16, device="cuda")
    for bad in (dict(k=k[:9]), dict(o=o[:, :3]), dict(v=v.float()), dict(q=q.cpu()),
                dict(lse=torch.empty((4, 9), device="cuda"))):
        args = dict(dict(q=q, k=k, v=v, o=o, lse=None), **bad)
        with pytest.raises((ValueError, TypeError)):
            cache.step(i32(torch, [10]), **args)
    assert cache.lens.tolist() == [0] and cache.free_pages() == 5
    cache.step(i32(torch, [10]), q, k, v, o)
    assert cache.lens.tolist() == [10]


def test_step_refuses_layouts_before_it_plans(torch):
    """Strides, alignment, rows that overlap and max_new, which the entry points
    behind the plan refuse too, leave the cache as it was."""
    from causal_streaming_softmax_gb300 import api
    q, k, v = packed_inputs(torch, 10, 4, 2, torch.float16, 17)
    cache = api.PagedCache(1, 4, 2, num_pages=5)
    o = torch.empty((10, 4, 64), dtype=torch.float16, device="cuda")
    room = torch.empty(10 * 4 * 72 + 8, dtype=torch.float16, device="cuda")
    floats = torch.empty(41, device="cuda")
    for bad in (dict(k=k[:, :1].expand(10, 2, 64)),               # a stride of 0
                dict(v=room.as_strided((10, 2, 64), (132, 66, 1))),  # not a multiple of 8
                dict(q=room.as_strided((10, 4, 64), (256, 64, 1), 4)),  # starts on 8 bytes
                dict(o=room.as_strided((10, 4, 64), (256, 64, 1), 1)),
                dict(o=room.as_strided((10, 4, 64), (64, 72, 1))),   # rows overlap
                dict(lse=floats[1:].view(4, 10)),
                dict(max_new=-1), dict(max_new=(1 << 30) + 1)):
        args = dict(dict(q=q, k=k, v=v, o=o), **bad)
        with pytest.raises(ValueError):
            cache.step(i32(torch, [10]), **args)
        assert cache.lens.tolist() == [0] and cache.free_pages() == 5
    lse = torch.empty((4, 10), device="cuda")
    cache.step(i32(torch, [10]), q, k, v, o, lse)
    assert cache.lens.tolist() == [10]
    check_packed(torch, q, k, v, [0, 10], True, o, lse)


FIRST_CALL = """
import torch
from causal_streaming_softmax_gb300 import api
g = torch.cuda.CUDAGraph()
cache = api.PagedCache(2, 8, 2, num_pages=40)
x = torch.randn(60, 12, 64, device="cuda", dtype=torch.float16)
q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
o = torch.zeros(60, 8, 64, device="cuda", dtype=torch.float16)
p = torch.zeros_like(o)
fresh = torch.tensor([60, 0], dtype=torch.int32, device="cuda")
done = torch.tensor([-1, -1], dtype=torch.int32, device="cuda")
cu = torch.tensor([0, 60, 60], dtype=torch.int32, device="cuda")
none = torch.empty(0, 12, 64, device="cuda", dtype=torch.float16)
torch.cuda.synchronize()
with torch.cuda.graph(g):
    cache.step(fresh, q, k, v, o, max_new=60)
    cache.step(done, none[:, :8], none[:, 8:10], none[:, 10:], none[:, :8])
    api.attn_packed_fwd(api.PackedShape(60, 2, 8, 2), q, k, v, cu, p)
for _ in range(3):
    o.zero_(), p.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert api.last_device_error() == 0
    assert cache.status() == 0 and cache.free_pages() == 40
    assert (o.float() - p.float()).abs().max() < 4e-3 and o.abs().max() > 0
print("fine")
"""


def test_first_calls_inside_a_capture(torch):
    """A process whose first calls are captured: nothing has been loaded or
    set up before."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


def test_a_captured_step_outlives_larger_steps(torch):
    """A captured token step replays after steps that need more workspace."""
    from causal_streaming_softmax_gb300 import api
    cache = api.PagedCache(1, 8, 2, num_pages=300)
    q, k, v = packed_inputs(torch, 3000, 8, 2, torch.float16, 18)
    o = torch.empty((3000, 8, 64), dtype=torch.float16, device="cuda")
    one, two = i32(torch, [1]), torch.empty((2, 1, 8, 64), dtype=torch.float16, device="cuda")
    cache.step(i32(torch, [500]), q[:500], k[:500], v[:500], o[:500], max_new=500)
    qs, ks, vs = q[500:501].clone(), k[500:501].clone(), v[500:501].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for x in two:
            cache.step(one, qs, ks, vs, x, max_new=1)
    g.replay()
    cache.step(i32(torch, [2000]), q[502:2502], k[502:2502], v[502:2502], o[502:2502])
    cache.step(i32(torch, [498]), q[2502:], k[2502:], v[2502:], o[2502:])
    junk = [torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda") for _ in range(20)]
    g.replay()
    torch.cuda.synchronize()
    assert all((j == -1).all() for j in junk)
    kk = torch.cat([k[:500], ks, ks, k[502:], ks, ks])
    vv = torch.cat([v[:500], vs, vs, v[502:], vs, vs])
    eo, _, to, _ = attend64(qs, kk, vv, torch.tensor([kk.shape[0]], device="cuda"))
    check(two[1], eo, to, "replayed step")
    assert cache.lens.tolist() == [kk.shape[0]] and cache.status() == 0


def test_both_marshalling_paths(torch, monkeypatch):
    """The calls through the native marshaller and through Python's checks
    (another stream, or a case the marshaller leaves) do the same."""
    from causal_streaming_softmax_gb300 import api
    q, k, v = packed_inputs(torch, 300, 8, 2, torch.bfloat16, 19)
    paged = paged_problem(torch, [(400, 1), (90, 30), (7, 1)], 8, 2, 16, torch.float16, 20, "rows")

    def everything():
        cache = api.PagedCache(2, 8, 2, num_pages=30, dtype=torch.bfloat16)
        o = torch.zeros((300, 8, 64), dtype=torch.bfloat16, device="cuda")
        cache.step(i32(torch, [200, 100]), q, k, v, o)
        return run_packed(torch, q, k, v, [0, 120, 300], o_layout="wide") + \
            run_packed(torch, q, k, v, [0, 120, 300], causal=False, lse=False)[:1] + \
            run_paged(torch, *paged[:6]) + (o, cache.k, cache.v, cache.table, cache.lens)

    api.load_library()
    assert api._native is not None
    native = everything()
    with monkeypatch.context() as m:
        m.setattr(api, "_native", None)
        python = everything()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, L = run_packed(torch, q, k, v, [0, 120, 300], stream=side)
    side.synchronize()
    for a, b in zip(native + (native[0],), python + (o,)):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_python_names_what_is_wrong(torch):
    from causal_streaming_softmax_gb300 import api
    n, H, Hkv = 10, 4, 2
    q, k, v = packed_inputs(torch, n, H, Hkv, torch.float16, 21)
    cu, o = i32(torch, [0, n]), torch.empty((n, H, 64), dtype=torch.float16, device="cuda")
    s = api.PackedShape(n, 1, H, Hkv)
    call = lambda **kw: api.attn_packed_fwd(**dict(dict(s=s, q=q, k=k, v=v, cu=cu, o=o), **kw))
    call()
    for kw, err, word in [
            (dict(q=q.bfloat16()), TypeError, "q must be torch.float16"),
            (dict(k=k[:9]), ValueError, "k must have shape"),
            (dict(v=v.cpu()), ValueError, "v must be a CUDA tensor"),
            (dict(cu=cu.long()), TypeError, "cu must be torch.int32"),
            (dict(cu=i32(torch, [0, 3, n])), ValueError, "cu must have shape"),
            (dict(o=o.transpose(1, 2).contiguous().transpose(1, 2)), ValueError, "dense in its last"),
            (dict(lse=torch.empty((n, H), device="cuda").t()), ValueError, "lse must be contiguous"),
            (dict(q=None), TypeError, "q must be a torch tensor"),
            (dict(s=api.PackedShape(n, 1, H, Hkv, dtype=torch.float32)), TypeError, "float32"),
            (dict(s=api.PackedShape(1 << 40, 1, H, Hkv)), ValueError, "shape"),
            (dict(s=api.PackedShape(n, 1, H, Hkv, scale=0.0)), api.AttnError, "admission"),
            (dict(o=o[:1].expand(n, H, 64)), api.AttnError, "admission"),
            (dict(q=torch.empty(n * H * 64 + 1, dtype=torch.float16, device="cuda")[1:]
                  .view(n, H, 64)), api.AttnError, "16-byte aligned")]:
        with pytest.raises(err, match=word):
            call(**kw)
    p = api.PagedShape(1, n, H, Hkv, 16, 4, 4, max_new=n)
    with pytest.raises(TypeError, match="ws must be"):
        api.attn_paged_fwd(p, q, torch.empty((4, Hkv, 16, 64), dtype=torch.float16, device="cuda"),
                           torch.empty((4, Hkv, 16, 64), dtype=torch.float16, device="cuda"),
                           i32(torch, [[0, 1, 2, 3]]), cu, i32(torch, [n]),
                           torch.empty(1 << 26, device="cuda"), o)
    with pytest.raises(api.AttnError, match="workspace"):
        api.attn_paged_fwd(p, q, torch.empty((4, Hkv, 16, 64), dtype=torch.float16, device="cuda"),
                           torch.empty((4, Hkv, 16, 64), dtype=torch.float16, device="cuda"),
                           i32(torch, [[0, 1, 2, 3]]), cu, i32(torch, [n]),
                           torch.empty(1 << 10, dtype=torch.uint8, device="cuda"), o)


def step_rows(torch, n, seed, H=8, Hkv=2):
    return [x.clone() for x in packed_inputs(torch, n, H, Hkv, torch.float16, seed)]


@pytest.mark.parametrize("captured", [1, 2, 3])
@pytest.mark.parametrize("between", [0, 1, 2, 3])
def test_captured_steps_between_eager_ones(torch, captured, between):
    """A graph of any number of steps replays after any number of eager steps:
    each step goes on from the lengths and pages that the one before it left."""
    from causal_streaming_softmax_gb300 import api
    cache = api.PagedCache(2, 8, 2, num_pages=60)
    hist = [[], []]

    def note(fresh, k, v):
        at = 0
        for i, f in enumerate(fresh):
            hist[i] += [(k[at + x], v[at + x]) for x in range(f)]
            at += f

    def eager(fresh, seed):
        n = sum(fresh)
        q, k, v = step_rows(torch, n, seed)
        cache.step(i32(torch, fresh), q, k, v, torch.empty_like(q), max_new=max(fresh))
        note(fresh, k, v)

    eager([37, 5], 1)
    one = i32(torch, [1, 1])
    rows = [step_rows(torch, 2, 10 + i) for i in range(captured)]
    outs = [torch.empty_like(r[0]) for r in rows]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for (q, k, v), o in zip(rows, outs):
            cache.step(one, q, k, v, o, max_new=1)
    for rep in range(3):
        g.replay()
        for (q, k, v), o in zip(rows, outs):
            note([1, 1], k, v)
        assert cache.lens.tolist() == [len(h) for h in hist], "replay %d" % rep
        for i in range(2):
            kk, vv = (torch.stack([h[j] for h in hist[i]]) for j in (0, 1))
            seen = torch.tensor([len(hist[i])], device="cuda")
            eo, _, to, _ = attend64(rows[-1][0][i:i + 1], kk, vv, seen)
            check(outs[-1][i:i + 1], eo, to, "replay %d request %d" % (rep, i))
        for x in range(between):
            eager([19, 1], 100 * rep + x)
        assert cache.lens.tolist() == [len(h) for h in hist]
        assert cache.status() == 0
        assert cache.free_pages() == 60 - sum(-(-len(h) // 16) for h in hist)


def test_status_follows_a_step_on_another_stream(torch):
    """status() and free_pages() wait for the last step, whichever stream it is on."""
    from causal_streaming_softmax_gb300 import api
    q, k, v = packed_inputs(torch, 50, 8, 2, torch.float16, 23)
    o, fresh, gone = torch.empty_like(q), i32(torch, [50]), i32(torch, [500])
    cache = api.PagedCache(1, 8, 2, num_pages=20)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # a tenth of a second
    cache.step(fresh, q, k, v, o, stream=side)
    assert cache.free_pages() == 20 - 4
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    cache.step(gone, q, k, v, o, stream=side)
    assert cache.status() == api.PLAN_PAGES | api.PLAN_WIDTH | api.PLAN_TOKENS
    assert cache.lens.tolist() == [50]


@pytest.mark.parametrize("heads", [(8, 2), (4, 4), (17, 1)])
@pytest.mark.parametrize("bound", [1, 3, 4, 5, 16, 20, 39])
def test_requests_with_more_new_tokens_than_the_bound_are_left_out(torch, heads, bound):
    """Their rows stay as they were, also where their keys are split over
    blocks; the other requests are right."""
    from causal_streaming_softmax_gb300 import api
    reqs = [(2000, 40), (500, bound), (64, 1), (9000, bound + 1), (33, bound)]
    q, kc, vc, table, cu, lens, _ = paged_problem(torch, reqs, heads[0], heads[1], 16,
                                                  torch.float16, 24)
    o, L = run_paged(torch, q, kc, vc, table, cu, lens, max_new=bound)
    assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX
    tt = torch.tensor(table, dtype=torch.int64, device="cuda")
    for i, (rows, eo, el, to, tl) in enumerate(paged64(q, kc, vc, tt, cu, lens)):
        if reqs[i][1] > bound:
            assert (o[rows] == SENTINEL).all() and (L[:, rows] == SENTINEL).all(), i
        else:
            check(o[rows], eo, to, "O of request %d" % i)
            check(L[:, rows], el, tl, "L of request %d" % i)


@pytest.mark.parametrize("bad", [-1, 9, 2 ** 31 - 1, -2 ** 31])
def test_plan_reports_a_retired_page_that_does_not_exist(torch, bad):
    """A finished request whose table row names no page of the pool."""
    from causal_streaming_softmax_gb300 import api
    got = run_plan(torch, [20, 3], [-1, 1], [6, 7, 8, -4, -4, -4, -4, -4, -4], [0, 3, 0, 0],
                   [[0, bad, 2], [4, 0, 0]], 1, 8, 3)
    assert api.last_device_error() == api.ATTN_ERR_DEVICE_INDEX
    assert got[0] == [0, 0, 1] and got[1] == [0, 4] and got[2] == [4 * 8 + 3]
    assert got[5] == [0, 6, 0, 0]


@pytest.mark.parametrize("new", [1, 40])
def test_a_workspace_that_something_else_writes(torch, new):
    """While another stream writes the workspace the outputs mean nothing, but
    nothing outside the rows is written and the next call is right."""
    from causal_streaming_softmax_gb300 import api
    q, kc, vc, table, cu, lens, _ = paged_problem(torch, [(3000, new), (4000, new)] * 4, 8, 2, 16,
                                                  torch.float16, 27)
    t = q.shape[0]
    s = api.PagedShape(8, t, 8, 2, 16, kc.shape[0], len(table[0]), max_new=new)
    ws = api.alloc_paged_workspace(s)
    room = torch.full((t + 64, 8, 64), SENTINEL, dtype=q.dtype, device="cuda")
    floats = torch.full((8 * t + 64,), SENTINEL, device="cuda")
    o, L = room[32:32 + t], floats[32:32 + 8 * t].view(8, t)
    args = (s, q, kc, vc, i32(torch, table), i32(torch, cu), i32(torch, lens), ws, o, L)
    junk = torch.randint(-2 ** 31, 2 ** 31 - 1, (ws.numel() // 4,), device="cuda", dtype=torch.int32,
                         generator=torch.Generator(device="cuda").manual_seed(1))
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(60):
        with torch.cuda.stream(other):
            for j in range(4):
                ws.view(torch.int32).copy_(junk if (i + j) % 2 else junk & 15)
        api.attn_paged_fwd(*args)
    torch.cuda.synchronize()
    assert api.last_device_error() in (0, api.ATTN_ERR_DEVICE_INDEX)
    for x in (room[:32], room[32 + t:], floats[:32], floats[32 + 8 * t:]):
        assert (x == SENTINEL).all()
    api.attn_paged_fwd(*args)
    check_paged(torch, q, kc, vc, table, cu, lens, o, L)


@pytest.mark.parametrize("heads", [(8, 2), (16, 1), (3, 3)])
@pytest.mark.parametrize("hi", [1, 5, 120])
def test_arrays_that_something_else_writes(torch, heads, hi):
    """While another stream writes the lengths, offsets and pages of a call its
    outputs mean nothing, but it ends, and nothing outside the rows is written;
    the next call is right."""
    from causal_streaming_softmax_gb300 import api
    H, Hkv = heads
    r = random.Random(hi)
    reqs = [(r.randint(hi, 3000), r.randint(1, hi)) for _ in range(40)]
    q, kc, vc, table, cu, lens, width = paged_problem(torch, reqs, H, Hkv, 16, torch.float16, 28)
    t, pages = q.shape[0], kc.shape[0]
    s = api.PagedShape(40, t, H, Hkv, 16, pages, width, max_new=hi)
    ws = api.alloc_paged_workspace(s)
    room = torch.full((t + 64, H, 64), SENTINEL, dtype=q.dtype, device="cuda")
    floats = torch.full((H * t + 64,), SENTINEL, device="cuda")
    o, L = room[32:32 + t], floats[32:32 + H * t].view(H, t)
    good = [i32(torch, x) for x in (table, cu, lens)]
    live = [x.clone() for x in good]
    others = []  # other lengths, offsets and pages, right and wrong ones
    for _ in range(6):
        at = sorted(r.randint(0, t) for _ in range(39))
        others.append([i32(torch, x) for x in (
            [[r.randint(-1, pages) for _ in range(width)] for _ in reqs],
            r.choice([[0] + at + [t], [r.randint(-9, t + 9) for _ in range(41)]]),
            [r.choice([0, 1, 16 * width, r.randint(0, 16 * width), -5, 2 ** 31 - 1]) for _ in reqs])])
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(60):
        with torch.cuda.stream(other):
            for j in range(5):
                for a, b in zip(live, others[(i + j) % 6]):
                    a.copy_(b)
        api.attn_paged_fwd(s, q, kc, vc, *live, ws, o, L)
    torch.cuda.synchronize()
    assert api.last_device_error() in (0, api.ATTN_ERR_DEVICE_INDEX)
    for x in (room[:32], room[32 + t:], floats[:32], floats[32 + H * t:]):
        assert (x == SENTINEL).all()
    api.attn_paged_fwd(s, q, kc, vc, *good, ws, o, L)
    check_paged(torch, q, kc, vc, table, cu, lens, o, L)


def test_plan_of_lengths_that_something_else_writes(torch):
    from causal_streaming_softmax_gb300 import api
    r = random.Random(30)
    B, page, width, N, tokens = 300, 8, 20, 4000, 9000
    s = api.PagedShape(B, tokens, 1, 1, page, N, width)
    room = torch.full((B * width + N + 2 * B + tokens + 600,), -77, dtype=torch.int32, device="cuda")
    at, parts, guards = 0, [], []
    for n in (B * width, N, B + 1, B, tokens, 4):
        guards.append(room[at:at + 64])
        parts.append(room[at + 64:at + 64 + n])
        at += 64 + n
    guards.append(room[at:])
    table, ring, cu, lens, slots, nxt = parts
    table.fill_(0), ring.copy_(torch.arange(N))
    state, fresh = i32(torch, [5, 2000, 0, 0]), i32(torch, [r.choice([0, 1, 30, -1]) for _ in range(B)])
    good = i32(torch, [3] * B)
    live, others = good.clone(), [i32(torch, [r.choice([0, 8, 100, 129, 130, -4, 2 ** 31 - 1, 7])
                                              for _ in range(B)]) for _ in range(6)]
    others += [i32(torch, [r.randint(0, 130) for _ in range(B)]) for _ in range(6)]
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(200):
        with torch.cuda.stream(other):
            for j in range(3):
                live.copy_(others[(i + j) % 12])
        api.attn_paged_plan(s, live, fresh, ring, state, table.view(B, width), cu, lens, slots, nxt)
    torch.cuda.synchronize()
    assert api.last_device_error() in (0, api.ATTN_ERR_DEVICE_INDEX)
    assert all((g == -77).all() for g in guards)
    ring.copy_(torch.arange(N)), table.fill_(0)
    api.attn_paged_plan(s, good, fresh, ring, state, table.view(B, width), cu, lens, slots, nxt)
    want = plan_host([3] * B, fresh.tolist(), list(range(N)), [5, 2000], [[0] * width] * B, tokens,
                     page, width)
    for g, w in zip((cu, lens, slots, ring, table.view(B, width), nxt), want):
        assert g.tolist() == list(w)


def test_the_native_marshaller_takes_ordinary_calls(torch):
    """Called directly: it makes the ordinary calls itself, and leaves alone,
    without doing anything, what it has to leave."""
    from causal_streaming_softmax_gb300 import api
    api.load_library()
    nat, H, Hkv, n = api._native, 8, 2, 40
    q, k, v = packed_inputs(torch, n, H, Hkv, torch.float16, 25)
    cu, o, L = i32(torch, [0, n]), torch.zeros_like(q), torch.zeros((H, n), device="cuda")
    s = api.PackedShape(n, 1, H, Hkv)
    assert nat.packed_fwd(s, q, k, v, cu, o, L) == 0
    assert nat.packed_fwd(s, q, k, v, cu, o, None) == 0
    check_packed(torch, q, k, v, [0, n], True, o, L)
    p = api.PagedShape(1, n, H, Hkv, 16, 5, 4, max_new=n)
    state = [i32(torch, x) for x in ([0], [n], list(range(5)), [0, 5, 0, 0], [[-1] * 4])]
    step = [torch.empty(x, dtype=torch.int32, device="cuda") for x in (2, 1, n, 4)]
    assert nat.paged_plan(p, *state, *step) == 0
    pools = [torch.zeros((5, Hkv, 16, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    assert nat.paged_store(p, k, v, step[2], *pools) == 0
    ws, o2, L2 = api.alloc_paged_workspace(p), torch.zeros_like(q), torch.zeros_like(L)
    assert nat.paged_fwd(p, q, *pools, state[4], step[0], step[1], ws, o2, L2) == 0
    check_packed(torch, q, k, v, [0, n], True, o2, L2)
    # an entry point's refusal comes back as its code
    assert nat.packed_fwd(s, q, k, v, cu, o[:1].expand(n, H, 64), None) == api.ATTN_ERR_SHAPE
    before = o.clone()
    for bad in (dict(q=q.cpu()), dict(q=q.bfloat16()), dict(k=k[:9]), dict(v=None),
                dict(cu=cu.long()), dict(cu=i32(torch, [0, 3, n])), dict(q=q.transpose(1, 2)),
                dict(L=L.t()), dict(s=api.PackedShape(1 << 40, 1, H, Hkv)), dict(s=None),
                dict(s=api.PackedShape(n, 1, H, Hkv, dtype=torch.float32)),
                dict(s=api.PackedShape(n, 1, H, Hkv, scale="1"))):
        a = dict(dict(s=s, q=q, k=k, v=v, cu=cu, o=o, L=L), **bad)
        assert nat.packed_fwd(*(a[x] for x in ("s", "q", "k", "v", "cu", "o", "L"))) is None, bad
    assert nat.paged_plan(p, state[0].cpu(), *state[1:], *step) is None
    assert nat.paged_store(p, k, v, step[2].long(), *pools) is None
    assert nat.paged_fwd(p, q, *pools, state[4], step[0], step[1], ws.float(), o2, L2) is None
    assert nat.paged_fwd(p, q) is None and torch.equal(before, o)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("new", [1, 2, 4])
@pytest.mark.parametrize("page", [8, 64, 256])
def test_bad_values_in_short_tables(torch, dtype, new, page):
    """NaN and infinities among visible keys where the table holds at most 256
    keys and every request is finished by one block."""
    reqs = [(200, new), (new, new), (129, 1), (128, new), (240, 1)]
    q, kc, vc, table, cu, lens, _ = paged_problem(torch, reqs, 8, 2, page, getattr(torch, dtype),
                                                  26, stale=NAN)
    table = [r[:256 // page] for r in table]
    for req, back, head, what in ((0, 1, 0, NAN), (0, 2, 1, math.inf), (1, 1, 1, -math.inf),
                                  (2, 1, 0, math.inf), (3, new, 1, NAN), (4, 240, 0, math.inf)):
        pos = lens[req] - back
        if pos >= 0:
            vc[table[req][pos // page], head, pos % page, 3 + back % 50] = what
    pos = lens[3] - 1
    kc[table[3][pos // page], 0, pos % page, 3] = NAN
    o, L = run_paged(torch, q, kc, vc, table, cu, lens)
    check_paged(torch, q, kc, vc, table, cu, lens, o, L)


def test_offsets_that_something_else_writes(torch):
    """The same of packed prompts."""
    from causal_streaming_softmax_gb300 import api
    H, Hkv, t, B = 8, 2, 3000, 50
    r = random.Random(31)
    q, k, v = packed_inputs(torch, t, H, Hkv, torch.float16, 32)
    room = torch.full((t + 64, H, 64), SENTINEL, dtype=q.dtype, device="cuda")
    floats = torch.full((H * t + 64,), SENTINEL, device="cuda")
    o, L = room[32:32 + t], floats[32:32 + H * t].view(H, t)
    ways = [[0] + sorted(r.randint(0, t) for _ in range(B - 1)) + [t] for _ in range(4)]
    good = i32(torch, ways[0])
    others = [i32(torch, w) for w in ways]
    others += [i32(torch, [r.choice([0, t, t + 1, -1, 2 ** 31 - 1, -2 ** 31, r.randint(0, t)])
                           for _ in range(B + 1)]) for _ in range(4)]
    live, other = good.clone(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(60):
        with torch.cuda.stream(other):
            for j in range(8):
                live.copy_(others[(3 * i + j) % 8])
        api.attn_packed_fwd(api.PackedShape(t, B, H, Hkv, causal=bool(i % 2)), q, k, v, live, o, L)
    torch.cuda.synchronize()
    assert api.last_device_error() in (0, api.ATTN_ERR_DEVICE_INDEX)
    for x in (room[:32], room[32 + t:], floats[:32], floats[32 + H * t:]):
        assert (x == SENTINEL).all()
    api.attn_packed_fwd(api.PackedShape(t, B, H, Hkv), q, k, v, good, o, L)
    check_packed(torch, q, k, v, ways[0], True, o, L)


@pytest.mark.parametrize("n", [1, 3, 40, 200])
def test_rows_whose_every_score_is_minus_infinity(torch, n):
    """Like rows that see no key; the rows that see another key too go on
    without the infinite one."""
    H, Hkv = 8, 2
    q, k, v = packed_inputs(torch, n, H, Hkv, torch.bfloat16, 33, "dense")
    q[..., 5] = -1.0
    k[0, :, 5] = math.inf
    outs = [run_packed(torch, q, k, v, [0, n])]
    if n > 1:
        outs.append(run_packed(torch, q, k, v, [0, 1, n]))
    pool = [torch.zeros((15, Hkv, 16, 64), dtype=q.dtype, device="cuda") for _ in range(2)]
    for p, x in zip(pool, (k, v)):
        for j in range(n):
            p[j // 16, :, j % 16] = x[j]
    outs.append(run_paged(torch, q, *pool, [list(range(15))], [0, n], [n]))
    for i, (o, L) in enumerate(outs):
        assert (o[0] == 0).all() and (L[:, 0] == -math.inf).all(), i
        assert torch.isfinite(o).all() and torch.isfinite(L[:, 1:]).all(), i
        if n > 1:
            eo, el, to, tl = attend64(q[1:], k[1:], v[1:], torch.arange(1, n, device="cuda"))
            check(o[1:], eo, to, "O")
            check(L[:, 1:], el, tl, "L")
