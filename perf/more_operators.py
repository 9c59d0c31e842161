"""The serving operators beside those of perf/operators.py: new tokens into the
paged cache with the position rotation applied on the way, in 16 bits and in
4, rows read back from a 4-bit cache, and attention over one.

A 4-bit pool is uint8 [pages][kv heads][page size / 8][288]: for every eight
tokens 8 x 32 bytes of codes (byte c holds channel c in its low and channel
c + 32 in its high half, each code + 8) and 8 x 2 scales in the cache's type
(channels 0..31 and 32..63).  A group of 32 channels with the extremum e (of
largest magnitude, the negative one of a tie) has the scale s = -e / 8, rounded
to three significant bits fewer than the type has, so that every value
code * s, code in -8..7, is exact in the type; code = x / s to nearest even.

Each case says what it stands for.  Where ``own`` is false ``run`` computes
the operator in elementary torch operations, in 32 bits; where it is true it
makes the calls a user makes of this package.
"""
import math
import random

import torch

own = False

D = 64
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
LN2 = math.log(2.0)
UNIT = 288  # bytes of eight tokens of a 4-bit pool
# of a scale: significant bits, and the largest magnitude
SCALES = {torch.float16: (8, 8160.0), torch.bfloat16: (5, 2.0 ** 123)}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one user's new token into a 16-bit cache: latency
        dict(name="append-one", op="append", dtype="bf16", heads=32, kv_heads=8, page=16, batch=1,
             lo=776, hi=776, decodes=1, new_lo=1, new_hi=1, pad=0, len_seed=21),
        # a server's ordinary token step
        dict(name="append-decode", op="append", dtype="f16", heads=32, kv_heads=8, page=16,
             batch=64, lo=17, hi=2048, decodes=64, new_lo=1, new_hi=1, pad=0, len_seed=22),
        # admitted prompts beside a few running requests, a padded token buffer
        dict(name="append-prompts", op="append", dtype="bf16", heads=32, kv_heads=8, page=16,
             batch=40, lo=0, hi=512, decodes=7, new_lo=100, new_hi=2000, pad=333, len_seed=23),
        # a small server's token step into a 4-bit cache
        dict(name="append4-decode", op="append4", dtype="bf16", heads=32, kv_heads=8, page=16,
             batch=8, lo=5, hi=200, decodes=8, new_lo=1, new_hi=1, pad=0, rotate=True, len_seed=24),
        # prompts of a model whose keys come without rotation into a 4-bit cache
        dict(name="append4-plain", op="append4", dtype="f16", heads=16, kv_heads=16, page=32,
             batch=6, lo=0, hi=100, decodes=0, new_lo=50, new_hi=700, pad=0, rotate=False,
             len_seed=25),
        # admitted prompts into a 4-bit cache
        dict(name="append4-prompts", op="append4", dtype="f16", heads=32, kv_heads=8, page=64,
             batch=24, lo=0, hi=512, decodes=4, new_lo=100, new_hi=2000, pad=77, rotate=True,
             len_seed=26),
        # one request's tokens read back, to hand it to another cache
        dict(name="load4-request", op="load4", dtype="bf16", kv_heads=8, page=16, slots=1111,
             spare=9000, len_seed=27),
        # a whole server's cache read back, some rows of the buffer without a slot
        dict(name="load4-many", op="load4", dtype="f16", kv_heads=4, page=64, slots=150000,
             spare=50000, len_seed=28),
        # one user, one token: the smallest serving step
        dict(name="decode4-one", op="paged4", dtype="bf16", heads=32, kv_heads=8, page=16, batch=1,
             lo=777, hi=777, decodes=1, new_lo=1, new_hi=1, lse=False, len_seed=29),
        # one user with a long history: few rows, a long axis
        dict(name="decode4-long", op="paged4", dtype="f16", heads=16, kv_heads=16, page=32, batch=2,
             lo=50000, hi=65536, decodes=2, new_lo=1, new_hi=1, lse=True, len_seed=30),
        # a large server's token step, every request at another length
        dict(name="decode4-large", op="paged4", dtype="bf16", heads=32, kv_heads=4, page=64,
             batch=256, lo=1024, hi=16384, decodes=256, new_lo=1, new_hi=1, lse=False, len_seed=31),
        # chunks of prompts beside running requests (continuous batching)
        dict(name="chunk4-mixed", op="paged4", dtype="f16", heads=32, kv_heads=8, page=16, batch=36,
             lo=2048, hi=8192, decodes=32, new_lo=301, new_hi=1024, lse=True, len_seed=32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append4", "append4", "load4", "paged4", "paged4", "paged4"])
    heads, kv_heads = rng.choice([(2, 1), (8, 8), (32, 8), (16, 16), (32, 4), (12, 2), (15, 5),
                                  (24, 1)])
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([8, 16, 16, 32, 64, 128])
    seed = rng.randrange(1 << 30)
    if op == "load4":
        return dict(op=op, dtype=dtype, kv_heads=kv_heads, page=page,
                    slots=_log_int(rng, 1, 600000 // kv_heads),
                    spare=_log_int(rng, 1, 100000 // kv_heads), len_seed=seed)
    hi = _log_int(rng, 1, 40000)
    lo = rng.choice([1, max(1, hi // 8), hi])
    batch = max(1, min(_log_int(rng, 1, 256), 8000000 // (hi * kv_heads)))
    decodes = rng.choice([batch, batch, batch // 2, 0])
    new_hi = _log_int(rng, 1, max(2, min(2000, 40000 // max(1, batch - decodes))))
    if op == "paged4":
        return dict(op=op, dtype=dtype, heads=heads, kv_heads=kv_heads, page=page, batch=batch,
                    lo=lo, hi=hi, decodes=decodes, new_lo=1, new_hi=new_hi,
                    lse=rng.random() < 0.5, len_seed=seed)
    case = dict(op=op, dtype=dtype, heads=heads, kv_heads=kv_heads, page=page,
                batch=min(batch, 40), lo=0, hi=min(hi, 1000), decodes=min(decodes, 40), new_lo=1,
                new_hi=min(new_hi, 1200), pad=rng.choice([0, rng.randint(1, 500)]), len_seed=seed)
    if op == "append4":
        case["rotate"] = rng.random() < 0.7
    return case


def _requests(case):
    """(cached, new) of each request."""
    r = random.Random(case["len_seed"])
    rows = []
    for i in range(case["batch"]):
        new = 1 if i < case["decodes"] else r.randint(case["new_lo"], case["new_hi"])
        cached = r.randint(case["lo"], case["hi"])
        if case["op"] == "paged4":  # lo..hi is what the attention reads, the new tokens among it
            cached = max(0, cached - new)
        rows.append((cached, new))
    r.shuffle(rows)
    return rows


def _up(n, p):
    return -(-n // p)


def _pages_of(case):
    """Pages of the pools of an append: the requests', and some to spare."""
    return sum(_up(c + n, case["page"]) for c, n in _requests(case)) + 5


def _positions(rows):
    """How many different positions the new tokens stand at."""
    n, at = 0, 0
    for a, b in sorted((c, c + n) for c, n in rows):
        n += max(0, b - max(a, at))
        at = max(at, b)
    return n


def work(case):
    g = case["kv_heads"]
    if case["op"] == "load4":
        rows = case["slots"] - case["slots"] // 10
        return {"bytes": rows * g * 2 * (36 + 128) + 4 * case["slots"], "flops": 2 * rows * g * D}
    rows, h = _requests(case), case["heads"]
    new = sum(n for _, n in rows)
    if case["op"] == "paged4":
        keys = sum(c + n for c, n in rows)
        pairs = sum(n * c + n * (n + 1) // 2 for c, n in rows)
        return {"bytes": 2 * D * 2 * h * new + 72 * g * keys + (4 * h * new if case["lse"] else 0)
                + 4 * sum(_up(c + n, case["page"]) for c, n in rows) + 8 * case["batch"],
                "flops": 4 * D * h * pairs}
    rotate = case.get("rotate", True)
    size = 4 * (new + case["pad"])  # the slots
    if rotate:  # q in and out, a row of both tables a position, offsets and lengths
        size += 2 * D * 2 * h * new + 256 * _positions(rows) + 8 * case["batch"]
    flops = 3 * D * (h + g) * new if rotate else 0
    if case["op"] == "append":
        return {"bytes": size + 2 * 2 * 2 * D * g * new, "flops": flops}
    # the pools come back as the values that they stand for
    back = _pages_of(case) * case["page"] * g * 2
    return {"bytes": size + 2 * g * new * (2 * D + 36) + back * (36 + 128),
            "flops": flops + 2 * 4 * D * g * new + back * D}


# --------------------------------------------------------------- the inputs
def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _scan(xs):
    out = [0]
    for x in xs:
        out.append(out[-1] + x)
    return out


def _i32(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def _tables(case, g, rows):
    """A pool of pages in random order, of which each request holds the pages
    of all its tokens.  Returns the table, its width and the pool's size."""
    p = case["page"]
    have = [_up(c + n, p) for c, n in rows]
    width, pages = max(1, max(have)), sum(have) + 5
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    first = torch.tensor(_scan(have)[:-1], device="cuda")
    at = (first[:, None] + col[None]).clamp(max=pages - 1)
    table = torch.where(col[None] < torch.tensor(have, device="cuda")[:, None], order[at], -1)
    return table.to(torch.int32).contiguous(), width, pages


def _pool4(g, pages, heads, page, dtype, outlier):
    """A 4-bit pool of random rows; ``outlier``: a few channels are larger, as
    those of keys are."""
    pool = torch.empty((pages, heads, page // 8, UNIT), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (heads * page * D))
    for a in range(0, pages, step):
        x = _randn(g, (min(step, pages - a), heads, page // 8, 8, D), dtype)
        if outlier:
            x[..., 5::16] *= 3
        codes, scales = _quantise(x.float(), dtype)
        pool[a:a + step, ..., :256] = codes.flatten(-2)
        pool[a:a + step, ..., 256:] = scales.flatten(-2).view(torch.uint8)
    return pool


def _prepare_append(case, g):
    rows = _requests(case)
    dt = DTYPES[case["dtype"]]
    h, hkv, p = case["heads"], case["kv_heads"], case["page"]
    new = [n for _, n in rows]
    table, width, pages = _tables(case, g, rows)
    slots = []
    for i, (c, n) in enumerate(rows):
        pos = torch.arange(c, c + n, device="cuda")
        slots.append(table[i, pos // p] * p + (pos % p).to(torch.int32))
    if case["pad"]:
        slots.append(torch.full((case["pad"],), -1, dtype=torch.int32, device="cuda"))
    t = sum(new) + case["pad"]
    # q, k and v are the column blocks of one fused projection's output
    qkv = _randn(g, (t, h + 2 * hkv, D), dt)
    qkv[:, :h] *= 2.0
    qkv[:, h:h + hkv, 5::16] *= 3.0
    far = max(c + n for c, n in rows)
    angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32)
    st = dict(case=case, slots=torch.cat(slots), cu=_i32(_scan(new)),
              lens=_i32([c + n for c, n in rows]), q=qkv[:, :h], k=qkv[:, h:h + hkv],
              v=qkv[:, h + hkv:], cos=angle.cos().float(), sin=angle.sin().float(),
              q_out=torch.zeros((t, h, D), dtype=dt, device="cuda"), pages=pages)
    if case["op"] == "append":
        st["kc"] = _randn(g, (pages, hkv, p, D), dt)
        st["vc"] = _randn(g, (pages, hkv, p, D), dt)
    else:
        st["kc"] = _pool4(g, pages, hkv, p, dt, True)
        st["vc"] = _pool4(g, pages, hkv, p, dt, False)
    if own:
        from causal_streaming_softmax_gb300 import api
        st["shape"] = api.PagedShape(len(rows), t, h, hkv, page_size=p, num_pages=pages,
                                     table_width=width, max_new=max(new), dtype=dt)
        if case["op"] == "append4":
            # every slot, to read the pools back
            st["every"] = torch.arange(pages * p, dtype=torch.int32, device="cuda")
            st["all"] = api.PagedShape(len(rows), pages * p, h, hkv, page_size=p, num_pages=pages,
                                       table_width=width, max_new=max(new), dtype=dt)
            st["kd"] = torch.empty((pages * p, hkv, D), dtype=dt, device="cuda")
            st["vd"] = torch.empty_like(st["kd"])
    return st


def _prepare_load(case, g):
    dt, hkv, p, n = DTYPES[case["dtype"]], case["kv_heads"], case["page"], case["slots"]
    pages = _up(n + case["spare"], p)
    slots = torch.randperm(pages * p, generator=g, device="cuda")[:n].to(torch.int32)
    none = torch.randperm(n, generator=g, device="cuda")[:n // 10]
    slots[none] = -1
    st = dict(case=case, slots=slots, kc=_pool4(g, pages, hkv, p, dt, True),
              vc=_pool4(g, pages, hkv, p, dt, False),
              k=torch.zeros((n, hkv, D), dtype=dt, device="cuda"),
              v=torch.zeros((n, hkv, D), dtype=dt, device="cuda"))
    if own:
        from causal_streaming_softmax_gb300 import api
        st["shape"] = api.PagedShape(1, n, hkv, hkv, page_size=p, num_pages=pages, table_width=1,
                                     dtype=dt)
    return st


def _prepare_paged(case, g):
    rows = _requests(case)
    dt = DTYPES[case["dtype"]]
    h, hkv, p = case["heads"], case["kv_heads"], case["page"]
    new = [n for _, n in rows]
    t = sum(new)
    table, width, pages = _tables(case, g, rows)
    st = dict(case=case, rows=rows, table=table, cu=_i32(_scan(new)),
              kv=_i32([c + n for c, n in rows]), q=_randn(g, (t, h, D), dt, 2.0),
              k=_pool4(g, pages, hkv, p, dt, True), v=_pool4(g, pages, hkv, p, dt, False))
    if own:
        from causal_streaming_softmax_gb300 import api
        s = api.PagedShape(len(rows), t, h, hkv, page_size=p, num_pages=pages, table_width=width,
                           max_new=max(new), dtype=dt)
        st["shape"] = s
        st["ws"] = api.alloc_paged_workspace(s)
        st["o"] = torch.empty((t, h, D), dtype=dt, device="cuda")
        st["lse"] = torch.empty((h, t), dtype=torch.float32, device="cuda") if case["lse"] else None
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"append": _prepare_append, "append4": _prepare_append, "load4": _prepare_load,
            "paged4": _prepare_paged}[case["op"]](case, g)


# -------------------------------------------------------------- plain forms
def _quantise(x, dtype):
    """Codes uint8 [..., 32] and scales [..., 2] of rows x [..., 64] in 32 bits."""
    keep, most = SCALES[dtype]
    x = x.unflatten(-1, (2, 32))
    mx, mn = x.amax(-1), x.amin(-1)
    s = torch.where(mx > -mn, -mx, -mn) / 8
    drop = 24 - keep  # to nearest, ties away from zero
    s = ((s.contiguous().view(torch.int32) + (1 << (drop - 1))) >> drop << drop).view(torch.float32)
    s = s.clamp(-most, most).to(dtype)
    s = torch.where(torch.isfinite(mx) & torch.isfinite(mn), s, float("nan"))
    sf = s.float()[..., None]
    code = torch.where((sf != 0) & torch.isfinite(sf), torch.round(x / sf), 0.0).clamp(-8, 7)
    code = (code + 8).to(torch.uint8)
    return code[..., 0, :] | code[..., 1, :] << 4, s


def _values(codes, scales):
    """The rows [..., 64] that codes [..., 32] and scales [..., 2] stand for, in 32 bits."""
    lo = ((codes & 15).float() - 8) * scales[..., :1].float()
    return torch.cat([lo, ((codes >> 4).float() - 8) * scales[..., 1:].float()], -1)


def _pool_values(pool, dtype):
    """The rows [..., heads, page, 64] of pages of a 4-bit pool."""
    scales = pool[..., 256:].contiguous().view(dtype).unflatten(-1, (8, 2))
    return _values(pool[..., :256].unflatten(-1, (8, 32)), scales).flatten(-3, -2)


def _places(pool, page, r):
    """Indices of the codes and of the scales' bytes of rows (page, r), every head."""
    i = page[:, None, None]
    h = torch.arange(pool.shape[1], device=pool.device)[None, :, None]
    u, r = (r // 8)[:, None, None], (r % 8)[:, None, None]
    return ((i, h, u, r * 32 + torch.arange(32, device=pool.device)),
            (i, h, u, 256 + r * 4 + torch.arange(4, device=pool.device)))


def _rotate(x, cos, sin):
    """Rows x [t, heads, 64] turned by the angles of their positions, in 32 bits."""
    a, b = x[..., :32].float(), x[..., 32:].float()
    c, s = cos[:, None], sin[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _at(st):
    """The tokens that have a slot, their slots, and their positions."""
    rows = (st["slots"] >= 0).nonzero().squeeze(1)
    req = torch.searchsorted(st["cu"][1:], rows.to(torch.int32), right=True)
    first = st["lens"][req] - (st["cu"][req + 1] - st["cu"][req])
    return rows, st["slots"][rows].long(), first + rows - st["cu"][req]


def _put4(pool, page, r, x, dtype):
    codes, scales = _places(pool, page, r)
    pool[codes], s = _quantise(x, dtype)
    pool[scales] = s.contiguous().view(torch.uint8)


def _plain_append(st):
    case, p, dt = st["case"], st["case"]["page"], st["q"].dtype
    rows, slot, pos = _at(st)
    page, r = slot // p, slot % p
    k, v = st["k"][rows].float(), st["v"][rows].float()
    if case.get("rotate", True):
        cos, sin = st["cos"][pos], st["sin"][pos]
        k = _rotate(k, cos, sin)
        st["q_out"][rows] = _rotate(st["q"][rows], cos, sin).to(dt)
    if case["op"] == "append":
        st["kc"][page, :, r] = k.to(dt)
        st["vc"][page, :, r] = v.to(dt)
        return st["q_out"], st["kc"], st["vc"]
    _put4(st["kc"], page, r, k, dt)
    _put4(st["vc"], page, r, v, dt)
    pools = [_pool_values(st[x], dt).to(dt).transpose(1, 2).flatten(0, 1) for x in ("kc", "vc")]
    return [st["q_out"]] + pools if case["rotate"] else pools


def _plain_load(st):
    p, dt = st["case"]["page"], st["k"].dtype
    rows = (st["slots"] >= 0).nonzero().squeeze(1)
    slot = st["slots"][rows].long()
    codes, scales = _places(st["kc"], slot // p, slot % p)
    st["k"][rows] = _values(st["kc"][codes], st["kc"][scales].view(dt)).to(dt)
    st["v"][rows] = _values(st["vc"][codes], st["vc"][scales].view(dt)).to(dt)
    return st["k"], st["v"]


def _softmax_product(s, v):
    mx = s.amax(-1, keepdim=True)
    e = torch.exp(s - mx)
    z = e.sum(-1, keepdim=True)
    return torch.matmul(e, v) / z, ((mx + torch.log(z)) / LN2).squeeze(-1)


def _plain_paged(st):
    """The requests of one token together, their keys padded to the longest;
    each chunk by itself, its scores being a matrix of its own size."""
    q, dt = st["q"], st["q"].dtype
    t, h, _ = q.shape
    hkv = st["case"]["kv_heads"]
    o = torch.empty((t, h, D), dtype=dt, device="cuda")
    lse = torch.empty((h, t), dtype=torch.float32, device="cuda")
    starts = _scan([n for _, n in st["rows"]])
    ones = [i for i, (_, n) in enumerate(st["rows"]) if n == 1]
    if ones:
        keys = max(st["rows"][i][0] + 1 for i in ones)
        row = torch.tensor(ones, device="cuda")
        at = st["cu"][row].long()
        ids = st["table"][row, :_up(keys, st["case"]["page"])].long().clamp(min=0)
        k, v = (_pool_values(st[x][ids], dt).transpose(1, 2).flatten(2, 3)[:, :, :keys]
                for x in "kv")
        s = torch.matmul(q[at].float().reshape(len(ones), hkv, h // hkv, D),
                         k.transpose(2, 3)) * D ** -0.5
        gone = torch.arange(keys, device="cuda")[None] >= st["kv"][row][:, None]
        r, e = _softmax_product(s.masked_fill(gone[:, None, None], float("-inf")), v)
        o[at] = r.reshape(len(ones), h, D).to(dt)
        lse[:, at] = e.reshape(len(ones), h).T
    for i, (c, n) in enumerate(st["rows"]):
        if n == 1:
            continue
        a, b, m = starts[i], starts[i + 1], c + n
        ids = st["table"][i, :_up(m, st["case"]["page"])].long()
        k, v = (_pool_values(st[x][ids], dt).transpose(0, 1).flatten(1, 2)[:, :m] for x in "kv")
        qi = q[a:b].float().reshape(n, hkv, h // hkv, D).permute(1, 2, 0, 3)
        s = torch.matmul(qi, k[:, None].transpose(2, 3)) * D ** -0.5
        gone = torch.arange(m, device="cuda")[None] > torch.arange(c, m, device="cuda")[:, None]
        r, e = _softmax_product(s.masked_fill(gone, float("-inf")), v[:, None])
        o[a:b] = r.permute(2, 0, 1, 3).reshape(n, h, D).to(dt)
        lse[:, a:b] = e.reshape(h, n)
    return (o, lse) if st["case"]["lse"] else o


def _own(st):
    from causal_streaming_softmax_gb300 import api
    case, s = st["case"], st["shape"]
    if case["op"] == "append":
        api.attn_paged_append(s, st["q"], st["k"], st["v"], st["cos"], st["sin"], st["slots"],
                              st["cu"], st["lens"], st["q_out"], st["kc"], st["vc"])
        return st["q_out"], st["kc"], st["vc"]
    if case["op"] == "append4":
        if case["rotate"]:
            api.attn_paged_append4(s, st["q"], st["k"], st["v"], st["cos"], st["sin"], st["slots"],
                                   st["cu"], st["lens"], st["q_out"], st["kc"], st["vc"])
        else:
            api.attn_paged_append4(s, None, st["k"], st["v"], None, None, st["slots"], None, None,
                                   None, st["kc"], st["vc"])
        api.attn_paged_load4(st["all"], st["every"], st["kc"], st["vc"], st["kd"], st["vd"])
        pools = [st["kd"], st["vd"]]
        return [st["q_out"]] + pools if case["rotate"] else pools
    if case["op"] == "load4":
        api.attn_paged_load4(s, st["slots"], st["kc"], st["vc"], st["k"], st["v"])
        return st["k"], st["v"]
    api.attn_paged_fwd4(s, st["q"], st["k"], st["v"], st["table"], st["cu"], st["kv"], st["ws"],
                        st["o"], st["lse"])
    return (st["o"], st["lse"]) if case["lse"] else st["o"]


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "append4": _plain_append, "load4": _plain_load,
            "paged4": _plain_paged}[state["case"]["op"]](state)


# ------------------------------------------------------ the values in 64 bits
def _exact_rows(unit, dtype):
    """Rows [..., 64] of the 36 bytes [..., 36] that hold each of them."""
    byte = unit[..., :32].to(torch.int64)
    s = unit[..., 32:].contiguous().view(dtype).double()
    return torch.cat([(byte % 16 - 8) * s[..., 0:1], (byte // 16 - 8) * s[..., 1:2]], -1)


def _exact_read(pool, page, r, dtype):
    """The rows [n, heads, 64] at places (page, r)."""
    u, r = r // 8, r % 8
    sub = pool[page, :, u]
    i = torch.arange(32, device=pool.device)
    n, h = sub.shape[:2]
    codes = sub.gather(2, (r[:, None, None] * 32 + i).expand(n, h, 32))
    scales = sub.gather(2, (256 + r[:, None, None] * 4 + i[:4]).expand(n, h, 4))
    return _exact_rows(torch.cat([codes, scales], 2), dtype)


def _exact_round(x, dtype):
    """What a 4-bit cache makes of rows x [n, heads, 64], in 64 bits."""
    keep, most = SCALES[dtype]
    out = torch.empty_like(x)
    for part in (slice(0, 32), slice(32, 64)):
        y = x[..., part]
        lo, hi = y.min(-1).values, y.max(-1).values
        e = torch.where(lo.abs() >= hi.abs(), lo, hi)
        # the scale's significand to `keep` bits, halves away from zero
        m, exp = torch.frexp(-e / 8)
        m = torch.sign(m) * torch.floor(m.abs() * 2.0 ** keep + 0.5) / 2.0 ** keep
        s = torch.ldexp(m, exp).clamp(-most, most).to(dtype).double()[..., None]
        s1 = torch.where(s == 0, 1.0, s)
        out[..., part] = torch.round(y / s1).clamp(-8, 7) * s
    return out


def _exact_append(case, st):
    p, dt, n = case["page"], st["q"].dtype, len(st["lens"])
    lens, cu = st["lens"].tolist(), st["cu"].tolist()
    pos = torch.cat([torch.arange(lens[i] - (cu[i + 1] - cu[i]), lens[i], device="cuda")
                     for i in range(n)])
    t = len(pos)
    slot = st["slots"][:t].long()
    k, v, q = (st[x][:t].double() for x in ("k", "v", "q"))
    if case.get("rotate", True):
        z = torch.complex(st["cos"].double(), st["sin"].double())[pos][:, None]
        turn = lambda x: torch.cat([(y := torch.complex(x[..., :32], x[..., 32:]) * z).real,
                                    y.imag], -1)
        k, q = turn(k), turn(q)
    q_out = st["q_out"].double()
    q_out[:t] = q
    if case["op"] == "append":
        kc, vc = st["kc"].double(), st["vc"].double()
        kc[slot // p, :, slot % p], vc[slot // p, :, slot % p] = k, v
        return q_out, kc, vc
    every = torch.arange(st["pages"] * p, device="cuda")
    pools = []
    for pool, x in ((st["kc"], k), (st["vc"], v)):
        rows = _exact_read(pool, every // p, every % p, dt)
        rows[slot] = _exact_round(x, dt)
        pools.append(rows)
    return [q_out] + pools if case["rotate"] else pools


def _exact_attend(q, k, v, seen):
    """One sequence, from the definition: q [n, H, D], k and v [m, Hkv, D],
    row i sees the first seen[i] keys."""
    n, h, _ = q.shape
    m, hkv, _ = k.shape
    o = torch.zeros((n, h, D), dtype=torch.float64, device=q.device)
    lse = torch.zeros((h, n), dtype=torch.float64, device=q.device)
    for head in range(h):
        kd, vd = k[:, head * hkv // h], v[:, head * hkv // h]
        step = max(1, (1 << 26) // m)
        for a in range(0, n, step):
            lim = seen[a:a + step]
            top = int(lim.max())
            x = q[a:a + step, head].double() @ kd[:top].T / math.sqrt(D)
            x[torch.arange(top, device=q.device)[None] >= lim[:, None]] = -math.inf
            z = torch.logsumexp(x, 1)
            o[a:a + step, head] = torch.exp(x - z[:, None]) @ vd[:top]
            lse[head, a:a + step] = z / math.log(2.0)
    return o, lse


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("append", "append4"):
        return _exact_append(case, st)
    p, dt = case["page"], DTYPES[case["dtype"]]
    if case["op"] == "load4":
        slot = st["slots"].long().clamp(min=0)
        gone = (st["slots"] < 0)[:, None, None]
        return tuple(_exact_read(st[x], slot // p, slot % p, dt).masked_fill(gone, 0.0)
                     for x in ("kc", "vc"))
    parts, at = [], 0
    for i, (c, n) in enumerate(st["rows"]):
        j = torch.arange(c + n, device="cuda")
        page, r = st["table"][i].long()[j // p], j % p
        k, v = (_exact_read(st[x], page, r, dt) for x in "kv")
        parts.append(_exact_attend(st["q"][at:at + n], k, v, j[c:] + 1))
        at += n
    o = torch.cat([x[0] for x in parts])
    return (o, torch.cat([x[1] for x in parts], 1)) if case["lse"] else o
