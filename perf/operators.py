"""The serving operators: attention over packed prompts, and the paged cache
(plan, store, attention of new tokens over the pages).

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


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one short prompt on a small model: latency
        dict(name="prompt-short", op="packed", dtype="f16", heads=2, kv_heads=1, causal=True,
             batch=1, lo=93, hi=93, len_seed=1),
        # a training or prefill batch of ragged prompts, grouped heads
        dict(name="prompt-ragged", op="packed", dtype="bf16", heads=32, kv_heads=8, causal=True,
             batch=16, lo=256, hi=4096, len_seed=2),
        # one long document
        dict(name="prompt-long", op="packed", dtype="f16", heads=32, kv_heads=4, causal=True,
             batch=1, lo=16384, hi=16384, len_seed=3),
        # one user, one token: the smallest serving step
        dict(name="decode-one", op="paged", dtype="bf16", heads=32, kv_heads=8, page=16, batch=1,
             lo=777, hi=777, decodes=1, new_lo=1, new_hi=1, lse=False, len_seed=4),
        # one user with a long history: few rows, a long axis
        dict(name="decode-long", op="paged", dtype="f16", heads=16, kv_heads=16, page=32, batch=2,
             lo=50000, hi=65536, decodes=2, new_lo=1, new_hi=1, lse=True, len_seed=5),
        # a server's ordinary token step, every request at another length
        dict(name="decode-batch", op="paged", dtype="f16", heads=32, kv_heads=8, page=16, batch=64,
             lo=17, hi=8192, decodes=64, new_lo=1, new_hi=1, lse=False, len_seed=6),
        # a large server's token step
        dict(name="decode-large", op="paged", dtype="bf16", heads=32, kv_heads=4, page=64,
             batch=256, lo=1024, hi=16384, decodes=256, new_lo=1, new_hi=1, lse=False, len_seed=7),
        # chunks of prompts beside running requests (continuous batching)
        dict(name="chunk-mixed", op="paged", dtype="bf16", heads=32, kv_heads=8, page=16, batch=36,
             lo=2048, hi=8192, decodes=32, new_lo=301, new_hi=1024, lse=True, len_seed=8),
        # tables and slots of a token step
        dict(name="plan-decode", op="plan", page=16, batch=64, lo=17, hi=8192, decodes=64,
             new_lo=1, new_hi=1, retire=0, pad=0, len_seed=9),
        # tables and slots of admitted prompts, others retired, a padded token buffer
        dict(name="plan-prompts", op="plan", page=16, batch=512, lo=0, hi=4096, decodes=256,
             new_lo=1, new_hi=1024, retire=100, pad=777, len_seed=10),
        # the new rows of a token step into the cache
        dict(name="store-decode", op="store", dtype="bf16", kv_heads=8, page=16, batch=64, lo=17,
             hi=2048, decodes=64, new_lo=1, new_hi=1, len_seed=11),
        # the rows of admitted prompts into the cache
        dict(name="store-prompts", op="store", dtype="f16", kv_heads=8, page=16, batch=40, lo=0,
             hi=512, decodes=7, new_lo=100, new_hi=2000, len_seed=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["packed", "packed", "paged", "paged", "paged", "plan", "store"])
    heads, kv_heads = rng.choice([(2, 1), (8, 8), (32, 8), (16, 16), (32, 4), (12, 2), (15, 5)])
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([16, 16, 32, 64, 128])
    seed = rng.randrange(1 << 30)
    if op == "packed":
        hi = _log_int(rng, 2, 12000)
        lo = rng.choice([1, max(1, hi // 8), hi])
        # no more pairs than the longest listed prompt has, over heads
        batch = max(1, min(_log_int(rng, 1, 64), 16384 ** 2 // (hi * hi), 60000 // hi))
        return dict(op=op, dtype=dtype, heads=heads, kv_heads=kv_heads,
                    causal=rng.random() < 0.8, batch=batch, lo=lo, hi=hi, len_seed=seed)
    hi = _log_int(rng, 1, 40000)
    lo = rng.choice([1, max(1, hi // 8), hi])
    batch = max(1, min(_log_int(rng, 1, 256), 8000000 // (hi * kv_heads)))
    decodes = rng.choice([batch, batch, batch // 2, 0])
    new_lo = 1
    new_hi = _log_int(rng, 1, max(2, min(2000, 60000 // max(1, batch - decodes))))
    if op == "plan":
        batch = _log_int(rng, 1, 512)
        decodes = batch // rng.choice([1, 2, 3])
        return dict(op=op, page=page, batch=batch, lo=0, hi=_log_int(rng, 1, 4000),
                    decodes=decodes, new_lo=1, new_hi=_log_int(rng, 1, 1000),
                    retire=rng.randint(0, batch // 3), pad=rng.choice([0, rng.randint(1, 999)]),
                    len_seed=seed)
    if op == "store":
        return dict(op=op, dtype=dtype, kv_heads=kv_heads, page=page, batch=min(batch, 40), lo=0,
                    hi=min(hi, 4000), decodes=min(decodes, 40), new_lo=new_lo,
                    new_hi=min(new_hi, 1500), len_seed=seed)
    return dict(op=op, dtype=dtype, heads=heads, kv_heads=kv_heads, page=page, batch=batch, lo=lo,
                hi=hi, decodes=decodes, new_lo=new_lo, new_hi=new_hi, lse=rng.random() < 0.5,
                len_seed=seed)


def _lengths(case):
    """Packed: the prompts' lengths."""
    r = random.Random(case["len_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _requests(case):
    """Paged: (cached, new) of each request; new is -1 for a retired one."""
    r = random.Random(case["len_seed"])
    rows = []
    for i in range(case["batch"]):
        new = 1 if i < case["decodes"] else r.randint(case["new_lo"], case["new_hi"])
        cached = r.randint(case["lo"], case["hi"])
        if case["op"] == "paged":  # lo..hi is what the attention reads, the new tokens among it
            cached = max(0, cached - new)
        rows.append([cached, new])
    for i in r.sample(range(case["batch"]), case.get("retire", 0)):
        rows[i][1] = -1
    r.shuffle(rows)
    return [tuple(x) for x in rows]


def _pairs(case):
    """Visible (query, key) pairs of one head."""
    if case["op"] == "packed":
        return sum(n * (n + 1) // 2 if case["causal"] else n * n for n in _lengths(case))
    return sum(n * c + n * (n + 1) // 2 for c, n in _requests(case))


def work(case):
    if case["op"] == "packed":
        t = sum(_lengths(case))
        h, g = case["heads"], case["kv_heads"]
        return {"bytes": 2 * D * t * (2 * h + 2 * g) + 4 * h * t + 4 * (case["batch"] + 1),
                "flops": 4 * D * h * _pairs(case)}
    rows = _requests(case)
    p = case["page"]
    new = sum(max(0, n) for _, n in rows)
    up = lambda x: -(-x // p)
    if case["op"] == "paged":
        h, g = case["heads"], case["kv_heads"]
        keys = sum(c + n for c, n in rows)
        return {"bytes": 2 * D * (2 * h * new + 2 * g * keys) + (4 * h * new if case["lse"] else 0)
                + 4 * sum(up(c + n) for c, n in rows) + 8 * case["batch"],
                "flops": 4 * D * h * _pairs(case)}
    if case["op"] == "plan":
        moved = sum(up(c + n) - up(c) if n >= 0 else up(c) for c, n in rows)
        return {"bytes": 16 * case["batch"] + 4 * (new + case["pad"]) + 8 * moved + 32, "flops": 0}
    return {"bytes": 2 * 2 * 2 * D * case["kv_heads"] * new + 4 * new, "flops": 0}


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


def _prepare_packed(case, g):
    lens = _lengths(case)
    t, h, hkv = sum(lens), case["heads"], case["kv_heads"]
    dt = DTYPES[case["dtype"]]
    # q, k and v are the column blocks of one fused projection's output
    qkv = _randn(g, (t, h + 2 * hkv, D), dt)
    qkv[:, :h] *= 2.0
    st = dict(case=case, lens=lens, q=qkv[:, :h], k=qkv[:, h:h + hkv], v=qkv[:, h + hkv:],
              cu=_i32(_scan(lens)))
    if own:
        from causal_streaming_softmax_gb300 import api
        st["shape"] = api.PackedShape(t, len(lens), h, hkv, causal=case["causal"], dtype=dt)
        st["o"] = torch.empty((t, h, D), dtype=dt, device="cuda")
        st["lse"] = torch.empty((h, t), dtype=torch.float32, device="cuda")
    return st


def _tables(case, g, rows, after):
    """A pool of pages in random order.  Each request holds the pages of its
    cached tokens (with ``after`` also those of its new ones); the rest are
    free.  Returns the table, its width, the pool's size and the free pages."""
    p = case["page"]
    up = lambda x: -(-x // p)
    have = [up(c + max(0, n)) if after else up(c) for c, n in rows]
    width = max(1, max(up(c + max(0, n)) for c, n in rows))
    extra = sum(up(c + max(0, n)) for c, n in rows) - sum(have)
    pages = sum(have) + extra + 5 + len(rows)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    have_t = torch.tensor(have, device="cuda")
    first = torch.tensor(_scan(have)[:-1], device="cuda")
    table = torch.where(col[None] < have_t[:, None],
                        order[(first[:, None] + col[None]).clamp(max=pages - 1)], -1)
    return table.to(torch.int32).contiguous(), width, pages, order[sum(have):].contiguous()


def _prepare_paged(case, g):
    rows = _requests(case)
    dt = DTYPES[case["dtype"]]
    h, hkv, p = case["heads"], case["kv_heads"], case["page"]
    new = [n for _, n in rows]
    t = sum(new)
    table, width, pages, _ = _tables(case, g, rows, after=True)
    st = dict(case=case, rows=rows, table=table, cu=_i32(_scan(new)),
              kv=_i32([c + n for c, n in rows]), q=_randn(g, (t, h, D), dt, 2.0),
              k=_randn(g, (pages, hkv, p, D), dt), v=_randn(g, (pages, hkv, p, D), dt))
    if own:
        from causal_streaming_softmax_gb300 import api
        s = api.PagedShape(len(rows), t, h, hkv, page_size=p, num_pages=pages, table_width=width,
                           max_new=max(new), dtype=dt)
        st["shape"] = s
        st["ws"] = api.alloc_paged_workspace(s)
        st["o"] = torch.empty((t, h, D), dtype=dt, device="cuda")
        st["lse"] = torch.empty((h, t), dtype=torch.float32, device="cuda") if case["lse"] else None
    return st


def _prepare_plan(case, g):
    rows = _requests(case)
    table, width, pages, free = _tables(case, g, rows, after=False)
    t = sum(max(0, n) for _, n in rows) + case["pad"]
    head = int(torch.randint(pages, (1,), generator=g, device="cuda"))
    ring = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(len(free), device="cuda")) % pages] = free
    st = dict(case=case, table=table, ring=ring, state=_i32([head, len(free), 0, 0]), tokens=t,
              cached=_i32([c for c, _ in rows]), new=_i32([n for _, n in rows]))
    if own:
        from causal_streaming_softmax_gb300 import api
        st["shape"] = api.PagedShape(len(rows), t, 1, 1, page_size=case["page"], num_pages=pages,
                                     table_width=width, max_new=max(n for _, n in rows))
        st["cu"] = torch.empty(len(rows) + 1, dtype=torch.int32, device="cuda")
        st["kv"] = torch.empty(len(rows), dtype=torch.int32, device="cuda")
        st["slots"] = torch.empty(t, dtype=torch.int32, device="cuda")
        st["next"] = torch.empty(4, dtype=torch.int32, device="cuda")
    return st


def _prepare_store(case, g):
    rows = _requests(case)
    dt = DTYPES[case["dtype"]]
    hkv, p = case["kv_heads"], case["page"]
    table, width, pages, _ = _tables(case, g, rows, after=True)
    slots = []
    for i, (c, n) in enumerate(rows):
        pos = torch.arange(c, c + n, device="cuda")
        slots.append(table[i, pos // p] * p + (pos % p).to(torch.int32))
    slots = torch.cat(slots)
    t = slots.numel()
    kv = _randn(g, (t, 2 * hkv, D), dt)  # the K and V columns of a projection's output
    st = dict(case=case, slots=slots, k=kv[:, :hkv], v=kv[:, hkv:],
              kc=_randn(g, (pages, hkv, p, D), dt), vc=_randn(g, (pages, hkv, p, D), dt))
    if own:
        from causal_streaming_softmax_gb300 import api
        st["shape"] = api.PagedShape(len(rows), t, hkv, hkv, page_size=p, num_pages=pages,
                                     table_width=width, max_new=max(n for _, n in rows), dtype=dt)
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"packed": _prepare_packed, "paged": _prepare_paged, "plan": _prepare_plan,
            "store": _prepare_store}[case["op"]](case, g)


# -------------------------------------------------------------- plain forms
def _attend(q, k, v, first, scale):
    """q [n, H, D] over k, v [m, Hkv, D] in 32 bits; query i sees the keys
    below first + i + 1 (every key where first is None)."""
    n, h, _ = q.shape
    m, hkv, _ = k.shape
    o = torch.empty((n, h, D), dtype=torch.float32, device=q.device)
    lse = torch.empty((h, n), dtype=torch.float32, device=q.device)
    kf = k.float().permute(1, 2, 0)
    vf = v.float().permute(1, 0, 2)
    step = max(1, (1 << 28) // max(1, m * h))
    for a in range(0, n, step):
        b = min(n, a + step)
        top = m if first is None else min(m, first + b)
        qf = q[a:b].float().reshape(b - a, hkv, h // hkv, D).permute(1, 2, 0, 3)
        s = torch.matmul(qf, kf[:, None, :, :top]) * scale
        if first is not None:
            i = torch.arange(first + a, first + b, device=q.device)
            j = torch.arange(top, device=q.device)
            s = s.masked_fill(j[None, :] > i[:, None], float("-inf"))
        mx = s.amax(-1, keepdim=True)
        e = torch.exp(s - mx)
        z = e.sum(-1, keepdim=True)
        r = torch.matmul(e, vf[:, None, :top]) / z
        o[a:b] = r.permute(2, 0, 1, 3).reshape(b - a, h, D)
        lse[:, a:b] = ((mx + torch.log(z)) / LN2).squeeze(-1).reshape(h, b - a)
    return o, lse


def _plain_packed(st):
    case, lens = st["case"], st["lens"]
    o, lse, at = [], [], 0
    for n in lens:
        r = _attend(st["q"][at:at + n], st["k"][at:at + n], st["v"][at:at + n],
                    0 if case["causal"] else None, D ** -0.5)
        o.append(r[0].to(st["q"].dtype))
        lse.append(r[1])
        at += n
    return torch.cat(o), torch.cat(lse, 1)


def _pages(cache, row, n, p):
    """The first n keys that a table row names, as [n, Hkv, D]."""
    idx = row[:-(-n // p)].long()
    return cache[idx].permute(0, 2, 1, 3).reshape(-1, cache.shape[1], D)[:n]


def _plain_paged(st):
    case, p = st["case"], st["case"]["page"]
    o, lse, at = [], [], 0
    for i, (c, n) in enumerate(st["rows"]):
        r = _attend(st["q"][at:at + n], _pages(st["k"], st["table"][i], c + n, p),
                    _pages(st["v"], st["table"][i], c + n, p), c, D ** -0.5)
        o.append(r[0].to(st["q"].dtype))
        lse.append(r[1])
        at += n
    return (torch.cat(o), torch.cat(lse, 1)) if case["lse"] else torch.cat(o)


def _plain_plan(st):
    p, t = st["case"]["page"], st["tokens"]
    cached, new, table, ring = (st[k].long() for k in ("cached", "new", "table", "ring"))
    n_pages = ring.numel()
    head, free = st["state"][0].long(), st["state"][1].long()
    add = new.clamp(min=0)
    gone = new < 0
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    cu = torch.cat([zero, add.cumsum(0)])
    kv = torch.where(gone, 0, cached + add)
    have = (cached + p - 1) // p
    need = torch.where(gone, 0, (cached + add + p - 1) // p - have)
    back = torch.where(gone, have, 0)
    first = need.cumsum(0) - need
    out = back.cumsum(0) - back
    taken, given = need.sum(), back.sum()
    col = torch.arange(table.shape[1], device="cuda")
    fresh = (col[None] >= have[:, None]) & (col[None] < (have + need)[:, None])
    at = (head + first[:, None] + col[None] - have[:, None]) % n_pages
    table = torch.where(fresh, ring[at], table)
    ret = gone[:, None] & (col[None] < have[:, None])
    to = (head + free + out[:, None] + col[None]) % n_pages
    ring = ring.clone()
    ring[to[ret]] = table[ret]
    tok = torch.arange(t, device="cuda")
    req = torch.searchsorted(cu[1:], tok, right=True)
    live = req < new.numel()
    req = req.clamp(max=new.numel() - 1)
    pos = cached[req] + tok - cu[req]
    page = table[req, (pos // p).clamp(max=table.shape[1] - 1)]
    slots = torch.where(live, page * p + pos % p, -1)
    nxt = torch.stack([(head + taken) % n_pages, free - taken + given, taken,
                       torch.zeros_like(taken)])
    return [x.to(torch.int32) for x in (cu, kv, table, slots, ring, nxt)]


def _plain_store(st):
    p = st["case"]["page"]
    s = st["slots"].long()
    st["kc"][s // p, :, s % p] = st["k"]
    st["vc"][s // p, :, s % p] = st["v"]
    return st["kc"], st["vc"]


def _own(st):
    from causal_streaming_softmax_gb300 import api
    op, s = st["case"]["op"], st["shape"]
    if op == "packed":
        api.attn_packed_fwd(s, st["q"], st["k"], st["v"], st["cu"], st["o"], st["lse"])
        return st["o"], st["lse"]
    if op == "paged":
        api.attn_paged_fwd(s, st["q"], st["k"], st["v"], st["table"], st["cu"], st["kv"], st["ws"],
                           st["o"], st["lse"])
        return (st["o"], st["lse"]) if st["case"]["lse"] else st["o"]
    if op == "plan":
        api.attn_paged_plan(s, st["cached"], st["new"], st["ring"], st["state"], st["table"],
                            st["cu"], st["kv"], st["slots"], st["next"])
        return [st["cu"], st["kv"], st["table"], st["slots"], st["ring"], st["next"]]
    api.attn_paged_store(s, st["k"], st["v"], st["slots"], st["kc"], st["vc"])
    return st["kc"], st["vc"]


def run(state):
    if own:
        return _own(state)
    return {"packed": _plain_packed, "paged": _plain_paged, "plan": _plain_plan,
            "store": _plain_store}[state["case"]["op"]](state)


# ------------------------------------------------------ the values in 64 bits
def _exact_rows(q, k, v, seen):
    """One sequence, from the definition: q [n, H, D], k and v [m, Hkv, D],
    row i sees the first seen[i] keys."""
    n, h, _ = q.shape
    m, hkv, _ = k.shape
    o = torch.zeros((n, h, D), dtype=torch.float64, device=q.device)
    lse = torch.zeros((h, n), dtype=torch.float64, device=q.device)
    for head in range(h):
        kd, vd = k[:, head * hkv // h].double(), v[:, head * hkv // h].double()
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
    if case["op"] in ("plan", "store"):
        return None  # whole numbers, and copies
    st = prepare(case, seed)
    parts, at = [], 0
    if case["op"] == "packed":
        for n in st["lens"]:
            rows = slice(at, at + n)
            i = torch.arange(1, n + 1, device="cuda")
            parts.append(_exact_rows(st["q"][rows], st["k"][rows], st["v"][rows],
                                     i if case["causal"] else torch.full_like(i, n)))
            at += n
    else:
        p = case["page"]
        for i, (c, n) in enumerate(st["rows"]):
            j = torch.arange(c + n, device="cuda")
            page, off = st["table"][i].long()[j // p], j % p
            parts.append(_exact_rows(st["q"][at:at + n], st["k"][page, :, off],
                                     st["v"][page, :, off], j[c:] + 1))
            at += n
    o = torch.cat([x[0] for x in parts])
    if case["op"] == "paged" and not case["lse"]:
        return o
    return o, torch.cat([x[1] for x in parts], 1)
