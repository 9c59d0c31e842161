"""Plain 64-bit forms of the packed and paged calls, and the tolerances that
follow from the roundings the kernels make.

Bound of one output element, with u = eps / 2 of the 16-bit type, P the
normalised weights and A = sum_j P_j |v_j|:
  u |O|            rounding of the stored output
  u A              P rounded to the type before its product with V
  2 d A            relative error d of the binary32 weights (numerator and sum)
  2^-25 sum |v_j|  binary16 only: weights below 2^-14 have a fixed spacing of
                   2^-24 (the running maximum's weight is 1, so l >= 1)
  2^-25            binary16 only: the same of the output
where d = ln 2 * (error of t) + 2^-21: the score's error is at most
64 * 2^-23 sum_d |q_d k_d| c (64 products, each sum rounded or cut to 24 bits)
plus 2^-23 |t| twice (scaling and the difference), and 2^-21 covers ex2, the
running rescales and the binary32 sums of P V (64 terms a tile, then tiles).
L's bound is the error of t + 2 d / ln 2 + 2^-22 |L|.
"""
import math

import torch

D = 64
LN2 = math.log(2.0)


def attend64(q, k, v, seen, scale=0.125):
    """q [n, H, 64], k, v [m, Hkv, 64]; row i sees the first seen[i] keys.
    Returns O, L (base 2) and their tolerances, in float64."""
    n, H, _ = q.shape
    m, Hkv, _ = k.shape
    g = H // Hkv
    u = torch.finfo(q.dtype).eps / 2
    f16 = q.dtype == torch.float16
    dev = q.device
    o = torch.zeros((n, H, D), dtype=torch.float64, device=dev)
    lse = torch.full((H, n), -math.inf, dtype=torch.float64, device=dev)
    otol = torch.zeros_like(o)
    ltol = torch.zeros_like(lse)
    if n == 0 or m == 0:
        return o, lse, otol, ltol
    mask = torch.arange(m, device=dev)[None] >= seen[:, None]
    some = (seen > 0)
    for h in range(H):
        qd = q[:, h].double()
        # a key that no row sees may hold anything: it takes no part
        used = (~mask).any(0)
        kd = torch.where(used[:, None], k[:, h // g].double(), 0.0)
        vd = torch.where(used[:, None], v[:, h // g].double(), 0.0)
        c = scale / LN2
        t = (qd @ kd.T) * c
        fin = torch.isfinite(kd).all(1)
        kabs = torch.where(fin[:, None], kd, 0.0).abs()
        qabs = torch.nan_to_num(qd, 0.0, 0.0, 0.0).abs()
        terr = (64 * 2.0 ** -23 * (qabs @ kabs.T) * c).masked_fill(mask, 0.0)
        terr = terr + 2 * 2.0 ** -23 * torch.nan_to_num(t, 0.0, 0.0, 0.0).abs().masked_fill(mask, 0)
        terr = terr.amax(1)
        t = t.masked_fill(mask, -math.inf)
        mx = t.amax(1).masked_fill(~some, 0.0)
        p = torch.exp2(t - mx[:, None])
        z = p.sum(1)
        w = p / z.clamp(min=1e-300)[:, None]
        # rows must not meet the values of keys that they do not see
        o_h = torch.zeros((n, D), dtype=torch.float64, device=dev)
        a_h = torch.zeros_like(o_h)
        s_h = torch.zeros_like(o_h)
        if torch.isfinite(vd).all():
            o_h, a_h = w @ vd, w @ vd.abs()
            s_h = (~mask).double() @ vd.abs()
        else:
            for i in range(n):
                x = int(seen[i])
                if x > 0:
                    o_h[i], a_h[i] = w[i, :x] @ vd[:x], w[i, :x] @ vd[:x].abs()
                    s_h[i] = vd[:x].abs().sum(0)
        d = LN2 * terr + 2.0 ** -21
        tol = u * o_h.abs() + (u + 2 * d[:, None]) * a_h
        if f16:
            tol = tol + 2.0 ** -25 * s_h + 2.0 ** -25
        o[:, h] = torch.where(some[:, None], o_h, 0.0)
        otol[:, h] = torch.where(some[:, None], tol, 0.0)
        L = mx + torch.log2(z)
        lse[h] = torch.where(some, L, -math.inf)
        ltol[h] = torch.where(some, terr + 2 * d / LN2 + 2.0 ** -22 * L.abs(), 0.0)
    return o, lse, otol, ltol


def check(got, want, tol, what):
    """Within tol where the value is finite, the same infinity or NaN elsewhere."""
    if want.numel() == 0:
        return
    got = got.double()
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), "%s: other infinities or NaN: %s" % (
        what, (torch.isfinite(got) != fin).nonzero()[:5].tolist())
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    err = torch.where(fin, (got - want).abs() - tol, -1.0)
    worst = int(err.argmax())
    assert float(err.max()) <= 0, "%s: off by %g more than its bound at %d: %g for %g" % (
        what, float(err.max()), worst, float(got.flatten()[worst]), float(want.flatten()[worst]))


def packed64(q, k, v, cu, causal, scale=0.125):
    """[(rows, O, L, tolerances)] of every sequence."""
    out = []
    for a, b in zip(cu[:-1], cu[1:]):
        i = torch.arange(1, b - a + 1, device=q.device)
        seen = i if causal else torch.full_like(i, b - a)
        out.append((slice(a, b),) + attend64(q[a:b], k[a:b], v[a:b], seen, scale))
    return out


def gather(pool, row, n):
    """The first n tokens that a table row names, [n, Hkv, 64]."""
    p = pool.shape[2]
    if n <= 0:
        return pool.new_zeros((0, pool.shape[1], D))
    j = torch.arange(n, device=pool.device)
    return pool[row.long()[j // p], :, j % p]


def paged64(q, kc, vc, table, cu, lens, scale=0.125):
    out = []
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        n, m = b - a, lens[i]
        seen = (m - n + 1 + torch.arange(n, device=q.device)).clamp(min=0)
        out.append((slice(a, b),) + attend64(q[a:b], gather(kc, table[i], m),
                                             gather(vc, table[i], m), seen, scale))
    return out


def plan_host(cached, fresh, ring, state, table, tokens, page, width):
    """attn_paged_plan on lists: (cu, lens, slots, ring, table, next)."""
    N, (head, free) = len(ring), state[:2]
    up = lambda x: -(-x // page)
    st = 0
    if not (0 <= head < N and 0 <= free <= N):
        st |= 8
    if any(c < 0 for c in cached):
        st |= 8
    cc = [max(c, 0) for c in cached]
    back = sum(up(c) for c, f in zip(cc, fresh) if f < 0)
    if free + back > N:
        st |= 8
    if any(up(c + max(f, 0)) > width for c, f in zip(cc, fresh)):
        st |= 2
    need = sum(up(c + f) - up(c) for c, f in zip(cc, fresh) if f >= 0)
    if need > free:
        st |= 1
    if sum(max(f, 0) for f in fresh) > tokens:
        st |= 4
    ring, table = list(ring), [list(r) for r in table]
    if st:
        return [0] * (len(cached) + 1), list(cached), [-1] * tokens, ring, table, \
            [head, free, 0, st]
    cu, lens, slots, taken, tail = [0], [], [], 0, 0
    for i, (c, f) in enumerate(zip(cached, fresh)):
        if f < 0:
            lens.append(0)
            cu.append(cu[-1])
            for x in range(up(c)):
                ring[(head + free + tail) % N] = table[i][x]
                tail += 1
            continue
        for x in range(up(c), up(c + f)):
            table[i][x] = ring[(head + taken) % N]
            taken += 1
        slots += [table[i][p // page] * page + p % page for p in range(c, c + f)]
        lens.append(c + f)
        cu.append(cu[-1] + f)
    slots += [-1] * (tokens - len(slots))
    return cu, lens, slots, ring, table, [(head + taken) % N, free - taken + tail, taken, 0]
