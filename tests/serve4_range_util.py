"""Attention over 4-bit pools whose magnitudes differ by key, by channel group and
by row: problems, and a bound that a row's own keys alone enter.

The bound of an output element of row i, head h (P the row's normalised weights, A =
sum_k P_k |v_k|, u = eps / 2 of the type, d the relative error of the weights):
  u |O|                       rounding of the stored output
  u A                         a weight times a scale in 16 bits: at most 2^-11
                              (binary16) or the type's own rounding
  2 d A                       as in serve_util
  sum_k min(P_k, 2^-25) |v_k| weights in binary16 where they are small: a key's
                              weight counts 2^10 times its scale over a unit, and no key
                              goes in whose scale lies below 2^-10 of the unit, so half a
                              spacing of 2^-24 is at most 2^-25 of its |v|; nothing is
                              lost that the key does not have
  2^-126 (sum_k |v_k| + 1)    the exponential gives no subnormal numbers
  2^-25                       binary16 only: spacing of the smallest outputs
Scores: 103 * 2^-23 * 23 c sum_d |q_d| s_d as in serve4_util (either channel group has
sums of its own), two roundings of t, and q in binary16.  A row's elements of a group
have a spacing of 2^-24 where the row's largest element counts 2^9 or more: half of
that is 2^-34 of it, or, where the group's own largest is the measure, 2^-21 of the
group's (a group further below than 2^12 is scaled by itself): the smaller of both,
twice for the rounding of the sum of q, times 23 s_d.
"""
import math
import random

import torch

from serve4_util import gather, pool_of, values
from serve_util import D, LN2


def attend4_own(q, k, ks, v, vs, seen, scale=0.125):
    """q [n, H, 64]; k, v [m, Hkv, 64] in 64 bits and K's scales' magnitudes; finite.
    O, L (base 2) and their bounds."""
    n, H, _ = q.shape
    m, Hkv, _ = k.shape
    g, dev = H // Hkv, q.device
    u = torch.finfo(q.dtype).eps / 2
    f16 = q.dtype == torch.float16
    o = torch.zeros((n, H, D), dtype=torch.float64, device=dev)
    lse = torch.full((H, n), -math.inf, dtype=torch.float64, device=dev)
    otol, ltol = torch.zeros_like(o), torch.zeros_like(lse)
    if n == 0 or m == 0:
        return o, lse, otol, ltol
    mask = torch.arange(m, device=dev)[None] >= seen[:, None]
    some = seen > 0
    c = scale / LN2
    for h in range(H):
        qd, kd, sd, vd = q[:, h].double(), k[:, h // g], ks[:, h // g], v[:, h // g]
        t = (qd @ kd.T) * c
        terr = 103 * 2.0 ** -23 * 23 * c * (qd.abs() @ sd.T)
        row = qd.abs().amax(1, keepdim=True)
        for part in (slice(0, 32), slice(32, 64)):
            own = qd[:, part].abs().amax(1, keepdim=True)
            off = torch.minimum(2.0 ** -33 * row, 2.0 ** -20 * own)
            terr = terr + 23 * c * off * sd[:, part].sum(1)
        terr = (terr + 2 * 2.0 ** -23 * t.abs()).masked_fill(mask, 0.0).amax(1)
        t = t.masked_fill(mask, -math.inf)
        mx = t.amax(1).masked_fill(~some, 0.0)
        p = torch.exp2(t - mx[:, None])
        z = p.sum(1)
        w = p / z.clamp(min=1e-300)[:, None]
        o_h, a_h, s_h = w @ vd, w @ vd.abs(), (~mask).double() @ vd.abs()
        d = LN2 * terr + 2.0 ** -21
        tol = u * o_h.abs() + (u + 2 * d[:, None]) * a_h + 2.0 ** -126 * (s_h + 1)
        tol = tol + w.clamp(max=2.0 ** -25) @ vd.abs()
        if f16:
            tol = tol + 2.0 ** -25
        o[:, h] = torch.where(some[:, None], o_h, 0.0)
        otol[:, h] = torch.where(some[:, None], tol, 0.0)
        L = mx + torch.log2(z)
        lse[h] = torch.where(some, L, -math.inf)
        ltol[h] = torch.where(some, terr + 2 * d / LN2 + 2.0 ** -22 * L.abs(), 0.0)
    return o, lse, otol, ltol


def own64(q, kc, vc, table, cu, lens, scale=0.125):
    """[(rows, O, L, bounds)] of every request over 4-bit pools."""
    (k, ks), (v, vs) = values(kc, q.dtype), values(vc, q.dtype)
    tt = torch.tensor(table, dtype=torch.int64, device=q.device)
    out = []
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        n, m = b - a, lens[i]
        seen = (m - n + 1 + torch.arange(n, device=q.device)).clamp(min=0)
        out.append((slice(a, b),) + attend4_own(q[a:b], *(gather(x, tt[i], m)
                                                          for x in (k, ks, v, vs)), seen, scale))
    return out


def problem(reqs, H, Hkv, page, dtype, seed, shape_k=None, shape_v=None, shape_q=None):
    """reqs: (keys in the cache, new tokens).  shape_k(i, x), shape_v(i, x): K and V
    [keys, Hkv, 64] of request i before they are quantised, binary64, changed in place;
    shape_q(q): the queries [rows, H, 64]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    up = [-(-n // page) for n, _ in reqs]
    order = list(range(sum(up) + 2))
    r.shuffle(order)
    width = max(1, max(up))
    table = [[order.pop() for _ in range(u)] + [-1] * (width - u) for u in up]
    pools = []
    for shape in (shape_k, shape_v):
        x = torch.randn((sum(up) + 2, page, Hkv, D), generator=g, device="cuda",
                        dtype=torch.float64)
        for i, (n, _) in enumerate(reqs):
            j = torch.arange(n, device="cuda")
            at = torch.tensor(table[i], device="cuda", dtype=torch.int64)[j // page]
            rows = x[at, j % page]
            if shape is not None:
                shape(i, rows)
            x[at, j % page] = rows
        pools.append(pool_of(x.transpose(1, 2).to(dtype), dtype))
    cu = [0]
    for _, n in reqs:
        cu.append(cu[-1] + n)
    q = 2 * torch.randn((cu[-1], H, D), generator=g, device="cuda", dtype=torch.float64)
    if shape_q is not None:
        shape_q(q)
    return q.to(dtype), pools[0], pools[1], table, cu, [n for n, _ in reqs]
