"""The 4-bit cache and the rotated append in plain torch, and the tolerances of
attention over 4 bits.

Rows in and out are compared bit for bit: the rotation's products and sums and a
code's quotient are single binary32 operations, a scale's roundings are exact in
64 bits, and code * scale is exact in the type.

Attention: the bound of serve_util with another error of the scores and of small
weights.  The kernel for few rows sums q * (code + 8) from a start of -8 sum q, so
that a term has up to |q| (15 + 8), and applies the scale afterwards: 64 products,
two starts and the sum of q (32 and two shuffles), each rounded or cut to 24 bits,
three roundings of the scaling: 103 * 2^-23 sum_d |q_d| 23 s_d c; q itself goes in
as binary16 with the row's largest element between 2^9 and 2^10, whose spacing of
2^-24 at the small end is 2^-34 of that: with the binary32 roundings above, 2^-33
max |q| sum_d 23 s_d c more.  The kernel for many rows forms exact 16-bit values
first, which is less.
Weights times V's scales are binary16 in the kernel for few rows, a weight of 1
counting 2^10 and the scales in a unit of at most the largest of them, S: spacing
2^-24, so a key's share of O is off by up to 2^-25 2^-10 8 S, the sum of weights
being at least one: 2^-32 n S.  The kernel for many rows rounds weights to the type
(binary16: 2^-25 sum |v_j|).
Weights below 2^-126 count as zero (the exponential gives no subnormal numbers), and
so may a subnormal product: 2^-126 (sum |v_j| + 1), which only an element whose
large values all have such weights comes near (one of 1.27e-38 did, where the bound
without the term is a quarter of that).
"""
import math

import torch

from serve_util import D, LN2

UNIT = 288
KEEP = {torch.float16: 8, torch.bfloat16: 5}
MOST = {torch.float16: 8160.0, torch.bfloat16: 2.0 ** 123}


def rotate(x, cos, sin):
    """Rows x [t, H, 64] in binary32, products and sums rounded one by one."""
    a, b = x[..., :32].float(), x[..., 32:].float()
    c, s = cos[:, None], sin[:, None]
    ac, bs, bc, as_ = a * c, b * s, b * c, a * s
    return torch.cat([ac - bs, bc + as_], -1)


def quantise(x, dtype):
    """x [..., 64] binary32 -> codes int64 [..., 64] in -8..7, scales [..., 2]."""
    g = x.double().unflatten(-1, (2, 32))
    fine = torch.isfinite(g).all(-1)
    g = torch.where(fine[..., None], g, 0.0)
    hi, lo = g.amax(-1), g.amin(-1)
    e = torch.where(lo.abs() >= hi.abs(), lo, hi)
    # the extremum over -8 to KEEP bits, halves away; below binary32's normal
    # numbers the bits that count are fixed
    frac, exp = torch.frexp(-e / 8)
    unit = torch.ldexp(torch.ones_like(e), exp.clamp(min=-125) - KEEP[dtype])
    s = torch.sign(frac) * torch.floor((e / 8).abs() / unit + 0.5) * unit
    s = s.clamp(-MOST[dtype], MOST[dtype]).to(dtype)
    s1 = s.float()[..., None]
    quot = torch.where(s1 != 0, g.float() / torch.where(s1 == 0, 1.0, s1), 0.0)
    codes = torch.round(quot).clamp(-8, 7).to(torch.int64)
    return codes.flatten(-2), torch.where(fine, s, float("nan"))


def pack(codes, scales):
    """Rows [..., 36] of bytes."""
    c = (codes + 8).unflatten(-1, (2, 32))
    both = (c[..., 0, :] + 16 * c[..., 1, :]).to(torch.uint8)
    return torch.cat([both, scales.contiguous().view(torch.uint8)], -1)


def row_bytes(pool):
    """A view-free copy [pages, heads, page, 36] of a pool's rows."""
    p, h, u, _ = pool.shape
    codes = pool[..., :256].reshape(p, h, u * 8, 32)
    return torch.cat([codes, pool[..., 256:].reshape(p, h, u * 8, 4)], -1)


def put(pool, page, row, data):
    """data [n, heads, 36] into rows (page, row)."""
    for i, (a, r) in enumerate(zip(page.tolist(), row.tolist())):
        pool[a, :, r // 8, r % 8 * 32:r % 8 * 32 + 32] = data[i, :, :32]
        pool[a, :, r // 8, 256 + r % 8 * 4:260 + r % 8 * 4] = data[i, :, 32:]


def values(pool, dtype):
    """[pages, heads, page, 64] in 64 bits and the scales' magnitudes, as wide."""
    b = row_bytes(pool)
    s = b[..., 32:].contiguous().view(dtype).double()
    c = b[..., :32].to(torch.int64)
    s = torch.cat([s[..., :1].expand(*c.shape), s[..., 1:].expand(*c.shape)], -1)
    return torch.cat([c % 16 - 8, c // 16 - 8], -1) * s, s.abs()


def pool_of(x, dtype):
    """A pool that holds rows x [pages, heads, page, 64]."""
    p, h, n, _ = x.shape
    b = pack(*quantise(x.float(), dtype)).reshape(p, h, n // 8, 8, 36)
    return torch.cat([b[..., :32].flatten(-2), b[..., 32:].flatten(-2)], -1).contiguous()


def attend4(q, k, ks, v, vs, seen, scale=0.125):
    """q [n, H, 64] 16-bit; k, v [m, Hkv, 64] in 64 bits and ks, vs their scales'
    magnitudes; row i sees the first seen[i] keys.  Returns O, L (base 2) and their
    tolerances."""
    n, H, _ = q.shape
    m, Hkv, _ = k.shape
    g = H // Hkv
    u = torch.finfo(q.dtype).eps / 2
    f16 = q.dtype == torch.float16
    dev = q.device
    o = torch.zeros((n, H, D), dtype=torch.float64, device=dev)
    lse = torch.full((H, n), -math.inf, dtype=torch.float64, device=dev)
    otol, ltol = torch.zeros_like(o), torch.zeros_like(lse)
    if n == 0 or m == 0:
        return o, lse, otol, ltol
    mask = torch.arange(m, device=dev)[None] >= seen[:, None]
    some = seen > 0
    used = (~mask).any(0)[:, None]
    c = scale / LN2
    for h in range(H):
        qd = q[:, h].double()
        kd, sd, vd = (torch.where(used, x[:, h // g], 0.0) for x in (k, ks, v))
        t = (qd @ kd.T) * c
        sd = torch.nan_to_num(sd, 0.0, 0.0, 0.0)
        terr = 103 * 2.0 ** -23 * 23 * c * (torch.nan_to_num(qd, 0.0, 0.0, 0.0).abs() @ sd.T)
        big = torch.nan_to_num(qd, 0.0, 0.0, 0.0).abs().amax(1, keepdim=True)
        terr = terr + 2.0 ** -33 * 23 * c * big * sd.sum(1)
        terr = terr + 2 * 2.0 ** -23 * torch.nan_to_num(t, 0.0, 0.0, 0.0).abs()
        terr = terr.masked_fill(mask, 0.0).amax(1)
        t = t.masked_fill(mask, -math.inf)
        mx = t.amax(1).masked_fill(~some, 0.0)
        p = torch.exp2(t - mx[:, None])
        z = p.sum(1)
        w = p / z.clamp(min=1e-300)[:, None]
        if torch.isfinite(vd).all():
            o_h, a_h, s_h = w @ vd, w @ vd.abs(), (~mask).double() @ vd.abs()
        else:
            o_h = torch.zeros((n, D), dtype=torch.float64, device=dev)
            a_h, s_h = torch.zeros_like(o_h), torch.zeros_like(o_h)
            for i in range(n):
                x = int(seen[i])
                if x > 0:
                    o_h[i], a_h[i] = w[i, :x] @ vd[:x], w[i, :x] @ vd[:x].abs()
                    s_h[i] = vd[:x].abs().sum(0)
        d = LN2 * terr + 2.0 ** -21
        tol = u * o_h.abs() + (u + 2 * d[:, None]) * a_h + 2.0 ** -126 * (s_h + 1)
        top = torch.nan_to_num(torch.where(used, vs[:, h // g], 0.0), 0.0, 0.0, 0.0).max()
        tol = tol + 2.0 ** -32 * m * top
        if f16:
            tol = tol + 2.0 ** -25 * s_h + 2.0 ** -25
        o[:, h] = torch.where(some[:, None], o_h, 0.0)
        otol[:, h] = torch.where(some[:, None], tol, 0.0)
        L = mx + torch.log2(z)
        lse[h] = torch.where(some, L, -math.inf)
        ltol[h] = torch.where(some, terr + 2 * d / LN2 + 2.0 ** -22 * L.abs(), 0.0)
    return o, lse, otol, ltol


def gather(pool, row, n):
    """The first n tokens that a table row names, [n, heads, 64]."""
    p = pool.shape[2]
    if n <= 0:
        return pool.new_zeros((0, pool.shape[1], D))
    j = torch.arange(n, device=pool.device)
    return pool[row.long()[j // p], :, j % p]


def paged4_64(q, kc, vc, table, cu, lens, scale=0.125):
    """[(rows, O, L, tolerances)] of every request over 4-bit pools."""
    k, ks = values(kc, q.dtype)
    v, vs = values(vc, q.dtype)
    out = []
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        n, m = b - a, lens[i]
        seen = (m - n + 1 + torch.arange(n, device=q.device)).clamp(min=0)
        out.append((slice(a, b),) + attend4(q[a:b], gather(k, table[i], m),
                                            gather(ks, table[i], m), gather(v, table[i], m),
                                            gather(vs, table[i], m), seen, scale))
    return out
