"""Attention in float64 with bounds per element, for inputs where the bounds of
lm_reference.py are wider than the operator's accuracy: the error of a capped
score is relative to the score, and masks are given as truth values."""

import math

import torch

BF = 2.0 ** -8
F32 = 2.0 ** -24
# A capped score c tanh(x / c) above the cap of 64.  Near zero (|x / c| < 1/4):
# the product, five rounded steps of the series and its first term left out
# (9e-9), below 2^-21 of the score.  Else 1 - 2 r with r = 1 / (exp(2 y) + 1):
# exponential and reciprocal are each good to 2^-23, so 1 - 2 r is off by at most
# 2 (r (1 - r) 2^-22 + r 3 2^-24) + 2^-24 < 4e-7 up to r = 0.63, that is 1.7e-6 of
# tanh(1/4), and by less of larger values.  2^-19 = 1.9e-6 covers both.
CAP = 2.0 ** -19


def _one(q, k, v, do, vis, dist, scale, cap, slope):
    """One head: q (sq, d), k and v (sk, d); results and bounds."""
    d, (sq, sk) = q.shape[1], vis.shape
    sums = (sk + d + 64) * F32
    x = q @ k.T * scale
    ex = (d + 8) * F32 * (q.abs() @ k.abs().T) * scale
    z, down = x, torch.ones_like(x)
    if cap:
        t = torch.tanh(x / cap)
        z, down = cap * t, 1 - t * t
        ex = ex + CAP * z.abs()
    z = z - slope * dist
    ex = ex + 4 * F32 * abs(slope) * dist
    live = vis.any(1)
    z = torch.where(vis, z, -math.inf)
    lse = torch.logsumexp(z, 1)
    p = torch.where(vis, torch.exp(z - torch.where(live, lse, 0.0)[:, None]), 0.0)
    # float32 exponents: their own rounding is relative to the size of z and lse
    ex = ex + 8 * F32 * (torch.where(vis, z.abs(), 0.0) + torch.where(live, lse.abs(), 0.0)[:, None] + 1)
    ex = torch.where(vis, ex, 0.0)
    elog = ex.amax(1) + sums
    ep = p * (ex + elog[:, None] + 4 * F32)
    o = p @ v
    eo = BF * o.abs() + (ep + p * (BF + sums)) @ v.abs()
    res, tol = {"out": o, "lse": lse}, {"out": eo * (1 + BF), "lse": torch.where(live, elog + 4 * F32 * lse.abs(), 0.0)}
    if do is not None:
        dp = do @ v.T
        delta = (do * o).sum(1, keepdim=True)
        ds = p * (dp - delta) * down
        edelta = (do.abs() * (eo + sums * o.abs())).sum(1, keepdim=True)
        eds = (ep * (dp - delta).abs() + p * (sums * (do.abs() @ v.abs().T) + edelta)) * down
        if cap:
            # 4 (r - r^2): r is off by 2^-22 at most, and the slope of this is at most 4
            eds = eds + p * (dp - delta).abs() * 2.0 ** -20
        eds = eds + ds.abs() * BF
        res |= {"dv": p.T @ do, "dq": scale * ds @ k, "dk": scale * ds.T @ q}
        rows = (sq + 64) * F32
        tol |= {"dv": (ep + p * (BF + rows)).T @ do.abs(), "dq": scale * (eds + sums * ds.abs()) @ k.abs(),
                "dk": scale * (eds + rows * ds.abs()).T @ q.abs()}
    return res, tol


def attention(q, k, v, dout, vis, pos, scale=None, softcap=0.0, slopes=None):
    """(results, bounds), float64 on the CPU: vis (b, sq, sk) truth values, pos
    (b, sq).  What no query sees and queries that see nothing may hold
    anything."""
    q, k, v = (t.detach().cpu().double() for t in (q, k, v))
    do = None if dout is None else dout.detach().cpu().double()
    b, sq, hq, d = q.shape
    sk, hkv = k.shape[1:3]
    grp = hq // hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    live, seen = vis.any(2), vis.any(1)
    q = torch.where(live[:, :, None, None], q, 0.0)
    k, v = (torch.where(seen[:, :, None, None], t, 0.0) for t in (k, v))
    if do is not None:
        do = torch.where(live[:, :, None, None], do, 0.0)
    shapes = {"out": q.shape, "lse": (b, hq, sq), "dq": q.shape, "dk": k.shape, "dv": k.shape}
    names = ("out", "lse") if do is None else tuple(shapes)
    res, tol = ({n: torch.zeros(shapes[n], dtype=torch.float64) for n in names} for _ in range(2))
    for n in range(b):
        dist = (pos[n][:, None] - torch.arange(sk)).abs().double()
        for h in range(hq):
            got = _one(q[n, :, h], k[n, :, h // grp], v[n, :, h // grp], None if do is None else do[n, :, h], vis[n],
                       dist, scale, softcap, 0.0 if slopes is None else float(slopes[h]))
            for to, one in zip((res, tol), got):
                for name, t in one.items():
                    if name == "lse":
                        to[name][n, h] = t
                    else:
                        to[name][n, :, h // grp if name in ("dk", "dv") else h] += t
    for name in names[2:]:
        tol[name] += BF * (res[name].abs() + tol[name])
    return res, tol
