"""Float64 definitions of the language-model operators, with bounds on how far
bfloat16 operands and float32 sums may move the results.

A rounding to bfloat16 is off by at most 2^-8 of the value (half a step), one
to float32 by 2^-24.  The bounds add up, for every output element, what the
documented roundings can do to it: the probabilities and the gradients of the
scores are rounded to bfloat16 once, the outputs once, and everything else is
float32 with sums of n terms off by at most n 2^-24 of the sum of magnitudes.
"""

import math

import torch

BF = 2.0 ** -8
F32 = 2.0 ** -24


def visible(b, sq, sk, causal=True, window=0, documents=None, prefix=None, lengths=None, starts=None):
    """(b, sq, sk) truth values and the query positions (b, sq)."""
    j = torch.arange(sk)
    vis = torch.zeros(b, sq, sk, dtype=torch.bool)
    pos = torch.zeros(b, sq, dtype=torch.long)
    for n in range(b):
        first = int(starts[n]) if starts is not None else sk - sq
        length = min(max(int(lengths[n]), 0), sk) if lengths is not None else sk
        for i in range(sq):
            p = first + i
            pos[n, i] = p
            see = torch.ones(sk, dtype=torch.bool)
            if causal:
                see &= j <= p
            if window:
                see &= (j - p).abs() < window
            if prefix is not None:
                see |= j < int(prefix[n])
            if documents is not None and sk:
                see &= documents[n] == documents[n][min(max(p, 0), sk - 1)]
            if lengths is not None:
                see &= j < length
                if p >= length:
                    see[:] = False
            vis[n, i] = see
    return vis, pos


def attention(q, k, v, dout=None, scale=None, causal=True, window=0, softcap=0.0, slopes=None, documents=None,
              prefix=None, lengths=None, starts=None):
    """(results, bounds): dicts of out, lse and, with dout, dq, dk, dv (float64, CPU)."""
    q, k, v = (t.detach().cpu().double() for t in (q, k, v))
    b, sq, hq, d = q.shape
    sk, hkv = k.shape[1:3]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    vis, pos = visible(b, sq, sk, causal, window, cpu(documents), cpu(prefix), cpu(lengths), cpu(starts))
    res = {"out": torch.zeros_like(q), "lse": torch.full((b, hq, sq), -math.inf, dtype=torch.float64)}
    tol = {"out": torch.zeros_like(q), "lse": torch.zeros(b, hq, sq, dtype=torch.float64)}
    if dout is not None:
        dout = dout.detach().cpu().double()
        for n, t in (("dq", q), ("dk", k), ("dv", v)):
            res[n], tol[n] = torch.zeros_like(t), torch.zeros_like(t)
    sums = (sk + d + 64) * F32
    for n in range(b):
        live = vis[n].any(1)
        seen = vis[n].any(0)
        for h in range(hq):
            u = h // (hq // hkv)
            # what nobody sees is padding: any value may be there
            qq = torch.where(live[:, None], q[n, :, h], 0.0)
            kk, vv = (torch.where(seen[:, None], t[n, :, u], 0.0) for t in (k, v))
            x = qq @ kk.T * scale
            ex = (d + 8) * F32 * (qq.abs() @ kk.abs().T) * scale
            z, slope = x, 1.0
            if softcap:
                th = torch.tanh(x / softcap)
                z, slope = softcap * th, 1 - th * th
                ex = ex + 2.0 ** -20 * softcap
            if slopes is not None:
                bias = float(slopes[h]) * (pos[n][:, None] - torch.arange(sk)).abs()
                z = z - bias
                ex = ex + 4 * F32 * bias.abs()
            z = torch.where(vis[n], z, -math.inf)
            lse = torch.logsumexp(z, 1) if sk else torch.full((sq,), -math.inf, dtype=torch.float64)
            p = torch.where(vis[n], torch.exp(z - torch.where(live, lse, 0.0)[:, None]), 0.0)
            # float32 exponents: their own rounding is relative to the size of z and lse
            ex = ex + 8 * F32 * (torch.where(vis[n], z.abs(), 0.0) + torch.where(live, lse.abs(), 0.0)[:, None] + 1)
            ex = torch.where(vis[n], ex, 0.0)
            elog = ex.amax(1) + sums if sk else torch.zeros(sq, dtype=torch.float64)
            ep = p * (ex + elog[:, None] + 4 * F32)     # without the rounding to bfloat16
            o = p @ vv
            eo = BF * o.abs() + (ep + p * (BF + sums)) @ vv.abs()
            res["out"][n, :, h], tol["out"][n, :, h] = o, eo
            res["lse"][n, h] = lse
            tol["lse"][n, h] = torch.where(live, elog + 4 * F32 * lse.abs(), 0.0)
            if dout is None:
                continue
            do = torch.where(live[:, None], dout[n, :, h], 0.0)
            dp = do @ vv.T
            delta = (do * o).sum(1, keepdim=True)
            ds = p * (dp - delta) * slope
            eds = (ep * (dp - delta).abs() + p * (sums * (do.abs() @ vv.abs().T) + (do.abs() * (eo + sums * o.abs())).sum(1, keepdim=True))) * slope
            if softcap:
                eds = eds + p * (dp - delta).abs() * 2.0 ** -20
            eds = eds + ds.abs() * BF
            res["dv"][n, :, u] += p.T @ do
            tol["dv"][n, :, u] += (ep + p * (BF + (sq * (hq // hkv) + 64) * F32)).T @ do.abs()
            res["dq"][n, :, h] = scale * ds @ kk
            tol["dq"][n, :, h] = scale * (eds + sums * ds.abs()) @ kk.abs()
            res["dk"][n, :, u] += scale * ds.T @ qq
            tol["dk"][n, :, u] += scale * (eds + (sq * (hq // hkv) + 64) * F32 * ds.abs()).T @ qq.abs()
    if dout is not None:
        for n in ("dq", "dk", "dv"):
            tol[n] += BF * (res[n].abs() + tol[n])
    tol["out"] += BF * tol["out"]
    return res, tol


def close(got, want, bound, name, floor=1e-30):
    """Every element within its bound; infinities in the same places."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin], want[~fin]), f"{name}: values that are not finite"
    off = torch.where(fin, (got - want).abs(), 0.0)
    bad = ~(off <= torch.where(fin, bound, 0.0) + floor)  # a NaN is bad
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} out of bounds, first at {at}: "
                             f"{got[tuple(at)].item()} for {want[tuple(at)].item()} +- {bound[tuple(at)].item()}")


def rotate_norm(x, w, table, positions, eps):
    x = x.detach().cpu().double()
    d = x.shape[-1]
    cs = table.cpu().double()[positions.cpu().long()][:, :, None]
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w.cpu().double()
    a, b = y[..., :d // 2], y[..., d // 2:]
    return torch.cat([a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1]], -1)
