"""Float64 definitions of the operators of a decoder layer (feed-forward block,
norms around a block, dropout), with bounds on how far their documented
roundings may move each element of the results.

A rounding to bfloat16 is off by at most 2^-8 of the value (half a step), one
to float32 by 2^-24; a float32 sum of n terms is off by at most n 2^-24 of the
sum of magnitudes, in any order.
"""

import math

import numpy as np
import torch

BF = 2.0 ** -8
F32 = 2.0 ** -24


def rounding(dtype):
    return BF if dtype is torch.bfloat16 else F32


# ------------------------------------------------------------ feed-forward

# largest |act'| and |act''| (relu: of either side of 0)
SLOPE = {"silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13, "relu": 1.0}
BEND = {"silu": 0.51, "gelu": 0.8, "gelu_tanh": 0.82, "relu": 0.0}


def act(name, g):
    """act(g) and its derivative, float64."""
    if name == "relu":
        return g.clamp(min=0), (g > 0).double()
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def feed_forward(x, wg, wu, wd, name, dout=None, dtype=torch.bfloat16):
    """(results, bounds): dicts of out, kept and, with dout, dx, dwg, dwu, dwd (float64, CPU)."""
    x, wg, wu, wd = (t.double().cpu() for t in (x, wg, wu, wd))
    n, width = x.shape
    hidden = wg.shape[0]
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = (width * F32 * (x.abs() @ w.abs().t()) for w in (wg, wu))
    a, da = act(name, g)
    h = a * u
    # a dozen float32 steps of act, whose exponential's argument is off by a few of its own
    steps = 16 * F32 * (1 + g.abs())
    eh = SLOPE[name] * eg * (u.abs() + eu) + a.abs() * eu + steps * h.abs() + F32 * u.abs()
    eh = eh + BF * (h.abs() + eh)
    out = h @ wd.t()
    eo = eh @ wd.abs().t() + hidden * F32 * (h.abs() + eh) @ wd.abs().t()
    eo = eo + BF * (out.abs() + eo)
    eg, eu = eg + BF * (g.abs() + eg), eu + BF * (u.abs() + eu)
    res = {"out": out, "kept": torch.stack([g, u, h])}
    bound = {"out": eo, "kept": torch.stack([eg, eu, eh])}
    if dout is None:
        return res, bound
    do = dout.double().cpu()
    dh = do @ wd
    edh = width * F32 * (do.abs() @ wd.abs())
    big = dh.abs() + edh
    dg, du = dh * u * da, dh * a
    edg = (u.abs() * da.abs() * edh + big * da.abs() * eu + big * (u.abs() + eu) * BEND[name] * eg
           + big * u.abs() * steps + F32 * big * u.abs())
    if name == "relu":
        edg = edg + torch.where(g.abs() <= eg, big * (u.abs() + eu), 0.0)
    edg = edg + BF * (dg.abs() + edg)
    edu = a.abs() * edh + big * SLOPE[name] * eg + steps * big * a.abs()
    edu = edu + BF * (du.abs() + edu)
    res["dx"] = dg @ wg + du @ wu
    e = edg @ wg.abs() + edu @ wu.abs()
    e = e + 2 * hidden * F32 * ((dg.abs() + edg) @ wg.abs() + (du.abs() + edu) @ wu.abs())
    bound["dx"] = e + BF * (res["dx"].abs() + e)
    for key, left, eleft, right, eright in (("dwg", dg, edg, x, None), ("dwu", du, edu, x, None), ("dwd", do, None, h, eh)):
        res[key] = left.t() @ right
        e = eleft.t() @ right.abs() if eleft is not None else left.abs().t() @ eright
        big_l = left.abs() + (0 if eleft is None else eleft)
        big_r = right.abs() + (0 if eright is None else eright)
        e = e + max(1, n) * F32 * big_l.t() @ big_r
        bound[key] = e + rounding(dtype) * (res[key].abs() + e)
    return res, bound


# ----------------------------------------------------------------- dropout

def philox(seed, block):
    """The four words of Philox4x32-10 for the counter (block, 0) under the key seed, from Python integers."""
    low = 0xFFFFFFFF
    c = [block & low, block >> 32 & low, 0, 0]
    k = [seed & low, seed >> 32 & low]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [b >> 32 ^ c[1] ^ k[0], b & low, a >> 32 ^ c[3] ^ k[1], a & low]
        k = [k[0] + 0x9E3779B9 & low, k[1] + 0xBB67AE85 & low]
    return c


def bits(seed, block):
    """The 16 bits of the 8 elements of a block."""
    return [w >> s & 0xFFFF for w in philox(seed, block) for s in (0, 16)]


def factors(n, p, seed, offset=0):
    """float64 factors of n elements: 0, or 65536 / (65536 - t)."""
    t = int(math.floor(p * 65536 + 0.5))
    seed, offset = seed & (1 << 64) - 1, offset & (1 << 64) - 1
    v = []
    for b in range((n + 7) // 8):
        v += bits(seed, (offset + b) & (1 << 64) - 1)
    keep = np.array(v[:n], dtype=np.int64) >= t
    return torch.from_numpy(keep).double() * (65536 / (65536 - t) if t < 65536 else 0.0)


# ---------------------------------------------------- norms around a block

def residual_norm(x, y=None, gate=None, scale=None, postw=None, prew=None, post=True, eps=1e-6, factor=None,
                  xo=None, dz=None, dxo=None):
    """Results and bounds of the forward pass (x_out, z) or, with dz, of the
    gradients at the stream xo; float64, CPU; x (batch, s, width); factor:
    dropout's, shaped as x.  The gate may be (width,), (batch, width) or full."""
    d = lambda t: None if t is None else t.double().cpu()  # noqa: E731
    src_x, src_y = x, y
    x, y, gate, scale, postw, prew, xo, dz, dxo = map(d, (x, y, gate, scale, postw, prew, xo, dz, dxo))
    width = x.shape[-1] if x is not None else xo.shape[-1]
    one = torch.ones(width, dtype=torch.float64)
    scale, prew = (one if scale is None else scale), (one if prew is None else prew)
    w1 = one if postw is None else postw
    step = F32 * (width + 16)  # of a norm: the sum of its squares, and a dozen operations
    gfull = 1.0
    if gate is not None:
        gfull = gate[:, None] if gate.dim() == 2 and src_y.dim() == 3 else gate
    if y is not None:
        f = torch.ones_like(y) if factor is None else factor
        r = (y.square().mean(-1, keepdim=True) + eps).rsqrt() if post else torch.ones(1, dtype=torch.float64)
        n = y * r * w1 * f
        en = step * n.abs()
    stream = rounding((src_x if src_x is not None else None).dtype) if dz is None else None
    if dz is None:
        v = x * scale + (gfull * n if y is not None else 0.0)
        mag = (x * scale).abs() + ((gfull * n).abs() if y is not None else 0.0)
        ev = 4 * F32 * mag + (abs(gfull) * en if y is not None else 0.0)
        rr = (v.square().mean(-1, keepdim=True) + eps).rsqrt()
        z = v * rr * prew
        # r' moves by at most r' times the relative move of the row's 2-norm
        move = (ev.square().sum(-1, keepdim=True).sqrt() / v.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-300))
        ez = ev * rr * prew.abs() + z.abs() * (step + move)
        zt = BF if (src_y.dtype if src_y is not None else src_x.dtype) is torch.bfloat16 else F32
        return {"x_out": v, "z": z}, {"x_out": ev + stream * (v.abs() + ev), "z": ez + zt * (z.abs() + ez)}
    rows = xo.numel() // width
    rr = (xo.square().mean(-1, keepdim=True) + eps).rsqrt()
    unit = xo * rr
    t = dz * prew
    m = (t * unit).mean(-1, keepdim=True)
    mm = (t * unit).abs().mean(-1, keepdim=True)
    e = rr * (t - unit * m) + (0.0 if dxo is None else dxo)
    ee = 2 * step * rr * (t.abs() + unit.abs() * mm) + 4 * F32 * e.abs() + (0.0 if dxo is None else F32 * dxo.abs())
    total = (0, 1)
    res = {"dx": e * scale, "dprew": (dz * unit).sum(total)}
    bound = {"dx": ee * scale.abs() + F32 * (e * scale).abs(),
             "dprew": (step + rows * F32) * (dz * unit).abs().sum(total)}
    if x is not None:
        res["dscale"] = (e * x).sum(total)
        bound["dscale"] = (ee * x.abs()).sum(total) + (rows + 2) * F32 * ((e.abs() + ee) * x.abs()).sum(total)
    if y is None:
        return res, bound
    dg = e * n
    edg = ee * n.abs() + (e.abs() + ee) * en + F32 * dg.abs()
    if gate is not None:
        if gate.dim() == 1:
            res["dgate"], bound["dgate"] = dg.sum(total), edg.sum(total) + rows * F32 * dg.abs().sum(total)
        elif gate.dim() == 2 and src_y.dim() == 3:
            res["dgate"], bound["dgate"] = dg.sum(1), edg.sum(1) + rows * F32 * dg.abs().sum(1)
        else:
            res["dgate"], bound["dgate"] = dg, edg
    dn = e * gfull * f
    edn = ee * abs(gfull) * f + 4 * F32 * dn.abs()
    if post:
        yu = y * r
        res["dpostw"] = (dn * yu).sum(total)
        bound["dpostw"] = (edn * yu.abs()).sum(total) + (step + rows * F32) * ((dn.abs() + edn) * yu.abs()).sum(total)
        u = dn * w1
        eu = edn * w1.abs() + F32 * u.abs()
        m = (u * yu).mean(-1, keepdim=True)
        em = (eu * yu.abs()).mean(-1, keepdim=True) + step * (u * yu).abs().mean(-1, keepdim=True)
        dy = r * (u - yu * m)
        edy = r * (eu + yu.abs() * em) + 2 * step * r * (u.abs() + yu.abs() * m.abs())
    else:
        dy, edy = dn, edn
    res["dy"], bound["dy"] = dy, edy
    return res, bound
