"""Cases of the language-model operators: attention, the norm and rotation of
queries and keys, and the embedding with its gradient.

Each case runs one operator as a training step, a prefill or a generation step
calls it.  ``run`` computes the plain form (elementary torch operations in
float32, rounded once at the end) or, with ``own`` set, calls
``newton_schulz_09_amd.lm``.  ``exact`` is the definition in float64, one head
or one array at a time.

Kinds of case

* ``forward``: attention of a prefill, a validation pass or a step of
  generation; outputs ``out`` (bfloat16) and ``lse`` (float32).
* ``train``: attention and its gradients; outputs ``out``, ``lse``, ``dq``,
  ``dk``, ``dv``.
* ``qk``: RMS norm of every query and key head with the rotation;
  ``qk_grad``: its gradients (inputs and both weights).
* ``embed``: scaled rows of the table; ``embed_grad``: the table's gradient.

Attention masks: ``causal``; ``window`` (0: none); ``cap`` (tanh cap, 0:
none); ``slopes`` (bias by distance); ``doc`` (mean document length, 0: one
document); ``prefix`` (share of the sequence that everybody sees); ``ragged``
(every sequence of the batch has its own length).
"""

import math
import random

import torch

own = False

DEV = "cuda"


def _attn(name, kind, b, sq, sk, hq, hkv, d, causal=True, window=0, cap=0.0, slopes=False, doc=0, prefix=0.0,
          ragged=False):
    return {"name": name, "kind": kind, "b": b, "sq": sq, "sk": sk, "hq": hq, "hkv": hkv, "d": d, "causal": causal,
            "window": window, "cap": cap, "slopes": slopes, "doc": doc, "prefix": prefix, "ragged": ragged}


def _qk(name, kind, b, s, hq, hkv, d, dtype, weights=True):
    return {"name": name, "kind": kind, "b": b, "s": s, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype,
            "weights": weights}


def _embed(name, kind, n, vocab, width, table, out):
    return {"name": name, "kind": kind, "n": n, "vocab": vocab, "width": width, "table": table, "out": out}


def listed():
    return [
        # one new token of one sequence with GPT-2 124M's heads: latency
        _attn("attn_one_token", "forward", 1, 1, 1023, 12, 12, 64),
        # a generation step of a full batch over long caches of unequal length, grouped heads, capped scores
        _attn("attn_generate", "forward", 32, 1, 16384, 32, 8, 128, cap=30.0, ragged=True),
        # a prefill: grouped heads, a prefix that all tokens see (instructions), odd length
        _attn("attn_prefill_prefix", "forward", 4, 4001, 4001, 32, 8, 128, prefix=0.2),
        # a GPT-2 124M layer of a training step (16 sequences of 1024)
        _attn("attn_train_124m", "train", 16, 1024, 1024, 12, 12, 64),
        # one packed sequence of many documents with a window and capped scores, as speedruns train
        _attn("attn_train_documents", "train", 1, 16384, 16384, 6, 6, 128, window=4096, cap=15.0, doc=2000),
        # GPT-2 1.5B's 25 heads with a bias by distance instead of a rotation, ragged batch, odd length
        _attn("attn_train_bias", "train", 3, 777, 777, 25, 25, 64, slopes=True, ragged=True),
        # queries and keys of a GPT-2 124M batch of 65536 tokens, and their gradients
        _qk("qk_124m", "qk", 64, 1024, 12, 12, 64, "bfloat16"),
        _qk("qk_grad_124m", "qk_grad", 64, 1024, 12, 12, 64, "bfloat16"),
        # one new token for each of 32 sequences, float32, grouped heads
        _qk("qk_one_token", "qk", 32, 1, 32, 8, 128, "float32", weights=False),
        # the batch's embeddings and the float32 table's gradient
        _embed("embed_124m", "embed", 65536, 50304, 768, "float32", "bfloat16"),
        _embed("embed_grad_124m", "embed_grad", 65536, 50304, 768, "float32", "bfloat16"),
        # a small odd batch of GPT-2 1.5B's width and vocabulary, bfloat16 throughout
        _embed("embed_grad_small", "embed_grad", 999, 50257, 1600, "bfloat16", "bfloat16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["forward", "forward", "train", "train", "qk", "qk_grad", "embed", "embed_grad"])
    if kind in ("forward", "train"):
        d = rng.choice([64, 64, 128, 128, 80])
        hkv = rng.choice([1, 2, 4, 8, 12])
        hq = hkv * rng.choice([1, 1, 2, 4])
        # generation: a few new tokens over a cache; otherwise whole sequences
        few = kind == "forward" and rng.random() < 0.5
        sk = _log(rng, 17, 16384 if few else 4096)
        sq = min(sk, rng.choice([1, 1, 2, 5])) if few else sk
        b = max(1, min(_log(rng, 1, 32), (1 << 23) // (sk * hkv) if few else 60000000 // (sk * sk * hq)))
        causal = few or rng.random() < 0.8
        c = _attn("", kind, b, sq, sk, hq, hkv, d, causal=causal)
        extra = rng.choice(["none", "window", "cap", "slopes", "doc", "prefix", "ragged", "all"])
        if extra in ("window", "all"):
            c["window"] = _log(rng, 8, max(9, sk))
        if extra in ("cap", "all"):
            c["cap"] = rng.choice([15.0, 30.0, 50.0])
        if extra in ("slopes", "all"):
            c["slopes"] = True
        if extra in ("doc", "all"):
            c["doc"] = _log(rng, 8, max(9, sk))
        if extra == "prefix" and causal:
            c["prefix"] = rng.uniform(0.05, 0.6)
        if extra in ("ragged", "all"):
            c["ragged"] = True
    elif kind in ("qk", "qk_grad"):
        d = rng.choice([64, 128, 80, 96])
        hkv = rng.choice([1, 2, 4, 8, 12])
        hq = hkv * rng.choice([1, 2, 4])
        s = _log(rng, 1, 4096)
        b = max(1, min(_log(rng, 1, 64), (1 << 26) // (s * d * (hq + hkv))))
        c = _qk("", kind, b, s, hq, hkv, d, rng.choice(["float32", "bfloat16", "bfloat16"]), rng.random() < 0.7)
    else:
        c = _embed("", kind, _log(rng, 1, 65536), _log(rng, 256, 50304), rng.choice([64, 100, 256, 640, 768]),
                   rng.choice(["float32", "bfloat16"]), rng.choice(["float32", "bfloat16"]))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _documents(rng, b, s, mean):
    """Document numbers of b packed sequences of s tokens (lengths spread about the mean)."""
    rows = []
    for _ in range(b):
        row, k = [], 0
        while len(row) < s:
            row += [k] * max(1, int(rng.uniform(0.2, 1.8) * mean))
            k += 1
        rows.append(row[:s])
    return rows


def _lengths(rng, b, lo, hi):
    return [rng.randint(max(1, lo), hi) for _ in range(b)]


def _layout(case, seed):
    """Host values of the masks: lengths, first positions, documents, prefixes."""
    rng = random.Random(seed)
    b, sq, sk = case["b"], case["sq"], case["sk"]
    lengths = _lengths(rng, b, sk // 2, sk) if case["ragged"] else None
    starts = None
    if lengths is not None:
        # a cache: the new tokens are the last ones; whole sequences: they start at 0 and the rest is padding
        starts = [max(0, n - sq) for n in lengths] if sq < sk else [0] * b
    docs = _documents(rng, b, sk, case["doc"]) if case["doc"] else None
    prefix = [int(case["prefix"] * sk * rng.uniform(0.8, 1.2)) for _ in range(b)] if case["prefix"] else None
    return lengths, starts, docs, prefix


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)

    def ints(v):
        return None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)

    kind = case["kind"]
    if kind in ("forward", "train"):
        b, sq, sk, hq, hkv, d = (case[n] for n in ("b", "sq", "sk", "hq", "hkv", "d"))
        lengths, starts, docs, prefix = _layout(case, seed)
        st = {"kind": kind, "causal": case["causal"], "window": case["window"], "softcap": case["cap"],
              "scale": 1.0 / math.sqrt(d), "lengths": ints(lengths), "starts": ints(starts),
              "documents": ints(docs), "prefix": ints(prefix), "slopes": None}
        if case["slopes"]:
            st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device=DEV)
        st["q"] = normal(b, sq, hq, d, std=1.5)
        st["k"] = normal(b, sk, hkv, d)
        if kind == "train":
            # v as it lies in the output of one projection of q, k and v
            st["v"] = normal(b, sk, hq + 2 * hkv, d)[:, :, hq + hkv:]
            st["dout"] = normal(b, sq, hq, d)
        else:
            st["v"] = normal(b, sk, hkv, d)
        return st
    if kind in ("qk", "qk_grad"):
        b, s, hq, hkv, d = (case[n] for n in ("b", "s", "hq", "hkv", "d"))
        dtype = getattr(torch, case["dtype"])
        # q and k as they lie in the output of one projection of q, k and v
        qkv = normal(b, s, hq + 2 * hkv, d, dtype=dtype, std=0.7)
        st = {"kind": kind, "q": qkv[:, :, :hq], "k": qkv[:, :, hq:hq + hkv], "eps": 1e-6, "qw": None, "kw": None}
        limit = 32768
        # the table a program builds once: (cos, sin) of position * base^(-2 i / d)
        freq = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d)
        angle = torch.arange(limit, dtype=torch.float64, device=DEV)[:, None] * freq
        st["table"] = torch.stack([angle.cos(), angle.sin()], dim=-1).float().contiguous()
        if case["weights"]:
            st["qw"] = 1.0 + normal(d, dtype=torch.float32, std=0.2)
            st["kw"] = 1.0 + normal(d, dtype=torch.float32, std=0.2)
        first = torch.randint(0, limit - s, (b, 1), generator=g, device=DEV)
        st["positions"] = (first + torch.arange(s, device=DEV)).to(torch.int32)
        if kind == "qk_grad":
            st["dq"] = normal(b, s, hq, d, dtype=dtype)
            st["dk"] = normal(b, s, hkv, d, dtype=dtype)
        return st
    n, vocab, width = case["n"], case["vocab"], case["width"]
    # token frequencies fall as 1 / rank, ranks dealt over the vocabulary
    rank = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    rank = (torch.exp(rank * math.log(vocab + 1)) - 1).long().clamp_(0, vocab - 1)
    deal = torch.randperm(vocab, generator=g, device=DEV)
    st = {"kind": kind, "tokens": deal[rank], "vocab": vocab, "scale": math.sqrt(width),
          "table_dtype": getattr(torch, case["table"]), "out_dtype": getattr(torch, case["out"])}
    if kind == "embed":
        st["table"] = normal(vocab, width, dtype=st["table_dtype"], std=0.02)
    else:
        st["dout"] = normal(n, width, dtype=st["out_dtype"])
    return st


# ---------------------------------------------------------------- the plain forms

def _visible(st, b, sq, sk):
    """Truth values (b, sq, sk): which keys each query sees."""
    j = torch.arange(sk, device=DEV)
    starts = st["starts"].long() if st["starts"] is not None else torch.full((b,), sk - sq, device=DEV)
    i = starts[:, None] + torch.arange(sq, device=DEV)
    dist = i[:, :, None] - j
    if st["causal"]:
        vis = dist >= 0
    else:
        vis = torch.ones_like(dist, dtype=torch.bool)
    if st["window"]:
        vis = vis & (dist < st["window"]) & (dist > -st["window"])
    if st["prefix"] is not None:
        vis = vis | (j < st["prefix"][:, None])[:, None, :]
    if st["documents"] is not None:
        mine = torch.gather(st["documents"], 1, i.clamp(0, sk - 1))
        vis = vis & (mine[:, :, None] == st["documents"][:, None, :])
    if st["lengths"] is not None:
        n = st["lengths"].long()[:, None]
        vis = vis & (i < n)[:, :, None] & (j < n)[:, None, :]
    return vis, dist


def _plain_attention(st):
    q, k, v = st["q"], st["k"], st["v"]
    b, sq, hq, d = q.shape
    sk, hkv = k.shape[1], k.shape[2]
    grp = hq // hkv
    vis, dist = _visible(st, b, sq, sk)
    # heads that share a key head are rows of one product
    qg = q.float().reshape(b, sq, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, grp * sq, d)
    kg = k.float().permute(0, 2, 1, 3).contiguous()
    vg = v.float().permute(0, 2, 1, 3).contiguous()
    s = torch.matmul(qg, kg.transpose(-1, -2).contiguous()).view(b, hkv, grp, sq, sk) * st["scale"]
    slope = 1.0
    if st["softcap"]:
        t = torch.tanh(s / st["softcap"])
        s = st["softcap"] * t
        slope = 1.0 - t * t
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, hkv, grp, 1, 1) * dist.abs().float()[:, None, None]
    s = s.masked_fill(~vis[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))
    p = p / torch.where(total > 0, total, torch.ones_like(total))

    def back(x, h):  # (b, hkv, h * s, d) -> (b, s, heads, d)
        return x.view(b, hkv, h, -1, d).permute(0, 3, 1, 2, 4).reshape(b, -1, hkv * h, d).to(torch.bfloat16)

    rows = p.view(b, hkv, grp * sq, sk)
    o = torch.matmul(rows, vg)
    out = {"out": back(o, grp), "lse": lse.reshape(b, hq, sq)}
    if st["kind"] == "forward":
        return out
    do = st["dout"].float().reshape(b, sq, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, grp * sq, d)
    dv = torch.matmul(rows.transpose(-1, -2).contiguous(), do)
    dp = torch.matmul(do, vg.transpose(-1, -2).contiguous()).view(b, hkv, grp, sq, sk)
    delta = (do * o).sum(-1).view(b, hkv, grp, sq, 1)
    ds = (p * (dp - delta) * slope * st["scale"]).view(b, hkv, grp * sq, sk)
    dq = torch.matmul(ds, kg)
    dk = torch.matmul(ds.transpose(-1, -2).contiguous(), qg)
    return {**out, "dq": back(dq, grp), "dk": back(dk, 1), "dv": back(dv, 1)}


def _cos_sin(st):
    cs = st["table"][st["positions"].long()][:, :, None]
    return cs[..., 0], cs[..., 1]


def _plain_qk_one(x, w, cos, sin, eps):
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w
    a, b = y.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(x.dtype)


def _plain_qk_grad_one(dz, x, w, cos, sin, eps):
    a, b = dz.float().chunk(2, -1)
    dy = torch.cat([a * cos + b * sin, b * cos - a * sin], -1)
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    unit = x * r
    dw = (dy * unit).sum((0, 1, 2)) if w is not None else None
    dy = dy * w if w is not None else dy
    dx = r * (dy - unit * (dy * unit).mean(-1, keepdim=True))
    return dx.to(dz.dtype), dw


def _named(**kw):
    return {n: t for n, t in kw.items() if t is not None}


def run(st):
    kind = st["kind"]
    if own:
        from newton_schulz_09_amd import lm
        if kind in ("forward", "train"):
            mask = {n: st[n] for n in ("scale", "causal", "window", "softcap", "slopes", "documents", "prefix",
                                       "lengths", "starts")}
            out, lse = lm.attention(st["q"], st["k"], st["v"], **mask)
            if kind == "forward":
                return {"out": out, "lse": lse}
            dq, dk, dv = lm.attention_backward(st["dout"], st["q"], st["k"], st["v"], out, lse, **mask)
            return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
        if kind == "qk":
            q, k = lm.qk_norm_rope(st["q"], st["k"], st["table"], positions=st["positions"], q_weight=st["qw"],
                                   k_weight=st["kw"], eps=st["eps"])
            return {"q": q, "k": k}
        if kind == "qk_grad":
            dq, dk, dqw, dkw = lm.qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], st["table"],
                                                        positions=st["positions"], q_weight=st["qw"],
                                                        k_weight=st["kw"], eps=st["eps"])
            return _named(dq=dq, dk=dk, dqw=dqw, dkw=dkw)
        if kind == "embed":
            return lm.embedding(st["tokens"], st["table"], scale=st["scale"], dtype=st["out_dtype"])
        return lm.embedding_backward(st["dout"], st["tokens"], st["vocab"], scale=st["scale"],
                                     dtype=st["table_dtype"])
    if kind in ("forward", "train"):
        return _plain_attention(st)
    if kind == "qk":
        cos, sin = _cos_sin(st)
        return {"q": _plain_qk_one(st["q"], st["qw"], cos, sin, st["eps"]),
                "k": _plain_qk_one(st["k"], st["kw"], cos, sin, st["eps"])}
    if kind == "qk_grad":
        cos, sin = _cos_sin(st)
        dq, dqw = _plain_qk_grad_one(st["dq"], st["q"], st["qw"], cos, sin, st["eps"])
        dk, dkw = _plain_qk_grad_one(st["dk"], st["k"], st["kw"], cos, sin, st["eps"])
        return _named(dq=dq, dk=dk, dqw=dqw, dkw=dkw)
    if kind == "embed":
        return (st["table"][st["tokens"]].float() * st["scale"]).to(st["out_dtype"])
    grad = torch.zeros(st["vocab"], st["dout"].shape[1], dtype=torch.float32, device=DEV)
    grad.index_add_(0, st["tokens"], st["dout"].float())
    return (grad * st["scale"]).to(st["table_dtype"])


# ---------------------------------------------------------------- work

def _pairs(case):
    """Query-key pairs that the masks leave, for one head (lengths and documents as seed 0 lays them out)."""
    lengths, starts, docs, prefix = _layout(case, 0)
    b, sq, sk, w = case["b"], case["sq"], case["sk"], case["window"]
    total = 0
    for n in range(b):
        end = lengths[n] if lengths else sk
        first = starts[n] if starts else sk - sq
        pre = prefix[n] if prefix else 0
        bounds = {}
        if docs:
            for j, x in enumerate(docs[n][:end]):
                bounds.setdefault(x, [j, j])[1] = j
        for i in range(max(0, first), min(end, first + sq)):
            lo, hi = (bounds[docs[n][i]][0], bounds[docs[n][i]][1] + 1) if docs else (0, end)
            a = max(lo, i - w + 1) if w else lo
            z = min(hi, i + 1) if case["causal"] else (min(hi, i + w) if w else hi)
            seen = max(0, z - a)
            p = min(pre, hi)
            if p > lo:  # the prefix keys below the span, and those above it
                seen += max(0, min(p, a) - lo) + max(0, p - max(z, lo))
            total += seen
    return total


def work(case):
    kind = case["kind"]
    size = {"float32": 4, "bfloat16": 2}
    if kind in ("forward", "train"):
        b, sq, sk, hq, hkv, d = (case[n] for n in ("b", "sq", "sk", "hq", "hkv", "d"))
        pairs = _pairs(case) * hq
        lengths = _layout(case, 0)[0]
        keys = sum(lengths) if lengths else b * sk
        q_bytes, kv_bytes, lse = 2 * b * sq * hq * d, 2 * keys * hkv * d, 4 * b * hq * sq
        if kind == "forward":
            return {"bytes": 2 * q_bytes + 2 * kv_bytes + lse, "flops": 4.0 * d * pairs}
        return {"bytes": 4 * q_bytes + 4 * kv_bytes + lse, "flops": 14.0 * d * pairs}
    if kind in ("qk", "qk_grad"):
        n = case["b"] * case["s"] * (case["hq"] + case["hkv"]) * case["d"]
        reads = 1 if kind == "qk" else 2
        # the table's row of each position, once
        table = min(case["b"] * case["s"], 32768) * case["d"] * 4
        return {"bytes": (reads + 1) * n * size[case["dtype"]] + table, "flops": (8 if kind == "qk" else 20) * n}
    n, width = case["n"], case["width"]
    # rows of the table that n tokens of these frequencies touch, on average
    share = 1.0 / torch.arange(1, case["vocab"] + 1, dtype=torch.float64) / math.log(case["vocab"] + 1)
    distinct = float((1.0 - (1.0 - share.clamp(max=1.0)) ** n).sum())
    if kind == "embed":
        return {"bytes": 8 * n + n * width * size[case["out"]] + distinct * width * size[case["table"]],
                "flops": n * width}
    return {"bytes": 8 * n + n * width * size[case["out"]] + case["vocab"] * width * size[case["table"]],
            "flops": 2 * n * width}


# ---------------------------------------------------------------- the definition in float64

def _exact_attention(case, st):
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    b, sq, hq, d = q.shape
    sk, hkv = k.shape[1:3]
    cap, scale = st["softcap"], st["scale"]
    train = st["kind"] == "train"
    out = torch.zeros(b, sq, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((b, hq, sq), -math.inf, dtype=torch.float64, device=DEV)
    grads = [torch.zeros_like(t) for t in (q, k, v)] if train else []
    do = st["dout"].double() if train else None
    key = torch.arange(sk, device=DEV)[None, :]
    for n in range(b):
        end = int(st["lengths"][n]) if st["lengths"] is not None else sk
        first = int(st["starts"][n]) if st["starts"] is not None else sk - sq
        pos = (first + torch.arange(sq, device=DEV))[:, None]
        hidden = (key > pos) if case["causal"] else torch.zeros(sq, sk, dtype=torch.bool, device=DEV)
        if case["window"]:
            hidden = hidden | ((pos - key).abs() >= case["window"])
        if st["prefix"] is not None:
            hidden = hidden & (key >= int(st["prefix"][n]))
        if st["documents"] is not None:
            doc = st["documents"][n]
            hidden = hidden | (doc[pos.clamp(0, sk - 1)] != doc[None, :])
        hidden = hidden | (key >= end) | (pos >= end)
        some = ~hidden.all(1)
        for h in range(hq):
            u = h // (hq // hkv)
            z = q[n, :, h] @ k[n, :, u].t() * scale
            th = None
            if cap:
                th = torch.tanh(z / cap)
                z = cap * th
            if st["slopes"] is not None:
                z = z - st["slopes"][h].double() * (pos - key).abs()
            z = z.masked_fill(hidden, -math.inf)
            lse[n, h] = torch.logsumexp(z, 1)
            w = torch.softmax(z, 1)
            w[~some] = 0.0
            o = w @ v[n, :, u]
            out[n, :, h] = o
            if train:
                g = do[n, :, h]
                grads[2][n, :, u] += w.t() @ g
                dz = w * (g @ v[n, :, u].t() - (g * o).sum(1, keepdim=True))
                if cap:
                    dz = dz * (1.0 - th.square())
                grads[0][n, :, h] = scale * (dz @ k[n, :, u])
                grads[1][n, :, u] += scale * (dz.t() @ q[n, :, h])
    res = {"out": out, "lse": lse}
    if train:
        res.update(dq=grads[0], dk=grads[1], dv=grads[2])
    return res


def _exact_qk(st):
    half = st["q"].shape[-1] // 2
    turn = torch.view_as_complex(st["table"].double().contiguous())[st["positions"].long()][:, :, None, :]

    def one(x, w):
        x = x.double()
        y = x / (x.square().mean(-1, keepdim=True) + st["eps"]).sqrt()
        y = y if w is None else y * w.double()
        z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)

    if st["kind"] == "qk":
        return {"q": one(st["q"], st["qw"]), "k": one(st["k"], st["kw"])}
    res = {}
    for name, x, dz, w, dname in (("dq", st["q"], st["dq"], st["qw"], "dqw"), ("dk", st["k"], st["dk"], st["kw"], "dkw")):
        x, dz = x.double(), dz.double()
        t = torch.complex(dz[..., :half].contiguous(), dz[..., half:].contiguous()) * turn.conj()
        t = torch.cat([t.real, t.imag], -1)
        norm = (x.square().mean(-1, keepdim=True) + st["eps"]).sqrt()
        if w is not None:
            res[dname] = (t * x / norm).sum((0, 1, 2))
            t = t * w.double()
        res[name] = t / norm - x * (t * x).sum(-1, keepdim=True) / (x.shape[-1] * norm ** 3)
    return res


def exact(case, seed):
    st = prepare(case, seed)
    kind = st["kind"]
    if kind in ("forward", "train"):
        return _exact_attention(case, st)
    if kind in ("qk", "qk_grad"):
        return _exact_qk(st)
    if kind == "embed":
        return st["scale"] * st["table"].double().index_select(0, st["tokens"])
    grad = torch.zeros(st["vocab"], st["dout"].shape[1], dtype=torch.float64, device=DEV)
    return grad.index_add_(0, st["tokens"], st["dout"].double()).mul_(st["scale"])
