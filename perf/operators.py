"""Cases of the encoder operators: attention over packed documents, rotary positions, and
the global gradient norm with clipping.

Each case is one call (or one forward and backward) as a retriever's program makes it:
encoding a query, encoding passages or pages for the index, a training step over them, and
the clipping of an encoder's gradients. `run` makes it with plain torch operations in
32 bits, or, where `own` is true, with this package's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- the cases
def _att(name, docs, lo, hi, heads, kv, dim, dtype, mask="all", prefix=0, cap=0.0, bias=False,
         train=False, fixed=False):
    """docs documents of lo..hi tokens each (drawn from the seed). mask: "all" (every token of
    the document), "causal" or "prefix" (the first `prefix` tokens, and the ones before).
    fixed: rows padded to hi tokens with per-document lengths, else packed with offsets."""
    c = {"op": "attention", "docs": docs, "lo": lo, "hi": hi, "heads": heads, "kv": kv,
         "dim": dim, "dtype": dtype, "mask": mask, "prefix": prefix, "cap": cap, "bias": bias,
         "train": train, "fixed": fixed}
    return dict(c, name=name) if name else c


def _rot(name, docs, lo, hi, heads, dim, rot, dtype, layout, factor=1.0, train=False,
         given=False):
    """Rotation of the first `rot` entries of each head; factor > 1 stretches the positions for
    long texts; given: positions are an input, else the token's index in its document."""
    c = {"op": "rotary", "docs": docs, "lo": lo, "hi": hi, "heads": heads, "dim": dim,
         "rot": rot, "dtype": dtype, "layout": layout, "factor": factor, "train": train,
         "given": given}
    return dict(c, name=name) if name else c


def _clip(name, layers, hidden, inner, vocab, dtype, max_norm):
    """Gradients of `layers` encoder layers, a token table and a 128-wide projection."""
    c = {"op": "clip", "layers": layers, "hidden": hidden, "inner": inner, "vocab": vocab,
         "dtype": dtype, "max_norm": max_norm}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one query of 32 tokens being encoded while a user waits: latency
        _att("attention query", 1, 32, 32, 12, 12, 64, "bf16"),
        # passages of ragged length encoded for the index
        _att("attention passages", 1024, 20, 300, 12, 12, 64, "bf16"),
        # page images as patches with a short text after them: prefix mask, tanh cap, one
        # shared key and value head, wide heads
        _att("attention pages", 48, 1030, 1061, 8, 1, 256, "bf16", "prefix", 1024, 50.0),
        # whole long documents with a causal encoder, shared heads and a distance bias
        _att("attention long", 2, 5003, 8191, 32, 8, 128, "fp16", "causal", bias=True),
        # a padded batch of short texts in full precision with a symmetric distance bias;
        # some rows have no token at all
        _att("train padded fp32", 48, 0, 77, 8, 8, 96, "fp32", bias=True, train=True,
             fixed=True),
        # a contrastive training step's passages
        _att("train passages", 512, 20, 300, 12, 12, 64, "bf16", train=True),
        # a training step over pages, shared heads, prefix mask and cap
        _att("train pages", 16, 1030, 1061, 16, 4, 128, "bf16", "prefix", 1024, 30.0,
             train=True),
        # queries' and keys' heads of one query
        _rot("rotary query", 1, 32, 32, 24, 64, 64, "bf16", "half"),
        # long texts with stretched positions, 32 query and 8 key heads in one call
        _rot("rotary long", 2, 20011, 32768, 40, 128, 128, "fp16", "half", 4.0),
        # training, part of the head, interleaved pairs, positions given
        _rot("rotary train fp32", 200, 20, 300, 16, 96, 32, "fp32", "interleaved", train=True,
             given=True),
        # only the projection after a frozen encoder is trained: latency
        _clip("clip projection", 0, 768, 0, 0, "fp32", 1.0),
        # a whole encoder: weights in bf16, norms and biases in fp32
        _clip("clip encoder", 12, 768, 2048, 30522, "bf16", 1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "train", "rotary", "clip"])
    if kind in ("attention", "train"):
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        dim = rng.choice([32, 64, 72, 96, 128, 256] if dtype != "fp32" else [32, 64, 80, 128])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4])
        hi = _log(rng, 16, 4096)
        lo = rng.choice([0, 1, hi // 8, hi // 2, hi])
        mask = rng.choice(["all", "all", "causal", "prefix"])
        # about as much as the listed training cases at most, and scores that fit the card in
        # plain form
        room = (1.5e9 if kind == "train" else 3e9) / (2 if dtype == "fp32" else 1)
        docs = max(1, min(_log(rng, 1, 600), int(room / (hi * hi * heads)),
                          int(1.5e8 / (hi * heads * dim))))
        return _att(None, docs, lo, hi, heads, kv, dim, dtype, mask,
                    rng.randrange(0, hi + 1) if mask == "prefix" else 0,
                    rng.choice([0.0, 0.0, 20.0, 50.0]), rng.random() < 0.3, kind == "train",
                    rng.random() < 0.3)
    if kind == "rotary":
        dim = rng.choice([32, 64, 96, 128, 256])
        rot = rng.choice([dim, dim, dim // 2, 16])
        heads = rng.choice([1, 5, 12, 16, 40])
        hi = _log(rng, 8, 32768)
        docs = max(1, min(_log(rng, 1, 500), int(2.5e8 / (hi * heads * dim))))
        return _rot(None, docs, rng.choice([1, hi // 4 + 1, hi]), hi, heads, dim, rot,
                    rng.choice(["bf16", "fp16", "fp32"]), rng.choice(["half", "interleaved"]),
                    rng.choice([1.0, 2.0, 8.0]), rng.random() < 0.4, rng.random() < 0.4)
    hidden = rng.choice([256, 320, 384, 512, 768, 896])
    return _clip(None, rng.randrange(0, 13), hidden, hidden * 2 + rng.randrange(0, 999),
                 rng.choice([0, 8001, 30522]), rng.choice(["bf16", "fp16", "fp32"]),
                 rng.choice([0.1, 1.0, 1e6]))


# ---------------------------------------------------------------- inputs
def _lengths(case, seed):
    """Token counts of the documents; they are the case's own (the same for every seed), so that
    passes over different inputs are equal work. The first is the longest and the second the
    shortest."""
    g = torch.Generator().manual_seed(77)
    n = torch.randint(case["lo"], case["hi"] + 1, (case["docs"],), generator=g)
    n[0] = case["hi"]
    if case["docs"] > 1:
        n[1] = case["lo"]
    if case["docs"] > 2 and case["docs"] < 2000:
        n = n[torch.randperm(case["docs"], generator=g)]
    return n


def _normal(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _prepare_attention(case, seed, g):
    n = _lengths(case, seed)
    dt, dim = TYPES[case["dtype"]], case["dim"]
    rows = (case["docs"], case["hi"]) if case["fixed"] else (int(n.sum()),)
    # queries, keys and values are views of one projection's output, as an encoder has them
    heads, kv = case["heads"], case["kv"]
    qkv = _normal(g, *rows, heads + 2 * kv, dim, dtype=dt)
    q, k, v = qkv.split([heads, kv, kv], dim=-2)
    if case["train"]:
        q, k, v = (x.detach().requires_grad_(True) for x in (q, k, v))
    off = torch.zeros(case["docs"] + 1, dtype=torch.int64)
    off[1:] = torch.cumsum(n, 0)
    return {
        "op": "attention", "q": q, "k": k, "v": v,
        "off": None if case["fixed"] else off.cuda(),
        "lens": n.to(torch.int32).cuda() if case["fixed"] else None,
        "most": int(n.max()),  # the longest document, known to whoever packed them
        "causal": case["mask"] != "all",
        "prefix": (torch.full((case["docs"],), case["prefix"], dtype=torch.int32,
                              device="cuda") if case["mask"] == "prefix" else None),
        "cap": case["cap"],
        "slopes": (torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)],
                                device="cuda") if case["bias"] else None),
        "scale": dim ** -0.5,
        "do": _normal(g, *rows, heads, dim, dtype=dt, std=0.01) if case["train"] else None,
    }


def _prepare_rotary(case, seed, g):
    n = _lengths(case, seed)
    total = int(n.sum())
    off = torch.zeros(case["docs"] + 1, dtype=torch.int64)
    off[1:] = torch.cumsum(n, 0)
    half = case["rot"] // 2
    # the table that a program makes once for its model; a stretched text divides it
    freq = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half) / case["factor"])
    pos = None
    if case["given"]:
        pos = torch.randint(0, 100000, (total,), generator=g, device="cuda", dtype=torch.int32)
    x = _normal(g, total, case["heads"], case["dim"], dtype=TYPES[case["dtype"]])
    return {
        "op": "rotary", "x": x.requires_grad_(case["train"]), "off": off.cuda(), "pos": pos,
        "freq": freq.float().cuda(), "layout": case["layout"],
        "mscale": 0.1 * math.log(case["factor"]) + 1.0,
        "dy": (_normal(g, total, case["heads"], case["dim"], dtype=TYPES[case["dtype"]])
               if case["train"] else None),
    }


def _shapes(case):
    """(shape, is it a matrix) of every gradient."""
    h, i = case["hidden"], case["inner"]
    layer = [((3 * h, h), True), ((h, h), True), ((i, h), True), ((h, i), True),
             ((h,), False), ((h,), False), ((i,), False), ((h,), False)]
    top = [((128, h), True), ((128,), False)]
    return layer * case["layers"] + ([((case["vocab"], h), True)] if case["vocab"] else []) + top


def _views(shapes, dtypes, flats):
    """The tensors of `shapes`, one after the other in the flat buffer of their type."""
    at = {d: 0 for d in flats}
    got = []
    for s, d in zip(shapes, dtypes):
        n = math.prod(s)
        got.append(flats[d][at[d]:at[d] + n].view(s))
        at[d] += n
    return got


def _prepare_clip(case, seed, g):
    shapes = [s for s, _ in _shapes(case)]
    low = TYPES[case["dtype"]]
    dtypes = [low if wide else torch.float32 for _, wide in _shapes(case)]
    sizes = {}
    for s, d in zip(shapes, dtypes):
        sizes[d] = sizes.get(d, 0) + math.prod(s)
    flats = {d: _normal(g, n, dtype=d, std=1e-3) for d, n in sizes.items()}
    outs = {d: torch.empty_like(f) for d, f in flats.items()}
    return {"op": "clip", "grads": _views(shapes, dtypes, flats),
            "outs": _views(shapes, dtypes, outs), "flat": list(outs.values()),
            "max_norm": case["max_norm"]}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"attention": _prepare_attention, "rotary": _prepare_rotary,
            "clip": _prepare_clip}[case["op"]](case, seed, g)


# ---------------------------------------------------------------- plain forms
def _tokens(s, total):
    """(document, index in it) of every packed token."""
    t = torch.arange(total, device="cuda")
    doc = torch.searchsorted(s["off"], t, right=True) - 1
    return doc, t - s["off"][doc]


def _pad(x, at, docs, most):
    """Packed rows [T, H, d] as [docs, H, most, d] in 32 bits, zeros where there is no token."""
    p = torch.zeros(docs * most, *x.shape[1:], device="cuda")
    p[at] = x.float()
    return p.view(docs, most, *x.shape[1:]).transpose(1, 2).contiguous()


def _plain_scores(s, q, k, lens, most, group):
    """Masked scores, and the factor of the cap's slope where there is one."""
    x = torch.matmul(q, k.repeat_interleave(group, 1).transpose(2, 3).contiguous()) * s["scale"]
    slope = None
    if s["cap"]:
        t = torch.tanh(x / s["cap"])
        x, slope = t * s["cap"], 1 - t * t
    i = torch.arange(most, device="cuda")
    if s["slopes"] is not None:
        far = (i[:, None] - i[None, :]).abs().float()
        x = x - s["slopes"].view(1, -1, 1, 1) * far
    seen = (i[None, :] < lens[:, None])[:, None, None, :]
    if s["causal"]:
        near = (i[None, :] <= i[:, None])[None, None]
        if s["prefix"] is not None:
            near = near | (i[None, :] < s["prefix"][:, None])[:, None, None, :]
        seen = seen & near
    return x.masked_fill(~seen, -math.inf), slope


def _plain_attention(s):
    q, k, v = (s[n].detach() for n in "qkv")
    group = q.shape[-2] // k.shape[-2]
    if s["lens"] is not None:
        docs, most = q.shape[:2]
        lens = s["lens"]
        qp, kp, vp = (x.float().transpose(1, 2).contiguous() for x in (q, k, v))
    else:
        docs, most = s["off"].numel() - 1, s["most"]
        lens = s["off"].diff()
        doc, idx = _tokens(s, q.shape[0])
        at = doc * most + idx
        qp, kp, vp = (_pad(x, at, docs, most) for x in (q, k, v))
    real = (torch.arange(most, device="cuda")[None, :] < lens[:, None])[:, None, :, None]
    x, slope = _plain_scores(s, qp, kp, lens, most, group)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    p = p / total.clamp_min(1e-37) * real
    o = torch.matmul(p, vp.repeat_interleave(group, 1))
    lse = (m + torch.log(total)).masked_fill(~real, -math.inf)[..., 0]

    def back(y, heads):  # [docs, H, most, d] to the inputs' layout
        y = y.transpose(1, 2).to(q.dtype)
        return y if s["lens"] is not None else y.reshape(docs * most, heads, -1)[at]

    if s["lens"] is None:
        lse = lse.transpose(1, 2).reshape(docs * most, -1)[at].t()
    else:
        lse = lse.transpose(0, 1).reshape(q.shape[2], -1)
    heads, kv = q.shape[-2], k.shape[-2]
    if s["do"] is None:
        return [back(o, heads), lse]
    g = (s["do"].float().transpose(1, 2).contiguous() if s["lens"] is not None
         else _pad(s["do"], at, docs, most)) * real
    dv = torch.matmul(p.transpose(2, 3).contiguous(), g)
    dp = torch.matmul(g, vp.repeat_interleave(group, 1).transpose(2, 3).contiguous())
    ds = p * (dp - (g * o).sum(-1, keepdim=True)) * s["scale"]
    if slope is not None:
        ds = ds * slope
    dq = torch.matmul(ds, kp.repeat_interleave(group, 1))
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), qp)
    dk, dv = (t.view(docs, kv, group, most, -1).sum(2) for t in (dk, dv))
    return [back(o, heads), back(dq, heads), back(dk, kv), back(dv, kv)]


def _plain_turn(x, cos, sin, layout, mscale):
    """The first 2 * cos.shape[-1] entries of each head turned, the others as they are."""
    half = cos.shape[-1]
    y = x.float()
    part, rest = y[..., :2 * half], y[..., 2 * half:]
    if layout == "half":
        a, b = part[..., :half], part[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned * mscale, rest], -1).to(x.dtype)


def _plain_rotary(s):
    x = s["x"].detach()
    pos = s["pos"] if s["pos"] is not None else _tokens(s, x.shape[0])[1]
    # 64 bits: at position 30000 an angle in 32 bits is off by 1e-3
    angle = pos.double()[:, None] * s["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    y = _plain_turn(x, cos, sin, s["layout"], s["mscale"])
    if s["dy"] is None:
        return [y]
    return [y, _plain_turn(s["dy"], cos, -sin, s["layout"], s["mscale"])]


def _plain_clip(s):
    # squares of small values are summed per tensor in 64 bits
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    c = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    [o.copy_(g.float() * c) for g, o in zip(s["grads"], s["outs"])]
    return s["flat"] + [norm.float()]


# ---------------------------------------------------------------- one pass
def _own_attention(s):
    import maxsim_scoring_fwd_amd as ms
    kw = dict(doc_offsets=s["off"], doc_lens=s["lens"], causal=s["causal"],
              prefix_lens=s["prefix"], softcap=s["cap"], slopes=s["slopes"], scale=s["scale"])
    if s["do"] is None:
        return list(ms.maxsim_attention(s["q"], s["k"], s["v"], **kw))
    o = ms.attention(s["q"], s["k"], s["v"], **kw)
    return [o.detach(), *torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["do"])]


def _own_rotary(s):
    import maxsim_scoring_fwd_amd as ms
    kw = dict(doc_offsets=s["off"] if s["pos"] is None else None, positions=s["pos"],
              layout=s["layout"], mscale=s["mscale"])
    if s["dy"] is None:
        return [ms.maxsim_rotary(s["x"], s["freq"], **kw)]
    y = ms.rotary(s["x"], s["freq"], **kw)
    return [y.detach(), *torch.autograd.grad(y, s["x"], s["dy"])]


def _own_clip(s):
    import maxsim_scoring_fwd_amd as ms
    norm = ms.maxsim_clip_grad_norm(s["grads"], s["max_norm"], out=s["outs"])
    return s["flat"] + [norm]


def run(state):
    op = state["op"]
    if own:
        return {"attention": _own_attention, "rotary": _own_rotary, "clip": _own_clip}[op](state)
    with torch.no_grad():
        return {"attention": _plain_attention, "rotary": _plain_rotary,
                "clip": _plain_clip}[op](state)


# ---------------------------------------------------------------- least work
def work(case):
    if case["op"] == "clip":
        low = BYTES[case["dtype"]]
        nbytes = sum(math.prod(s) * (low if wide else 4) for s, wide in _shapes(case))
        count = sum(math.prod(s) for s, _ in _shapes(case))
        return {"bytes": 2 * nbytes, "flops": 3 * count}
    n = _lengths(case, 0)
    rows = case["docs"] * case["hi"] if case.get("fixed") else int(n.sum())
    size = BYTES[case["dtype"]]
    if case["op"] == "rotary":
        x = rows * case["heads"] * case["dim"]
        turns = 2 if case["train"] else 1
        return {"bytes": 2 * x * size * turns,
                "flops": 3 * rows * case["heads"] * case["rot"] * turns}
    n = n.double()
    pairs = n * n
    if case["mask"] != "all":
        free = torch.clamp(n, max=case["prefix"])  # rows and keys of the prefix see each other
        pairs = free * free + (n - free) * free + (n - free) * (n - free + 1) / 2
    pairs = float(pairs.sum()) * case["heads"]
    q = rows * case["heads"] * case["dim"] * size
    kv = 2 * rows * case["kv"] * case["dim"] * size
    lse = rows * case["heads"] * 4
    if not case["train"]:
        return {"bytes": 2 * q + kv + lse, "flops": 4 * case["dim"] * pairs}
    # the forward, then q, k, v, o, do in and dq, dk, dv out; four further products
    return {"bytes": 2 * q + kv + 4 * q + 2 * kv + 2 * lse, "flops": 14 * case["dim"] * pairs}


# ---------------------------------------------------------------- 64 bits
def _exact_attention(case, s):
    q, k, v = (s[n].detach() for n in "qkv")
    heads, kv = case["heads"], case["kv"]
    n = _lengths(case, 0).tolist()
    if case["fixed"]:
        starts = [b * case["hi"] for b in range(case["docs"])]
        flat = lambda x: x.reshape(-1, *x.shape[2:])  # noqa: E731
        q, k, v = flat(q), flat(k), flat(v)
        do = flat(s["do"]) if s["do"] is not None else None
    else:
        starts = [sum(n[:b]) for b in range(len(n))]
        do = s["do"]
    rows = q.shape[0]
    f64 = dict(dtype=torch.float64, device="cuda")
    o = torch.zeros(rows, heads, case["dim"], **f64)
    lse = torch.full((heads, rows), -math.inf, **f64)
    dq, dk, dv = torch.zeros_like(o), torch.zeros(k.shape, **f64), torch.zeros(k.shape, **f64)
    for b, (t0, len_b) in enumerate(zip(starts, n)):
        if not len_b:
            continue
        i = torch.arange(len_b, device="cuda")
        hide = torch.zeros(len_b, len_b, dtype=torch.bool, device="cuda")
        if case["mask"] != "all":
            hide = i[None, :] > i[:, None]
            if case["mask"] == "prefix":
                hide[:, :case["prefix"]] = False
        far = (i[:, None] - i[None, :]).abs().double()
        rows_b = slice(t0, t0 + len_b)
        per = max(1, int(2e8 // (len_b * len_b)))  # heads at a time
        for h0 in range(0, heads, per):
            hs = torch.arange(h0, min(heads, h0 + per), device="cuda")
            ks = hs // (heads // kv)
            qb, kb, vb = (x[rows_b].double().transpose(0, 1)
                          for x in (q[:, hs], k[:, ks], v[:, ks]))
            x = qb @ kb.transpose(1, 2) * case["dim"] ** -0.5
            y = case["cap"] * torch.tanh(x / case["cap"]) if case["cap"] else x
            if case["bias"]:
                y = y - s["slopes"].double()[hs][:, None, None] * far
            y = y.masked_fill(hide, -math.inf)
            z = torch.logsumexp(y, -1)
            w = torch.exp(y - z[..., None])
            ob = w @ vb
            o[rows_b, h0:h0 + per] = ob.transpose(0, 1)
            lse[h0:h0 + per, rows_b] = z
            if do is None:
                continue
            g = do[rows_b][:, hs].double().transpose(0, 1)
            dw = w * (g @ vb.transpose(1, 2) - (g * ob).sum(-1, keepdim=True))
            if case["cap"]:
                dw = dw * (1 - torch.tanh(x / case["cap"]) ** 2)
            dw = dw * case["dim"] ** -0.5
            dq[rows_b, h0:h0 + per] = (dw @ kb).transpose(0, 1)
            dk[rows_b].index_add_(1, ks, (dw.transpose(1, 2) @ qb).transpose(0, 1))
            dv[rows_b].index_add_(1, ks, (w.transpose(1, 2) @ g).transpose(0, 1))
    if do is None:
        return [o.view(s["q"].shape), lse]
    return [o.view(s["q"].shape), dq.view(s["q"].shape), dk.view(s["k"].shape),
            dv.view(s["k"].shape)]


def _exact_rotary(case, s):
    n = _lengths(case, 0)
    if s["pos"] is None:
        pos = torch.cat([torch.arange(int(m)) for m in n]).double().cuda()
    else:
        pos = s["pos"].double()
    angle = torch.outer(pos, s["freq"].double())
    turn = torch.polar(torch.full_like(angle, s["mscale"]), angle)[:, None, :]
    half = case["rot"] // 2

    def turned(x, by):
        y = x.detach().double().clone()
        if case["layout"] == "half":
            a, b = y[..., :half].clone(), y[..., half:2 * half].clone()
        else:
            a, b = y[..., 0:2 * half:2].clone(), y[..., 1:2 * half:2].clone()
        z = torch.complex(a, b) * by
        if case["layout"] == "half":
            y[..., :half], y[..., half:2 * half] = z.real, z.imag
        else:
            y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
        return y

    out = [turned(s["x"], turn)]
    return out if s["dy"] is None else out + [turned(s["dy"], turn.conj())]


def _exact_clip(case, s):
    squares = 0.0
    for g in s["grads"]:
        squares += float(torch.linalg.vector_norm(g.double())) ** 2
    norm = math.sqrt(squares)
    factor = min(1.0, case["max_norm"] / (norm + 1e-6))
    flat = {}
    for g in s["grads"]:
        flat.setdefault(g.dtype, []).append(g.double().flatten() * factor)
    parts = [torch.cat(flat[f.dtype]) for f in s["flat"]]
    return parts + [torch.tensor(norm, dtype=torch.float64)]


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"attention": _exact_attention, "rotary": _exact_rotary,
                "clip": _exact_clip}[case["op"]](case, s)
