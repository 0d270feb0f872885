"""Cases of further operators around the scoring: the encoder's norm with the residual's addition
(and its 8-bit output for the index), dropout, the cross entropy over a vocabulary with its
gradients, and 4-bit microscaled vectors with the scores of documents stored in them.

Each case is one call (or one forward and backward) as a retriever's program makes it: encoding
a query, encoding passages for the index, a training step of the encoder, searching an index of
4-bit vectors. `run` makes it with plain torch operations in 32 bits, or, where `own` is true,
with this package's entry points.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
LEFT_OUT = -100  # label of a token that is not trained on


# ---------------------------------------------------------------- the cases
def _norm(name, rows, d, dtype, wtype="fp32", residual=True, p=0.0, train=False, int8=False):
    """rows token vectors of d entries; weights in wtype; p: dropout before the addition."""
    c = {"op": "norm", "rows": rows, "d": d, "dtype": dtype, "wtype": wtype,
         "residual": residual, "p": p, "train": train, "int8": int8}
    return dict(c, name=name) if name else c


def _drop(name, rows, d, dtype, p, train=False):
    c = {"op": "dropout", "rows": rows, "d": d, "dtype": dtype, "p": p, "train": train}
    return dict(c, name=name) if name else c


def _loss(name, rows, vocab, d, dtype, share=1.0, scale=1.0, train=False):
    """share: the part of the rows that has a label, the others are left out."""
    c = {"op": "loss", "rows": rows, "vocab": vocab, "d": d, "dtype": dtype, "share": share,
         "scale": scale, "train": train}
    return dict(c, name=name) if name else c


def _quant(name, rows, d, dtype):
    c = {"op": "quantise", "rows": rows, "d": d, "dtype": dtype}
    return dict(c, name=name) if name else c


def _score(name, queries, docs, lo, hi, d, layout):
    """layout: "fixed" (documents of hi tokens), "lens" (padded to hi, lo..hi of them count) or
    "packed" (documents of lo..hi tokens, one after the other)."""
    c = {"op": "score", "queries": queries, "docs": docs, "lo": lo, "hi": hi, "d": d,
         "layout": layout}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a layer's norm for one query of 32 tokens while a user waits: latency
        _norm("norm query", 32, 768, "bf16"),
        # the projected vectors of packed passages on their way into an 8-bit index
        _norm("norm index 8 bits", 163877, 128, "bf16", residual=False, int8=True),
        # a layer's norm in a training step over packed passages, with dropout before the addition
        _norm("norm train", 81907, 768, "bf16", p=0.1, train=True),
        # dropout on the embeddings of a few short texts, an odd number of entries
        _drop("dropout texts", 101, 513, "fp16", 0.1),
        # dropout on the inner activations of a feed-forward layer in a training step
        _drop("dropout train", 81907, 2048, "bf16", 0.1, train=True),
        # how likely the tokens of one query are: latency, one read of the token table
        _loss("loss query", 32, 30522, 768, "bf16"),
        # a training step in which every token has a label
        _loss("loss train", 8192, 30522, 768, "bf16", train=True),
        # masked-token training: 15 in 100 tokens have a label, an odd vocabulary
        _loss("loss train masked", 20011, 50021, 512, "fp16", share=0.15, train=True),
        # the vectors of one query into 4 bits
        _quant("quantise query", 32, 128, "bf16"),
        # the vectors of a batch of passages into 4 bits, and back as the values stored
        _quant("quantise passages", 1638401, 128, "bf16"),
        # one query against a small collection of passages of ragged length
        _score("score packed", 32, 20000, 20, 300, 96, "packed"),
        # one query against a hundred thousand documents
        _score("score fixed", 32, 100000, 128, 128, 128, "fixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "dropout", "loss", "loss", "quantise", "score", "score"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if kind == "norm":
        d = rng.choice([_log(rng, 16, 4096), 64 * rng.randrange(1, 33), 128, 768])
        rows = max(1, min(_log(rng, 1, 200000), int(6e7 / d / BYTES[dtype] * 2)))
        residual, int8 = rng.random() < 0.7, rng.random() < 0.3
        train = not int8 and rng.random() < 0.6
        return _norm(None, rows, d, dtype, rng.choice(["fp32", dtype]), residual,
                     rng.choice([0.0, 0.1, 0.3]) if train and residual else 0.0, train, int8)
    if kind == "dropout":
        d = _log(rng, 8, 4096)
        rows = max(1, min(_log(rng, 1, 200000), int(1.6e8 / d / BYTES[dtype] * 2)))
        return _drop(None, rows, d, dtype, rng.choice([0.1, 0.25, 0.5]), rng.random() < 0.6)
    if kind == "loss":
        d = 8 * rng.randrange(4, 113)
        vocab = _log(rng, 500, 130000)
        train, share = rng.random() < 0.6, rng.choice([1.0, 1.0, 0.5, 0.15])
        room = 1.9e11 / (10 if dtype == "fp32" else 1)
        rows = max(1, min(_log(rng, 1, 32768), int(room / (d * vocab * share)),
                          int(1e9 / vocab)))
        return _loss(None, rows, vocab, d, dtype, share, rng.choice([1.0, 0.5, 5.0]), train)
    if kind == "quantise":
        d = 32 * rng.randrange(1, 33)
        return _quant(None, max(1, min(_log(rng, 1, 2000000), int(2e8 / d))), d, dtype)
    d = rng.choice([32, 64, 96, 128, 128, 256, 512])
    hi = _log(rng, 8, 1500)
    queries = rng.choice([1, 8, 17, 32, 33, 64, 200])
    docs = max(1, min(_log(rng, 10, 100000), int(1.6e9 / d / hi), int(4e8 / queries / hi)))
    return _score(None, queries, docs,
                  rng.choice([0, 1, hi // 4, hi // 2]), hi, d,
                  rng.choice(["fixed", "lens", "packed"]))


# ---------------------------------------------------------------- inputs
def _normal(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _rng_state(seed):
    """The generator's state as a program keeps it on the device: key and step."""
    return torch.tensor([0x9E3779B97F4A7C15 * (seed + 1) % (1 << 63), 1000 + seed],
                        dtype=torch.int64, device="cuda")


def _prepare_norm(case, seed, g):
    rows, d, dt = case["rows"], case["d"], TYPES[case["dtype"]]
    train = case["train"]
    x = _normal(g, rows, d, dtype=dt).requires_grad_(train)
    r = None
    if case["residual"]:
        r = _normal(g, rows, d, dtype=dt, std=2.0).requires_grad_(train)
    w = (1 + _normal(g, d, std=0.1)).to(TYPES[case["wtype"]]).requires_grad_(train)
    return {"op": "norm", "x": x, "r": r, "w": w, "p": case["p"], "rng": _rng_state(seed),
            "int8": case["int8"],
            "dy": _normal(g, rows, d, dtype=dt, std=0.01) if train else None,
            "dh": _normal(g, rows, d, dtype=dt, std=0.01) if train and r is not None else None}


def _prepare_dropout(case, seed, g):
    rows, d, dt = case["rows"], case["d"], TYPES[case["dtype"]]
    return {"op": "dropout", "x": _normal(g, rows, d, dtype=dt).requires_grad_(case["train"]),
            "p": case["p"], "rng": _rng_state(seed),
            "dy": _normal(g, rows, d, dtype=dt, std=0.01) if case["train"] else None}


def _labelled(case):
    """How many rows have a label: the case's own, the same for every seed."""
    return max(1, int(round(case["rows"] * case["share"])))


def _prepare_loss(case, seed, g):
    rows, vocab, d, dt = case["rows"], case["vocab"], case["d"], TYPES[case["dtype"]]
    h = _normal(g, rows, d, dtype=dt).requires_grad_(case["train"])
    w = _normal(g, vocab, d, dtype=dt, std=2.0 * d ** -0.5).requires_grad_(case["train"])
    labels = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    without = torch.randperm(rows, generator=g, device="cuda")[_labelled(case):]
    labels[without] = LEFT_OUT
    # the gradient of the mean over the rows that have a label
    dl = torch.full((rows,), 1.0 / _labelled(case), device="cuda")
    return {"op": "loss", "h": h, "w": w, "labels": labels, "scale": case["scale"],
            "dl": dl if case["train"] else None}


def _prepare_quantise(case, seed, g):
    # token vectors of unit length, as the projection leaves them
    x = _normal(g, case["rows"], case["d"])
    x = x / x.square().sum(-1, keepdim=True).sqrt()
    return {"op": "quantise", "x": x.to(TYPES[case["dtype"]])}


def _lengths(case):
    """Token counts of the documents; they are the case's own (the same for every seed)."""
    if case["layout"] == "fixed":
        return torch.full((case["docs"],), case["hi"])
    g = torch.Generator().manual_seed(77)
    n = torch.randint(case["lo"], case["hi"] + 1, (case["docs"],), generator=g)
    n[0] = case["hi"]
    if case["docs"] > 1:
        n[1] = case["lo"]
    return n


def _stored(g, rows, d):
    """(codes, scales) of `rows` unit vectors, as an index holds them: two entries a byte, the
    first in the low half, and one byte of exponent for 32 entries."""
    codes = torch.empty(rows, d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, d // 32, dtype=torch.uint8, device="cuda")
    step = 1 << 20
    for a in range(0, rows, step):
        x = _normal(g, min(step, rows - a), d)
        code, k = _plain_codes(x / x.square().sum(-1, keepdim=True).sqrt())
        codes[a:a + step] = code[:, 0::2] | code[:, 1::2] << 4
        scales[a:a + step] = k + 127
    return codes, scales


def _prepare_score(case, seed, g):
    n = _lengths(case)
    packed = case["layout"] == "packed"
    rows = int(n.sum()) if packed else case["docs"] * case["hi"]
    q, qs = _stored(g, case["queries"], case["d"])
    c, s = _stored(g, rows, case["d"])
    off = torch.zeros(case["docs"] + 1, dtype=torch.int64)
    off[1:] = torch.cumsum(n, 0)
    if not packed:
        c = c.view(case["docs"], case["hi"], -1)
        s = s.view(case["docs"], case["hi"], -1)
    return {"op": "score", "q": q, "qs": qs, "c": c, "s": s,
            "off": off.cuda() if packed else None,
            "lens": n.to(torch.int32).cuda() if case["layout"] == "lens" else None}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"norm": _prepare_norm, "dropout": _prepare_dropout, "loss": _prepare_loss,
            "quantise": _prepare_quantise, "score": _prepare_score}[case["op"]](case, seed, g)


# ---------------------------------------------------------------- plain forms
def _plain_words(rng, blocks, call=0):
    """Philox4x32 with 7 rounds: the four 32-bit words of blocks 0 .. blocks - 1, [blocks, 4]. The
    key is rng[0], the counter (block, block >> 32, rng[1], call)."""
    low = 0xFFFFFFFF
    at = torch.arange(blocks, device=rng.device)
    a, b = at & low, at >> 32
    c, d = torch.zeros_like(a) + (rng[1] & low), torch.full_like(a, call)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low

    def one(a, b, c, d, i):
        # products mod 2^64: their two 32-bit halves are right whatever the sign
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        return ((q >> 32) & low ^ b ^ (k0 + i * 0x9E3779B9) & low, q & low,
                (p >> 32) & low ^ d ^ (k1 + i * 0xBB67AE85) & low, p & low)
    a, b, c, d = one(a, b, c, d, 0)
    a, b, c, d = one(a, b, c, d, 1)
    a, b, c, d = one(a, b, c, d, 2)
    a, b, c, d = one(a, b, c, d, 3)
    a, b, c, d = one(a, b, c, d, 4)
    a, b, c, d = one(a, b, c, d, 5)
    a, b, c, d = one(a, b, c, d, 6)
    return torch.stack([a, b, c, d], 1)


def _plain_factor(rng, p, rows, d):
    """0 or 1 / (1 - p) for every entry [rows, d]: each has 16 bits of its own, 8 entries of a row a
    block; p counts in steps of 2^-16."""
    least = round(p * 65536)
    blocks = -(-d // 8)
    w = _plain_words(rng, rows * blocks)
    u = torch.stack([w & 0xFFFF, w >> 16], 2).view(rows, blocks * 8)[:, :d]
    return (u >= least).float() * (65536 / (65536 - least))


def _plain_norm(s):
    x, r, w = (t.detach() if t is not None else None for t in (s["x"], s["r"], s["w"]))
    keep = _plain_factor(s["rng"], s["p"], *x.shape) if s["p"] else None
    u = x.float() if keep is None else x.float() * keep
    u = u if r is None else u + r.float()
    h = u.to(x.dtype)  # what is handed on, and what the norm is of
    u = h.float()
    rstd = torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
    n = u * rstd
    y = n * w.float()
    if s["int8"]:
        scale = y.abs().amax(-1, keepdim=True) / 127
        code = torch.round(y / scale.clamp_min(1e-30))
        return [(code * scale).to(torch.bfloat16), scale[:, 0], h]
    if s["dy"] is None:
        return [y.to(x.dtype), h]
    dy = s["dy"].float()
    g = dy * w.float()
    dr = rstd * (g - n * (g * n).mean(-1, keepdim=True))
    dr = dr if s["dh"] is None else dr + s["dh"].float()
    dw = (dy * n).sum(0).to(w.dtype)
    dx = (dr if keep is None else dr * keep).to(x.dtype)
    return [y.to(x.dtype), h, dx] + ([] if r is None else [dr.to(x.dtype)]) + [dw]


def _plain_dropout(s):
    x = s["x"].detach()
    keep = _plain_factor(s["rng"], s["p"], 1, x.numel()).view(x.shape)
    y = (x.float() * keep).to(x.dtype)
    return [y] if s["dy"] is None else [y, (s["dy"].float() * keep).to(x.dtype)]


def _plain_loss(s):
    h, w, labels = s["h"].detach(), s["w"].detach(), s["labels"]
    rows = torch.nonzero((labels >= 0) & (labels < w.shape[0]))[:, 0]  # the others are left out
    hv, wf, lv = h[rows].float(), w.float(), labels[rows]
    z = torch.matmul(hv, wf.t()) * s["scale"]
    m = z.amax(-1, keepdim=True)
    lse = m + torch.exp(z - m).sum(-1, keepdim=True).log()
    loss = torch.zeros(h.shape[0], device=h.device)
    loss[rows] = (lse - z.gather(1, lv[:, None]))[:, 0]
    if s["dl"] is None:
        return [loss, torch.full_like(loss, -math.inf).index_copy(0, rows, lse[:, 0])]
    p = torch.exp(z - lse)
    p.scatter_add_(1, lv[:, None], torch.full_like(lse, -1.0))
    p = p * (s["dl"][rows, None] * s["scale"])
    dh = torch.zeros(h.shape, device=h.device)
    dh[rows] = torch.matmul(p, wf)
    dw = torch.matmul(p.t(), hv)
    return [loss, dh.to(h.dtype), dw.to(w.dtype)]


# what the 16 codes stand for, low three bits the magnitude, the fourth the sign
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _power(k):
    """2^k in 64 bits, for whole numbers: exact, which torch's exp2 is not everywhere."""
    return (k.long() + 1023 << 52).view(torch.float64)


def _plain_codes(x):
    """(4-bit codes [rows, d], exponents [rows, d / 32]) of x in 32 bits: 32 entries share a power
    of two, that of the largest over 4; entries go to the nearest, ties to the even code."""
    b = x.unflatten(-1, (-1, 32))
    _, e = torch.frexp(b.abs().amax(-1))  # 2^(e - 1) <= amax < 2^e
    k = torch.where(b.abs().amax(-1) > 0, (e - 3).clamp(-127, 127), -127)
    a = b.double().abs() * _power(-k)[..., None]
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5).byte())
    code = code | torch.signbit(b).byte() << 3
    return code.flatten(-2), k


def _plain_quantise(s):
    x = s["x"]
    code, k = _plain_codes(x.float())
    values = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=x.device)
    v = values[code.int()].unflatten(-1, (-1, 32)) * _power(k).float()[..., None]
    return [v.flatten(-2).to(x.dtype)]


def _plain_values(codes, scales):
    """Stored vectors in 32 bits."""
    values = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pairs = torch.stack([values.repeat(16), values.repeat_interleave(16)], 1)  # of a byte's halves
    v = pairs[codes.int()].flatten(-2).unflatten(-1, (-1, 32))
    return (v * _power(scales.int() - 127).float()[..., None]).flatten(-2)


def _plain_score(s):
    q, v = _plain_values(s["q"], s["qs"]), _plain_values(s["c"], s["s"])
    x = torch.matmul(v.view(-1, v.shape[-1]), q.t())  # [tokens, queries]
    if s["off"] is not None:
        docs = s["off"].numel() - 1
        doc = torch.searchsorted(s["off"], torch.arange(x.shape[0], device="cuda"), right=True) - 1
        m = torch.full((docs, x.shape[1]), -math.inf, device="cuda")
        m = m.scatter_reduce(0, doc[:, None].expand_as(x), x, "amax")
    else:
        docs, nd = s["c"].shape[:2]
        x = x.view(docs, nd, -1)
        if s["lens"] is not None:
            pad = torch.arange(nd, device="cuda")[None, :] >= s["lens"][:, None]
            x = x.masked_fill(pad[..., None], -math.inf)
        m = x.amax(1)
    return [m.sum(1)]


# ---------------------------------------------------------------- one pass
def _own_norm(s):
    import maxsim_scoring_fwd_amd as ms
    if s["int8"]:
        code, scale, h = ms.maxsim_rms_norm_i8(s["x"], s["w"], residual=s["r"], eps=EPS)
        v = torch.empty(code.shape, dtype=torch.bfloat16, device=code.device)
        return [torch.mul(code, scale[:, None], out=v), scale, h]
    kw = dict(residual=s["r"], eps=EPS, dropout=s["p"], rng=s["rng"] if s["p"] else None)
    if s["dy"] is None:
        return list(ms.maxsim_rms_norm(s["x"], s["w"], **kw)[:2])
    y, h = ms.rms_norm(s["x"], s["w"], **kw)
    if s["r"] is None:
        got = torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
    else:
        got = torch.autograd.grad((y, h), (s["x"], s["r"], s["w"]), (s["dy"], s["dh"]))
    return [y.detach(), h.detach(), *got]


def _own_dropout(s):
    import maxsim_scoring_fwd_amd as ms
    if s["dy"] is None:
        return [ms.maxsim_dropout(s["x"], s["p"], s["rng"])]
    y = ms.dropout(s["x"], s["p"], s["rng"])
    return [y.detach(), *torch.autograd.grad(y, s["x"], s["dy"])]


def _own_loss(s):
    import maxsim_scoring_fwd_amd as ms
    if s["dl"] is None:
        return list(ms.maxsim_linear_cross_entropy(s["h"], s["w"], s["labels"], scale=s["scale"]))
    loss = ms.linear_cross_entropy(s["h"], s["w"], s["labels"], scale=s["scale"])
    return [loss.detach(), *torch.autograd.grad(loss, (s["h"], s["w"]), s["dl"])]


def _own_quantise(s):
    import maxsim_scoring_fwd_amd as ms
    codes, scales = ms.maxsim_quantize_mx4(s["x"])
    return [ms.maxsim_dequantize_mx4(codes, scales, s["x"].dtype)]


def _own_score(s):
    import maxsim_scoring_fwd_amd as ms
    return [ms.maxsim_score_mx4(s["q"], s["qs"], s["c"], s["s"], doc_offsets=s["off"],
                                doc_lens=s["lens"])]


def run(state):
    op = state["op"]
    if own:
        return {"norm": _own_norm, "dropout": _own_dropout, "loss": _own_loss,
                "quantise": _own_quantise, "score": _own_score}[op](state)
    with torch.no_grad():
        return {"norm": _plain_norm, "dropout": _plain_dropout, "loss": _plain_loss,
                "quantise": _plain_quantise, "score": _plain_score}[op](state)


# ---------------------------------------------------------------- least work
def work(case):
    if case["op"] == "norm":
        n, size = case["rows"] * case["d"], BYTES[case["dtype"]]
        into = 2 if case["residual"] else 1
        if case["int8"]:
            return {"bytes": n * (size * into + 1 + (size if into == 2 else 0)) + 4 * case["rows"],
                    "flops": 6 * n}
        tensors = 2 * into  # x, residual; y, h
        if case["train"]:
            # the gradients of y and h come in, those of x and the residual go out
            tensors += 2 * into
        return {"bytes": tensors * n * size + 3 * case["d"] * BYTES[case["wtype"]],
                "flops": (14 if case["train"] else 4) * n}
    if case["op"] == "dropout":
        n = case["rows"] * case["d"] * (2 if case["train"] else 1)
        return {"bytes": 2 * n * BYTES[case["dtype"]], "flops": n}
    if case["op"] == "loss":
        m, size = _labelled(case), BYTES[case["dtype"]]
        h, w = case["rows"] * case["d"] * size, case["vocab"] * case["d"] * size
        products = m * case["vocab"] * case["d"] * 2
        if not case["train"]:
            return {"bytes": m * case["d"] * size + w + 12 * case["rows"], "flops": products}
        # logits once for the sums and once for the gradients, since they are not kept
        return {"bytes": 2 * (h + w) + 16 * case["rows"], "flops": 4 * products}
    if case["op"] == "quantise":
        n = case["rows"] * case["d"]
        # in, codes and scales out; and those in, values out
        return {"bytes": 2 * n * BYTES[case["dtype"]] + 2 * (n // 2 + n // 32), "flops": 4 * n}
    tokens = int(_lengths(case).sum())
    row = case["d"] // 2 + case["d"] // 32
    return {"bytes": (tokens + case["queries"]) * row + 12 * case["docs"],
            "flops": 2 * tokens * case["queries"] * case["d"]}


# ---------------------------------------------------------------- 64 bits
def _exact_factor(s, rows, d, p):
    """As _plain_factor, with unsigned integers on the host."""
    key, step = (int(v) for v in s["rng"].tolist())
    mask, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    nb = (d + 7) // 8
    n = np.arange(rows * nb, dtype=np.uint64)
    x = [n & mask, n >> sh, np.full_like(n, step & 0xFFFFFFFF), np.zeros_like(n)]
    k = [key & 0xFFFFFFFF, key >> 32 & 0xFFFFFFFF]
    for _ in range(7):
        m0, m1 = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [m1 >> sh ^ x[1] ^ np.uint64(k[0]), m1 & mask, m0 >> sh ^ x[3] ^ np.uint64(k[1]),
             m0 & mask]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    bits = np.stack(x, 1).astype(np.uint32).view(np.uint16)  # low half first
    least = round(p * 65536)
    keep = torch.from_numpy((bits.reshape(rows, nb * 8) >= least)[:, :d]).cuda()
    return keep.double() * 65536 / (65536 - least)


def _exact_norm(case, s):
    x, r, w = (None if t is None else t.detach().double() for t in (s["x"], s["r"], s["w"]))
    f = _exact_factor(s, case["rows"], case["d"], case["p"]) if case["p"] else 1.0
    h = x * f
    if r is not None:
        h += r
    h = h.to(s["x"].dtype).double()
    size = torch.sqrt((h * h).sum(1, keepdim=True) / case["d"] + EPS)
    hat = h / size
    if case["int8"]:
        big = torch.max(torch.abs(hat * w), 1, keepdim=True).values / 127
        code = torch.round(torch.where(big > 0, hat * w / big, torch.zeros_like(hat)))
        return [code * big, big[:, 0], h]
    if not case["train"]:
        return [hat * w, h]
    dy = s["dy"].double()
    dw = torch.einsum("nd,nd->d", dy, hat)
    dhat = dy * w
    dh = (dhat - hat * torch.einsum("nd,nd->n", dhat, hat)[:, None] / case["d"]) / size
    if s["dh"] is not None:
        dh += s["dh"].double()
    return [hat * w, h, dh * f] + ([dh] if r is not None else []) + [dw]


def _exact_dropout(case, s):
    f = _exact_factor(s, 1, case["rows"] * case["d"], case["p"]).view(case["rows"], case["d"])
    out = [s["x"].detach().double() * f]
    return out if s["dy"] is None else out + [s["dy"].double() * f]


def _exact_loss(case, s):
    h, w, y = s["h"].detach().double(), s["w"].detach().double(), s["labels"]
    loss = torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
    lse = torch.full_like(loss, -math.inf)  # of a row that is left out
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    counted = torch.arange(case["rows"], device="cuda")[y >= 0]
    for t in counted.split(max(1, int(2e8 // case["vocab"]))):
        z = case["scale"] * (h[t] @ w.T)
        logp = torch.log_softmax(z, 1)
        one = torch.arange(len(t), device="cuda")
        loss[t] = -logp[one, y[t]]
        lse[t] = torch.logsumexp(z, 1)
        if s["dl"] is None:
            continue
        z = torch.exp(logp)
        z[one, y[t]] -= 1
        z *= case["scale"] * s["dl"][t].double()[:, None]
        dh[t] = z @ w
        dw += z.T @ h[t]
    return [loss, lse] if s["dl"] is None else [loss, dh, dw]


def _powers():
    """2^-127 .. 2^127 in 64 bits."""
    return torch.tensor([2.0 ** k for k in range(-127, 128)], dtype=torch.float64, device="cuda")


def _exact_quantise(case, s):
    x = s["x"].double().view(case["rows"], -1, 32)
    big = x.abs().max(2, keepdim=True).values
    # a quarter of the largest power of two that is not above the block's largest entry
    powers = _powers()
    unit = powers[torch.searchsorted(powers, big / 4, right=True) - 1]
    # the grid is 1/2 up to 2, 1 up to 4, 2 up to 6: round halves to even on each part
    v = torch.abs(x / unit)
    g = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    v = torch.clamp(torch.round(v / g) * g, max=6.0)
    return [(torch.sign(x) * v * unit).view(case["rows"], -1)]


def _exact_values(codes, scales):
    c = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
    mantissa, exponent = c % 2, c // 2 % 4
    v = torch.where(exponent > 0, (2 + mantissa) * 2.0 ** (exponent - 2).double(), mantissa * 0.5)
    v = torch.where(c >= 8, -v, v)
    return v * _powers()[scales.int()].repeat_interleave(32, -1)


def _exact_score(case, s):
    q = _exact_values(s["q"], s["qs"])
    n = _lengths(case).tolist()
    c, e = (t.view(-1, t.shape[-1]) for t in (s["c"], s["s"]))
    start, total = [], 0
    for k in n:
        start.append(total)
        total += k if case["layout"] == "packed" else case["hi"]
    out = []
    per = max(1, (1 << 21) // case["hi"])  # documents at a time
    for a in range(0, case["docs"], per):
        lens = torch.tensor(n[a:a + per], device="cuda")
        first = torch.tensor(start[a:a + per], device="cuda")
        j = torch.arange(case["hi"], device="cuda")
        seen = j[None, :] < lens[:, None]
        at = torch.where(seen, first[:, None] + j[None, :], 0)
        lo = int(first[0])
        hi = start[a + per] if a + per < case["docs"] else total
        x = torch.zeros(1, case["queries"], dtype=torch.float64, device="cuda")
        if hi > lo:
            x = _exact_values(c[lo:hi], e[lo:hi]) @ q.T
        x = x[torch.where(seen, at - lo, 0)].masked_fill(~seen[..., None], -math.inf)
        out.append(x.max(1).values.sum(1))
    return [torch.cat(out)]


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"norm": _exact_norm, "dropout": _exact_dropout, "loss": _exact_loss,
                "quantise": _exact_quantise, "score": _exact_score}[case["op"]](case, s)
