"""Attention within documents on the GPU against a plain 64-bit implementation, element by
element within bounds that count the kernels' roundings (encoder_ref.attention)."""
import math

import numpy as np
import pytest

import encoder_ref as ref
from gpu_util import ms, say

pytestmark = pytest.mark.gpu


def T():
    import torch
    return torch


def dt(name):
    t = T()
    return {"bf16": t.bfloat16, "fp16": t.float16, "fp32": t.float32}[name]


def check(what, got, want, tol):
    got = ref.as64(got).reshape(want.shape)
    ninf = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), ninf), f"{what}: -inf pattern differs"
    got, want, tol = got[~ninf], want[~ninf], tol[~ninf]
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    if got.size == 0:
        return
    err = np.abs(got - want)
    worst = int(np.argmax(err / np.maximum(tol, 1e-300)))
    say(f"  {what}: worst error {err[worst]:.3e} of {tol[worst]:.3e} allowed, "
        f"norm-wise {np.linalg.norm(err) / max(np.linalg.norm(want), 1e-300):.2e}")
    assert np.all(err <= tol), f"{what}: {int((err > tol).sum())} of {err.size} out of bounds"


def inputs(seed, lens, heads, kv, d, dtype, fixed, std=1.0):
    """q, k, v as views of one projection's output, grad_o, and the layout's arguments."""
    t = T()
    g = t.Generator().manual_seed(seed)
    n = t.tensor(lens)
    rows = (len(lens), fixed) if fixed else (int(n.sum()),)
    qkv = (t.randn(*rows, heads + 2 * kv, d, generator=g) * std).to(dtype).cuda()
    q, k, v = qkv.split([heads, kv, kv], dim=-2)
    do = (t.randn(*rows, heads, d, generator=g) * 0.03).to(dtype).cuda()
    if fixed:
        lay = dict(doc_lens=n.to(t.int32).cuda())
        docs = ref.spans(len(lens) * fixed, lens=lens, nd=fixed)
    else:
        off = t.zeros(len(lens) + 1, dtype=t.int64)
        off[1:] = t.cumsum(n, 0)
        lay = dict(doc_offsets=off.cuda())
        docs = ref.spans(int(n.sum()), offsets=off.tolist())
    return q, k, v, do, lay, docs


def run_case(q, k, v, do, lay, docs, dtype, causal=False, prefix=None, cap=0.0, slopes=None,
             scale=None):
    t = T()
    kw = dict(lay, causal=causal, softcap=cap, scale=scale,
              prefix_lens=None if prefix is None else t.tensor(prefix, dtype=t.int32).cuda(),
              slopes=None if slopes is None else t.tensor(slopes, dtype=t.float32).cuda())
    o, lse = ms().maxsim_attention(q, k, v, **kw)
    grads = ms().maxsim_attention_backward(do, q, k, v, o, lse, **kw)
    t.cuda.synchronize()
    flat = lambda x: ref.as64(x).reshape(-1, x.shape[-2], x.shape[-1])  # noqa: E731
    s32 = None if slopes is None else np.float32(slopes).astype(np.float64)
    want = ref.attention(flat(q), flat(k), flat(v), docs, causal, prefix, cap, s32, scale,
                         flat(do), dtype)
    check("o", o, want["o"], want["tol_o"])
    check("lse", lse, want["lse"], want["tol_lse"])
    for name, got in zip(("dq", "dk", "dv"), grads):
        check(name, got, want[name], want["tol_" + name])
    return o, lse, grads


LENGTHS = {
    "ragged": [1, 0, 37, 128, 5, 129, 64, 0, 200],
    "tiny": [1, 2, 3, 0, 1],
    "one": [1],
    "long": [700, 33],
    "turns": [423, 290, 517],  # whole tiles that begin and end anywhere in a ring of four
    "edges": [31, 32, 33, 63, 64, 65, 127, 128, 129],
}

CASES = [
    # lengths, heads, kv, d, dtype, fixed, causal, prefix, cap, bias
    ("ragged", 4, 4, 64, "bf16", 0, False, False, 0.0, False),
    ("ragged", 4, 2, 64, "fp16", 0, True, False, 0.0, False),
    ("ragged", 2, 1, 128, "fp32", 0, True, True, 0.0, True),
    ("edges", 3, 3, 32, "bf16", 0, True, True, 0.0, False),
    ("edges", 4, 1, 96, "fp16", 0, False, False, 20.0, True),
    ("edges", 2, 2, 80, "fp32", 0, False, False, 5.0, False),
    ("tiny", 6, 2, 72, "bf16", 0, True, True, 30.0, True),
    ("tiny", 1, 1, 8, "fp32", 0, False, False, 0.0, False),
    ("tiny", 1, 1, 8, "fp16", 0, True, False, 0.0, True),
    ("one", 12, 12, 64, "bf16", 0, False, False, 0.0, False),
    ("one", 2, 1, 256, "fp16", 0, True, False, 0.0, False),
    ("long", 8, 2, 128, "bf16", 0, True, False, 0.0, True),
    ("long", 4, 1, 256, "bf16", 0, True, True, 50.0, False),
    ("long", 2, 1, 256, "fp16", 0, False, False, 0.0, False),
    ("long", 2, 2, 64, "fp32", 0, True, False, 0.0, False),
    ("long", 3, 1, 160, "bf16", 0, False, False, 0.0, True),
    ("ragged", 4, 4, 64, "bf16", 200, False, False, 0.0, False),
    ("ragged", 4, 2, 128, "fp16", 201, True, True, 0.0, True),
    ("edges", 2, 1, 96, "fp32", 130, True, True, 10.0, True),
    ("tiny", 2, 2, 40, "bf16", 3, False, False, 0.0, True),
    ("long", 2, 1, 256, "bf16", 701, True, False, 0.0, False),
    ("turns", 6, 2, 64, "bf16", 0, False, False, 0.0, False),
    ("turns", 3, 1, 64, "fp16", 0, True, False, 20.0, False),
    ("turns", 3, 1, 128, "fp16", 0, True, True, 30.0, True),
    ("turns", 6, 2, 128, "bf16", 0, False, False, 30.0, False),
    ("turns", 3, 1, 128, "bf16", 0, False, False, 0.0, False),
    ("turns", 2, 1, 128, "fp32", 0, False, False, 0.0, True),
    ("turns", 3, 1, 128, "fp32", 0, True, False, 15.0, False),
    ("turns", 4, 2, 96, "bf16", 0, False, False, 30.0, True),
    ("turns", 2, 1, 256, "fp16", 0, False, False, 30.0, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_against_64_bits(case):
    name, heads, kv, d, dtype, fixed, causal, pre, cap, bias = case
    say("case:", case)
    lens = LENGTHS[name]
    x = inputs(7 + d + heads, lens, heads, kv, d, dt(dtype), fixed)
    prefix = [(5 * b + n // 3) % (n + 2) for b, n in enumerate(lens)] if pre else None
    slopes = [2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)] if bias else None
    run_case(*x, dt(dtype), causal, prefix, cap, slopes)


def test_padding_holds_anything():
    """Rows past a document's length hold NaN and infinities in q, k, v and grad_o; the results
    are those of clean padding, and zeros / -inf in the padding."""
    t = T()
    lens = [0, 3, 64, 77, 31, 100]
    for dtype in ("bf16", "fp16", "fp32"):
        say("case: dirty padding", dtype)
        q, k, v, do, lay, docs = inputs(3, lens, 4, 2, 64, dt(dtype), 100)
        clean = run_case(q, k, v, do, lay, docs, dt(dtype), causal=True)
        pad = t.arange(100)[None, :] >= t.tensor(lens)[:, None]
        dirty = [x.clone() for x in (q, k, v, do)]
        for x, val in zip(dirty, (math.nan, math.inf, math.nan, -math.inf)):
            x[pad.cuda()] = val
        o, lse = ms().maxsim_attention(*dirty[:3], **lay, causal=True)
        g = ms().maxsim_attention_backward(dirty[3], *dirty[:3], o, lse, **lay, causal=True)
        t.cuda.synchronize()
        assert t.equal(o, clean[0]) and t.equal(lse, clean[1])
        for a, b in zip(g, clean[2]):
            assert t.equal(a, b)
        assert not o[pad.cuda()].any() and t.isneginf(lse.view(4, 6, 100)[:, pad]).all()


def test_tokens_of_no_document():
    """Offsets that begin after the first token and end before the last: the tokens outside get
    zeros and -inf, the others what they get alone."""
    t = T()
    q, k, v, do, lay, docs = inputs(11, [140, 3, 150], 4, 2, 64, t.bfloat16, 0)
    off = t.tensor([130, 143, 143, 160], dtype=t.int64)
    docs = ref.spans(293, offsets=off.tolist())
    say("case: offsets inside the token range")
    o, lse, grads = run_case(q, k, v, do, dict(doc_offsets=off.cuda()), docs, t.bfloat16)
    assert not o[:130].any() and not o[160:].any() and not grads[1][160:].any()
    none = t.zeros(1, dtype=t.int64).cuda()
    o, lse = ms().maxsim_attention(q, k, v, none)  # no document at all
    assert not o.any() and t.isneginf(lse).all()


@pytest.mark.parametrize("kind", ["ragged", "clustered", "empty tail", "growing", "single tokens"])
def test_many_documents(kind):
    """Thousands of documents of uneven lengths: every tile finds its own. With q = 0 a token's
    result is its document's mean of v, and lse the logarithm of its length."""
    t = T()
    rng = np.random.default_rng(3)
    n = {"ragged": rng.integers(0, 40, 5000), "clustered": np.where(rng.random(4000) < 0.9, 0, 300),
         "empty tail": np.r_[np.full(3, 3000), np.zeros(3000, int)], "growing": np.arange(0, 600),
         "single tokens": np.ones(3000, int)}[kind]
    off = np.r_[0, np.cumsum(n)]
    rows = int(off[-1])
    v = t.randn(rows, 1, 64, generator=t.Generator().manual_seed(5))
    say("case: many documents", kind, rows)
    o, lse = ms().maxsim_attention(t.zeros(rows, 2, 64, device="cuda"), t.zeros(rows, 1, 64, device="cuda"),
                                   v.cuda(), t.from_numpy(off).cuda())
    x = v[:, 0].double().numpy()
    sums = np.r_[np.zeros((1, 64)), np.cumsum(x, 0)]
    doc = np.repeat(np.arange(len(n)), n)
    want = ((sums[off[1:]] - sums[off[:-1]]) / np.maximum(n, 1)[:, None])[doc]
    # n sums of n terms in 32 bits, and the weights' own division
    tol = (n[doc][:, None] + 4) * ref.U32 * np.abs(x).max()
    got = ref.as64(o)
    assert np.all(np.abs(got - want[:, None]) <= tol[:, None])
    assert np.all(np.abs(ref.as64(lse) - np.log(n[doc])) <= 1e-5)


@pytest.mark.parametrize("dtype, d, heads, kv, causal, cap, bias", [
    ("bf16", 128, 8, 2, True, 0.0, True), ("fp16", 128, 4, 4, False, 30.0, False),
    ("bf16", 64, 16, 16, False, 0.0, False), ("fp16", 64, 16, 8, True, 20.0, True),
    ("bf16", 96, 8, 1, False, 0.0, True), ("fp16", 72, 12, 3, True, 0.0, False),
    ("bf16", 32, 32, 4, True, 0.0, True)])
def test_long_batches(dtype, d, heads, kv, causal, cap, bias):
    """Enough long documents for several rounds of workgroups on every CU: single heads of some of
    them, in the batch and alone, against 64 bits."""
    t = T()
    lens = [1100, 700, 1025, 513, 1400, 900, 640] * 4
    q, k, v, do, lay, docs = inputs(77, lens, heads, kv, d, dt(dtype), 0)
    slopes = t.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)]).cuda() if bias else None
    kw = dict(causal=causal, softcap=cap, slopes=slopes)
    say("case: long batch", dtype, d, heads)
    o, lse = ms().maxsim_attention(q, k, v, **lay, **kw)
    for b in (0, 3, 27):
        t0, n = docs[b]
        rows = slice(t0, t0 + n)
        alone = ms().maxsim_attention(q[rows], k[rows], v[rows], t.tensor([0, n]).cuda(), **kw)
        s64 = None if slopes is None else ref.as64(slopes)
        for h in (0, heads - 1):
            g = h // (heads // kv)
            want = ref.attention(ref.as64(q[rows, h:h + 1]), ref.as64(k[rows, g:g + 1]),
                                 ref.as64(v[rows, g:g + 1]), [(0, n)], causal, None, cap,
                                 None if s64 is None else s64[h:h + 1], dtype=dt(dtype))
            for got, gl in ((o[rows, h:h + 1], lse[h, rows]), (alone[0][:, h:h + 1], alone[1][h])):
                check("o", got, want["o"], want["tol_o"])
                check("lse", gl[None], want["lse"], want["tol_lse"])


def test_any_strides():
    """Heads before tokens, gaps between rows, an offset start: the same bits as contiguous."""
    t = T()
    B, N, H, KV, d = 3, 90, 4, 2, 64
    g = t.Generator().manual_seed(2)
    q = t.randn(B, H, N, d, generator=g).bfloat16().cuda().transpose(1, 2)
    big = t.randn(B, N + 5, 2 * KV + 1, d + 24, generator=g).bfloat16().cuda()
    k, v = big[:, 3:N + 3, :KV, 8:d + 8], big[:, 2:N + 2, KV + 1:, 16:d + 16]
    lens = t.tensor([90, 11, 64], dtype=t.int32).cuda()
    say("case: strides")
    a = ms().maxsim_attention(q, k, v, doc_lens=lens, causal=True)
    b = ms().maxsim_attention(q.contiguous(), k.contiguous(), v.contiguous(), doc_lens=lens, causal=True)
    assert all(t.equal(x, y) for x, y in zip(a, b))
    ga = ms().maxsim_attention_backward(a[0], q, k, v, *a, doc_lens=lens, causal=True)
    gb = ms().maxsim_attention_backward(a[0], q.contiguous(), k.contiguous(), v.contiguous(), *a,
                                        doc_lens=lens, causal=True)
    assert all(t.equal(x, y) for x, y in zip(ga, gb))


def test_large_scores_and_scale():
    """Scores of several hundred, where a weight is all or nothing, and a scale of one's own."""
    t = T()
    for dtype in ("bf16", "fp32"):
        x = inputs(21, [150, 40], 2, 1, 64, dt(dtype), 0, std=6.0)
        say("case: large scores", dtype)
        run_case(*x, dt(dtype), scale=0.31)


def test_small_gradients_fp16():
    """Gradients of 1e-6 over several hundred keys: dS far below fp16's normal range."""
    t = T()
    q, k, v, do, lay, docs = inputs(23, [600], 2, 1, 64, t.float16, 0)
    do = (do.float() * 2.0 ** -9).half()
    say("case: small gradients")
    o, lse = ms().maxsim_attention(q, k, v, **lay)
    dq, dk, dv = ms().maxsim_attention_backward(do * 512, q, k, v, o, lse, **lay)
    eq, ek, ev = ms().maxsim_attention_backward(do, q, k, v, o, lse, **lay)
    # a power of two less, so that what is not lost scales: the two differ by their own last
    # rounding, which for results of 1e-6 is half a subnormal step
    for a, b in ((dq, eq), (dk, ek), (dv, ev)):
        a = a.float() / 512
        assert bool(((a - b.float()).abs() <= 2.0 ** -25 + 2.0 ** -10 * a.abs()).all())


def test_autograd_and_partial_gradients():
    t = T()
    q, k, v, do, lay, docs = inputs(31, [50, 0, 70], 4, 2, 64, t.bfloat16, 0)
    o, lse = ms().maxsim_attention(q, k, v, **lay, causal=True)
    want = ms().maxsim_attention_backward(do, q, k, v, o, lse, **lay, causal=True)
    leaves = [x.detach().clone().requires_grad_(True) for x in (q, k, v)]
    y = ms().attention(*leaves, **lay, causal=True)
    assert t.equal(y, o)
    y.backward(do)
    for a, b in zip(leaves, want):
        assert t.equal(a.grad, b)
    # a broadcast gradient (stride 0), and only some inputs asking
    qq = q.detach().clone().requires_grad_(True)
    ms().attention(qq, k.detach(), v.detach(), **lay, causal=True).sum().backward()
    ones = t.ones_like(o)
    assert t.equal(qq.grad, ms().maxsim_attention_backward(ones, q, k, v, o, lse, **lay, causal=True)[0])
    vv = v.detach().clone().requires_grad_(True)
    ms().attention(q.detach(), k.detach(), vv, **lay, causal=True).backward(do)
    assert t.equal(vv.grad, want[2])


def test_no_tokens():
    t = T()
    q = t.empty(0, 4, 64, dtype=t.bfloat16, device="cuda")
    off = t.zeros(3, dtype=t.int64).cuda()
    o, lse = ms().maxsim_attention(q, q, q, off)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    g = ms().maxsim_attention_backward(q, q, q, q, o, lse, off)
    assert all(x.shape == q.shape for x in g)


def test_same_bits_again_and_on_another_stream_and_in_a_graph():
    t = T()
    for dtype in ("bf16", "fp16"):
        q, k, v, do, lay, docs = inputs(41, [200, 3, 0, 150, 77], 8, 2, 64, dt(dtype), 0)
        o, lse = ms().maxsim_attention(q, k, v, **lay)
        want = [o, lse, *ms().maxsim_attention_backward(do, q, k, v, o, lse, **lay)]
        t.cuda.synchronize()
        for _ in range(3):
            o, lse = ms().maxsim_attention(q, k, v, **lay)
            got = [o, lse, *ms().maxsim_attention_backward(do, q, k, v, o, lse, **lay)]
            assert all(t.equal(a, b) for a, b in zip(got, want))
        side = t.cuda.Stream()
        o, lse = ms().maxsim_attention(q, k, v, **lay, stream=side)
        got = [o, lse, *ms().maxsim_attention_backward(do, q, k, v, o, lse, **lay, stream=side)]
        side.synchronize()
        assert all(t.equal(a, b) for a, b in zip(got, want))
        outs = [t.empty_like(x) for x in want]
        ws = t.empty(ms().attention_backward_workspace_size(q.shape[0], 8), dtype=t.uint8, device="cuda")

        def step():
            ms().maxsim_attention(q, k, v, **lay, out=outs[0], lse=outs[1])
            ms().maxsim_attention_backward(do, q, k, v, outs[0], outs[1], **lay, dq=outs[2],
                                           dk=outs[3], dv=outs[4], workspace=ws)
        step()
        t.cuda.synchronize()
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            step()
        for _ in range(3):
            for x in outs:
                x.fill_(float("nan"))
            ws.fill_(255)
            t.cuda.synchronize()
            graph.replay()
            t.cuda.synchronize()
            assert all(t.equal(a, b) for a, b in zip(outs, want))


def test_unsupported_head_is_an_error():
    t = T()
    q = t.zeros(4, 1, 192, device="cuda")
    with pytest.raises(ms().MaxSimError) as e:
        ms().maxsim_attention(q, q, q, t.tensor([0, 4]).cuda())
    assert e.value.status == -5
    q = t.zeros(4, 1, 65, device="cuda", dtype=t.bfloat16)[..., 1:]
    with pytest.raises(ms().MaxSimError) as e:  # rows that are not a multiple of 16 bytes apart
        ms().maxsim_attention(q, q, q, t.tensor([0, 4]).cuda())
    assert e.value.status == -4


def test_tokens_of_no_document_hold_anything():
    """A packed buffer whose ends hold no document: whatever lies there, the results are those of
    clean ends, fp16's small gradients included, whose scale is taken from grad_o and v."""
    t = T()
    for dtype in ("bf16", "fp16", "fp32"):
        q, k, v, do, lay, docs = inputs(13, [140, 3, 150], 4, 2, 64, dt(dtype), 0)
        off = t.tensor([130, 143, 143, 260], dtype=t.int64)
        docs = ref.spans(293, offsets=off.tolist())
        do = (do.float() * 2.0 ** -9).to(dt(dtype))
        say("case: anything outside the offsets", dtype)
        clean = run_case(q, k, v, do, dict(doc_offsets=off.cuda()), docs, dt(dtype))
        for value in (6e4, math.inf, math.nan):
            dirty = [x.clone() for x in (q, k, v, do)]
            for x in dirty:
                x[:130] = value
                x[260:] = -value
            kw = dict(doc_offsets=off.cuda())
            o, lse = ms().maxsim_attention(*dirty[:3], **kw)
            g = ms().maxsim_attention_backward(dirty[3], *dirty[:3], o, lse, **kw)
            t.cuda.synchronize()
            for a, b in zip((o, lse, *g), (clean[0], clean[1], *clean[2])):
                assert t.equal(a, b), value


@pytest.mark.parametrize("dtype, d, heads, kv, causal, bias", [
    ("bf16", 64, 4, 2, False, False), ("bf16", 256, 2, 1, True, True), ("fp16", 96, 3, 1, True, True),
    ("fp16", 128, 2, 2, False, False), ("fp16", 32, 2, 1, False, True), ("fp32", 128, 2, 1, True, False),
    ("bf16", 96, 4, 4, False, False), ("fp32", 32, 2, 1, False, True)])
def test_caps_far_above_the_scores(dtype, d, heads, kv, causal, bias):
    """A cap far above every score changes the scores by less than they are rounded by, so the
    results are within the bounds of a call without a cap, however large it is."""
    t = T()
    x = inputs(51 + d, [1, 70, 0, 200, 33], heads, kv, d, dt(dtype), 0)
    q, k, v, do, lay, docs = x
    slopes = np.float32([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)]) if bias else None
    args = (*(ref.as64(y) for y in (q, k, v)), docs, causal, None)
    s64 = None if slopes is None else slopes.astype(np.float64)
    bound = ref.attention(*args, 0.0, s64, None, ref.as64(do), dt(dtype))
    for cap in (1e3, 1e4, 1e5, 1e6, 1e8, 1e20, 1e35, 3.4e38):
        say("case: far cap", cap, dtype, d)
        want = ref.attention(*args, cap, s64, None, ref.as64(do), dt(dtype))
        kw = dict(lay, causal=causal, softcap=cap, slopes=None if slopes is None else t.tensor(slopes).cuda())
        o, lse = ms().maxsim_attention(q, k, v, **kw)
        grads = ms().maxsim_attention_backward(do, q, k, v, o, lse, **kw)
        t.cuda.synchronize()
        for name, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
            check(name, got, want[name], bound["tol_" + name])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cap", [1e-42, 511.0, 513.0])
def test_caps_that_scores_reach(cap, dtype):
    """Scores of up to twice the cap on either side of the two forms of the tanh, and caps so small
    that every score saturates."""
    say("case: reached cap", cap, dtype)
    q, k, v, do, lay, docs = inputs(61, [90, 40], 2, 1, 64, dt(dtype), 0)
    q[3] = 0  # scores of exactly 0
    run_case(q, k, v, do, lay, docs, dt(dtype), cap=cap, scale=40.0 if cap > 1 else None)
