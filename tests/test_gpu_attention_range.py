"""Attention at the ends of its range: the backward over several rounds of workgroups, lengths and
offsets that are clamped, tensors past 4 GiB."""
import numpy as np
import pytest

import encoder_ref as ref
from gpu_util import ms, say
from test_gpu_attention import check, dt, inputs, run_case

pytestmark = pytest.mark.gpu


def T():
    import torch
    return torch


@pytest.mark.parametrize("dtype, d, heads, kv, causal, cap, bias", [
    ("bf16", 128, 8, 2, True, 0.0, True), ("fp16", 128, 4, 4, False, 30.0, False),
    ("bf16", 64, 16, 16, False, 0.0, False), ("fp16", 64, 16, 8, True, 20.0, True),
    ("bf16", 256, 4, 1, False, 0.0, False), ("fp16", 96, 8, 4, False, 30.0, True),
    ("fp32", 128, 4, 2, True, 0.0, False), ("fp32", 64, 8, 8, False, 15.0, True)])
def test_backward_of_long_batches(dtype, d, heads, kv, causal, cap, bias):
    """Enough long documents for several rounds of workgroups on every CU: the gradients of one
    key/value head of some of them against 64 bits."""
    t = T()
    lens = [1100, 700, 1025, 513, 1400, 900, 640] * 4
    q, k, v, do, lay, docs = inputs(78, lens, heads, kv, d, dt(dtype), 0)
    slopes = t.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)]).cuda() if bias else None
    kw = dict(causal=causal, softcap=cap, slopes=slopes)
    say("case: backward of a long batch", dtype, d, heads)
    o, lse = ms().maxsim_attention(q, k, v, **lay, **kw)
    grads = ms().maxsim_attention_backward(do, q, k, v, o, lse, **lay, **kw)
    t.cuda.synchronize()
    group = heads // kv
    s64 = None if slopes is None else ref.as64(slopes)
    for b, g in ((0, 0), (3, kv - 1), (27, kv // 2)):
        rows, H, G = slice(docs[b][0], sum(docs[b])), slice(g * group, (g + 1) * group), slice(g, g + 1)
        want = ref.attention(*(ref.as64(x) for x in (q[rows, H], k[rows, G], v[rows, G])),
                             [(0, docs[b][1])], causal, None, cap, None if s64 is None else s64[H],
                             None, ref.as64(do[rows, H]), dt(dtype))
        for name, got, at in zip(("o", "dq", "dk", "dv"), (o, *grads), (H, H, G, G)):
            check(name, got[rows, at], want[name], want["tol_" + name])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_lengths_are_clamped(dtype):
    """Lengths below 0 and above nd, prefixes below 0 and above the length."""
    t = T()
    given, lens = [-7, 300, 90, 2 ** 31 - 1, -2 ** 31, 33], [0, 90, 90, 90, 0, 33]
    q, k, v, do, _, docs = inputs(5, lens, 4, 2, 64, dt(dtype), 90)
    lay = dict(doc_lens=t.tensor(given, dtype=t.int32).cuda())
    say("case: clamped lengths", dtype)
    run_case(q, k, v, do, lay, docs, dt(dtype))
    prefix = [5, -3, 2 ** 31 - 1, 40, 7, 1000]
    run_case(q, k, v, do, lay, docs, dt(dtype), causal=True, prefix=prefix)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_offsets_are_clamped(dtype):
    """Offsets before the first token and past the last."""
    t = T()
    q, k, v, do, _, _ = inputs(6, [300], 4, 2, 64, dt(dtype), 0)
    given = [-2 ** 62, -5, 40, 170, 170, 300, 2 ** 40, 2 ** 62]
    real = np.clip(given, 0, 300).tolist()
    say("case: clamped offsets", dtype)
    run_case(q, k, v, do, dict(doc_offsets=t.tensor(given).cuda()), ref.spans(300, offsets=real), dt(dtype),
             causal=True)


@pytest.mark.parametrize("fixed", [False, True])
def test_tensors_past_4_gib(fixed):
    """Documents on either side of 4 GiB and at the end of tensors of 5 GiB get what they get alone,
    forwards and backwards."""
    t = T()
    heads, d, n, docs = 32, 128, 75, 8200
    assert docs * n * heads * d * 2 > 5e9
    g = t.Generator(device="cuda").manual_seed(3)
    q, k, v, do = (t.randn(docs, n, heads, d, generator=g, device="cuda", dtype=t.bfloat16) for _ in range(4))
    off = (t.arange(docs + 1) * n).cuda()
    flat = (lambda x: x) if fixed else (lambda x: x.flatten(0, 1))
    kw = {} if fixed else dict(doc_offsets=off)
    say("case: 5 GiB,", "fixed" if fixed else "packed")
    args = [flat(x) for x in (q, k, v)]
    o, lse = ms().maxsim_attention(*args, **kw)
    grads = ms().maxsim_attention_backward(flat(do), *args, o, lse, **kw)
    t.cuda.synchronize()
    edge = 2 ** 32 // (n * heads * d * 2)
    for b in (0, edge // 2, edge, edge + 1, docs - 1):
        one = [flat(x[b:b + 1].clone()) for x in (q, k, v, do)]
        few = {} if fixed else dict(doc_offsets=off[:2])
        a, z = ms().maxsim_attention(*one[:3], **few)
        alone = (a, *ms().maxsim_attention_backward(one[3], *one[:3], a, z, **few))
        for x, y in zip((o, *grads), alone):
            assert t.equal(x.view(docs, n, heads, d)[b], y.view(n, heads, d)), b
        assert t.equal(lse.view(heads, docs, n)[:, b], z)
