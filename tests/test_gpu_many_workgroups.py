"""Calls with more work than one launch may have threads (2^32), and tensors of more than 2^31
elements."""
import numpy as np
import pytest

import encoder_ref as ref
from gpu_util import ms, say

pytestmark = pytest.mark.gpu


def test_attention_over_hundreds_of_thousands_of_documents():
    """One token a document: it sees itself alone, so o is v and dv is grad_o to the bit, lse its
    score, and dq and dk vanish up to the roundings of two equal sums of d products. A longer
    document at the end gets what it gets alone."""
    import torch as t
    docs, heads, d, tail = 600_000, 32, 8, 200
    n = docs + tail
    assert (docs + 2) * heads > 2 ** 24
    g = t.Generator(device="cuda").manual_seed(9)
    q, k, v, do = (t.randn(n, heads, d, generator=g, device="cuda").bfloat16() for _ in range(4))
    off = t.cat([t.arange(docs + 1), t.tensor([n])]).cuda()
    say("case: attention over", docs, "documents")
    o, lse = ms().maxsim_attention(q, k, v, off)
    dq, dk, dv = ms().maxsim_attention_backward(do, q, k, v, o, lse, off)
    t.cuda.synchronize()
    one = slice(0, docs)
    assert t.equal(o[one], v[one]) and t.equal(dv[one], do[one])
    scale = d ** -0.5
    x, size = ((y * z).sum(-1).t()[:, one] * scale for y, z in ((q.float(), k.float()),
                                                               (q.float().abs(), k.float().abs())))
    # both sums of d products, and a few roundings of the score itself
    assert bool(((lse[:, one] - x).abs() <= (2 * d + 8) * ref.U32 * size).all())
    sums = (do.float().abs() * v.float().abs()).sum(-1, keepdim=True) * (2 * d + 8) * ref.U32 * scale
    for got, other in ((dq, k), (dk, q)):
        bound = sums * other.float().abs() * (1 + ref.HALF_STEP[t.bfloat16]) + ref.TINY[t.bfloat16]
        assert bool((got[one].float().abs() <= bound[one]).all())
    alone = [y[docs:].clone() for y in (q, k, v, do)]
    whole = t.tensor([0, tail]).cuda()
    a, b = ms().maxsim_attention(*alone[:3], whole)
    assert t.equal(a, o[docs:]) and t.equal(b, lse[:, docs:])
    grads = ms().maxsim_attention_backward(alone[3], *alone[:3], a, b, whole)
    assert all(t.equal(y, z[docs:]) for y, z in zip(grads, (dq, dk, dv)))


def test_rotary_over_a_billion_tokens():
    import torch as t
    n = 2 ** 30 + 12345
    x = t.empty(n, 1, 2, dtype=t.bfloat16, device="cuda")
    x[..., 0], x[..., 1] = 0.75, -0.5
    say("case: rotary over", n, "tokens")
    y = ms().maxsim_rotary(x, t.ones(1, device="cuda"))
    t.cuda.synchronize()
    for at in (0, 2 ** 29 - 500, 2 ** 29, 2 ** 30 - 500, 2 ** 30, n - 1000):
        pos = np.arange(at, at + 1000)
        want = ref.turned(np.tile([0.75, -0.5], (1000, 1, 1)), pos, np.ones(1), "half", 1.0)
        # output rounding; sine and cosine off by at most 4e-7, two products and a sum
        tol = ref.HALF_STEP[t.bfloat16] * np.abs(want) + 1.25 * (4e-7 + 6 * ref.U32)
        assert np.all(np.abs(ref.as64(y[at:at + 1000]) - want) <= tol), at
    # every token is there: turning keeps a pair's length (0.9014) up to two roundings of it
    for part in y.split(2 ** 27):
        assert bool(((part.float().square().sum(-1).sqrt() - 0.9014).abs() < 0.01).all())


def test_clipping_of_two_billion_elements():
    """All of one value but the last, whose square is as large as the others' together."""
    import torch as t
    n = 2 ** 31 + 777
    x = t.ones(n, dtype=t.bfloat16, device="cuda")
    x[-1] = 2.0 ** 15.5  # rounded to 46336
    last = float(x[-1])
    norm = (n - 1 + last ** 2) ** 0.5
    say("case: clipping of", n, "elements")
    got = ms().maxsim_clip_grad_norm([x], 1.0)
    assert abs(float(got) - norm) <= 2 * ref.U32 * norm
    want = t.tensor([1 / (norm + 1e-6), last / (norm + 1e-6)], dtype=t.float64)
    # the factor and the product round to 32 bits, the result to its type
    tol = (ref.HALF_STEP[t.bfloat16] + 3 * ref.U32) * want
    assert bool(((x[:-1].amin().double().cpu() - want[0]).abs() <= tol[0]))
    assert bool(((x[:-1].amax().double().cpu() - want[0]).abs() <= tol[0]))
    assert bool(((x[-1].double().cpu() - want[1]).abs() <= tol[1]))
