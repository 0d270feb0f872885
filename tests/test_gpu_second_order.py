"""Gradients of gradients: right, or an error; a term is never left out without one."""
import pytest

from gpu_util import ms, say

pytestmark = pytest.mark.gpu


def T():
    import torch
    return torch


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_gradients_of_gradients(layout):
    """With y the turned x and R the turning, the gradient of sum(y^2 w) is R^T (2 w R x), and that
    of its squared length |h|^2 is 2 R^T (2 w R h): three turnings there and three back."""
    t = T()
    say("case: rotary twice", layout)
    g = t.Generator().manual_seed(4)
    x = t.randn(50, 3, 64, generator=g).cuda().requires_grad_(True)
    w = t.randn(50, 3, 64, generator=g).cuda()
    freq = (10000.0 ** (-t.arange(16, dtype=t.float64) / 16)).float().cuda()
    off = t.tensor([0, 20, 50]).cuda()
    kw = dict(doc_offsets=off, layout=layout, mscale=1.2)
    h, = t.autograd.grad((ms().rotary(x, freq, **kw).square() * w).sum(), x, create_graph=True)
    got, = t.autograd.grad(h.square().sum(), x)
    turn = lambda z, back: ms().maxsim_rotary(z, freq, inverse=back, **kw)  # noqa: E731
    lin = lambda z: turn(2 * w * turn(z, False), True)  # noqa: E731
    x = x.detach()
    # the same turnings in the same order: some 20 roundings of 32 bits apart, of values that a
    # turning mixes in pairs
    want = 2 * lin(lin(x))
    assert bool(((got - want).abs() <= 1e-5 * want.abs().max()).all())


def first_order(f, *inputs):
    """f(*inputs), a sum, has right first gradients under create_graph, other terms may be
    differentiated again beside them, and what depends on the gradients themselves is an error."""
    t = T()
    want = t.autograd.grad(f(*inputs), inputs)
    got = t.autograd.grad(f(*inputs), inputs, create_graph=True)
    assert all(t.equal(a, b) and b.requires_grad for a, b in zip(want, got))
    x = inputs[0]
    both = f(*inputs) + x.float().pow(3).sum()
    g, = t.autograd.grad(both, x, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        t.autograd.grad(g.float().square().sum(), x)
    x2 = x.detach().clone().requires_grad_(True)
    h, = t.autograd.grad(x2.float().pow(3).sum() + f(*inputs), x2, create_graph=True)
    assert t.equal(t.autograd.grad(h.float().sum(), x2)[0], (6 * x2.float()).to(x2.dtype))


def test_attention_gradients_of_gradients_are_an_error():
    t = T()
    say("case: attention twice")
    g = t.Generator().manual_seed(6)
    q, k, v = (t.randn(60, h, 64, generator=g).cuda().requires_grad_(True) for h in (4, 2, 2))
    off = t.tensor([0, 25, 60]).cuda()
    first_order(lambda *x: ms().attention(*x, off).sum(), q, k, v)
    first_order(lambda *x: (ms().attention(*x, off, causal=True).square()).sum(), q, k, v)
    # one input alone
    g, = t.autograd.grad(ms().attention(q, k.detach(), v.detach(), off).sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        g.sum().backward()


def test_maxsim_gradients_of_gradients_are_an_error():
    t = T()
    say("case: maxsim twice")
    g = t.Generator().manual_seed(8)
    Q = t.randn(16, 64, generator=g).cuda().requires_grad_(True)
    D = t.randn(90, 64, generator=g).cuda().requires_grad_(True)
    off = t.tensor([0, 25, 90]).cuda()
    first_order(lambda *x: ms().maxsim(*x, off).sum(), Q, D)
    first_order(lambda *x: ms().maxsim(*x, off).square().sum(), Q, D)
