"""Rotary positions and clipping by the global norm on the GPU against 64 bits."""
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


def rotary_bound(x, want, freq, layout, mscale, dtype):
    """Output rounding, and in 32 bits: sine and cosine (each off by at most 4e-7), two products
    and a sum."""
    half = len(freq)
    A = slice(0, half) if layout == "half" else slice(0, 2 * half, 2)
    B = slice(half, 2 * half) if layout == "half" else slice(1, 2 * half, 2)
    tol = np.zeros_like(x)
    both = (np.abs(x[..., A]) + np.abs(x[..., B])) * mscale * (4e-7 + 6 * ref.U32)
    tol[..., A] = both
    tol[..., B] = both
    tol += ref.HALF_STEP[dtype] * np.abs(want) * (tol > 0) + ref.TINY[dtype] * (tol > 0)
    return tol


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n, heads, d, rot, dtype, where, mscale", [
    (1, 1, 64, 64, "bf16", "docs", 1.0),
    (32, 24, 64, 64, "bf16", "docs", 1.0),
    (301, 5, 96, 32, "fp32", "given", 1.1),
    (301, 3, 128, 128, "fp16", "docs", 1.2),
    (77, 40, 128, 64, "bf16", "index", 1.0),
    (50, 3, 36, 18, "fp16", "given", 1.0),     # odd pairs: entries one by one
    (50, 2, 34, 34, "fp32", "docs", 1.0),
    (13, 2, 256, 16, "bf16", "given", 1.0),
    (9, 1, 1024, 1024, "bf16", "docs", 1.0),
    (2000, 2, 32, 16, "fp32", "docs", 0.9),
])
def test_rotary(n, heads, d, rot, dtype, where, mscale, layout):
    t = T()
    say("case: rotary", n, heads, d, rot, dtype, where, layout)
    g = t.Generator().manual_seed(n + d)
    x = t.randn(n, heads, d, generator=g).to(dt(dtype)).cuda()
    freq = (10000.0 ** (-t.arange(rot // 2, dtype=t.float64) / (rot // 2))).float()
    kw, pos = {}, np.arange(n)
    if where == "given":
        p = t.randint(-5, 100000, (n,), generator=g, dtype=t.int32)
        kw, pos = dict(positions=p.cuda()), p.numpy()
    elif where == "docs":
        cuts = sorted(set([0, 0, n // 3, n // 3 + 1, n // 2, n]))
        off = t.tensor([0, 0] + cuts[1:], dtype=t.int64)  # an empty document first
        kw = dict(doc_offsets=off.cuda())
        pos = np.concatenate([np.arange(b - a) for a, b in zip(off[:-1].tolist(), off[1:].tolist())])
    y = ms().maxsim_rotary(x, freq.cuda(), layout=layout, mscale=mscale, **kw)
    back = ms().maxsim_rotary(x, freq.cuda(), layout=layout, mscale=mscale, inverse=True, **kw)
    t.cuda.synchronize()
    for got, sign in ((y, 1.0), (back, -1.0)):
        want = ref.turned(ref.as64(x), pos, freq.double().numpy(), layout, mscale, sign)
        err = np.abs(ref.as64(got) - want)
        tol = rotary_bound(ref.as64(x), want, freq, layout, mscale, dt(dtype))
        say(f"  worst {np.max(err):.2e}")
        assert np.all(err <= tol)
    assert t.equal(y[..., rot:], x[..., rot:])
    leaf = x.clone().requires_grad_(True)
    z = ms().rotary(leaf, freq.cuda(), layout=layout, mscale=mscale, **kw)
    assert t.equal(z, y)
    dy = t.randn(n, heads, d, generator=g).to(dt(dtype)).cuda()
    z.backward(dy)
    assert t.equal(leaf.grad, ms().maxsim_rotary(dy, freq.cuda(), layout=layout, mscale=mscale,
                                                 inverse=True, **kw))


def test_rotary_strides_in_place_and_far_offsets():
    t = T()
    freq = (10000.0 ** (-t.arange(32, dtype=t.float64) / 32)).float().cuda()
    buf = t.randn(70, 9, 64, device="cuda").bfloat16()
    q = buf[:, :5]  # the query heads of one projection's output
    want = ms().maxsim_rotary(q.contiguous(), freq)
    say("case: rotary on a view, then in place")
    assert t.equal(ms().maxsim_rotary(q, freq), want)
    rest = buf[:, 5:].clone()
    assert ms().maxsim_rotary(q, freq, out=q) is q
    assert t.equal(q, want) and t.equal(buf[:, 5:], rest)
    x = t.randn(20, 64, 4, device="cuda").transpose(1, 2)  # entries not side by side
    with pytest.raises(ValueError):
        ms().maxsim_rotary(x, freq)
    # a broadcast gradient
    leaf = t.randn(20, 2, 64, device="cuda", requires_grad=True)
    ms().rotary(leaf, freq).sum().backward()
    assert t.equal(leaf.grad, ms().maxsim_rotary(t.ones_like(leaf), freq, inverse=True))
    assert ms().maxsim_rotary(buf[:0], freq).shape == (0, 9, 64)


def test_rotary_graph_and_stream():
    t = T()
    freq = (10000.0 ** (-t.arange(32, dtype=t.float64) / 32)).float().cuda()
    x = t.randn(333, 6, 64, device="cuda").half()
    off = t.tensor([0, 100, 333]).cuda()
    want = ms().maxsim_rotary(x, freq, off)
    out = t.empty_like(x)
    side = t.cuda.Stream()
    t.cuda.synchronize()
    got = ms().maxsim_rotary(x, freq, off, stream=side)
    side.synchronize()
    assert t.equal(got, want)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        ms().maxsim_rotary(x, freq, off, out=out)
    for _ in range(3):
        out.fill_(float("nan"))
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(out, want)


def grads(shapes, dtypes, seed=0, std=1e-3):
    t = T()
    g = t.Generator().manual_seed(seed)
    return [(t.randn(*s, generator=g) * std).to(dt(d)).cuda() for s, d in zip(shapes, dtypes)]


@pytest.mark.parametrize("max_norm", [0.0, 1e-3, 1e6])
@pytest.mark.parametrize("shapes, dtypes", [
    ([(1,)], ["fp32"]),
    ([(7, 3), (0,), (128, 320), (5,)], ["bf16", "fp32", "fp16", "fp32"]),
    ([(16384,), (16385,), (16383,)], ["fp16", "bf16", "fp32"]),
    ([(0,), (0, 4)], ["fp32", "bf16"]),
    ([(3,)] * 300 + [(100, 100)], ["fp32", "bf16", "fp16"] * 100 + ["bf16"]),
    ([(5_000_001,), (77,)], ["bf16", "fp32"]),
    ([(3,)] * 130 + [(17_000_003,), (9,)], ["fp16"] * 130 + ["bf16", "fp32"]),
])
def test_clip(shapes, dtypes, max_norm):
    t = T()
    say("case: clip", len(shapes), shapes[:4], max_norm)
    gs = grads(shapes, dtypes)
    norm, want = ref.clipped([ref.as64(x) for x in gs], max_norm)
    outs = [t.full_like(x, float("nan")) for x in gs]
    got = ms().maxsim_clip_grad_norm(gs, max_norm, out=outs)
    again = [x.clone() for x in gs]
    inplace = ms().maxsim_clip_grad_norm(again, max_norm)
    t.cuda.synchronize()
    assert got.shape == () and abs(float(got) - norm) <= 2 * ref.U32 * norm
    assert t.equal(got, inplace)
    for o, a, g, w in zip(outs, again, gs, want):
        assert t.equal(o, a)
        # the factor and the product round to 32 bits, the result to its type
        tol = (ref.HALF_STEP[g.dtype] + 3 * ref.U32) * np.abs(w) + ref.TINY[g.dtype]
        assert np.all(np.abs(ref.as64(o) - w) <= tol)
    if max_norm == 1e6:
        assert all(t.equal(o, g) for o, g in zip(outs, gs))


def test_clip_extremes():
    """Squares past fp32's range, views that start anywhere, NaN and infinity."""
    t = T()
    say("case: clip extremes")
    big = t.full((1000,), 1e30, device="cuda")
    assert abs(float(ms().maxsim_clip_grad_norm([big], 1.0)) / (1e30 * math.sqrt(1000)) - 1) < 1e-6
    assert abs(float(big[0]) * math.sqrt(1000) - 1) < 1e-6
    flat = t.randn(1000, device="cuda").half()
    odd = flat[3:778]  # 2-byte aligned only
    norm, want = ref.clipped([ref.as64(odd)], 0.5)
    before = flat.clone()
    got = ms().maxsim_clip_grad_norm([odd], 0.5)
    assert abs(float(got) - norm) <= 2 * ref.U32 * norm
    assert t.equal(flat[:3], before[:3]) and t.equal(flat[778:], before[778:])
    assert np.all(np.abs(ref.as64(odd) - want[0]) <= (2.0 ** -11 + 3 * ref.U32) * np.abs(want[0]) + 2.0 ** -25)
    x = t.ones(100, device="cuda")
    x[7] = math.nan
    y = t.ones(10, device="cuda")
    assert math.isnan(float(ms().maxsim_clip_grad_norm([x, y], 1.0))) and t.isnan(y).all()
    x = t.ones(100, device="cuda")
    x[7] = math.inf
    assert math.isinf(float(ms().maxsim_clip_grad_norm([x], 1.0)))
    assert math.isnan(float(x[7])) and float(x[0]) == 0.0
    g = [t.zeros(5, device="cuda")]
    assert float(ms().maxsim_clip_grad_norm(g, 1.0)) == 0.0 and not g[0].any()


def test_clip_same_bits_graph_and_stream():
    t = T()
    gs = grads([(700, 333), (5,), (3000,)], ["bf16", "fp32", "fp16"])
    outs = [t.empty_like(x) for x in gs]
    norm = t.empty((), device="cuda")
    ws = t.empty(ms().clip_grad_norm_workspace_size(3), dtype=t.uint8, device="cuda")
    want_norm = ms().maxsim_clip_grad_norm(gs, 1e-3, out=outs)
    want = [x.clone() for x in outs]
    side = t.cuda.Stream()
    t.cuda.synchronize()
    ms().maxsim_clip_grad_norm(gs, 1e-3, out=outs, stream=side)
    side.synchronize()
    assert all(t.equal(a, b) for a, b in zip(outs, want))
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        ms().maxsim_clip_grad_norm(gs, 1e-3, out=outs, norm=norm, workspace=ws)
    for _ in range(3):
        for x in outs:
            x.fill_(float("nan"))
        ws.fill_(255)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(norm, want_norm) and all(t.equal(a, b) for a, b in zip(outs, want))


def test_clip_leaves_out_parameters_without_a_gradient():
    t = T()
    gs = grads([(70, 33), (5,), (300,)], ["bf16", "fp32", "fp16"])
    outs = [t.empty_like(x) for x in gs]
    want_norm = ms().maxsim_clip_grad_norm(gs, 1e-3, out=outs)
    kept = t.full((4,), 7.0, device="cuda")
    got = [t.empty_like(x) for x in gs]
    say("case: clip with None")
    norm = ms().maxsim_clip_grad_norm([gs[0], None, *gs[1:], None], 1e-3,
                                      out=[got[0], kept, *got[1:], None])
    assert t.equal(norm, want_norm) and all(t.equal(a, b) for a, b in zip(got, outs))
    assert bool((kept == 7.0).all())
    inplace = [x.clone() for x in gs]
    assert t.equal(ms().maxsim_clip_grad_norm([None, *inplace], 1e-3), want_norm)
    assert all(t.equal(a, b) for a, b in zip(inplace, outs))
