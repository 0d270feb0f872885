"""The operators together, as a program uses them: the example's masked-token training step against
plain operators, its index in 8 and 4 bits, and a step of all of them captured in a graph."""
import importlib.util
import math
import os

import pytest
import torch

import maxsim_scoring_fwd_amd as ms
from test_gpu_example import plain_attention, plain_rotary

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_encoder.py")
    spec = importlib.util.spec_from_file_location("train_encoder", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_norm(x, w, residual=None, eps=1e-6, dropout=0.0, rng=None, call=0):
    h = x.double()
    if dropout:  # the mask itself is checked elsewhere
        h = h * ms.maxsim_dropout(torch.ones_like(x), dropout, rng, call).double()
    if residual is not None:
        h = h + residual.double()
    y = h * (h.square().mean(-1, keepdim=True) + eps).rsqrt() * w.double()
    return y.to(x.dtype), h.to(x.dtype)


def plain_loss(h, w, labels, scale=1.0):
    z = scale * (h.double() @ w.double().t())
    keep = labels >= 0
    picked = z.gather(1, labels.clamp(min=0)[:, None])[:, 0]
    return torch.where(keep, torch.logsumexp(z, 1) - picked, torch.zeros_like(picked)).float()


def test_masked_step_matches_plain_operators(example, monkeypatch):
    """Loss and gradients with the norm, rotary positions, attention and the loss replaced by 64-bit
    torch, in fp32 storage, dropout included. Some 40 sums of up to 1024 terms follow each other,
    each off by 2^-24 * sqrt(1024), as in the retrieval step but without its temperature."""
    print("case: masked step against plain operators", flush=True)
    monkeypatch.setattr(example, "BF16", torch.float32)
    tol = 40 * 32 * 2.0 ** -24 * 4
    torch.manual_seed(0)
    encoder = example.Encoder(500).cuda()
    data = example.masked_batch(5, 500, torch.Generator().manual_seed(3))
    masks = torch.tensor([77, 3], device="cuda")

    def step():
        encoder.zero_grad()
        loss = encoder.masked_loss(*data, 0.2, masks)
        loss.backward()
        return float(loss.detach()), [p.grad.double().clone() for p in encoder.parameters() if p.grad is not None]

    loss, grads = step()
    for name, f in (("rotary", plain_rotary), ("attention", plain_attention), ("rms_norm", plain_norm),
                    ("linear_cross_entropy", plain_loss)):
        monkeypatch.setattr(example.ms, name, f)
    want_loss, want = step()
    assert len(grads) == len(want) == len(list(encoder.parameters())) - 1  # all but the projection
    assert abs(loss - want_loss) <= tol * want_loss
    for g, w in zip(grads, want):
        assert float((g - w).norm()) <= tol * float(w.norm())


def test_trains_with_masks_and_searches_every_index(example):
    print("case: example, masked steps and indexes", flush=True)
    losses, encoder = example.train(30, masked=20, report=lambda line: print(line, flush=True))
    assert all(math.isfinite(x) for x in losses)
    for kind in ("bf16", "int8", "mx4"):
        found, best = example.search(encoder, index=kind)
        assert 0 <= found <= 20 and len(set(best)) == 5 and all(0 <= b < 200 for b in best)


def test_index_scores_are_those_of_the_vectors_it_stands_for(example):
    """Scores of an 8-bit and a 4-bit index against those of the values that its codes stand for."""
    g = torch.Generator().manual_seed(4)
    D = torch.nn.functional.normalize(torch.randn(500, 128, generator=g), dim=-1).bfloat16().cuda()
    Q = torch.nn.functional.normalize(torch.randn(32, 128, generator=g), dim=-1).bfloat16().cuda()
    off = torch.tensor([0, 100, 101, 300, 500], device="cuda")
    for kind in ("int8", "mx4"):
        index = example.Index(D, off, kind)
        values = {"int8": lambda c, s: c.double() * s.double()[:, None],
                  "mx4": lambda c, s: ms.maxsim_dequantize_mx4(c, s).double()}[kind]
        q, d = values(*index.store(Q)), values(*index.stored)
        want = torch.stack([(q @ d[a:b].t()).max(1).values.sum() for a, b in zip(off.tolist()[:-1], off.tolist()[1:])])
        # 32 sums of 128 products in 32 bits
        tol = 2.0 ** -24 * 140 * float((q.abs() @ d.abs().t()).max() * 32)
        assert float((index.scores(Q).double() - want).abs().max()) <= tol


@pytest.mark.parametrize("kind", ["bf16", "int8", "mx4"])
def test_search_finds_what_plain_scores_find(example, monkeypatch, kind):
    """Each query of a search: its scores are those of the vectors that the index stands for in 64 bits, and the
    documents found and the best five are the plain scores' own, but where two of them are as near to
    each other as the sums' rounding."""
    print("case: search", kind, flush=True)
    _, encoder = example.train(5, masked=5, report=lambda line: None)
    values = {"bf16": lambda x: x.double(), "int8": lambda c, s: c.double() * s.double()[:, None],
              "mx4": lambda c, s: ms.maxsim_dequantize_mx4(c, s).double()}[kind]
    scores, plain, tol = example.Index.scores, [], 0.0

    def checked(index, Q):
        nonlocal tol
        got = scores(index, Q)
        s = values(*index.store(Q)) @ values(*index.stored).t()
        off = index.offsets.tolist()
        plain.append(torch.stack([s[:, a:b].max(1).values.sum() for a, b in zip(off[:-1], off[1:])]))
        # unit vectors (in 8 bits sqrt(128) long): 32 sums of 128 products in 32 bits
        tol = max(tol, 2.0 ** -24 * 140 * 32 * (128.0 if kind == "int8" else 1.0) * 1.25)
        assert float((got.double() - plain[-1]).abs().max()) <= tol
        return got
    monkeypatch.setattr(example.Index, "scores", checked)
    found, best = example.search(encoder, index=kind)
    assert len(plain) == 20
    first = [(float(p[i]), float(torch.cat([p[:i], p[i + 1:]]).max())) for i, p in enumerate(plain)]
    assert sum(a > b + 2 * tol for a, b in first) <= found <= sum(a >= b - 2 * tol for a, b in first)
    p = plain[-1]
    assert len(set(best)) == 5
    order = torch.sort(p, descending=True).values[:5]
    assert float((p[best] - order).abs().max()) <= 2 * tol


def test_a_whole_step_captured():
    """Norm, rotary positions, attention, norm, loss, and all their gradients in one graph: replays
    are the eager step's bits, with the masks of each replay's own step."""
    print("case: a whole step captured", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    n, H, d, V = 700, 4, 64, 900
    dim = H * d

    def rand(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()
    x, r, w1, w2, table = rand(n, dim), rand(n, dim), rand(dim), rand(dim), rand(V, dim, std=0.1)
    off = torch.tensor([0, 200, 201, 500, n], device="cuda")
    y = torch.randint(-200, V, (n,), generator=g, device="cuda")
    dl, rng = torch.rand(n, generator=g, device="cuda"), torch.tensor([5, 0], device="cuda")
    freq = (100.0 ** -torch.linspace(0, 1, d // 2)).cuda()
    out = [torch.empty_like(x), torch.empty_like(w1), torch.empty_like(table), torch.empty(n, device="cuda")]

    def step():
        a, h, s = ms.maxsim_rms_norm(x, w1, r, dropout=0.1, rng=rng, call=0)
        t = ms.maxsim_rotary(a.view(n, H, d), freq, off)
        o, lse = ms.maxsim_attention(t, t, a.view(n, H, d), off)
        b, h2, s2 = ms.maxsim_rms_norm(o.view(n, dim), w2, h, dropout=0.1, rng=rng, call=1)
        loss, z = ms.maxsim_linear_cross_entropy(b, table, y)
        db, _ = ms.maxsim_linear_cross_entropy_backward(dl, b, table, y, z, dw=out[2])
        do, dh, _ = ms.maxsim_rms_norm_backward(db, h2, w2, s2, dropout=0.1, rng=rng, call=1)
        dq, dk, dv = ms.maxsim_attention_backward(do.view(n, H, d), t, t, a.view(n, H, d), o, lse, off)
        da = ms.maxsim_rotary(dq + dk, freq, off, inverse=True) + dv
        ms.maxsim_rms_norm_backward(da.view(n, dim), h, w1, s, dh, 0.1, rng, 0, dx=out[0], dweight=out[1])
        out[3].copy_(loss)

    def bits():
        torch.cuda.synchronize()
        return [t.clone() for t in out]
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = []
    for _ in range(4):
        rng[1] += 1
        step()
        want = bits()
        for t in out:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(bits(), want))
        assert not any(torch.equal(want[0], s) for s in seen)
        seen.append(want[0])
