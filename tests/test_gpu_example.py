"""The example encoder: trains, searches, and its gradients are those of plain torch operators."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_encoder.py")
    spec = importlib.util.spec_from_file_location("train_encoder", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_trains_and_searches(example):
    print("case: example, 100 steps", flush=True)
    before, _ = example.search(example.train(0)[1])
    losses, encoder = example.train(100, report=lambda line: print(line, flush=True))
    assert all(math.isfinite(x) for x in losses)
    assert sum(losses[-20:]) < 0.8 * sum(losses[:20])
    found, best = example.search(encoder)
    assert found > before and len(best) == 5


def plain_rotary(x, freq, offsets):
    off = offsets.tolist()
    pos = torch.cat([torch.arange(b - a, device=x.device) for a, b in zip(off[:-1], off[1:])])
    ang = pos[:, None].double() * freq.double()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x.double().chunk(2, dim=-1)
    return torch.cat([a * c - b * s, a * s + b * c], dim=-1).to(x.dtype)


def plain_attention(q, k, v, offsets):
    off = offsets.tolist()
    g = q.shape[1] // k.shape[1]
    outs = []
    for a, b in zip(off[:-1], off[1:]):
        qd, kd, vd = (t[a:b].double().transpose(0, 1).contiguous() for t in (q, k, v))
        kd, vd = kd.repeat_interleave(g, 0), vd.repeat_interleave(g, 0)
        p = torch.softmax(torch.bmm(qd, kd.transpose(1, 2).contiguous()) * q.shape[-1] ** -0.5, -1)
        outs.append(torch.bmm(p, vd).transpose(0, 1))
    return torch.cat(outs).to(q.dtype)


def test_step_matches_plain_operators(example, monkeypatch):
    """The same loss and gradients with rotary and attention replaced by 64-bit torch, in fp32
    storage: in bf16 a rounding that changes which document token is a query token's best would
    change the gradient by all of that token's share. Some 40 sums of up to 1024 terms follow each
    other, each off by 2^-24 * sqrt(1024), and the temperature multiplies the scores by 20."""
    print("case: example, one step against plain operators", flush=True)
    monkeypatch.setattr(example, "BF16", torch.float32)
    tol = 40 * 32 * 20 * 2.0 ** -24
    torch.manual_seed(0)
    encoder = example.Encoder(500).cuda()
    data = example.batch(6, 500, 32, torch.Generator().manual_seed(3))

    def step():
        encoder.zero_grad()
        loss = example.loss_of(encoder, *data, 32)
        loss.backward()
        return float(loss.detach()), [p.grad.double().clone() for p in encoder.parameters()]

    loss, grads = step()
    monkeypatch.setattr(example.ms, "rotary", plain_rotary)
    monkeypatch.setattr(example.ms, "attention", plain_attention)
    want_loss, want = step()
    assert abs(loss - want_loss) <= tol * want_loss
    for g, w in zip(grads, want):
        assert float((g - w).norm()) <= tol * float(w.norm())
