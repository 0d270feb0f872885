"""The norm, dropout, the cross entropy and the 4-bit vectors captured in graphs, on other streams,
and at the ends of their range: tensors past 4 GiB, steps that change between replays."""
import numpy as np
import pytest
import torch

import maxsim_scoring_fwd_amd as ms
import train_ref as ref
from encoder_ref import as64

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def rand(*shape, dtype=BF16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def norm_step():
    x, r, w, gy, gh = rand(999, 200), rand(999, 200, seed=1), rand(200, seed=2), rand(999, 200, seed=3), rand(999, 200, seed=4)
    rng = torch.tensor([3, 4], device="cuda")
    out = [torch.empty_like(x), torch.empty_like(x), torch.empty(999, device="cuda"), torch.empty_like(x),
           torch.empty_like(x), torch.empty_like(w)]
    ws = torch.empty(ms.rms_norm_backward_workspace_size(999, 200), dtype=torch.uint8, device="cuda")

    def step():
        ms.maxsim_rms_norm(x, w, r, 1e-6, 0.2, rng, 1, out[0], out[1], out[2])
        ms.maxsim_rms_norm_backward(gy, out[1], w, out[2], gh, 0.2, rng, 1, dx=out[3], dresidual=out[4],
                                    dweight=out[5], workspace=ws)
    return step, out, rng


def drop_step():
    x, rng = rand(100001), torch.tensor([3, 4], device="cuda")
    out = [torch.empty_like(x)]
    return lambda: ms.maxsim_dropout(x, 0.3, rng, 5, out[0]), out, rng


def loss_step(n, share):
    h, w = rand(n, 72), rand(3001, 72, seed=1)
    y = torch.randint(0, 3001, (n,), device="cuda")
    y[torch.rand(n, device="cuda") >= share] = -100
    dl = torch.rand(n, device="cuda")
    out = [torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(h), torch.empty_like(w)]
    ws = torch.empty(max(ms.linear_cross_entropy_backward_workspace_size(n, 3001, 72, BF16),
                         ms.linear_cross_entropy_workspace_size(n, 3001, 72, BF16)), dtype=torch.uint8, device="cuda")

    def step():  # both calls share a workspace, one after the other
        ms.maxsim_linear_cross_entropy(h, w, y, 1.0, out[0], out[1], ws)
        ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, out[1], 1.0, dh=out[2], dw=out[3], workspace=ws)
    return step, out, None


def index_step():
    x, w, q = rand(5000, 128), rand(128, seed=1, dtype=torch.float32), rand(32, 128, seed=2)
    off = torch.tensor([0, 17, 17, 3000, 5000], device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    code, scale = torch.empty(5000, 128, dtype=torch.int8, device="cuda"), torch.empty(5000, device="cuda")
    c, s, cq, sq = (torch.empty(*z, **u8) for z in ((5000, 64), (5000, 4), (32, 64), (32, 4)))
    out = [code, scale, c, s, torch.empty(4, device="cuda"), torch.empty_like(x)]

    def step():
        ms.maxsim_rms_norm_i8(x, w, out=code, scale=scale)
        ms.maxsim_quantize_mx4(x, c, s)
        ms.maxsim_quantize_mx4(q, cq, sq)
        ms.maxsim_score_mx4(cq, sq, c, s, off, out=out[4])
        ms.maxsim_dequantize_mx4(c, s, BF16, out[5])
    return step, out, None


STEPS = {"norm": norm_step, "dropout": drop_step, "loss": lambda: loss_step(1500, 0.5),
         "loss of few rows": lambda: loss_step(40, 0.9), "loss of many rows": lambda: loss_step(9001, 0.8),
         "index": index_step}


def bits(t):
    return t.detach().cpu().view(torch.uint8).clone() if t.numel() else t.cpu()


@pytest.mark.parametrize("name", list(STEPS))
def test_graph_replays_match_eager(name):
    """Replays of a captured step, with eager work between and outputs overwritten before each; where
    there is a generator its step goes up between replays, and the masks with it."""
    print("case: captured", name, flush=True)
    step, outs, rng = STEPS[name]()
    step()
    torch.cuda.synchronize()
    eager = [bits(t) for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for replay in range(5):
        for t in outs:
            t.view(torch.uint8).fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, bits(t)) for a, t in zip(eager, outs)), f"{name}: replay {replay}"
        if rng is not None:
            rng[1] += 1
        step()
        torch.cuda.synchronize()
        again = [bits(t) for t in outs]
        assert all(torch.equal(a, b) for a, b in zip(eager, again)) == (rng is None)
        eager = again


N, D = 4096, 128


@pytest.fixture(scope="module")
def data():
    x, r, w, q = rand(N, D), rand(N, D, seed=1), rand(D, seed=2), rand(32, D, seed=3)
    rng, y = torch.tensor([3, 4], device="cuda"), torch.randint(-500, 2000, (N,), device="cuda")
    V = rand(2000, D, seed=4)
    _, h, rstd = ms.maxsim_rms_norm(x, w, r)
    loss, lse = ms.maxsim_linear_cross_entropy(x, V, y)
    c, s = ms.maxsim_quantize_mx4(x)
    long = torch.randn(8192, 8192, device="cuda")
    torch.mm(long, long)
    torch.cuda.synchronize()
    return dict(x=x, r=r, w=w, q=q, rng=rng, y=y, V=V, h=h, rstd=rstd, lse=lse, c=c, s=s, long=long,
                dl=torch.rand(N, device="cuda"))


CALLS = {
    "norm": lambda z, s: ms.maxsim_rms_norm(z["x"], z["w"], z["r"], 1e-6, 0.1, z["rng"], stream=s),
    "norm 8 bits": lambda z, s: ms.maxsim_rms_norm_i8(z["x"], z["w"], z["r"], stream=s),
    "norm backward": lambda z, s: ms.maxsim_rms_norm_backward(z["r"], z["h"], z["w"], z["rstd"], z["x"], 0.1, z["rng"], stream=s),
    "dropout": lambda z, s: [ms.maxsim_dropout(z["x"], 0.1, z["rng"], stream=s)],
    "loss": lambda z, s: ms.maxsim_linear_cross_entropy(z["x"], z["V"], z["y"], stream=s),
    "loss backward": lambda z, s: ms.maxsim_linear_cross_entropy_backward(z["dl"], z["x"], z["V"], z["y"], z["lse"], stream=s),
    "quantise": lambda z, s: ms.maxsim_quantize_mx4(z["x"], stream=s),
    "values": lambda z, s: [ms.maxsim_dequantize_mx4(z["c"], z["s"], BF16, stream=s)],
    "score": lambda z, s: [ms.maxsim_score_mx4(z["c"][:32], z["s"][:32], z["c"].view(64, 64, -1), z["s"].view(64, 64, -1), stream=s)],
}


@pytest.mark.parametrize("as_int", [False, True])
@pytest.mark.parametrize("name", list(CALLS))
def test_buffers_of_another_stream(data, name, as_int):
    """A call on another stream neither writes to blocks that the current stream still reads, nor
    are its results handed out before the current stream is past them."""
    print("case: another stream", name, flush=True)
    call = CALLS[name]
    want = [t.clone() for t in call(data, None)]
    side = torch.cuda.Stream()
    handle = side.cuda_stream if as_int else side
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.full_like(t, 3) for t in want]
    torch.cuda.synchronize()
    for _ in range(4):
        torch.mm(data["long"], data["long"])
    kept = [t.clone() for t in old]
    at = {t.data_ptr() for t in old}
    del old
    got = call(data, handle)
    assert not at & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(bool((t == 3).all()) for t in kept)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = call(data, handle)
    side.synchronize()
    for _ in range(4):
        torch.mm(data["long"], data["long"])
    kept = [t.clone() for t in got]
    at = {t.data_ptr() for t in got}
    del got
    again = call(data, handle)
    assert not at & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))
    assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_two_calls_at_once(data):
    """Two losses and two norms on two streams at the same time."""
    want = [[t.clone() for t in CALLS[n](data, None)] for n in ("loss backward", "norm backward")]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in sides:
            got.append([CALLS[n](data, s) for n in ("loss backward", "norm backward")])
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_norm_and_dropout_past_4_gib():
    n, d = 2300003, 1000  # 4.6 GB
    x = rand(1000, d).repeat(n // 1000 + 1, 1)[:n]
    w, rng = rand(d, seed=1), torch.tensor([9, 9], device="cuda")
    y, _, rstd = ms.maxsim_rms_norm(x, w)
    want = ms.maxsim_rms_norm(x[:1000], w)
    assert torch.equal(y[n - 3:], want[0][n % 1000 - 3:n % 1000]) and torch.equal(y[2000000:2001000], want[0])
    dx = ms.maxsim_rms_norm_backward(y, x, w, rstd, dx=y, want_dweight=False, want_dresidual=False)[0]
    want = ms.maxsim_rms_norm_backward(want[0], x[:1000], w, want[2], want_dweight=False, want_dresidual=False)[0]
    assert torch.equal(dx[2299000:2300000], want)
    del dx, rstd
    ms.maxsim_dropout(x, 0.5, rng, out=y)
    first = (n - 5) * d
    keep, up = ref.kept(rng.tolist(), 0, 0.5, 1, 5 * d, first // 8)
    assert first % 8 == 0
    z = torch.where(torch.from_numpy(keep).view(5, d), x[n - 5:].cpu().float() * torch.tensor(up), torch.zeros(())).to(BF16)
    assert torch.equal(y[n - 5:].cpu(), z)


def test_loss_past_4_gib():
    """A vocabulary of 4.6 GB, and rows whose gradients pass 4 GiB."""
    V, d = 4500001, 512
    w = rand(500, d).repeat(V // 500 + 1, 1)[:V] * 0.05
    w[V - 1] = 0.5 * rand(d, seed=5)
    h = rand(40, d, seed=6)
    y = torch.arange(40, device="cuda") * 100000
    y[7] = V - 1
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y)
    z = h.double() @ w[:500].double().t()
    count = torch.full((500,), V // 500, device="cuda", dtype=torch.float64)
    count[:V % 500 - 1] += 1  # the last entry is another
    last = h.double() @ w[V - 1].double()
    want = torch.logsumexp(torch.cat([z + count.log(), last[:, None]], 1), 1)
    picked = z[torch.arange(40), y % 500]
    picked[7] = last[7]
    # sums of 4.5 million exponentials in parts of 32 and 128, a logit's error of 512 products
    size = (h.double().abs() @ w[:500].double().abs().t()).max()
    tol = 2.0 ** -24 * (float(size) * 600 + V / 128 / 32 + 600)
    assert float((lse.double() - want).abs().max()) <= tol and float((loss.double() - (want - picked)).abs().max()) <= 2 * tol


def test_index_past_4_gib():
    n = 50000003  # tokens of 128: 6.4 GB of values, 3.2 GB of codes; scores' codes repeated past 4 GiB
    x = rand(1000, 128)
    c, s = ms.maxsim_quantize_mx4(x)
    want = ms.maxsim_dequantize_mx4(c, s, BF16)
    big = x.repeat(n // 1000 + 1, 1)[:n]
    C, S = ms.maxsim_quantize_mx4(big)
    assert torch.equal(C[n - 3:], c[n % 1000 - 3:n % 1000]) and torch.equal(S[40000000:40001000], s)
    ms.maxsim_dequantize_mx4(C, S, BF16, out=big)
    assert torch.equal(big[49999000:50000000], want) and torch.equal(big[n - 3:], want[n % 1000 - 3:n % 1000])
    del big
    C, S = torch.cat([C, C]), torch.cat([S, S])
    off = torch.tensor([0, 1000, 2000, 2 * n - 100, 2 * n - 60, 2 * n], device="cuda")
    got = ms.maxsim_score_mx4(c[:20], s[:20], C, S, off)
    tail = torch.cat([c, c, c])[n % 1000 + 900:][:100], torch.cat([s, s, s])[n % 1000 + 900:][:100]
    small = ms.maxsim_score_mx4(c[:20], s[:20], *tail, torch.tensor([0, 40, 100], device="cuda"))
    one = ms.maxsim_score_mx4(c[:20], s[:20], c, s, torch.tensor([0, 1000], device="cuda"))
    assert torch.equal(got[3:], small) and torch.equal(got[:1], one) and torch.equal(got[2:3], one)
