"""The cross entropy and its gradients where the table, its gradient, the rows, theirs, or the parts that
they are joined from pass 4 GiB."""
import math

import numpy as np
import pytest
import torch

import maxsim_scoring_fwd_amd as ms
import train_ref as ref
from encoder_ref import HALF_STEP, TINY, U32, as64

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def rand(*shape, dtype=BF16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def weights(z, L, hot, size, d):
    """P before its gradient, and how far it may be off: the logit's error, the lse's rounding and the
    exponential's."""
    p = np.exp(z - L)
    return p - hot, p * ((d + 12) * U32 * size + 12 * U32 * (np.abs(z) + np.abs(L) + 1))


def check_dw(dw_v, h, w_v, v, labels, L, g, dtype):
    """Gradients dw_v of the entries numbered v, whose vectors are w_v, against 64 bits; every row counts."""
    H, u = as64(h), HALF_STEP[dtype]
    least = 2.0 ** -38 * np.abs(g).max() if dtype == FP16 else 2.0 ** -133
    got = as64(dw_v)
    for i, (e, W) in enumerate(zip(v, as64(w_v))):
        p, off = weights(H @ W, L, labels == e, np.abs(H) @ np.abs(W), H.shape[1])
        P, tP = p * g, np.abs(g) * (off + np.abs(p) * (u + len(H) * U32)) + least
        want = P @ H
        ref.close(got[i], want, tP @ np.abs(H) + u * np.abs(want) + TINY[dtype], f"dw of entry {e}")


V, D = 4500001, 512
EDGE = 4194304  # 4 GiB of rows of 512 in 16 bits


@pytest.fixture(scope="module")
def table():
    """500 vectors over and over, and another one at the end."""
    w = rand(500, D).repeat(V // 500 + 1, 1)[:V] * 0.05
    w[V - 1] = 0.5 * rand(D, seed=5)
    return w


def test_gradient_of_a_large_table(table):
    print("case: dw past 4 GiB", flush=True)
    w, n = table, 40
    h = rand(n, D, seed=6)
    y = torch.arange(n, device="cuda") * 100000 + 7
    y[7], y[8], y[9], y[10] = V - 1, EDGE - 1, EDGE, EDGE + 100
    dl = torch.linspace(-1, 2, n, device="cuda")
    _, lse = ms.maxsim_linear_cross_entropy(h, w, y)
    dw = torch.full_like(w, 3.0)
    ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse, want_dh=False, dw=dw)
    # the vocabulary goes in 5 pieces of 7032 tiles of 128
    v = sorted({0, 1, EDGE - 2, EDGE - 1, EDGE, EDGE + 1, V - 2, V - 1, *y.tolist(),
                *(900096 * k + i for k in range(1, 5) for i in (-1, 0))})
    check_dw(dw[v], h, w[v], v, y.cpu().numpy(), as64(lse), as64(dl), BF16)
    # entries with the same vector that are no row's label have the same gradient, bit for bit
    for e in y.tolist():
        if e < V - 1:
            dw[e] = dw[500 + e % 500]
    assert bool((dw[:V - 1].view(-1, 500, D) == dw[500:1000]).all())


def test_few_rows_of_a_large_table(table):
    """The kernel for up to 32 rows, with labels at both ends of the table."""
    print("case: few rows, table past 4 GiB", flush=True)
    w, n = table, 32
    h = rand(n, D, seed=6)
    y = torch.arange(n, device="cuda") * 140000
    y[7], y[8], y[9] = V - 1, EDGE - 1, EDGE
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y)
    z = h.double() @ w[:500].double().t()
    count = torch.full((500,), V // 500, device="cuda", dtype=torch.float64)
    count[:V % 500 - 1] += 1  # the last entry is another
    last = h.double() @ w[V - 1].double()
    want = torch.logsumexp(torch.cat([z + count.log(), last[:, None]], 1), 1)
    picked = z[torch.arange(n), y % 500]
    picked[7] = last[7]
    # sums of 4.5 million exponentials in parts of 32 and 128, a logit's error of 512 products
    size = (h.double().abs() @ w[:500].double().abs().t()).max()
    tol = 2.0 ** -24 * (float(size) * 600 + V / 128 / 32 + 600)
    assert float((lse.double() - want).abs().max()) <= tol and float((loss.double() - (want - picked)).abs().max()) <= 2 * tol


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
def test_rows_gradients_from_a_large_table(dtype):
    """dh = P w over a table of 4.4 GB, exactly. Rows of zeros have 2^22 equal logits, so that P is 2^-22
    times a gradient of a power of two, and p - 1 rounds to -1 at the label; with a table of zeros and
    ones every sum is a multiple of 2^-22 of up to 23 bits, which 32 bits hold."""
    print("case: dh from a table past 4 GiB", dtype, flush=True)
    n, vocab, d = 40, 1 << 22, 520
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(0, 2, (vocab, d), generator=g, device="cuda", dtype=torch.uint8).to(dtype)
    h = torch.zeros(n, d, device="cuda", dtype=dtype)
    y = torch.arange(n, device="cuda") * 107374 + 3
    y[5], y[6], y[7] = vocab - 1, (1 << 32) // (2 * d), 0
    dl = 2.0 ** -(torch.arange(n, device="cuda") % 5 + 2).float()
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y)
    assert float((lse - 22 * math.log(2)).abs().max()) <= 2.0 ** -18  # 22 log 2, which has steps of 2^-20
    dw = torch.full_like(w, 3.0)
    dh, _ = ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse, dw=dw)
    ones = torch.stack([w[a:a + (1 << 18)].double().sum(0) for a in range(0, vocab, 1 << 18)]).sum(0)
    label = w[y].double()
    want = dl.double()[:, None] * ((ones - label) * 2.0 ** -22 - label)
    assert torch.equal(dh, want.to(dtype))
    assert not dw.any()  # of rows of zeros


def test_parts_of_a_large_tables_gradient():
    """Many rows of few entries: dw's tiles are fewer than the workgroups and go in two parts, piece by piece
    of the vocabulary, up to past 4 GiB of it. The lse is the formula's, rounded."""
    print("case: parts of dw past 4 GiB", flush=True)
    n, d, vocab = 4352, 64, (1 << 25) + 1000
    w = rand(1000, d).repeat(vocab // 1000 + 1, 1)[:vocab] * 0.25
    h = rand(n, d, seed=1)
    y = torch.randint(0, vocab, (n,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    edge = 1 << 25  # 4 GiB of rows of 64
    y[0], y[1], y[2], y[3] = 0, edge - 1, edge, vocab - 1
    dl = torch.rand(n, device="cuda") / n
    count = torch.full((1000,), vocab // 1000, device="cuda", dtype=torch.float64)
    count[:vocab % 1000] += 1
    lse = torch.logsumexp(h.double() @ w[:1000].double().t() + count.log(), 1).float()
    dw = torch.full_like(w, 3.0)
    ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse, want_dh=False, dw=dw)
    # edges of tiles of 128, of which a piece has some 481
    v = sorted({0, 127, 128, edge - 1, edge, edge + 1, vocab - 2, vocab - 1,
                *(128 * t - i for t in (480, 481, 482, 963, 130000, 262144) for i in (0, 1)), *y[4:12].tolist()})
    check_dw(dw[v], h, w[v], v, y.cpu().numpy(), as64(lse), as64(dl), BF16)
    assert bool(torch.isfinite(dw).all())
    again = torch.full_like(w, 5.0)
    ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse, want_dh=False, dw=again)
    assert torch.equal(again, dw)


def test_many_rows():
    """2^22 rows of 520 entries, the most: h, its gathered copy and dh pass 4 GiB each, and dh's parts, whole
    tiles of 256 columns, take 12.9 GB."""
    print("case: rows past 4 GiB", flush=True)
    n, vocab, d = 1 << 22, 300, 520
    h = rand(1 << 12, d).repeat(1 << 10, 1)
    h[n - 1] = rand(d, seed=7)
    w = rand(vocab, d, seed=1) * 0.1
    y = torch.randint(0, vocab, (n,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    y[5] = -100
    dl = torch.rand(n, device="cuda")
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y)
    dh, _ = ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse, want_dw=False)
    edge = (1 << 32) // (2 * d)
    rows = [0, 1, 4, 5, 6, n // 2, edge - 1, edge, edge + 1, n - 2, n - 1]
    want = ref.loss(as64(h[rows]), as64(w), y[rows].cpu().numpy(), 1.0, as64(dl[rows]), BF16)
    ref.close(loss[rows], want["loss"], want["tol_loss"], "loss")
    ref.close(lse[rows], want["lse"], want["tol_lse"], "lse")
    ref.close(dh[rows], want["dh"], want["tol_dh"], "dh")
    # rows with the same vector and label have the same loss
    same = y[: 1 << 12].eq(y.view(-1, 1 << 12))
    same[-1, -1] = same[0, 5] = False
    got = loss.view(-1, 1 << 12)
    assert bool((got.eq(got[0]) | ~same).all())
    assert bool(torch.isfinite(dh).all()) and not dh[5].any()
