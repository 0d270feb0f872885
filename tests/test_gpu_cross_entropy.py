"""The cross entropy over a vocabulary and its gradients against a 64-bit reference."""
import math

import numpy as np
import pytest
import torch

import maxsim_scoring_fwd_amd as ms
import train_ref as ref
from encoder_ref import as64

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def make(n, vocab, d, dtype, share=1.0, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = (torch.randn(n, d, generator=g, device="cuda") * std).to(dtype)
    w = (torch.randn(vocab, d, generator=g, device="cuda") * 2 * d ** -0.5).to(dtype)
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    y[torch.rand(n, generator=g, device="cuda") >= share] = -100
    return h, w, y


def check(h, w, y, scale=1.0, dl=None, backward=True):
    n = h.shape[0]
    if dl is None:
        dl = torch.linspace(-1, 2, n, device="cuda") / n
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y, scale)
    want = ref.loss(as64(h), as64(w), y.cpu().numpy(), scale, as64(dl) if backward else None, h.dtype)
    ref.close(loss, want["loss"], want["tol_loss"], "loss")
    ref.close(lse, want["lse"], want["tol_lse"], "lse")
    if backward:
        dh, dw = ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse, scale)
        ref.close(dh, want["dh"], want["tol_dh"], "dh")
        ref.close(dw, want["dw"], want["tol_dw"], "dw")
    return loss, lse


@pytest.mark.parametrize("n, vocab, d, dtype, share", [
    (1, 1, 8, BF16, 1.0),          # one entry: loss 0
    (1, 300, 64, BF16, 1.0),
    (7, 1000, 40, FP16, 1.0),      # a last step along d that is not whole
    (33, 257, 72, BF16, 1.0),      # one entry past a tile, one row past a small tile
    (32, 700, 104, FP16, 0.8),     # as many rows as the smallest tile has
    (31, 129, 52, FP32, 1.0),
    (128, 300, 200, FP32, 0.9),    # as many as the next one
    (128, 1000, 96, FP16, 1.0),
    (64, 777, 256, FP32, 1.0),
    (65, 500, 320, BF16, 1.0),     # the first size of the large tiles
    (129, 255, 24, FP16, 0.5),
    (200, 5000, 768, BF16, 0.7),
    (300, 1025, 1032, FP32, 0.15),
    (1023, 511, 128, FP16, 0.9),
    (1025, 513, 36, FP32, 0.5),    # more rows than one count
    (3000, 700, 88, BF16, 0.02),
    (300, 50001, 24, BF16, 1.0),   # tiles of 256 rows: more than 384 of them
    (257, 27000, 72, FP16, 0.8),
    (513, 17001, 36, FP32, 1.0),
    (3000, 5001, 40, BF16, 0.3),
])
def test_against_reference(n, vocab, d, dtype, share):
    print("case: cross entropy", n, vocab, d, dtype, share, flush=True)
    check(*make(n, vocab, d, dtype, share, seed=n), scale=0.7 if n % 2 else 1.0)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
@pytest.mark.parametrize("n", [20, 40, 300, 25000])
def test_rows_left_out_hide_what_they_hold(n, dtype):
    """NaN and infinities in rows without a label change nothing; labels of all sizes that are none."""
    h, w, y = make(n, 400, 96, dtype, 0.6, seed=3)
    out = y < 0
    bad = torch.tensor([-1, -100, 400, 1 << 40, -(1 << 63), (1 << 63) - 1], device="cuda")
    y[out] = bad[torch.arange(int(out.sum()), device="cuda") % 6]
    dl = torch.rand(n, device="cuda") + 0.5
    want = [*ms.maxsim_linear_cross_entropy(h, w, y)]
    want += ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, want[1])
    check(h, w, y, dl=dl)
    x = h.clone()
    x[out] = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda", dtype=dtype).repeat(32)
    dl = torch.where(out, torch.full_like(dl, float("nan")), dl)
    got = [*ms.maxsim_linear_cross_entropy(x, w, y)]
    got += ms.maxsim_linear_cross_entropy_backward(dl, x, w, y, got[1])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert not got[0][out].any() and (got[1][out] == -float("inf")).all() and not got[2][out].any()


@pytest.mark.parametrize("n", [1, 64, 65, 2000, 9000])
def test_no_row_counts(n):
    h, w, _ = make(n, 300, 64, BF16)
    y = torch.full((n,), -100, device="cuda")
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y)
    assert not loss.any() and (lse == -float("inf")).all()
    dh, dw = ms.maxsim_linear_cross_entropy_backward(torch.ones(n, device="cuda"), h, w, y, lse,
                                                     dh=torch.ones_like(h), dw=torch.ones_like(w))
    assert not dh.any() and not dw.any()


def test_no_rows():
    h, w = torch.zeros(0, 64, device="cuda"), torch.ones(300, 64, device="cuda")
    y = torch.zeros(0, dtype=torch.int64, device="cuda")
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y)
    dh, dw = ms.maxsim_linear_cross_entropy_backward(loss, h, w, y, lse, dw=w.clone())
    assert loss.shape == lse.shape == (0,) and dh.shape == (0, 64) and not dw.any()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
@pytest.mark.parametrize("size", [1e-7, 1e3])
def test_sizes_of_gradients(size, dtype):
    """Gradients of the losses far from 1, some 0, of both signs; fp16's results may pass its range."""
    h, w, y = make(150, 700, 64, dtype, 0.8, seed=9)
    dl = torch.linspace(-1, 1, 150, device="cuda") * size
    dl[::7] = 0
    if dtype == FP16 and size > 1:
        w *= 0.05  # so that dh stays in range
        h *= 0.05
    check(h, w, y, 2.0, dl)


def test_large_logits():
    """Scores of some thousands: the exponentials of all but a few are 0."""
    h, w, y = make(200, 1000, 128, FP32, seed=4, std=8.0)
    check(h, w, y, 20.0)


def test_one_direction_only_and_given_buffers():
    h, w, y = make(100, 333, 64, BF16, 0.7)
    dl = torch.rand(100, device="cuda")
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y)
    dh, dw = ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse)
    a = ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse, want_dw=False)
    b = ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse, want_dh=False)
    assert a[1] is None and b[0] is None and torch.equal(a[0], dh) and torch.equal(b[1], dw)
    size = ms.linear_cross_entropy_backward_workspace_size(100, 333, 64, BF16)
    ws = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    big = torch.full((337, 64), 3.0, dtype=BF16, device="cuda")
    top = torch.full((104, 64), 3.0, dtype=BF16, device="cuda")
    ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse, dh=top[2:102], dw=big[2:335], workspace=ws[:size])
    assert torch.equal(top[2:102], dh) and torch.equal(big[2:335], dw)
    assert (top[[0, 1, 102, 103]] == 3).all() and (big[[0, 1, 335, 336]] == 3).all() and (ws[size:] == 0x5A).all()
    size = ms.linear_cross_entropy_workspace_size(100, 333, 64, BF16)
    ws = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    outs = torch.full((2, 104), 3.0, device="cuda")
    ms.maxsim_linear_cross_entropy(h, w, y, loss=outs[0, :100], lse=outs[1, :100], workspace=ws[:size])
    assert torch.equal(outs[0, :100], loss) and torch.equal(outs[1, :100], lse)
    assert (outs[:, 100:] == 3).all() and (ws[size:] == 0x5A).all()


@pytest.mark.parametrize("vocab", [4001, 9001])  # tiles of 128 and of 256 rows
def test_repeated_calls_give_the_same_bits(vocab):
    h, w, y = make(3000, vocab, 264, BF16, 0.9)
    dl = torch.rand(3000, device="cuda")
    first = [*ms.maxsim_linear_cross_entropy(h, w, y)]
    first += ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, first[1])
    for _ in range(4):
        loss, lse = ms.maxsim_linear_cross_entropy(h, w, y)
        again = [loss, lse, *ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def part_of_gradients(h, w, y, lse, dl, scale, dh, dw, rows, vocab):
    """dh of some rows and dw of some entries against 64 bits, with the lse given (it is checked
    elsewhere): each needs one row or column of P."""
    n, V = len(y), w.shape[0]
    H, W, labels, L, g = as64(h), as64(w), y.cpu().numpy(), as64(lse), as64(dl)
    ok = (labels >= 0) & (labels < V)
    u = ref.HALF_STEP[h.dtype]
    f = np.where(ok, g * scale, 0)
    least = 2.0 ** -38 * np.abs(f).max() if h.dtype == FP16 else 2.0 ** -133

    def weights(z, L, hot, size):
        """P before its gradient, and how far it may be off: the logit's error, the lse's rounding and
        the exponential's."""
        p = np.exp(z - L)
        off = p * ((h.shape[1] + 12) * ref.U32 * size + 12 * ref.U32 * (np.abs(z) + np.abs(L) + 1))
        return p - hot, off
    for i in rows:
        if not ok[i]:
            assert not dh[i].any()
            continue
        p, off = weights(scale * (W @ H[i]), L[i], np.arange(V) == labels[i], scale * (np.abs(W) @ np.abs(H[i])))
        P, tP = p * f[i], np.abs(f[i]) * (off + np.abs(p) * (u + V * ref.U32)) + least
        want = P @ W
        ref.close(dh[i], want, tP @ np.abs(W) + u * np.abs(want) + ref.TINY[h.dtype], f"dh of row {i}")
    for v in vocab:
        p, off = weights(scale * (H[ok] @ W[v]), L[ok], labels[ok] == v, scale * (np.abs(H[ok]) @ np.abs(W[v])))
        P, tP = p * f[ok], np.abs(f[ok]) * (off + np.abs(p) * (u + n * ref.U32)) + least
        want = P @ H[ok]
        ref.close(dw[v], want, tP @ np.abs(H[ok]) + u * np.abs(want) + ref.TINY[h.dtype], f"dw of entry {v}")


@pytest.mark.parametrize("n, vocab, d, dtype, share", [
    (20011, 14001, 64, BF16, 1.0),    # more than one piece of the vocabulary
    (9000, 33001, 40, FP16, 0.95),    # the same with a part of the rows left out
    (9001, 16001, 20, FP32, 1.0),
    (40000, 20001, 32, BF16, 0.1),    # pieces for all rows, one for those that count
])
def test_pieces_of_the_vocabulary(n, vocab, d, dtype, share):
    print("case: pieces", n, vocab, d, dtype, share, flush=True)
    h, w, y = make(n, vocab, d, dtype, share, seed=n)
    dl = torch.rand(n, device="cuda") / n
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y)
    dh, dw = ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse)
    rows = [0, 1, n // 2, n - 1]
    want = ref.loss(as64(h[rows]), as64(w), y[rows].cpu().numpy(), 1.0)
    ref.close(loss[rows], want["loss"], want["tol_loss"], "loss")
    ref.close(lse[rows], want["lse"], want["tol_lse"], "lse")
    edge = [c + i for c in range(0, vocab, 128) for i in (0, 127) if c % 1024 == 0 or abs(c - vocab / 2) < 400]
    edge = [v for v in edge if v < vocab] + [vocab - 1]
    part_of_gradients(h, w, y, lse, dl, 1.0, dh, dw, rows, edge)
    assert torch.isfinite(dh).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("n, vocab, d, dtype, share", [
    (4100, 300, 128, BF16, 1.0),
    (8192, 129, 264, FP16, 0.97),
    (2500, 513, 36, FP32, 0.9),
    (9000, 100, 512, BF16, 0.03),     # as many rows, few that count
])
def test_many_rows_of_a_small_vocabulary(n, vocab, d, dtype, share):
    """So few tiles of dw that their sums over the rows go in parts; each direction alone too, within
    the workspace."""
    print("case: many rows", n, vocab, d, dtype, share, flush=True)
    h, w, y = make(n, vocab, d, dtype, share, seed=n)
    dl = torch.linspace(-1, 2, n, device="cuda") / n
    loss, lse = check(h, w, y, 0.8, dl)
    want = ref.loss(as64(h), as64(w), y.cpu().numpy(), 0.8, as64(dl), h.dtype)
    size = ms.linear_cross_entropy_backward_workspace_size(n, vocab, d, dtype)
    for dh, dw in ((True, False), (False, True), (True, True)):
        ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every type
        got = ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse, 0.8, dh, dw, workspace=ws[:size])
        for g, name in zip(got, ("dh", "dw")):
            if g is not None:
                ref.close(g, want[name], want["tol_" + name], name)
        assert (ws[size:] == 0xFF).all()


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
@pytest.mark.parametrize("n", [300, 1009])
def test_a_means_gradients_keep_their_size(n, dtype):
    """1 / n is no number of 16 bits, and its rounding would move all gradients by up to half a step:
    what they are along the exact ones is within 2^-13. (P at a label is p - 1, rounded to -1: p is some
    2^-14. All other roundings point anywhere, and average over 19200 entries and more.)"""
    h, w, y = make(n, 20000, 64, dtype, seed=n, std=0.25)
    dl = torch.full((n,), 1.0 / n, device="cuda")
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y)
    dh = ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse)[0]
    want = ref.loss(as64(h), as64(w), y.cpu().numpy(), 1.0, as64(dl), dtype)["dh"]
    assert abs((as64(dh) * want).sum() / (want * want).sum() - 1) <= 2.0 ** -13


def test_few_tiles_in_several_pieces():
    n, vocab, d = 70001, 4200, 64
    h, w, y = make(n, vocab, d, BF16, seed=8)
    dl = torch.rand(n, device="cuda") / n
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y)
    dh, dw = ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse)
    part_of_gradients(h, w, y, lse, dl, 1.0, dh, dw, [0, 35000, n - 1], [*range(0, vocab, 127), vocab - 1])
    again = ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=str)
def test_autograd(dtype):
    h, w, y = make(77, 200, 64, dtype, 0.7)
    h.requires_grad_(), w.requires_grad_()
    count = (y >= 0).sum()
    loss = ms.linear_cross_entropy(h, w, y, 1.5)
    got = torch.autograd.grad(loss.sum() / count, (h, w))  # an expanded gradient
    l, lse = ms.maxsim_linear_cross_entropy(h.detach(), w.detach(), y, 1.5)
    want = ms.maxsim_linear_cross_entropy_backward(torch.ones_like(l) / count, h.detach(), w.detach(), y, lse, 1.5)
    assert torch.equal(loss.detach(), l) and all(torch.equal(a, b) for a, b in zip(got, want))
    (dh,) = torch.autograd.grad(ms.linear_cross_entropy(h, w.detach(), y, 1.5).sum() / count, h)
    assert torch.equal(dh, want[0])
    (g,) = torch.autograd.grad(ms.linear_cross_entropy(h, w, y).sum(), h, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        g.sum().backward()


def test_gradients_against_differences():
    """fp32 values along a direction: central differences of step 2^-5 are off by its square (the
    loss's third derivatives along a unit-size direction are below 1) and by some 2^-22 of the loss
    over 2^-5."""
    h, w, y = make(50, 300, 64, FP32, 0.8, seed=2)
    dl = torch.rand(50, device="cuda") - 0.3
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y)
    g = ms.maxsim_linear_cross_entropy_backward(dl, h, w, y, lse)
    e = 2.0 ** -5
    for i in (0, 1):
        t = torch.randn(g[i].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i))
        t /= 8  # rows of about unit length
        side = []
        for s in (e, -e):
            a = [h, w]
            a[i] = a[i] + s * t
            side.append(float((ms.maxsim_linear_cross_entropy(*a, y)[0].double() * dl).sum()))
        got, want = (side[0] - side[1]) / (2 * e), float((g[i].double() * t).sum())
        size = float((g[i].double() * t).abs().sum()) + float(dl.abs().sum())
        assert abs(got - want) <= size * (e * e + 2.0 ** -22 / e * 8)


def rows_with_a_leader(scale, n=300, vocab=700, seed=0):
    """h and w of whole numbers, so that products are exact: each row's logits are 0 but those of entry a, some
    hundreds, and b, `gap` units below; all others' exponentials are nothing beside theirs."""
    g = np.random.default_rng(seed)
    d = 16
    w, h = np.zeros((vocab, d)), np.zeros((n, d))
    # 8 pairs of entries: pair k answers to column 2 k with `up` and column 2 k + 1 with 1 for a, 0 for b
    a, b = 10 + 80 * np.arange(8), 50 + 80 * np.arange(8)
    w[a, 2 * np.arange(8)] = w[b, 2 * np.arange(8)] = 64
    w[a, 2 * np.arange(8) + 1] = 1
    k = np.arange(n) % 8
    gap = g.integers(1, 30, n)
    h[np.arange(n), 2 * k] = g.integers(1, 5, n) * 1.0 + np.ceil(100 / scale / 64)
    h[np.arange(n), 2 * k + 1] = gap
    return h, w, a[k], b[k], gap


@pytest.mark.parametrize("scale", [0.7, 1.0, 3.3, 5.0, 11.1])
@pytest.mark.parametrize("n", [20, 100, 300])
def test_losses_of_large_logits_are_rounded_once(n, scale):
    """Statistics of logits of some hundreds, where a loss is a small difference of them: a result's own
    rounding, and for the two exponentials, their sum and its logarithm some steps of 2^-23."""
    scale = float(np.float32(scale))
    h, w, a, b, gap = rows_with_a_leader(scale, n)
    top, below = (h * w[a]).sum(1) * scale, (h * w[b]).sum(1) * scale
    more = np.log1p(np.exp(below - top))
    for dtype in (FP32, BF16):
        H, W = (torch.from_numpy(t).to(dtype).cuda() for t in (h, w))
        assert np.array_equal(as64(H), h) and np.array_equal(as64(W), w)
        for label, z in ((a, top), (b, below)):
            loss, lse = ms.maxsim_linear_cross_entropy(H, W, torch.from_numpy(label).cuda(), scale)
            ref.close(lse, top + more, ref.U32 * (top + more) + 6 * 2.0 ** -23, "lse")
            want = top - z + more
            ref.close(loss, want, ref.U32 * want + 6 * 2.0 ** -23, "loss")


@pytest.mark.parametrize("scale", [0.7, 1.0, 3.3, 5.0, 11.1])
def test_gradients_of_large_logits(scale):
    """fp32: with the lse given, each weight is exp(z - lse) to within some steps of 2^-23 of itself, however
    large z and lse are."""
    scale = float(np.float32(scale))
    h, w, a, b, gap = rows_with_a_leader(scale, 64, seed=1)
    top, below = (h * w[a]).sum(1) * scale, (h * w[b]).sum(1) * scale
    lse = torch.from_numpy(top + np.log1p(np.exp(below - top))).float()
    L, dl = as64(lse), np.random.default_rng(2).random(64)
    dl = as64(torch.from_numpy(dl).float())
    one = np.arange(64)
    P = np.zeros((64, 700))
    P[one, a], P[one, b] = np.exp(top - L), np.exp(below - L)
    size = P.copy()
    P[one, b] -= 1
    size[one, b] += 1
    P, size = P * (dl * scale)[:, None], size * (dl * scale)[:, None]
    to = dict(dtype=FP32, device="cuda")
    dh, dw = ms.maxsim_linear_cross_entropy_backward(torch.tensor(dl, **to), torch.tensor(h, **to), torch.tensor(w, **to),
                                                     torch.from_numpy(b).cuda(), lse.cuda(), scale)
    # the difference's rounding, its factor's, the exponential's, the subtraction's and the gradient's
    off = 8 * 2.0 ** -23
    gone = 700 * np.exp(-90)  # all other weights
    ref.close(dh, P @ w, (off + 4 * ref.U32) * (size @ np.abs(w)) + 64 * gone, "dh")
    ref.close(dw, P.T @ h, (off + 64 * ref.U32) * (size.T @ np.abs(h)) + 64 * 64 * gone, "dw")


@pytest.mark.parametrize("n", [1, 32, 100])
def test_small_products_behind_a_large_one_are_kept(n):
    """fp32, up to 128 rows: 2^24 and then halves. Two halves at a time are below half a step of 2^24 and
    would all be lost; groups of 16 are 8, four steps, and only the first group's are."""
    d, vocab, scale = 1024, 300, 2.0 ** -20
    w = torch.zeros(vocab, d, device="cuda")
    w[7] = 0.5
    w[7, 0] = 2.0 ** 24
    h = torch.ones(n, d, device="cuda")
    y = torch.full((n,), 3, device="cuda")
    loss, lse = ms.maxsim_linear_cross_entropy(h, w, y, scale)
    z = scale * (2.0 ** 24 + (d - 1) / 2)
    want = z + math.log1p((vocab - 1) * math.exp(-z))
    tol = 8 * scale + ref.U32 * want + 6 * 2.0 ** -23
    assert float((loss.double() - want).abs().max()) <= tol and float((lse.double() - want).abs().max()) <= tol
