"""The norm with the residual's addition, its 8-bit form and its gradients, and dropout, against
64-bit references."""
import math

import numpy as np
import pytest
import torch

import maxsim_scoring_fwd_amd as ms
import train_ref as ref
from encoder_ref import HALF_STEP, TINY, U32, as64

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
SIZES = [1, 3, 8, 31, 64, 77, 128, 257, 512, 513, 768, 1000, 1024, 1025, 2048, 2056, 4096, 8192]


def rand(*shape, dtype=torch.float32, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def rng_of(key=-5, step=7):
    return torch.tensor([key, step], dtype=torch.int64, device="cuda")


def rows_of(d):
    return {1: 300, 3: 33, 128: 1001, 768: 67}.get(d, 5)


def handed_on(x, residual, keep, up, dtype):
    """h, bit for bit: one product and one sum in 32 bits, one rounding."""
    h = x.float().cpu()
    if keep is not None:
        h = torch.where(torch.from_numpy(keep).view(h.shape), h * torch.tensor(up), torch.zeros(()))
    if residual is not None:
        h = h + residual.float().cpu()
    return h.to(dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("d", SIZES)
def test_norm_and_gradients(d, dtype):
    n = rows_of(d)
    for case, (residual, p, wtype) in enumerate([(False, 0.0, torch.float32), (True, 0.0, dtype),
                                                 (True, 0.3, torch.float32), (False, 0.1, dtype)]):
        print("case: norm", d, dtype, residual, p, wtype, flush=True)
        x = rand(n, d, dtype=dtype, seed=d)
        r = rand(n, d, dtype=dtype, seed=d + 1, std=3) if residual else None
        w = rand(d, dtype=wtype, seed=d + 2)
        rng = rng_of(d, case)
        y, h, rstd = ms.maxsim_rms_norm(x, w, r, 1e-6, p, rng if p else None, call=case)
        keep, up = ref.kept(rng.tolist(), case, p, n, d) if p else (None, 1)
        if residual or p:
            assert torch.equal(h.cpu(), handed_on(x, r, keep, up, dtype))
        else:
            assert h is x
        want, tol, wr = ref.norm(as64(h), as64(w), 1e-6, dtype)
        ref.close(y, want, tol, "y")
        ref.close(rstd, wr[:, 0], wr[:, 0] * 32 * U32, "rstd")
        gy, gh = rand(n, d, dtype=dtype, seed=d + 3), rand(n, d, dtype=dtype, seed=d + 4)
        dx, dr, dw = ms.maxsim_rms_norm_backward(gy, h, w, rstd, gh, p, rng if p else None, case)
        g = ref.norm_backward(as64(h), as64(w), 1e-6, as64(gy), as64(gh),
                              keep * np.float64(up) if p else 1.0, dtype, wtype)
        ref.close(dr, g["dresidual"], g["tol_dresidual"], "dresidual")
        ref.close(dx, g["dx"], g["tol_dx"], "dx")
        ref.close(dw, g["dw"], g["tol_dw"], "dw")
        assert (dx is dr) == (not p)
        only = ms.maxsim_rms_norm_backward(gy, h, w, rstd, None, p, rng if p else None, case, want_dx=False,
                                           want_dresidual=False)
        assert only[0] is None and only[1] is None and torch.equal(only[2], dw)


def test_many_rows_share_the_weights_gradient():
    n, d = 20011, 96
    x, w, gy = rand(n, d, dtype=torch.bfloat16), rand(d), rand(n, d, dtype=torch.bfloat16, seed=1)
    y, h, rstd = ms.maxsim_rms_norm(x, w)
    got = ms.maxsim_rms_norm_backward(gy, h, w, rstd)
    g = ref.norm_backward(as64(x), as64(w), 1e-6, as64(gy), 0.0, 1.0, torch.bfloat16, torch.float32)
    ref.close(got[2], g["dw"], g["tol_dw"], "dw")
    for _ in range(2):
        assert torch.equal(ms.maxsim_rms_norm_backward(gy, h, w, rstd)[2], got[2])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("d", [1, 7, 32, 128, 200, 768, 1024, 8192])
def test_norm_in_8_bits(d, dtype):
    n = rows_of(d)
    for residual in (False, True):
        print("case: norm 8 bits", d, dtype, residual, flush=True)
        x, w = rand(n, d, dtype=dtype, seed=d), rand(d, seed=d + 2)
        r = rand(n, d, dtype=dtype, seed=d + 1) if residual else None
        if n > 3:
            x[3] = 0
            if residual:
                r[3] = 0
        code, scale, h = ms.maxsim_rms_norm_i8(x, w, r)
        y, tol, _ = ref.norm(as64(h), as64(w), 1e-6, torch.float32)
        most = np.abs(y).max(1)
        # scale: y's error and one division; a code: half a step of the scale, and its own roundings
        ref.close(scale, most / 127, most / 127 * 40 * U32 + TINY[torch.float32], "scale")
        ref.close(as64(code) * as64(scale)[:, None], y, most[:, None] / 127 * (0.5 + 127 * 40 * U32), "values")
        assert int(code.abs().max()) <= 127 and (n <= 3 or (not code[3].any() and scale[3] == 0))


def test_8_bit_rows_of_other_sizes():
    """Tiny rows keep their codes, a row with a NaN or an infinity says so in its scale."""
    x = torch.ones(5, 16, device="cuda")
    w = torch.full((16,), 2.0 ** -120, device="cuda")
    w[1] = 2.0 ** -121
    x[1, 3] = float("nan")
    x[2, 3] = float("inf")
    code, scale, _ = ms.maxsim_rms_norm_i8(x, w, eps=0.0)
    assert code[0].tolist() == [127, 64] + [127] * 14
    assert torch.isnan(scale[1]) and torch.isnan(scale[2]) and not code[1:3].any()
    y, _, _ = ms.maxsim_rms_norm(x, w, eps=0.0)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 3]) and torch.isfinite(y[0]).all()


def codes_of(y, scale):
    """y / scale to the nearest, ties to even. The quotient in 64 bits: a product of a scale of 24 bits and a
    code and a half of 8 is exact there, and a fp32 y that is not that product is off by 2^-25 of it."""
    return np.rint(as64(y) / as64(scale)[:, None])


def test_8_bit_codes_are_the_nearest_ones():
    """Entries on the halves between two codes and fp32's neighbours of those, for scales of many
    mantissas (127: ties are exact), beside entries of any size. Rows of ones keep their weights: the
    mean of 1024 squares is 1."""
    x = torch.ones(1, 1024, device="cuda")
    for i in range(40):
        most = torch.tensor(127.0 if i % 8 == 0 else 1 + i / 40, device="cuda") * 2.0 ** (i - 20)
        unit = float(ms.maxsim_rms_norm_i8(x[:, :1], most[None], eps=0.0)[1])
        assert abs(unit - float(most) / 127) <= 2 ** -23 * unit
        half = (torch.arange(-127, 127, device="cuda") + 0.5) * unit
        ends = [torch.nextafter(half, torch.full_like(half, s * math.inf)) for s in (1, -1)]
        w = torch.cat([most[None], half, *ends, rand(1024 - 1 - 3 * 254, seed=i).clamp(-1, 1) * most])
        code, scale, _ = ms.maxsim_rms_norm_i8(x, w, eps=0.0)
        y = ms.maxsim_rms_norm(x, w, eps=0.0)[0]
        assert torch.equal(y[0], w) and float(scale) == unit
        assert np.array_equal(as64(code), codes_of(y, scale)), f"scale {float(scale)}"


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("d", [7, 64, 200, 768, 2056])
def test_8_bit_codes_of_every_form(d, dtype):
    """The same for rows as they come; fp32 rows of the same values have the same y."""
    x, w = rand(500, d, dtype=dtype, seed=d), rand(d, seed=d + 1)
    code, scale, _ = ms.maxsim_rms_norm_i8(x, w)
    y = ms.maxsim_rms_norm(x.float(), w)[0]
    most = np.abs(as64(y)).max(1)
    assert (np.abs(as64(scale) - most / 127) <= 2 ** -23 * most / 127).all()
    assert np.array_equal(as64(code), codes_of(y, scale))


def test_8_bit_rows_at_both_ends_of_the_range():
    """Rows whose largest entry's reciprocal is no normal number, or whose scale is none, keep their
    codes."""
    x = torch.ones(1, 64, device="cuda")
    for e in (-140, -127, -110, -101, -100, -99, 99, 100, 101, 125, 126, 127):
        w = (torch.arange(64, device="cuda") * 2 + 1).double() * 2.0 ** e / 127
        w = w.float()  # the largest is 2^e, up to a rounding
        code, scale, _ = ms.maxsim_rms_norm_i8(x, w, eps=0.0)
        most = as64(w).max()
        assert np.array_equal(as64(code)[0], np.rint(as64(w) / most * 127)), f"2^{e}"
        assert abs(float(scale) - most / 127) <= 2 * U32 * most / 127 + TINY[torch.float32]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_strides_and_shapes(dtype):
    """Rows of a wider tensor, tensors of more dimensions, addresses that are only the type's."""
    wide = rand(40, 3 * 96 + 1, dtype=dtype)
    w = rand(96)
    for first in (0, 1, 96, 193):
        x = wide[:, first:first + 96]
        r = rand(40, 200, dtype=dtype, seed=9)[:, 5:101]
        got = ms.maxsim_rms_norm(x, w, r)
        want = ms.maxsim_rms_norm(x.contiguous(), w, r.contiguous())
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        y, h, rstd = ms.maxsim_rms_norm(x, w)
        gy = rand(40, 96, dtype=dtype, seed=3)
        a, b = (ms.maxsim_rms_norm_backward(gy, t, w, rstd) for t in (x, x.contiguous()))
        assert all(torch.equal(i, j) for i, j in zip(a, b))
    x = rand(4, 5, 96, dtype=dtype)
    y, h, rstd = ms.maxsim_rms_norm(x, w, x)
    flat = ms.maxsim_rms_norm(x.view(20, 96), w, x.view(20, 96))
    assert y.shape == h.shape == x.shape and rstd.shape == (4, 5)
    assert torch.equal(y.view(20, 96), flat[0]) and torch.equal(rstd.view(20), flat[2])
    one = ms.maxsim_rms_norm(x[0, 0], w)
    assert torch.equal(one[0], ms.maxsim_rms_norm(x[0], w)[0][0])
    same = ms.maxsim_rms_norm(x[:1, :1].expand(4, 5, 96).reshape(20, 96), w)[0]
    assert torch.equal(same[0], same[19])
    shared = ms.maxsim_rms_norm(x[0, :1].expand(7, 96), w)[0]  # one row, seven times
    assert torch.equal(shared, same[:7])


def test_in_place_and_untouched_memory():
    x, r, w = rand(9, 77, dtype=torch.bfloat16), rand(9, 77, dtype=torch.bfloat16, seed=1), rand(77)
    want = ms.maxsim_rms_norm(x, w, r)
    buf = torch.full((11, 77), 3.0, dtype=torch.bfloat16, device="cuda")
    ms.maxsim_rms_norm(x, w, r, out=buf[1:10])
    assert torch.equal(buf[1:10], want[0]) and (buf[[0, 10]] == 3).all()
    y, h, _ = ms.maxsim_rms_norm(x, w, r, out=x, out_h=r)
    assert y is x and h is r and torch.equal(x, want[0]) and torch.equal(r, want[1])


def test_no_rows():
    w = rand(64)
    x = rand(0, 64, dtype=torch.bfloat16)
    y, h, rstd = ms.maxsim_rms_norm(x, w, x)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dw = ms.maxsim_rms_norm_backward(x, h, w, rstd, dweight=torch.ones(64, device="cuda"))[2]
    assert not dw.any()
    assert ms.maxsim_rms_norm_i8(x, w)[0].shape == (0, 64)
    assert ms.maxsim_dropout(x, 0.5, rng_of()).shape == (0, 64)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n", [1, 7, 8, 9, 255, 4096, 8191, 100003, 1 << 20])
def test_dropout(n, dtype):
    for i, p in enumerate((0.1, 0.5, 0.0, 1.0, 1e-6, 0.999)):
        print("case: dropout", n, dtype, p, flush=True)
        x = rand(n, dtype=dtype, seed=n)
        rng = rng_of(-(1 << 63) + n, (1 << 33) + i)
        y = ms.maxsim_dropout(x, p, rng, call=i)
        assert torch.equal(y.cpu(), ref.dropped(x, rng.tolist(), i, p))
        z = x.clone()
        assert torch.equal(ms.maxsim_dropout(z, p, rng, call=i, out=z), y)


def test_dropout_hides_what_it_drops_and_takes_any_address():
    x = torch.full((1001,), float("nan"), device="cuda", dtype=torch.bfloat16)
    y = ms.maxsim_dropout(x[1:], 0.5, rng_of())
    keep, _ = ref.kept(rng_of().tolist(), 0, 0.5, 1, 1000)
    assert torch.equal(torch.isnan(y).cpu(), torch.from_numpy(keep)[0]) and not y[~torch.isnan(y)].any()
    x = rand(1001, dtype=torch.bfloat16)
    assert torch.equal(ms.maxsim_dropout(x[1:], 0.5, rng_of()).cpu(), ref.dropped(x[1:], rng_of().tolist(), 0, 0.5))


def test_calls_steps_and_keys_are_independent():
    """Shares of kept entries and of agreements between two masks: each within 5 standard deviations
    of what independent bits give."""
    n, p = 1 << 20, 0.25
    x = torch.ones(n, device="cuda")
    masks = [ms.maxsim_dropout(x, p, rng_of(k, s), call=c) > 0
             for k, s, c in ((1, 1, 0), (2, 1, 0), (1, 2, 0), (1, 1, 1), (1 + (1 << 32), 1, 0))]
    for i, a in enumerate(masks):
        assert abs(float(a.double().mean()) - 0.75) <= 5 * (0.75 * 0.25 / n) ** 0.5
        for b in masks[:i]:
            same = 0.75 ** 2 + 0.25 ** 2
            assert abs(float((a == b).double().mean()) - same) <= 5 * (same * (1 - same) / n) ** 0.5


def test_autograd():
    """Gradients through the wrappers are the entry points'; dropout's go to any order, the norm's
    gradients cannot be differentiated again."""
    x, r, w = rand(33, 200).requires_grad_(), rand(33, 200, seed=1).requires_grad_(), rand(200, seed=2).requires_grad_()
    gy, gh, rng = rand(33, 200, seed=3), rand(33, 200, seed=4), rng_of()
    y, h = ms.rms_norm(x, w, r, dropout=0.2, rng=rng, call=3)
    got = torch.autograd.grad((y, h), (x, r, w), (gy, gh))
    a = ms.maxsim_rms_norm(x.detach(), w.detach(), r.detach(), dropout=0.2, rng=rng, call=3)
    want = ms.maxsim_rms_norm_backward(gy, a[1], w.detach(), a[2], gh, 0.2, rng, 3)
    assert all(torch.equal(i, j) for i, j in zip(got, want))
    y, h = ms.rms_norm(x, w, r)
    (h * gh).sum().backward()  # only h is used
    assert torch.equal(x.grad, gh) and torch.equal(r.grad, gh) and not w.grad.any()
    y, h = ms.rms_norm(x, w)
    assert h is x
    (g,) = torch.autograd.grad(y, x, gy, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        g.sum().backward()
    y, h = ms.rms_norm(x, w, r)
    gx, gr = torch.autograd.grad((y, h), (x, r), (gy, gh), create_graph=True)
    assert torch.equal(gx, gr)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        (gx + gr).sum().backward()
    z = ms.dropout(x, 0.5, rng)
    (g,) = torch.autograd.grad((z * z).sum(), x, create_graph=True)
    (g2,) = torch.autograd.grad(g.sum(), x)
    keep = ms.maxsim_dropout(torch.ones_like(x), 0.5, rng)
    assert torch.equal(g2, 2 * keep * keep)
    both = (x.detach() * 1).requires_grad_()
    y, h = ms.rms_norm(both, w, both, dropout=0.2, rng=rng)  # the same leaf twice
    (g,) = torch.autograd.grad((y, h), both, (gy, gh))
    y1, h1 = ms.rms_norm(x.detach().requires_grad_(), w, x.detach(), dropout=0.2, rng=rng)
    a = ms.maxsim_rms_norm(x.detach(), w.detach(), x.detach(), dropout=0.2, rng=rng)
    dx, dr, _ = ms.maxsim_rms_norm_backward(gy, a[1], w.detach(), a[2], gh, 0.2, rng)
    assert torch.equal(g, dx + dr)


def test_step_changed_before_the_backward_is_an_error():
    x, rng = rand(8, 8).requires_grad_(), rng_of()
    y = ms.dropout(x, 0.5, rng)
    rng[1] += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_gradients_against_differences():
    """fp32 values along one direction: central differences of step 2^-6 are off by its square (the
    norm's third derivatives are of the size of its first here) and by 2^-24 of the sum over 2^-6."""
    n, d = 16, 64
    x, r, w = rand(n, d), rand(n, d, seed=1), rand(d, seed=2)
    gy, gh, rng = rand(n, d, seed=3), rand(n, d, seed=4), rng_of()
    y, h, rstd = ms.maxsim_rms_norm(x, w, r, dropout=0.25, rng=rng)
    dx, dr, dw = ms.maxsim_rms_norm_backward(gy, h, w, rstd, gh, 0.25, rng)
    e = 2.0 ** -6
    for g, at in ((dx, 0), (dr, 1), (dw, 2)):
        t = rand(*g.shape, seed=5 + at)
        side = []
        for s in (e, -e):
            a = [x, r, w]
            a[at] = a[at] + s * t
            y2, h2, _ = ms.maxsim_rms_norm(a[0], a[2], a[1], dropout=0.25, rng=rng)
            side.append(float((y2.double() * gy).sum() + (h2.double() * gh).sum()))
        got, want = (side[0] - side[1]) / (2 * e), float((g.double() * t).sum())
        scale = float((g.double() * t).abs().sum())
        assert abs(got - want) <= scale * (4 * e * e + 2.0 ** -24 / e * 16)
