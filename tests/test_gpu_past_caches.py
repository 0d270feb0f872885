"""The norm, dropout and the 4-bit conversion where a call moves more than 256 MiB in a 16-bit type and
passes the caches by, and the weight's gradient over several rounds of rows."""
import numpy as np
import pytest
import torch

import maxsim_scoring_fwd_amd as ms
import train_ref as ref
from encoder_ref import HALF_STEP, TINY, U32, as64

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
CACHE = 256 << 20


def rand(*shape, dtype=FP32, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def weight_gradient(h, gy, wdtype):
    """sum of gy * h * rstd over the rows in 64 bits, and its bound: a lane adds up the rows of its rounds (1024
    workgroups of 256 threads, 16 to 256 of them to a row), then come a workgroup's groups (16 at most) and
    the workgroups' sums, 16 in turn and 6 steps across."""
    n, d = h.shape
    groups = 256 // (16 if d <= 512 else 32 if d <= 1024 else 64 if d <= 2048 else 256)
    chain = -(-n // (1024 * groups)) + 16 + 16 + 6
    rel = (ref.NORM_CHAIN / 2 + 8) * U32  # of h * rstd, as in the reference
    dw, size = torch.zeros(2, d, dtype=torch.float64, device="cuda")
    for a in range(0, n, 1 << 15):
        x = h[a:a + (1 << 15)].double()
        t = gy[a:a + (1 << 15)].double() * x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt()
        dw += t.sum(0)
        size += t.abs().sum(0)
    dw, size = as64(dw), as64(size)
    return dw, size * (chain * U32 + rel) + HALF_STEP[wdtype] * np.abs(dw) + TINY[wdtype]


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
@pytest.mark.parametrize("n, d", [(262201, 128), (43711, 768), (16403, 2048), (8209, 4096)])
def test_norm_and_gradients(n, d, dtype):
    """With a residual, dropout, a gradient of h and all three gradients: h of every row bit for bit, the
    weight's gradient whole, the others at rows of both ends and the middle."""
    print("case: norm past the caches", n, d, dtype, flush=True)
    assert n * d * 2 * 4 > CACHE  # x, residual, h and y; the backward moves one tensor more
    wdtype = FP32 if d % 256 else dtype
    x, r = rand(n, d, dtype=dtype, seed=1), rand(n, d, dtype=dtype, seed=2, std=2.0)
    gy, gh, w = rand(n, d, dtype=dtype, seed=3), rand(n, d, dtype=dtype, seed=4), rand(d, dtype=wdtype, seed=5)
    rng = torch.tensor([-17, 5], device="cuda")
    y, h, rstd = ms.maxsim_rms_norm(x, w, r, 1e-6, 0.1, rng, 3)
    # d is a multiple of 8, so that the masks are those of the whole tensor; fp32 goes through the caches
    assert torch.equal(h, (ms.maxsim_dropout(x.float(), 0.1, rng, 3) + r.float()).to(dtype))
    dx, dr, dw = ms.maxsim_rms_norm_backward(gy, h, w, rstd, gh, 0.1, rng, 3)
    want, tol = weight_gradient(h, gy, wdtype)
    ref.close(dw, want, tol, "dw")
    for first in (0, n // 2, n - 37):
        at = slice(first, first + 37)
        want, tol, wr = ref.norm(as64(h[at]), as64(w), 1e-6, dtype)
        ref.close(y[at], want, tol, "y")
        ref.close(rstd[at], wr[:, 0], wr[:, 0] * 32 * U32, "rstd")
        keep, up = ref.kept(rng.tolist(), 3, 0.1, 37, d, first * (d // 8))
        g = ref.norm_backward(as64(h[at]), as64(w), 1e-6, as64(gy[at]), as64(gh[at]), keep * np.float64(up), dtype, wdtype)
        ref.close(dr[at], g["dresidual"], g["tol_dresidual"], "dresidual")
        ref.close(dx[at], g["dx"], g["tol_dx"], "dx")
    # rows do not depend on each other: halves, which go through the caches, have the same bits
    y, h, rstd = ms.maxsim_rms_norm(x, w, r)
    dx, _, _ = ms.maxsim_rms_norm_backward(gy, h, w, rstd, gh, want_dweight=False)
    half = n // 2 + 1
    for a, b in ((0, half), (half, n)):
        p = ms.maxsim_rms_norm(x[a:b], w, r[a:b])
        assert all(torch.equal(i[a:b], j) for i, j in zip((y, h, rstd), p))
        q = ms.maxsim_rms_norm_backward(gy[a:b], h[a:b], w, rstd[a:b], gh[a:b], want_dweight=False)
        assert torch.equal(dx[a:b], q[0])


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
@pytest.mark.parametrize("n, d", [(33001, 128), (33001, 127), (8200, 768), (8200, 767), (4100, 2048), (4100, 2041),
                                  (2051, 4096), (2051, 4001)])
def test_gradients_over_several_rounds_of_rows(n, d, dtype):
    """More rows than the backward's workgroups take at once, in groups of 16, 32, 64 and 256 lanes."""
    print("case: rounds", n, d, dtype, flush=True)
    x, gy, gh = (rand(n, d, dtype=dtype, seed=s) for s in (1, 2, 3))
    w, rng = rand(d, seed=4), torch.tensor([6, 7], device="cuda")
    y, h, rstd = ms.maxsim_rms_norm(x, w, x, 1e-6, 0.2, rng, 1)
    dx, dr, dw = ms.maxsim_rms_norm_backward(gy, h, w, rstd, gh, 0.2, rng, 1)
    keep, up = ref.kept(rng.tolist(), 1, 0.2, n, d)
    g = ref.norm_backward(as64(h), as64(w), 1e-6, as64(gy), as64(gh), keep * np.float64(up), dtype, FP32)
    ref.close(dr, g["dresidual"], g["tol_dresidual"], "dresidual")
    ref.close(dx, g["dx"], g["tol_dx"], "dx")
    want, tol = weight_gradient(h, gy, FP32)
    ref.close(dw, want, tol, "dw")
    again = ms.maxsim_rms_norm_backward(gy, h, w, rstd, gh, 0.2, rng, 1)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dr, dw)))


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
def test_dropout(dtype):
    """Every entry against the fp32 kernel, which goes through the caches: one product in 32 bits, then one
    rounding. The ends against the generator itself."""
    n = (1 << 26) + 43
    assert 2 * n * 2 > CACHE
    x, rng = rand(n, dtype=dtype), torch.tensor([1 << 40, 3], device="cuda")
    for p in (0.1, 0.0):
        y = ms.maxsim_dropout(x, p, rng, 2)
        assert torch.equal(y, ms.maxsim_dropout(x.float(), p, rng, 2).to(dtype))
        first = (n - 1003) // 8 * 8
        for a, b in ((0, 1000), (first, n)):
            keep, up = ref.kept(rng.tolist(), 2, p, 1, b - a, a // 8)
            want = torch.where(torch.from_numpy(keep)[0], x[a:b].cpu().float() * torch.tensor(up), torch.zeros(()))
            assert torch.equal(y[a:b].cpu(), want.to(dtype))
        z = x.clone()
        assert torch.equal(ms.maxsim_dropout(z, p, rng, 2, out=z), y)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=str)
@pytest.mark.parametrize("n, d", [(840001, 128), (1120005, 96)])
def test_4_bit_vectors(n, d, dtype):
    """Codes, exponents and values are those of the halves, which go through the caches."""
    assert n * d // 8 * (16 + 4) > CACHE > n // 2 * d // 8 * (16 + 4) + CACHE // 8
    x = rand(n, d, dtype=dtype) * torch.logspace(-2, 2, n, device="cuda")[:, None].to(dtype)
    codes, scales = ms.maxsim_quantize_mx4(x)
    values = ms.maxsim_dequantize_mx4(codes, scales, dtype)
    half = n // 2
    for a, b in ((0, half), (half, n)):
        c, s = ms.maxsim_quantize_mx4(x[a:b])
        assert torch.equal(codes[a:b], c) and torch.equal(scales[a:b], s)
        c, s = codes[a:b].clone(), scales[a:b].clone()
        assert torch.equal(values[a:b], ms.maxsim_dequantize_mx4(c, s, dtype))
    want, k = ref.mx4(as64(x[n - 100:]))
    assert np.array_equal(ref.unpack(codes[n - 100:]), want)
    assert torch.equal(values[n - 100:].cpu(), torch.from_numpy(ref.mx4_values(want, k)).to(dtype))


def test_more_rows_than_one_launch_takes():
    """2^28 rows of 3 entries fill a launch's grid; the ones behind them go in another."""
    print("case: rows of two launches", flush=True)
    n, d = (1 << 28) + 1000, 3
    x = rand(1000, d, dtype=BF16).repeat(n // 1000 + 1, 1)[:n]
    w, rng = rand(d, seed=1), torch.tensor([4, 9], device="cuda")
    y, h, rstd = ms.maxsim_rms_norm(x, w, None, 1e-6, 0.5, rng, 2)
    code, scale, _ = ms.maxsim_rms_norm_i8(x, w)
    small = ms.maxsim_rms_norm_i8(x[:1000], w)
    for first in (0, (1 << 28) - 500, (1 << 28), n - 1000):
        at = slice(first, first + 1000)
        keep, up = ref.kept(rng.tolist(), 2, 0.5, 1000, d, first)
        want = torch.where(torch.from_numpy(keep), x[at].cpu().float() * torch.tensor(up), torch.zeros(()))
        assert torch.equal(h[at].cpu(), want.to(BF16))
        want, tol, wr = ref.norm(as64(h[at]), as64(w), 1e-6, BF16)
        ref.close(y[at], want, tol, "y")
        ref.close(rstd[at], wr[:, 0], wr[:, 0] * 32 * U32, "rstd")
        turn = first % 1000
        assert torch.equal(code[at], small[0].roll(-turn, 0)) and torch.equal(scale[at], small[1].roll(-turn, 0))
    gy = x[:1000].flip(0).repeat(n // 1000 + 1, 1)[:n]
    dx, _, _ = ms.maxsim_rms_norm_backward(gy, h, w, rstd, None, 0.5, rng, 2, want_dresidual=False, want_dweight=False)
    for first in (0, (1 << 28) - 500, n - 1000):
        at = slice(first, first + 1000)
        keep, up = ref.kept(rng.tolist(), 2, 0.5, 1000, d, first)
        g = ref.norm_backward(as64(h[at]), as64(w), 1e-6, as64(gy[at]), 0.0, keep * np.float64(up), BF16, FP32)
        ref.close(dx[at], g["dx"], g["tol_dx"], "dx")
