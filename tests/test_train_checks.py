"""The norm, dropout, the cross entropy over a vocabulary and the 4-bit vectors without a GPU: what
the binding and the C entry points refuse, sizes of workspaces, and the test reference itself:
its generator against published numbers, its gradients against differences."""
import numpy as np
import pytest
import torch

import maxsim_scoring_fwd_amd as ms
import train_ref as ref
from test_encoder_checks import On0, On1, refuses

bf, f16, f32, i8, u8, i32, i64 = (torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.uint8,
                                  torch.int32, torch.int64)
OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, DEVICE = 0, -1, -2, -3, -4, -5, -7
P = 0x10000  # a 16-byte aligned stand-in address; never dereferenced by these calls


@pytest.fixture(scope="module")
def L():
    return ms.lib()


def Z(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


RNG = torch.zeros(2, dtype=i64)


# ---------------------------------------------------------------- the binding
def test_norm_binding_refuses():
    x, w = Z(10, 64), Z(64)
    norm = ms.maxsim_rms_norm
    for f in (norm, ms.maxsim_rms_norm_i8):
        refuses("must be a torch.Tensor", f, [1.0], w)
        refuses("x must have dtype", f, x.int(), w)
        refuses("weight must have dtype", f, x, w.half())
        refuses("weight must have shape", f, x, Z(32))
        refuses("must be a torch.Tensor", f, x, None)
        refuses("residual must have dtype", f, x, w, x.half())
        refuses("residual must have shape", f, x, w, Z(9, 64))
        refuses("eps must not be negative", f, x, w, eps=-1.0)
        refuses("eps must not be negative", f, x, w, eps=float("nan"))
        refuses("side by side", f, Z(64, 10).t(), w)
        refuses("one distance", f, Z(5, 4, 64)[:, :3], w)
        refuses("h is x itself", f, x, w, out_h=x)
        refuses("out_h must have", f, x, w, x, out_h=Z(9, 64))
        refuses("scale must have|rstd must have", f, x, w, **{"scale" if f is not norm else "rstd": Z(10)})
        refuses("out must have", f, x, w, out=Z(9, 64))
        refuses("device tensor", f, x, w)
        refuses("at least one entry", f, torch.zeros((), dtype=bf), w)
        refuses("at least one entry", f, Z(4, 0), Z(0))
    refuses("needs rng", norm, x, w, dropout=0.5)
    refuses("must lie in", norm, x, w, dropout=1.5, rng=RNG)
    refuses("must lie in", norm, x, w, dropout=float("nan"), rng=RNG)
    refuses("rng must have dtype", norm, x, w, dropout=0.5, rng=RNG.int())
    refuses("rng must have shape", norm, x, w, dropout=0.5, rng=RNG[:1])
    refuses("call must lie in", norm, x, w, dropout=0.5, rng=RNG, call=-1)
    refuses("call must lie in", norm, x, w, call=1 << 31)
    back = ms.maxsim_rms_norm_backward
    r = Z(10, dtype=f32)
    refuses("grad_y must have", back, Z(9, 64), x, w, r)
    refuses("grad_h must have", back, x, x, w, r, Z(10, 64, dtype=f32))
    refuses("rstd must have", back, x, x, w, Z(10))
    refuses("dx must have", back, x, x, w, r, dx=Z(9, 64))
    refuses("dresidual must have", back, x, x, w, r, dresidual=Z(10, 64, dtype=f16))
    refuses("dweight must have", back, x, x, w, r, dweight=Z(64, dtype=f32))
    refuses("workspace must have", back, x, x, w, r, workspace=Z(64))
    refuses("needs rng", back, x, x, w, r, dropout=0.1)
    refuses("device tensor", back, x, x, w, r)


def test_norm_of_a_number_is_refused():
    for f in (ms.maxsim_rms_norm, ms.maxsim_rms_norm_i8, ms.rms_norm):
        refuses("rows of at least one entry", f, Z(()), Z(()))


def test_dropout_binding_refuses():
    x, drop = Z(10, 64), ms.maxsim_dropout
    refuses("x must have dtype", drop, x.int(), 0.5, RNG)
    refuses("needs rng", drop, x, 0.0, None)
    refuses("must lie in", drop, x, -0.1, RNG)
    refuses("rng must have", drop, x, 0.1, Z(2))
    refuses("call must lie in", drop, x, 0.1, RNG, -1)
    refuses("out must have", drop, x, 0.1, RNG, out=Z(64, 10))
    refuses("contiguous", drop, Z(64, 10).t(), 0.1, RNG)
    refuses("device tensor", drop, x, 0.1, RNG)


def test_loss_binding_refuses():
    h, w, y = Z(10, 64), Z(100, 64), torch.zeros(10, dtype=i64)
    loss, back = ms.maxsim_linear_cross_entropy, ms.maxsim_linear_cross_entropy_backward
    r = Z(10, dtype=f32)
    for f in (lambda h, w, y, scale=1.0, **k: loss(h, w, y, scale, **k),
              lambda h, w, y, scale=1.0, **k: back(r, h, w, y, r, scale, **k)):
        refuses("h must have dtype", f, h.int(), w, y)
        refuses("2 dimensions", f, Z(2, 5, 64), w, y)
        refuses("w must have dtype", f, h, w.half(), y)
        refuses("w has d = 32", f, h, Z(100, 32), y)
        refuses("at least one row", f, h, Z(0, 64), y)
        refuses("labels must have dtype", f, h, w, y.int())
        refuses("labels must have shape", f, h, w, y[:9])
        refuses("scale must be", f, h, w, y, 0.0)
        refuses("scale must be", f, h, w, y, float("inf"))
        refuses("scale must be", f, h, w, y, float("nan"))
        refuses("workspace must have", f, h, w, y, workspace=Z(4))
        refuses("device tensor", f, h, w, y)
    refuses("loss must have", loss, h, w, y, loss=Z(10))
    refuses("lse must have", loss, h, w, y, lse=Z(9, dtype=f32))
    refuses("grad_loss must have", back, Z(10), h, w, y, r)
    refuses("lse must have", back, r, h, w, y, Z(9, dtype=f32))
    refuses("dh must have", back, r, h, w, y, r, dh=Z(10, 64, dtype=f32))
    refuses("dw must have", back, r, h, w, y, r, dw=Z(99, 64))


def test_mx4_binding_refuses():
    quant, values, score = ms.maxsim_quantize_mx4, ms.maxsim_dequantize_mx4, ms.maxsim_score_mx4
    refuses("x must have dtype", quant, Z(4, 64).int())
    refuses("whole 32", quant, Z(4, 48))
    refuses("whole 32", quant, Z(4, 0))
    refuses("codes must have", quant, Z(4, 64), Z(4, 64, dtype=u8))
    refuses("scales must have", quant, Z(4, 64), None, Z(4, 1, dtype=u8))
    refuses("device tensor", quant, Z(4, 64))
    c, s = Z(4, 32, dtype=u8), Z(4, 2, dtype=u8)
    refuses("codes must have dtype", values, c.to(i8), s)
    refuses("whole 16", values, Z(4, 24, dtype=u8), s)
    refuses("scales must have shape", values, c, Z(4, 3, dtype=u8))
    refuses("unsupported dtype", values, c, s, torch.float64)
    refuses("out must have", values, c, s, f32, Z(4, 64))
    refuses("device tensor", values, c, s)
    D, ds, off = Z(10, 32, dtype=u8), Z(10, 2, dtype=u8), torch.tensor([0, 4, 10])
    F, fs = D.view(2, 5, 32), ds.view(2, 5, 2)
    refuses("Q must have", score, c.view(2, 2, 32), s, D, ds, off)
    refuses("q_scale must have", score, c, ds, D, ds, off)
    refuses("D must have", score, c, s, D, ds)
    refuses("D must have", score, c, s, F, fs, off)
    refuses("d_scale must have", score, c, s, D, s, off)
    refuses("D has d = 32", score, c, s, Z(10, 16, dtype=u8), Z(10, 1, dtype=u8), off)
    refuses("doc_offsets must have dtype", score, c, s, D, ds, off.int())
    refuses(">= 1 entries", score, c, s, D, ds, off[:0])
    refuses("not both", score, c, s, D, ds, off, torch.zeros(2, dtype=i32))
    refuses("doc_lens must have dtype", score, c, s, F, fs, doc_lens=torch.zeros(2, dtype=i64))
    refuses("doc_lens must have shape", score, c, s, F, fs, doc_lens=torch.zeros(3, dtype=i32))
    refuses("out must", score, c, s, F, fs, out=Z(3, dtype=f32))
    refuses("device tensor", score, c, s, F, fs)


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0)
    here, there = (lambda t: t.as_subclass(On0)), (lambda t: t.as_subclass(On1))

    def each(fn, args, **rest):
        for name in args:
            kw = {n: (there if n == name else here)(t) for n, t in args.items()}
            refuses(f"{name} is on cuda:1, expected cuda:0", fn, **kw, **rest)
    x, r = Z(10, 64), Z(10, dtype=f32)
    each(lambda **k: ms.maxsim_rms_norm(here(x), **k),
         dict(weight=Z(64), residual=x, rng=RNG, out=x, out_h=x, rstd=r), dropout=0.5)
    each(lambda **k: ms.maxsim_rms_norm_i8(here(x), **k),
         dict(weight=Z(64), residual=x, out=Z(10, 64, dtype=i8), out_h=x, scale=r))
    each(lambda **k: ms.maxsim_rms_norm_backward(h=here(x), **k),
         dict(grad_y=x, weight=Z(64), rstd=r, grad_h=x, rng=RNG, dx=x, dresidual=x, dweight=Z(64),
              workspace=Z(1 << 16, dtype=u8)), dropout=0.5)
    each(lambda **k: ms.maxsim_dropout(here(x), 0.5, **k), dict(rng=RNG, out=x))
    y = torch.zeros(10, dtype=i64)
    each(lambda **k: ms.maxsim_linear_cross_entropy(here(x), **k),
         dict(w=Z(100, 64), labels=y, loss=r, lse=r, workspace=Z(1 << 16, dtype=u8)))
    each(lambda **k: ms.maxsim_linear_cross_entropy_backward(h=here(x), **k),
         dict(grad_loss=r, w=Z(100, 64), labels=y, lse=r, dh=x, dw=Z(100, 64), workspace=Z(16, dtype=u8)))
    c, s = Z(10, 32, dtype=u8), Z(10, 2, dtype=u8)
    each(lambda **k: ms.maxsim_quantize_mx4(here(x), **k), dict(codes=c, scales=s))
    each(lambda **k: ms.maxsim_dequantize_mx4(here(c), dtype=bf, **k), dict(scales=s, out=x))
    each(lambda **k: ms.maxsim_score_mx4(here(c), **k),
         dict(q_scale=s, D=c, d_scale=s, doc_offsets=torch.tensor([0, 4, 10]), out=Z(2, dtype=f32)))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    refuses("the current device is cuda:1", ms.maxsim_dropout, here(x), 0.5, here(RNG), out=here(x))
    refuses("the current device is cuda:1", ms.maxsim_rms_norm, here(x), here(Z(64)), out=here(x), rstd=here(r))


# ---------------------------------------------------------------- the C entry points
def test_norm_c_entries_refuse(L):
    def f(x=P, xs=64, res=P, n=10, d=64, dt=0, w=P, wdt=2, eps=1e-6, p=0.0, rng=None, call=0, y=P, h=P, rstd=P):
        return L.maxsim_rms_norm(x, xs, res, 64, n, d, dt, w, wdt, eps, p, rng, call, y, h, rstd, None)
    assert f(x=None) == NULL and f(w=None) == NULL and f(y=None) == NULL and f(h=None) == NULL
    assert f(p=0.5) == NULL and f(res=None, h=None, p=0.5, rng=P) == NULL
    assert f(x=P + 1) == ALIGN and f(res=P + 1) == ALIGN and f(w=P + 2) == ALIGN and f(rstd=P + 2) == ALIGN
    assert f(p=0.5, rng=P + 4) == ALIGN and f(y=P + 1) == ALIGN and f(h=P + 1) == ALIGN
    assert f(dt=3) == DTYPE and f(wdt=1) == DTYPE and f(dt=2, wdt=0) == DTYPE
    assert f(n=-1) == SHAPE and f(d=0) == SHAPE and f(eps=-1.0) == SHAPE and f(eps=float("nan")) == SHAPE
    assert f(n=(1 << 31) + 1) == SHAPE
    assert f(p=-0.5) == SHAPE and f(p=1.5) == SHAPE and f(p=float("nan")) == SHAPE and f(call=-1) == SHAPE
    assert f(d=8193) == UNSUP and f(n=0, x=None) == OK

    def g(x=P, d=64, n=10, dt=0, wdt=0, eps=0.0, codes=P, scale=P, h=P, res=P):
        return L.maxsim_rms_norm_i8(x, 64, res, 64, n, d, dt, P, wdt, eps, codes, scale, h, None)
    assert g(codes=None) == NULL and g(scale=None) == NULL and g(h=None) == NULL and g(x=None) == NULL
    assert g(scale=P + 1) == ALIGN and g(d=9000) == UNSUP and g(eps=-1.0) == SHAPE and g(dt=9) == DTYPE
    assert g(n=0) == OK

    def b(gy=P, gh=P, h=P, n=10, d=64, dt=0, w=P, wdt=0, rstd=P, p=0.0, rng=None, call=0, dx=P, dr=P, dw=P, ws=P,
          size=1 << 20):
        return L.maxsim_rms_norm_backward(gy, gh, h, 64, n, d, dt, w, wdt, rstd, p, rng, call, dx, dr, dw, ws, size,
                                          None)
    assert b(gy=None) == NULL and b(h=None) == NULL and b(rstd=None) == NULL and b(ws=None) == NULL
    assert b(w=None) == NULL and b(p=0.1) == NULL
    assert b(size=255) == SHAPE and b(ws=P + 2) == ALIGN and b(dx=P + 1) == ALIGN and b(rstd=P + 1) == ALIGN
    assert b(p=2.0) == SHAPE and b(call=-1) == SHAPE and b(d=10000) == UNSUP and b(wdt=1) == DTYPE
    assert b(dx=None, dr=None, dw=None) == OK and b(n=0, dw=None) == OK
    size = L.maxsim_rms_norm_backward_workspace_size
    assert size(0, 64) == 0 and size(10, 0) == 0 and size(10, 9000) == 0 and size(10, 64) >= 256


def test_dropout_c_entry_refuses(L):
    def f(x=P, n=10, dt=0, p=0.5, rng=P, call=0, out=P):
        return L.maxsim_dropout(x, n, dt, p, rng, call, out, None)
    assert f(x=None) == NULL and f(rng=None) == NULL and f(out=None) == NULL
    assert f(x=P + 1) == ALIGN and f(rng=P + 4) == ALIGN and f(dt=2, out=P + 2) == ALIGN
    assert f(dt=3) == DTYPE and f(n=-1) == SHAPE and f(p=1.1) == SHAPE and f(p=-1.0) == SHAPE
    assert f(p=float("nan")) == SHAPE and f(call=-1) == SHAPE and f(n=1 << 41) == SHAPE
    assert f(n=0, x=None) == OK


def test_loss_c_entries_refuse(L):
    size, back_size = (L.maxsim_linear_cross_entropy_workspace_size,
                       L.maxsim_linear_cross_entropy_backward_workspace_size)

    def f(h=P, w=P, y=P, n=10, v=100, d=64, dt=0, scale=1.0, loss=P, lse=P, ws=P, room=1 << 40):
        return L.maxsim_linear_cross_entropy(h, w, y, n, v, d, dt, scale, loss, lse, ws, room, None)

    def g(grad=P, h=P, w=P, y=P, lse=P, n=10, v=100, d=64, dt=0, scale=1.0, dh=P, dw=P, ws=P, room=1 << 40):
        return L.maxsim_linear_cross_entropy_backward(grad, h, w, y, lse, n, v, d, dt, scale, dh, dw, ws, room, None)
    for e in (f, g):
        assert e(h=None) == NULL and e(w=None) == NULL and e(y=None) == NULL and e(ws=None) == NULL
        assert e(lse=None) == NULL
        assert e(h=P + 8) == ALIGN and e(w=P + 8) == ALIGN and e(y=P + 4) == ALIGN and e(ws=P + 8) == ALIGN
        assert e(dt=3) == DTYPE and e(n=-1) == SHAPE and e(v=0) == SHAPE and e(d=0) == SHAPE
        assert e(d=12) == SHAPE and e(dt=2, d=6) == SHAPE and e(d=16392) == SHAPE
        assert e(n=(1 << 22) + 1) == SHAPE and e(v=(1 << 26) + 1) == SHAPE and e(n=1 << 22, v=1 << 26) == SHAPE
        for bad in (0.0, -1.0, float("inf"), float("nan")):
            assert e(scale=bad) == SHAPE
    assert f(loss=None) == NULL and f(loss=P + 2) == ALIGN
    assert f(room=size(10, 100, 64, 0) - 1) == SHAPE and g(room=back_size(10, 100, 64, 0) - 1) == SHAPE
    assert g(grad=None) == NULL and g(dh=P + 8) == ALIGN and g(dw=P + 8) == ALIGN
    assert f(n=0) == OK and g(dh=None, dw=None) == OK and g(n=0, dw=None) == OK
    for s in (size, back_size):
        assert s(0, 100, 64, 0) == 0 and s(10, 100, 12, 0) == 0 and s(10, 100, 64, 5) == 0
        assert s(10, 100, 64, 0) > 0
    # P's room is bounded, however large the vocabulary: 512 MiB of it, dh's parts, the gathered rows
    assert back_size(32768, 130000, 768, 0) < (512 << 20) + 2 * 32768 * 768 * 4 + 32768 * 768 * 2 + (192 << 20)
    assert size(32768, 130000, 768, 0) < 32768 * 130000 * 4 // 50


@pytest.mark.parametrize("n, vocab, d, dt", [(1, 1, 8, 0), (40, 4500001, 512, 0), (130, 100000, 128, 0),
                                             (8192, 30522, 768, 0), (200000, 1000, 64, 0), (1 << 22, 1000, 8, 1),
                                             (32768, 30522, 256, 2), (9000, 100, 512, 2)])
def test_backward_workspace_of_the_loss_is_what_the_header_says(L, n, vocab, d, dt):
    """A copy of the rows, a piece of P, dh's sums and dw's parts, each as stated, and 20 bytes a row and some
    lines beside them."""
    def up(x, by):
        return -(-x // by) * by
    eb = 4 if dt == 2 else 2
    rows, tile = up(n, 256), 256 * 128 * 4
    piece = max(min(512 << 20, rows * up(vocab, 128) * eb), rows * 128 * eb)
    sums = max(up(n, 128) * up(d, 256) * 4, 128 << 20)
    size = L.maxsim_linear_cross_entropy_backward_workspace_size(n, vocab, d, dt)
    assert size <= n * up(d * eb, 64) + piece + sums + (128 << 20) + 20 * n + 4096
    # and no less than a whole tile of everything
    assert size >= n * d * eb + min(piece, rows * 128 * eb) + up(n, 128) * up(d, 256) * 4 >= tile


def test_mx4_c_entries_refuse(L):
    def q(x=P, n=4, d=64, dt=0, c=P, s=P):
        return L.maxsim_quantize_mx4(x, n, d, dt, c, s, None)

    def v(c=P, s=P, n=4, d=64, dt=0, x=P):
        return L.maxsim_dequantize_mx4(c, s, n, d, dt, x, None)
    for e in (q, v):
        assert e(x=None) == NULL and e(c=None) == NULL and e(s=None) == NULL
        assert e(x=P + 8) == ALIGN and e(c=P + 8) == ALIGN and e(dt=4) == DTYPE
        assert e(d=48) == SHAPE and e(d=16) == SHAPE and e(d=1056) == SHAPE and e(n=-1) == SHAPE and e(n=0) == OK

    def f(Q=P, qs=P, q=32, D=P, ds=P, off=P, n=10, nd=0, lens=None, d=128, out=P):
        return L.maxsim_score_mx4(Q, qs, q, D, ds, off, n, nd, lens, d, out, None)
    assert f(Q=None) == NULL and f(qs=None) == NULL and f(D=None) == NULL and f(ds=None) == NULL and f(out=None) == NULL
    assert f(q=0) == SHAPE and f(q=1025) == SHAPE and f(d=48) == SHAPE and f(d=1056) == SHAPE and f(n=-1) == SHAPE
    assert f(off=None) == SHAPE and f(lens=P) == UNSUP
    assert f(Q=P + 8) == ALIGN and f(D=P + 8) == ALIGN and f(out=P + 2) == ALIGN and f(off=P + 4) == ALIGN
    assert f(off=None, nd=4, lens=P + 2) == ALIGN
    assert f(q=513, d=256) == UNSUP and f(q=129, d=1024) == UNSUP and f(q=257, d=300 - 300 % 32) == UNSUP
    assert f(n=0) == OK


def test_4_bit_scores_of_no_documents_need_no_address(L):
    def f(Q=None, qs=None, q=32, D=None, ds=None, off=None, nd=4, lens=None, d=128, out=None):
        return L.maxsim_score_mx4(Q, qs, q, D, ds, off, 0, nd, lens, d, out, None)
    assert f() == OK and f(off=P) == OK and f(Q=P, qs=P, lens=P) == OK
    assert f(q=0) == SHAPE and f(nd=0) == SHAPE and f(d=48) == SHAPE and f(off=P, lens=P) == UNSUP
    assert f(q=129, d=1024) == UNSUP


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
def test_valid_calls_without_gpu_report_a_device_error(L):
    assert L.maxsim_rms_norm(P, 64, P, 64, 10, 64, 0, P, 2, 1e-6, 0.1, P, 0, P, P, P, None) == DEVICE
    assert L.maxsim_rms_norm_i8(P, 64, None, 0, 10, 64, 0, P, 2, 1e-6, P, P, None, None) == DEVICE
    assert L.maxsim_rms_norm_backward(P, None, P, 64, 10, 64, 0, P, 0, P, 0.0, None, 0, P, P, P, P, 1 << 20,
                                      None) == DEVICE
    assert L.maxsim_dropout(P, 10, 0, 0.5, P, 0, P, None) == DEVICE
    assert L.maxsim_linear_cross_entropy(P, P, P, 10, 100, 64, 0, 1.0, P, P, P, 1 << 40, None) == DEVICE
    assert L.maxsim_linear_cross_entropy_backward(P, P, P, P, P, 10, 100, 64, 0, 1.0, P, P, P, 1 << 40,
                                                  None) == DEVICE
    assert L.maxsim_quantize_mx4(P, 4, 64, 0, P, P, None) == DEVICE
    assert L.maxsim_dequantize_mx4(P, P, 4, 64, 0, P, None) == DEVICE
    assert L.maxsim_score_mx4(P, P, 32, P, P, P, 10, 0, None, 128, P, None) == DEVICE


# ---------------------------------------------------------------- the reference
def test_reference_generator_against_published_numbers():
    """The known answers that the generator's authors publish with it, for 10 rounds and 7."""
    zero, ones = ([0] * 4, [0] * 2), ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2)
    pi = ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0])
    assert ref.philox(*zero, 10) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox(*ones, 10) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox(*pi, 10) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]
    assert ref.philox(*zero, 7) == [0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48]
    # and the arrays of it that the masks come from
    rng, call = (-3, (7 << 32) + 5), 9
    keep, up = ref.kept(rng, call, 0.25, 3, 13)
    assert keep.shape == (3, 13) and up == np.float32(4 / 3)
    for r in range(3):
        for e in range(13):
            key = (1 << 64) - 3
            w = ref.philox([r * 2 + e // 8, 0, 5, 9], [key & ref.M32, key >> 32], 7)
            u = w[e % 8 // 2] >> 16 * (e % 2) & 0xFFFF
            assert keep[r, e] == (u >= 16384)


def differences(f, x, g, step=1e-5):
    """f's slope along a direction (64-bit central differences) against the gradient's: their truncation
    is some 1e-10 of the third derivative and their rounding 1e-11."""
    t = np.random.default_rng(8).standard_normal(x.shape)
    got = (f(x + step * t) - f(x - step * t)) / (2 * step)
    want = float((g * t).sum())
    assert abs(got - want) <= 1e-7 * max(1.0, float(np.abs(g * t).sum()))


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(5)
    x, r, w, gy, gh = (rng.standard_normal(s) for s in ((7, 24), (7, 24), (24,), (7, 24), (7, 24)))
    keep, up = ref.kept((3, 4), 0, 0.3, 7, 24)
    f = keep * np.float64(up)

    def value(x, r, w):
        h = r + x * f
        return float((ref.norm(h, w, 1e-6, f32)[0] * gy).sum() + (h * gh).sum())
    g = ref.norm_backward(r + x * f, w, 1e-6, gy, gh, f, f32, f32)
    differences(lambda v: value(v, r, w), x, g["dx"])
    differences(lambda v: value(x, v, w), r, g["dresidual"])
    differences(lambda v: value(x, r, v), w, g["dw"])
    h, w, dl = rng.standard_normal((6, 8)), rng.standard_normal((11, 8)), rng.standard_normal(6)
    y = np.array([3, 10, -1, 0, 11, 3])
    g = ref.loss(h, w, y, 0.7, dl)
    differences(lambda v: float((ref.loss(v, w, y, 0.7)["loss"] * dl).sum()), h, g["dh"])
    differences(lambda v: float((ref.loss(h, v, y, 0.7)["loss"] * dl).sum()), w, g["dw"])


def test_reference_of_4_bits():
    """A block's entries by hand: its largest is 6, so that the unit is 1."""
    x = np.zeros((1, 32))
    x[0, :12] = [6.0, -0.25, 0.26, 0.75, 1.25, -1.75, 2.5, 3.5, 5.0, 5.1, 0.0, -3.4]
    code, k = ref.mx4(x)
    assert k.tolist() == [[0]]
    assert code[0, :12].tolist() == [7, 8, 1, 2, 2, 8 + 4, 4, 6, 6, 7, 0, 8 + 5]
    x[0, 0] = 7.9  # saturates
    assert ref.mx4(x)[0][0, 0] == 7 and ref.mx4(x * 2.0 ** -9)[1][0, 0] == -9
