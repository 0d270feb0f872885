"""Attention, rotary positions and clipping without a GPU: what the binding and the C entry
points refuse, sizes of workspaces, and the test reference's gradients against differences."""
import ctypes

import numpy as np
import pytest
import torch

import encoder_ref as ref
import maxsim_scoring_fwd_amd as ms

bf, f16, f32, i32, i64 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.int64
OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, DEVICE = 0, -1, -2, -3, -4, -5, -7
P = 0x10000  # a 16-byte aligned stand-in address; never dereferenced by these calls


@pytest.fixture(scope="module")
def L():
    return ms.lib()


def Z(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


def refuses(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


OFF = torch.tensor([0, 4, 10], dtype=i64)


def test_attention_binding_refuses():
    q, k = Z(10, 4, 64), Z(10, 2, 64)
    att = ms.maxsim_attention
    refuses("k must have dtype", att, q, k.half(), k, OFF)
    refuses("q must have dtype", att, q.int(), k, k, OFF)
    refuses("v has shape", att, q, k, Z(9, 2, 64), OFF)
    refuses("k has shape", att, q, Z(10, 2, 32), k, OFF)
    refuses("k has 2 heads, v has 1", att, q, k, Z(10, 1, 64), OFF)
    refuses("cannot share", att, q, Z(10, 3, 64), Z(10, 3, 64), OFF)
    refuses("3 dimensions", att, Z(2, 5, 4, 64), k, k, OFF)
    refuses("4 dimensions", att, q, k, k)
    refuses("doc_offsets must have dtype", att, q, k, k, OFF.int())
    refuses("at least|>= 1 entries", att, q, k, k, OFF[:0])
    refuses("not both", att, q, k, k, OFF, torch.zeros(2, dtype=i32))
    refuses("needs causal", att, q, k, k, OFF, prefix_lens=torch.zeros(2, dtype=i32))
    refuses("prefix_lens must have", att, q, k, k, OFF, causal=True, prefix_lens=torch.zeros(2, dtype=i64))
    refuses("prefix_lens must have shape", att, q, k, k, OFF, causal=True,
            prefix_lens=torch.zeros(3, dtype=i32))
    refuses("slopes must have dtype", att, q, k, k, OFF, slopes=Z(4))
    refuses("slopes must have shape", att, q, k, k, OFF, slopes=Z(2, dtype=f32))
    refuses("scale must be positive", att, q, k, k, OFF, scale=-1.0)
    refuses("scale must be positive", att, q, k, k, OFF, scale=float("nan"))
    refuses("softcap must be", att, q, k, k, OFF, softcap=-2.0)
    refuses("softcap must be", att, q, k, k, OFF, softcap=float("inf"))
    refuses("side by side", att, Z(10, 64, 4).transpose(1, 2), k, k, OFF)
    refuses("device tensor", att, q, k, k, OFF)
    Q, K = Z(2, 5, 4, 64), Z(2, 5, 2, 64)
    refuses("doc_lens must have dtype", att, Q, K, K, None, torch.zeros(2, dtype=i64))
    refuses("doc_lens must have shape", att, Q, K, K, None, torch.zeros(3, dtype=i32))
    bwd = ms.maxsim_attention_backward
    refuses("device tensor", bwd, q, q, k, k, q, Z(4, 10, dtype=f32), OFF)


def test_rotary_binding_refuses():
    x, f = Z(10, 4, 64), Z(32, dtype=f32)
    rot = ms.maxsim_rotary
    refuses("x must have dtype", rot, x.int(), f)
    refuses("3 dimensions", rot, Z(10, 64), f)
    refuses("freq must have dtype", rot, x, f.double())
    refuses("33 entries", rot, x, Z(33, dtype=f32))
    refuses("0 entries", rot, x, Z(0, dtype=f32))
    refuses("layout must be", rot, x, f, layout="pairs")
    refuses("not both", rot, x, f, OFF, torch.zeros(10, dtype=i32))
    refuses("positions must have dtype", rot, x, f, positions=torch.zeros(10, dtype=i64))
    refuses("positions must have shape", rot, x, f, positions=torch.zeros(9, dtype=i32))
    refuses("side by side", rot, Z(10, 64, 4).transpose(1, 2), f)
    refuses("device tensor", rot, x, f)


def test_clip_binding_refuses():
    clip = ms.maxsim_clip_grad_norm
    refuses("at least one", clip, [], 1.0)
    refuses("holds 1 tensors", clip, [Z(3), Z(4)], 1.0, out=[Z(3)])
    refuses("negative", clip, [Z(3)], -1.0)
    refuses("negative", clip, [Z(3)], float("nan"))
    refuses("unsupported dtype", clip, [torch.zeros(3, dtype=torch.float64)], 1.0)
    refuses("contiguous", clip, [Z(4, 6).t()], 1.0)
    refuses("device tensor", clip, [Z(3)], 1.0)


def desc(**k):
    """maxsim_attention_desc as the header lays it out."""
    t = dict(data=P, token_stride=4 * 64, head_stride=64, doc_stride=5 * 4 * 64)
    f = [x for n in "qkv" for x in {**t, **k.pop(n, {})}.values()]
    base = dict(doc_offsets=P, doc_lens=0, n_tokens=10, n_docs=2, prefix_lens=0, slopes=0, nd=0,
                n_heads=4, n_kv_heads=4, d=64, dtype=0, causal=0, softcap=0.0, scale=0.125)
    assert set(k) <= set(base)
    return ms._ATTENTION_DESC.pack(*(x or 0 for x in f), *(x or 0 for x in {**base, **k}.values()))


def test_attention_c_entry_refuses(L):
    def f(o=P, lse=P, **k):
        return L.maxsim_attention(desc(**k), o, lse, None)
    assert L.maxsim_attention(None, P, P, None) == NULL
    assert f(o=None) == NULL and f(lse=None) == NULL
    assert f(q=dict(data=None)) == NULL
    assert f(o=P + 8) == ALIGN and f(lse=P + 2) == ALIGN and f(doc_offsets=P + 4) == ALIGN
    assert f(k=dict(data=P + 2)) == ALIGN
    assert f(k=dict(token_stride=4)) == ALIGN
    assert f(v=dict(head_stride=12)) == ALIGN
    assert f(q=dict(token_stride=-256)) == SHAPE
    assert f(q=dict(token_stride=1 << 24)) == SHAPE
    assert f(dtype=5) == DTYPE
    assert f(d=60) == SHAPE and f(d=264) == SHAPE and f(d=0) == SHAPE
    assert f(n_kv_heads=3) == SHAPE and f(n_heads=0) == SHAPE
    assert f(n_tokens=1 << 31) == SHAPE and f(n_tokens=-1) == SHAPE
    assert f(scale=0.0) == SHAPE and f(scale=float("inf")) == SHAPE and f(softcap=-1.0) == SHAPE
    assert f(prefix_lens=P) == UNSUP
    assert f(doc_lens=P) == UNSUP
    assert f(doc_offsets=None, nd=4) == SHAPE          # 2 documents of 4 are not 10 tokens
    assert f(n_tokens=0, q=dict(data=None)) == OK      # nothing to do
    assert f(doc_offsets=None, nd=0, n_tokens=0) == OK

    def g(dq=P, dk=P, dv=P, ws=P, n=1 << 20, **k):
        return L.maxsim_attention_backward(desc(**k), P, P, P, dq, dk, dv, ws, n, None)
    assert g(ws=None) == NULL and g(ws=P + 8) == ALIGN and g(n=100) == SHAPE
    assert g(dk=None) == NULL and g(dv=None) == NULL
    assert g(dq=P + 8) == ALIGN
    assert g(dq=None, dk=None, dv=None) == OK
    assert L.maxsim_attention_backward_workspace_size(-1, 4) == 0
    assert L.maxsim_attention_backward_workspace_size(10, 0) == 0
    assert L.maxsim_attention_backward_workspace_size(10, 4) >= 160


def test_rotary_c_entry_refuses(L):
    def f(x=P, n=10, heads=4, d=64, ts=256, hs=64, dt=0, freq=P, rot=64, layout=0, off=None, docs=0,
          pos=None, out=P):
        return L.maxsim_rotary(x, n, heads, d, ts, hs, dt, freq, rot, layout, 1.0, 0, off, docs, pos,
                               out, ts, hs, None)
    assert f(x=None) == NULL and f(freq=None) == NULL and f(out=None) == NULL
    assert f(x=P + 1) == ALIGN and f(freq=P + 2) == ALIGN and f(pos=P + 2) == ALIGN
    assert f(off=P + 4, docs=1) == ALIGN
    assert f(dt=4) == DTYPE
    assert f(rot=0) == SHAPE and f(rot=66) == SHAPE and f(rot=31) == SHAPE
    assert f(d=63, rot=32) == SHAPE and f(d=1026) == SHAPE and f(heads=0) == SHAPE
    assert f(heads=2048) == SHAPE
    assert f(n=-1) == SHAPE and f(n=0) == OK
    assert f(layout=2) == UNSUP
    assert f(off=P, docs=1, pos=P) == UNSUP


def test_clip_c_entry_refuses(L):
    one = lambda v, t: (t * 1)(v)  # noqa: E731
    src, num, dt = one(P, ctypes.c_uint64), one(5, ctypes.c_int64), one(0, ctypes.c_int32)

    def f(src=src, out=None, num=num, dt=dt, n=1, mx=1.0, norm=P, ws=P, size=1 << 20):
        return L.maxsim_clip_grad_norm(src, out, num, dt, n, mx, norm, ws, size, None)
    assert f(src=None) == NULL and f(norm=None) == NULL and f(ws=None) == NULL
    assert f(src=one(0, ctypes.c_uint64)) == NULL
    assert f(src=one(P + 1, ctypes.c_uint64)) == ALIGN and f(ws=P + 4) == ALIGN
    assert f(norm=P + 2) == ALIGN
    assert f(num=one(-1, ctypes.c_int64)) == SHAPE and f(n=-1) == SHAPE
    assert f(mx=-1.0) == SHAPE and f(mx=float("nan")) == SHAPE and f(size=8) == SHAPE
    assert f(dt=one(7, ctypes.c_int32)) == DTYPE
    size = L.maxsim_clip_grad_norm_workspace_size
    assert size(-1) == 0 and size(0) == size(1) > 0 and size(1000) > size(10)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU error path")
def test_valid_calls_without_gpu_report_a_device_error(L):
    assert L.maxsim_attention(desc(), P, P, None) == DEVICE
    assert L.maxsim_attention_backward(desc(), P, P, P, P, P, P, P, 1 << 20, None) == DEVICE
    assert L.maxsim_rotary(P, 10, 4, 64, 256, 64, 0, P, 64, 0, 1.0, 0, None, 0, None, P, 256, 64,
                           None) == DEVICE


@pytest.mark.parametrize("causal, prefix, cap, bias", [
    (False, None, 0.0, False), (True, None, 0.0, True), (True, [3, 0, 9], 4.0, False),
    (False, None, 2.5, True)])
def test_reference_gradients_against_differences(causal, prefix, cap, bias):
    """64-bit central differences: with a step of 1e-5 their truncation is about 1e-10 of the
    third derivative and their rounding 1e-11; 1e-7 leaves room for both."""
    rng = np.random.default_rng(5)
    docs = [(0, 6), (6, 1), (7, 8)]
    q, k, v = (rng.standard_normal((15, h, 8)) for h in (4, 2, 2))
    do = rng.standard_normal(q.shape)
    slopes = np.array([0.5, 0.1, 0.0, 0.3]) if bias else None
    kw = dict(docs=docs, causal=causal, prefix=prefix, cap=cap, slopes=slopes)
    g = ref.attention(q, k, v, do=do, **kw)
    for name, at in (("dq", 0), ("dk", 1), ("dv", 2)):
        x = [q, k, v]
        step = rng.standard_normal(x[at].shape)
        side = []
        for e in (1e-5, -1e-5):
            y = list(x)
            y[at] = x[at] + e * step
            side.append(float((ref.attention(*y, **kw)["o"] * do).sum()))
        got, want = (side[0] - side[1]) / 2e-5, float((g[name] * step).sum())
        assert abs(got - want) <= 1e-7 * max(1.0, float(np.abs(g[name] * step).sum()))


def test_attention_c_entry_refuses_more_documents_than_it_counts(L):
    for n in (1 << 31, (1 << 63) - 1):
        assert L.maxsim_attention(desc(n_docs=n), P, P, None) == SHAPE
    assert L.maxsim_attention(desc(n_docs=(1 << 31) - 8), P, P, None) == SHAPE  # times 4 heads


def test_clip_binding_refuses_what_is_no_tensor():
    clip = ms.maxsim_clip_grad_norm
    refuses("at least one", clip, [None, None], 1.0)
    refuses("must be a tensor", clip, [Z(3), 2.0], 1.0)
    refuses("must be a tensor", clip, [Z(3), Z(4)], 1.0, out=[Z(3), None])
    refuses("must be a tensor", clip, [Z(3), None, 2.0], 1.0)
    refuses("device tensor", clip, [Z(3), None], 1.0)


class On0(torch.Tensor):
    """A tensor that says it is on device 0; calls that have to be refused never read it."""
    index = 0
    is_cuda = True

    def get_device(self):
        return self.index


class On1(On0):
    index = 1


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0)
    here, there = (lambda t: t.as_subclass(On0)), (lambda t: t.as_subclass(On1))
    q = here(Z(10, 4, 64))
    off = here(OFF)
    args = dict(doc_offsets=OFF, prefix_lens=torch.zeros(2, dtype=i32), slopes=Z(4, dtype=f32),
                out=Z(10, 4, 64), lse=Z(4, 10, dtype=f32))
    for name in args:
        kw = {n: (there if n == name else here)(t) for n, t in args.items()}
        refuses(f"{name} is on cuda:1, expected cuda:0", ms.maxsim_attention, q, q, q, causal=True, **kw)
    refuses("v is on cuda:1", ms.maxsim_attention, q, q, there(q), off)
    Q = here(Z(2, 5, 4, 64))
    refuses("doc_lens is on cuda:1", ms.maxsim_attention, Q, Q, Q, doc_lens=there(torch.zeros(2, dtype=i32)))
    args = dict(grad_o=Z(10, 4, 64), o=Z(10, 4, 64), lse=Z(4, 10, dtype=f32), dq=Z(10, 4, 64),
                dk=Z(10, 4, 64), dv=Z(10, 4, 64), workspace=torch.zeros(1 << 16, dtype=torch.uint8))
    for name in args:
        kw = {n: (there if n == name else here)(t) for n, t in args.items()}
        refuses(f"{name} is on cuda:1", ms.maxsim_attention_backward, q=q, k=q, v=q, doc_offsets=off, **kw)
    args = dict(freq=Z(32, dtype=f32), doc_offsets=OFF, out=Z(10, 4, 64))
    for name in args:
        kw = {n: (there if n == name else here)(t) for n, t in args.items()}
        refuses(f"{name} is on cuda:1", ms.maxsim_rotary, q, **kw)
    refuses("positions is on cuda:1", ms.maxsim_rotary, q, here(Z(32, dtype=f32)),
            positions=there(torch.zeros(10, dtype=i32)), out=q)
    # all of them on one device that is not the current one
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    refuses("the current device is cuda:1", ms.maxsim_rotary, q, here(Z(32, dtype=f32)), out=q)
    refuses("the current device is cuda:1", ms.maxsim_attention, q, q, q, off, out=here(Z(10, 4, 64)),
            lse=here(Z(4, 10, dtype=f32)))


@pytest.mark.gpu
def test_clipping_on_another_device_is_refused(monkeypatch):
    g = [torch.ones(5, device="cuda")]
    norm, ws = torch.zeros((), device="cuda"), torch.zeros(1 << 14, dtype=torch.uint8, device="cuda")
    for name, t in (("norm", norm), ("workspace", ws)):
        kw = dict(dict(norm=norm, workspace=ws), **{name: t.as_subclass(On1)})
        refuses(f"{name} is on cuda:1", ms.maxsim_clip_grad_norm, g, 1.0, **kw)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    refuses("the current device is cuda:1", ms.maxsim_clip_grad_norm, g, 1.0, norm=norm, workspace=ws)
