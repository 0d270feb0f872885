"""Calls on another stream than the current one: the buffers made inside a call are ordered on
both streams. The allocator gives a block that was freed on a stream to that stream's next request
at once, with work on it still queued, so a buffer for another stream has to come from that
stream's own memory, and one that the caller reads on the current stream is not to be handed out
again before the current stream is past that."""
import pytest

from gpu_util import ms, say

pytestmark = pytest.mark.gpu

N, H, D = 4096, 4, 64


def T():
    import torch
    return torch


@pytest.fixture(scope="module")
def data():
    t = T()
    g = t.Generator().manual_seed(5)
    q, k, v, do = (t.randn(N, H, D, generator=g).bfloat16().cuda() for _ in range(4))
    off = t.tensor([0, 1000, 2500, N]).cuda()
    o, lse = ms().maxsim_attention(q, k, v, off)
    freq = (10000.0 ** (-t.arange(D // 2, dtype=t.float64) / (D // 2))).float().cuda()
    long = t.randn(8192, 8192, device="cuda")
    out = t.empty_like(q)
    Q, docs = do[:32, 0].contiguous(), q[:, 0].contiguous()
    arg = ms().maxsim_score_argmax(Q, docs, off)[2]
    scoring = dict(Q=Q, docs=docs, arg=arg, do_scores=t.randn(3, device="cuda"),
                   book=t.randn(8, 256, D // 8, generator=g).cuda())
    t.mm(long, long)  # whatever its first call prepares
    t.cuda.synchronize()
    return dict(q=q, k=k, v=v, do=do, off=off, o=o, lse=lse, freq=freq, long=long, out=out, **scoring)


def attention(x, stream):
    return list(ms().maxsim_attention(x["q"], x["k"], x["v"], x["off"], stream=stream))


def backward(x, stream):
    return list(ms().maxsim_attention_backward(x["do"], x["q"], x["k"], x["v"], x["o"], x["lse"],
                                               x["off"], stream=stream))


def rotary(x, stream):
    return [ms().maxsim_rotary(x["q"], x["freq"], x["off"], stream=stream)]


def clip(x, stream):
    return [ms().maxsim_clip_grad_norm([x["q"]], 0.5, out=[x["out"]], stream=stream)]


def score(x, stream):
    return [ms().maxsim_score(x["Q"], x["docs"], x["off"], stream=stream),
            ms().maxsim_score_fixed(x["Q"], x["docs"].view(64, 64, D), stream=stream)]


def argmax(x, stream):
    return list(ms().maxsim_score_argmax(x["Q"], x["docs"], x["off"], stream=stream))


def batch(x, stream):
    return [ms().maxsim_score_batch(x["Q"].view(2, 16, D), x["docs"].view(64, 64, D),
                                    stream=stream)]


def score_backward(x, stream):
    return list(ms().maxsim_backward(x["Q"], x["docs"], x["arg"], x["do_scores"], x["off"],
                                     stream=stream))


def topk(x, stream):
    return list(ms().maxsim_topk(x["long"][0], 5, stream=stream))


def pq(x, stream):
    return [ms().maxsim_pq_tables(x["Q"], x["book"], stream=stream)]


CALLS = [attention, backward, rotary, clip, score, argmax, batch, score_backward, topk, pq]


def handle(t, stream, as_int):
    return stream.cuda_stream if as_int else stream


@pytest.mark.parametrize("as_int", [False, True])
@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_buffers_freed_on_the_current_stream_are_left_alone(data, call, as_int):
    """A tensor of each buffer's size is read by the current stream behind long work and freed
    before it is read: a call on another stream must not write to its block."""
    t = T()
    say("case: freed on the current stream", call.__name__)
    want = [x.clone() for x in call(data, None)]
    side = t.cuda.Stream()
    t.cuda.synchronize()
    t.cuda.empty_cache()
    old = [t.full_like(x, 3.0) for x in want]
    t.cuda.synchronize()
    for _ in range(4):
        t.mm(data["long"], data["long"])
    kept = [x.clone() for x in old]
    at = {x.data_ptr() for x in old}
    del old
    got = call(data, handle(t, side, as_int))
    assert not at & {x.data_ptr() for x in got}
    t.cuda.synchronize()
    assert all(bool((x == 3.0).all()) for x in kept)
    assert all(t.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_results_read_on_the_current_stream_are_kept(data, call):
    """Results of a call on another stream, read by the current stream behind long work and
    dropped: the next call on that stream must not write to their blocks before."""
    t = T()
    say("case: read on the current stream", call.__name__)
    want = [x.clone() for x in call(data, None)]
    side = t.cuda.Stream()
    t.cuda.synchronize()
    got = call(data, side)
    side.synchronize()
    for _ in range(4):
        t.mm(data["long"], data["long"])
    kept = [x.clone() for x in got]
    at = {x.data_ptr() for x in got}
    del got
    again = call(data, side)
    assert not at & {x.data_ptr() for x in again}
    t.cuda.synchronize()
    assert all(t.equal(a, b) for a, b in zip(kept, want))
    assert all(t.equal(a, b) for a, b in zip(again, want))


def test_current_stream_without_torchs_private_functions(data, monkeypatch):
    t = T()
    say("case: public stream functions")
    side = t.cuda.Stream()
    for stream in (t.cuda.current_stream(), side):
        with t.cuda.stream(stream):
            handles = []
            for raw in (True, False):
                monkeypatch.setattr(ms(), "_RAW_STREAMS", raw)
                handles.append((ms()._current_device(), ms()._stream(None)))
            assert handles[0] == handles[1] == (t.cuda.current_device(), stream.cuda_stream)
    want = rotary(data, None)
    t.cuda.synchronize()
    monkeypatch.setattr(ms(), "_RAW_STREAMS", False)
    assert t.equal(rotary(data, None)[0], want[0]) and t.equal(attention(data, None)[0], data["o"])
