"""Microscaled 4-bit vectors: codes and exponents bit for bit, and the scores of documents stored
in them against a 64-bit reference."""
import numpy as np
import pytest
import torch

import maxsim_scoring_fwd_amd as ms
import train_ref as ref
from encoder_ref import as64

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def rand(*shape, dtype=torch.float32, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def same_codes(x):
    codes, scales = ms.maxsim_quantize_mx4(x)
    want, k = ref.mx4(as64(x).reshape(-1, x.shape[-1]))
    assert np.array_equal(ref.unpack(codes).reshape(want.shape), want)
    assert np.array_equal(scales.cpu().numpy().reshape(k.shape), k + 127)
    values = ref.mx4_values(want, k).reshape(x.shape)
    assert np.array_equal(as64(ms.maxsim_dequantize_mx4(codes, scales)), values)
    back = ms.maxsim_dequantize_mx4(codes, scales, x.dtype)
    assert torch.equal(back.cpu(), torch.from_numpy(values).to(x.dtype))
    return codes, scales


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("n, d", [(1, 32), (3, 64), (17, 96), (1001, 128), (5, 1024)])
def test_quantise(n, d, dtype):
    print("case: quantise", n, d, dtype, flush=True)
    same_codes(rand(n, d, dtype=dtype, seed=n) * torch.logspace(-2, 2, n, device="cuda", dtype=dtype)[:, None])


def test_every_boundary():
    """Each value, each half between two, and their fp32 neighbours, at exponents from the smallest
    normal numbers' to the largest's."""
    v = torch.tensor(sorted({*ref.E2M1, *((ref.E2M1[1:] + ref.E2M1[:-1]) / 2), 7.0}), dtype=torch.float32)
    up = torch.nextafter(v, torch.tensor(8.0))
    down = torch.nextafter(v, torch.tensor(0.0))
    v = torch.cat([v, up, down])
    v = torch.cat([v, -v])
    rows = []
    for e in (-120, -60, -1, 0, 1, 60, 125 - 1):
        for a in range(0, len(v), 31):
            part = v[a:a + 31]
            row = torch.zeros(32)
            row[1:1 + len(part)] = part
            row[0] = 6.5  # the block's exponent is that of 4 .. 8
            rows.append(row * 2.0 ** e)
    same_codes(torch.stack(rows).cuda())


def test_small_blocks_zeros_and_what_is_no_number():
    x = torch.zeros(6, 64, device="cuda")
    x[0, 5] = -0.0
    x[1, :32] = torch.arange(32, device="cuda") * 2.0 ** -149   # subnormal numbers
    x[1, 32:] = torch.arange(32, device="cuda") * 2.0 ** -131
    x[2, 7] = 3.0e38
    same_codes(x)
    x[3, 40] = float("nan")
    x[4, 3] = float("inf")
    x[4, 40] = -1.0
    codes, scales = ms.maxsim_quantize_mx4(x)
    assert scales[3].tolist() == [0, 255] and scales[4, 0] == 255 and scales[4, 1] == 125
    assert not codes[3].any() and not codes[4, :16].any() and codes[4, 16:].any()
    v = ms.maxsim_dequantize_mx4(codes, scales)
    assert torch.isnan(v[3, 32:]).all() and torch.isnan(v[4, :32]).all() and v[4, 40] == -1


def scores(q_len, lens, d, layout, seed=0):
    nd = max(max(lens), 1)
    q = rand(q_len, d, seed=seed) * torch.logspace(-1, 1, q_len, device="cuda")[:, None]
    rows = sum(lens) if layout == "packed" else len(lens) * nd
    x = rand(max(rows, 1), d, seed=seed + 1)[:rows] * torch.logspace(-1, 1, max(rows, 1), device="cuda")[:rows, None]
    Q, qs = ms.maxsim_quantize_mx4(q)
    D, ds = ms.maxsim_quantize_mx4(x)
    vq, vd = as64(ms.maxsim_dequantize_mx4(Q, qs)), as64(ms.maxsim_dequantize_mx4(D, ds))
    if layout == "packed":
        off = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int64, device="cuda")
        got = ms.maxsim_score_mx4(Q, qs, D, ds, off)
        docs = [vd[a:b] for a, b in zip(off.tolist()[:-1], off.tolist()[1:])]
    else:
        n = len(lens)
        t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        got = ms.maxsim_score_mx4(Q, qs, D.view(n, nd, -1), ds.view(n, nd, -1), doc_lens=t if layout == "lens" else None)
        docs = [vd[b * nd:b * nd + (k if layout == "lens" else nd)] for b, k in enumerate(lens)]
    want, tol = ref.mx4_scores(vq, docs)
    ref.close(got, want, tol, "scores")


@pytest.mark.parametrize("layout", ["packed", "lens", "fixed"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 256, 288, 512, 640, 1024])
def test_scores(d, layout):
    for q_len in (1, 16, 17, 33, 64):
        print("case: 4-bit scores", d, layout, q_len, flush=True)
        scores(q_len, [5, 0, 1, 16, 17, 40, 0, 128, 33], d, layout, seed=q_len)


@pytest.mark.parametrize("q_len, d", [(65, 128), (129, 96), (300, 128), (1024, 128), (512, 256), (100, 512), (128, 1024)])
def test_scores_of_long_queries(q_len, d):
    print("case: 4-bit scores, long query", q_len, d, flush=True)
    scores(q_len, [5, 0, 1, 16, 17, 140], d, "packed")
    scores(q_len, [7, 31, 0], d, "lens")


def test_many_documents():
    rng = np.random.default_rng(3)
    scores(32, rng.integers(0, 90, 9001).tolist(), 64, "packed")
    scores(20, [48] * 30011, 32, "fixed")


def test_empty_collections():
    """No documents, and documents without a token, in tensors that have no address."""
    Q, qs = ms.maxsim_quantize_mx4(rand(32, 128))

    def empty(*shape):
        return torch.empty(shape, dtype=torch.uint8, device="cuda")
    zeros = torch.zeros(5, dtype=torch.int64, device="cuda")
    assert empty(0, 64).data_ptr() == 0
    assert ms.maxsim_score_mx4(Q, qs, empty(0, 7, 64), empty(0, 7, 4)).shape == (0,)
    lens = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert ms.maxsim_score_mx4(Q, qs, empty(0, 7, 64), empty(0, 7, 4), doc_lens=lens).shape == (0,)
    assert ms.maxsim_score_mx4(Q, qs, empty(0, 64), empty(0, 4), zeros[:1]).shape == (0,)
    D, ds = ms.maxsim_quantize_mx4(rand(0, 128))
    got = ms.maxsim_score_mx4(Q, qs, D, ds, zeros)
    assert got.tolist() == [-float("inf")] * 4
    Q, qs = ms.maxsim_quantize_mx4(rand(100, 128))  # its operands from LDS
    assert ms.maxsim_score_mx4(Q, qs, D, ds, zeros).tolist() == [-float("inf")] * 4
    for d in (32, 64, 512):
        Q, qs = ms.maxsim_quantize_mx4(rand(20, d))
        D, ds = ms.maxsim_quantize_mx4(rand(0, d))
        assert ms.maxsim_score_mx4(Q, qs, D, ds, zeros).tolist() == [-float("inf")] * 4


@pytest.mark.parametrize("d", [32, 64, 128, 512])
def test_blocks_that_are_no_number_stay_in_their_document(d):
    """A NaN in one token leaves its own document's score undefined, and every other as it is."""
    lens = [20, 70, 64, 5, 0, 33]
    x = rand(sum(lens), d, seed=d)
    off = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int64, device="cuda")
    for q_len in (20, 70):
        Q, qs = ms.maxsim_quantize_mx4(rand(q_len, d))
        want = ms.maxsim_score_mx4(Q, qs, *ms.maxsim_quantize_mx4(x), off)
        for b, at in ((1, 20), (1, 89), (2, 100), (5, 191)):
            bad = x.clone()
            bad[at, 3] = float("nan")
            got = ms.maxsim_score_mx4(Q, qs, *ms.maxsim_quantize_mx4(bad), off)
            others = [i for i in range(len(lens)) if i != b]
            assert torch.equal(got[others], want[others])
    fixed = x[:180].view(6, 30, d)
    Q, qs = ms.maxsim_quantize_mx4(rand(20, d))
    want = ms.maxsim_score_mx4(Q, qs, *ms.maxsim_quantize_mx4(fixed))
    bad = fixed.clone()
    bad[2, 29, d - 1] = float("inf")
    got = ms.maxsim_score_mx4(Q, qs, *ms.maxsim_quantize_mx4(bad))
    assert torch.equal(got[[0, 1, 3, 4, 5]], want[[0, 1, 3, 4, 5]])
