"""The cross entropy over a vocabulary and its gradients against a 64-bit reference."""
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
    (64, 777, 256, FP32, 1.0),
    (65, 500, 320, BF16, 1.0),     # the first size of the large tiles
    (129, 255, 24, FP16, 0.5),
    (200, 5000, 768, BF16, 0.7),
    (300, 1025, 1032, FP32, 0.15),
    (1023, 511, 128, FP16, 0.9),
    (1025, 513, 36, FP32, 0.5),    # more rows than one count
    (3000, 700, 88, BF16, 0.02),
])
def test_against_reference(n, vocab, d, dtype, share):
    print("case: cross entropy", n, vocab, d, dtype, share, flush=True)
    check(*make(n, vocab, d, dtype, share, seed=n), scale=0.7 if n % 2 else 1.0)
