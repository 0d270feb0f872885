"""Plain 64-bit implementations of the norm with the residual's addition, dropout, the cross
entropy over a vocabulary and the 4-bit vectors, with bounds on what the kernels may be off by.
Test infrastructure: CPU, numpy, straight from the formulas."""
from __future__ import annotations

import math

import numpy as np
import torch

from encoder_ref import HALF_STEP, TINY, U32, as64

M32 = 0xFFFFFFFF


def philox(counter, key, rounds):
    """The generator in whole numbers of any size: counter of four and key of two 32-bit words."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & M32, (p >> 32) ^ c[3] ^ k[1], p & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def kept(rng, call, p, rows, d, first_block=0):
    """(which entries [rows, d] are kept, what they are multiplied by in fp32)."""
    key, step = int(rng[0]) & (1 << 64) - 1, int(rng[1]) & M32
    least = int(np.rint(p * 65536))
    per = -(-d // 8)
    at = first_block + np.arange(rows * per, dtype=np.uint64)
    c = [at & np.uint64(M32), at >> np.uint64(32), np.full_like(at, step), np.full_like(at, call)]
    k0, k1 = key & M32, key >> 32
    for _ in range(7):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & np.uint64(M32),
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & np.uint64(M32)]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    u = np.stack([w >> np.uint64(s) & np.uint64(0xFFFF) for w in c for s in (0, 16)], 1)
    keep = (u.reshape(rows, per * 8)[:, :d] >= least)
    return keep, np.float32(65536 / (65536 - least)) if least < 65536 else np.float32(0)


def dropped(x: torch.Tensor, rng, call, p) -> torch.Tensor:
    """Dropout of x, bit for bit: one product in 32 bits, one rounding."""
    keep, up = kept(rng, call, p, 1, x.numel())
    v = x.detach().cpu().float() * torch.tensor(up)
    return torch.where(torch.from_numpy(keep).view(x.shape), v, torch.zeros(())).to(x.dtype)


# Longest chain of additions in a norm's reductions: 32 entries of a lane, then 8 steps across lanes.
NORM_CHAIN = 48


def norm(h, w, eps, dtype):
    """y of rows h [n, d] in 64 bits (as the kernel hands it on), and its bound."""
    rstd = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    y = h * rstd * w
    # the mean is off by its chain, rstd by half of that and three roundings, y by two more
    rel = (NORM_CHAIN / 2 + 8) * U32
    return y, np.abs(y) * (HALF_STEP[dtype] + rel) + TINY[dtype], rstd


def norm_backward(h, w, eps, gy, gh, factor, dtype, wdtype):
    """dict of dresidual, dx, dw and their bounds; factor: dropout's, or 1."""
    rows, d = h.shape
    rstd = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    n, g = h * rstd, gy * w
    dot = (g * n).mean(1, keepdims=True)
    dr = rstd * (g - n * dot) + gh
    rel = (NORM_CHAIN / 2 + 8) * U32
    tdot = (NORM_CHAIN + 4) * U32 * np.abs(g * n).mean(1, keepdims=True) + rel * np.abs(g * n).mean(1, keepdims=True)
    # rstd's error, n's, the product's, the difference's, and the sum with gh
    tdr = rstd * (np.abs(g) * (2 * rel) + np.abs(n) * (np.abs(dot) * 3 * rel + tdot)) + 2 * U32 * (np.abs(dr) + np.abs(gh))
    u, tiny = HALF_STEP[dtype], TINY[dtype]
    dw = (gy * n).sum(0)
    tdw = np.abs(gy * n).sum(0) * ((rows + 200) * U32 + rel) + HALF_STEP[wdtype] * np.abs(dw) + TINY[wdtype]
    dx = dr * factor
    return {"dresidual": dr, "tol_dresidual": tdr + u * np.abs(dr) + tiny, "dx": dx,
            "tol_dx": tdr * factor + (u + 2 * U32) * np.abs(dx) + tiny, "dw": dw, "tol_dw": tdw}


def loss(h, w, labels, scale, dl=None, dtype=torch.float32):
    """dict of loss and lse (and dh and dw with dl, the losses' gradient) in 64 bits, with bounds."""
    n, d = h.shape
    V = w.shape[0]
    ok = (labels >= 0) & (labels < V)
    r = {"loss": np.zeros(n), "lse": np.full(n, -math.inf), "tol_loss": np.zeros(n), "tol_lse": np.zeros(n)}
    r["dh"], r["dw"] = np.zeros(h.shape), np.zeros(w.shape)
    r["tol_dh"], r["tol_dw"] = np.zeros(h.shape), np.full(w.shape, TINY[dtype])
    if not ok.any():
        return r
    H, y = h[ok], labels[ok]
    one = np.arange(len(y))
    z = scale * (H @ w.T)
    dz = (d + 6) * U32 * scale * (np.abs(H) @ np.abs(w).T) + 4 * U32 * np.abs(z)
    m = z.max(1, keepdims=True)
    lse = m[:, 0] + np.log(np.exp(z - m).sum(1))
    # the sum: its chain (128 entries of a lane, the tiles' parts), the exponentials (two units of
    # 2^-23 and their argument's rounding), the logarithm and its factor
    size = np.abs(z).max(1)
    tlse = dz.max(1) + U32 * (128 + V / 32 + 40) + 8 * U32 * (size + 1) + 4 * U32 * np.abs(lse)
    r["loss"][ok], r["lse"][ok] = lse - z[one, y], lse
    r["tol_lse"][ok] = tlse
    r["tol_loss"][ok] = tlse + dz[one, y] + 4 * U32 * np.abs(z[one, y])
    if dl is None:
        return r
    p = np.exp(z - lse[:, None])
    rel = dz + tlse[:, None] + 8 * U32 * (np.abs(z) + np.abs(lse[:, None]) + 1)
    tp = p * rel
    p[one, y] -= 1
    f = (dl[ok] * scale)[:, None]
    u = HALF_STEP[dtype]
    P = p * f
    # rounding of P as an operand; fp16 scaled so that the largest gradient is 2^14 or more
    least = {torch.float16: 2.0 ** -38 * np.abs(f).max()}.get(dtype, 2.0 ** -133)
    tP = np.abs(f) * (tp + 2 * U32 * np.abs(p)) + np.abs(P) * u * (dtype != torch.float32) + least
    dh, dw = P @ w, P.T @ H
    r["dh"][ok], r["dw"] = dh, dw
    r["tol_dh"][ok] = (tP + V * U32 * np.abs(P)) @ np.abs(w) + u * np.abs(dh) + TINY[dtype]
    r["tol_dw"] = (tP + len(y) * U32 * np.abs(P)).T @ np.abs(H) + u * np.abs(dw) + TINY[dtype]
    return r


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def mx4(x):
    """(codes [rows, d] one entry each, exponents [rows, d / 32]) of finite x, entry by entry against
    the halves between neighbouring values."""
    rows, d = x.shape
    b = x.reshape(rows, d // 32, 32)
    most = np.abs(b).max(2)
    _, e = np.frexp(most)
    k = np.where(most > 0, np.maximum(e - 3, -127), -127)
    v = np.abs(b) * np.ldexp(1.0, -k)[..., None]
    middle = (E2M1[1:] + E2M1[:-1]) / 2
    above, at = (v[..., None] > middle).sum(-1), (v[..., None] == middle)
    # a tie goes to the even code
    code = above + (at & (np.arange(7) % 2 == 1)).any(-1)
    return (code | np.signbit(b) << 3).reshape(rows, d).astype(np.uint8), k


def mx4_values(codes, k):
    v = np.where(codes & 8, -1, 1) * E2M1[codes & 7]
    return (v.reshape(*k.shape, 32) * np.ldexp(1.0, k)[..., None]).reshape(codes.shape)


def unpack(packed):
    p = packed.cpu().numpy()
    return np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], -1)


def mx4_scores(q, docs):
    """(scores, bounds) of documents, a list of [tokens, d] in 64 bits."""
    out, tol = [], []
    for d in docs:
        if not len(d):
            out.append(-math.inf)
            tol.append(0.0)
            continue
        s = q @ d.T
        # each product is exact; up to 1024 / 32 steps of sums, then one over the query tokens
        t = (q.shape[1] + 4) * U32 * (np.abs(q) @ np.abs(d).T).max(1)
        out.append(s.max(1).sum())
        tol.append(t.sum() + len(q) * U32 * np.abs(s.max(1)).sum())
    return np.array(out), np.array(tol)


def close(got, want, tol, what=""):
    got = as64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), f"{what}: other values than finite ones"
    off = np.abs(got[fine] - want[fine]) - np.broadcast_to(tol, want.shape)[fine]
    assert not np.isnan(got[fine]).any(), f"{what}: NaN"
    assert off.size == 0 or off.max() <= 0, f"{what}: {off.max()} past the bound"
