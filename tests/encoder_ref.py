"""Plain 64-bit implementations of the encoder operators (attention within documents with its
gradients, rotary positions, clipping), with bounds on what the kernels may be off by. Test
infrastructure: CPU, one document and head at a time, straight from the formulas."""
from __future__ import annotations

import math

import numpy as np
import torch

# half a step of each storage type, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -24
# least absolute step of results that fall below the type's normal range, halved
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def as64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to("cpu").double().numpy()


def spans(n_rows, offsets=None, lens=None, nd=None):
    """(first row, tokens) of every document."""
    if offsets is not None:
        return [(int(a), int(b - a)) for a, b in zip(offsets[:-1], offsets[1:])]
    n = n_rows // nd if nd else 0
    return [(b * nd, nd if lens is None else min(max(int(lens[b]), 0), nd)) for b in range(n)]


def hidden(n, causal, prefix):
    i = np.arange(n)
    if not causal:
        return np.zeros((n, n), bool)
    return (i[None, :] > i[:, None]) & (i[None, :] >= prefix)


def attention(q, k, v, docs, causal=False, prefix=None, cap=0.0, slopes=None, scale=None, do=None,
              dtype=torch.float32):
    """q [rows, H, d], k and v [rows, KV, d] in 64 bits, docs from spans(). Returns a dict with
    o, lse (and dq, dk, dv with do), and for each a bound `tol_...` on the error of a kernel
    that sums in 32 bits, rounds the weights and their gradients to `dtype` before the products
    and the results to it after them."""
    rows, H, d = q.shape
    KV = k.shape[1]
    group = H // KV
    scale = d ** -0.5 if scale is None else scale
    u, tiny = HALF_STEP[dtype], TINY[dtype]
    r = {"o": np.zeros(q.shape), "lse": np.full((H, rows), -math.inf),
         "tol_o": np.zeros(q.shape), "tol_lse": np.zeros((H, rows))}
    for n, like in (("dq", q), ("dk", k), ("dv", v)):
        r[n], r["tol_" + n] = np.zeros(like.shape), np.zeros(like.shape)
    for b, (t0, n) in enumerate(docs):
        if n == 0:
            continue
        hide = hidden(n, causal, 0 if prefix is None else int(prefix[b]))
        far = np.abs(np.arange(n)[:, None] - np.arange(n)[None, :]).astype(np.float64)
        R = slice(t0, t0 + n)
        for h in range(H):
            Q, K, V = q[R, h], k[R, h // group], v[R, h // group]
            x = Q @ K.T * scale
            y, slope = x, 1.0
            if cap:
                t = np.tanh(x / cap)
                y, slope = cap * t, 1 - t * t
            if slopes is not None:
                y = y - float(slopes[h]) * far
            # a score's error: the 32-bit product, a few roundings of it and of the bias, and
            # the tanh, which is off by at most 3 units of 2^-23 of the cap
            ds = (d + 4) * U32 * scale * (np.abs(Q) @ np.abs(K).T) + 8 * U32 * np.abs(y)
            if cap:
                ds = ds + 6 * U32 * cap
            if slopes is not None:
                ds = ds + 4 * U32 * abs(float(slopes[h])) * far
            y = np.where(hide, -math.inf, y)
            m = y.max(1, keepdims=True)
            e = np.exp(y - m)
            z = m[:, 0] + np.log(e.sum(1))
            p = np.exp(y - z[:, None])
            # relative error of a weight: its score's, the exponential's (argument and result),
            # and the sum's, as far as any visible score is off
            dsm = np.where(hide, 0, ds).max(1, keepdims=True)
            w = 2 * dsm + 2 * U32 * (np.where(hide, 0, np.abs(y - m)).max(1, keepdims=True) + 8) + n * U32
            o = p @ V
            pv = p @ np.abs(V)
            wp = p * (u + w) + tiny * (4 if dtype == torch.float16 else 1)
            tol_o = u * np.abs(o) + wp @ np.abs(V) + n * U32 * pv + tiny
            r["o"][R, h], r["tol_o"][R, h] = o, tol_o
            r["lse"][h, R] = z
            r["tol_lse"][h, R] = (w[:, 0] + 4 * U32 * np.abs(z) + 4 * U32)
            if do is None:
                continue
            G = do[R, h]
            dP = G @ V.T
            delta = (G * o).sum(1, keepdims=True)
            dS = p * (dP - delta) * slope
            # delta is taken from the rounded o
            tdelta = (np.abs(G) * tol_o).sum(1, keepdims=True) + d * U32 * np.abs(G) @ np.abs(o).T.max(1, keepdims=True)
            tdP = (d + 4) * U32 * (np.abs(G) @ np.abs(V).T)
            slope_err = 8 * U32 + (12 * U32 if cap else 0)
            tdS = (np.abs(dS) * (u + 2 * w + 16 * U32)
                   + p * (tdP + tdelta) * (1 + w)
                   + p * np.abs(dP - delta) * slope_err
                   + (2.0 ** -24 * np.abs(dS).max() if dtype == torch.float16 else 0))
            acc = (n * group + 8) * U32
            dq = dS @ K * scale
            r["dq"][R, h] = dq
            r["tol_dq"][R, h] = (u * np.abs(dq) + scale * ((tdS + acc * np.abs(dS)) @ np.abs(K))
                                 + tiny)
            kv = h // group
            r["dk"][R, kv] += dS.T @ Q * scale
            r["tol_dk"][R, kv] += scale * ((tdS + acc * np.abs(dS)).T @ np.abs(Q)) + tiny
            r["dv"][R, kv] += p.T @ G
            r["tol_dv"][R, kv] += ((wp + p * acc).T @ np.abs(G)) + tiny
        for n_ in ("dk", "dv"):
            r["tol_" + n_][R] += u * np.abs(r[n_][R])
    return r


def turned(x, pos, freq, layout, mscale, sign=1.0):
    """x [rows, H, d] in 64 bits with its first 2 len(freq) entries turned."""
    half = len(freq)
    angle = pos.astype(np.float64)[:, None] * freq[None, :]
    c, s = np.cos(angle)[:, None], sign * np.sin(angle)[:, None]
    y = x.copy()
    A = slice(0, half) if layout == "half" else slice(0, 2 * half, 2)
    B = slice(half, 2 * half) if layout == "half" else slice(1, 2 * half, 2)
    a, b = x[..., A], x[..., B]
    y[..., A], y[..., B] = mscale * (a * c - b * s), mscale * (b * c + a * s)
    return y


def clipped(tensors, max_norm):
    """(norm, scaled tensors) in 64 bits."""
    norm = math.sqrt(sum(float((t ** 2).sum()) for t in tensors))
    f = max_norm / (norm + 1e-6)
    f = 1.0 if f > 1 else f
    return norm, [t * f for t in tensors]
