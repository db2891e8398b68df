"""Root-mean-square norm with 8-bit outputs, 8-bit integers and their product,
and the router's balance loss.

TEST INFRASTRUCTURE ONLY (see the package docstring): plain restatements in
float64; quantize_int8 follows float32 steps with IEEE rounding, as the other
quantizers do, and the integer product is exact.

* Norm: h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd w.
* INT8: s = max(amax, 1e-12) * RN(1 / 127) per row, q = rint(x / s), ties to even
  (the scale of the worked example's INT8 row).
* Product: C = (the exact integer sum, rounded to float32) * sa * sb, each
  product rounded to float32.
* Balance: p = softmax over the experts above -inf, n tokens with one,
  f = counts E / (n k), loss = coeff sum f mean(p).
"""
from __future__ import annotations

import numpy as np

from .formats import F32_1E_12


def rms_norm(x, weight=None, residual=None, eps: float = 1e-6):
    """-> (y, h, rstd), float64."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + np.float64(np.float32(eps)))
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    return h * rstd[:, None] * w, h, rstd


def rms_norm_backward(d_y, h, rstd, weight=None, d_h=None):
    """-> (d_x, d_weight), float64, at the given rstd."""
    d_y, h, r = (np.asarray(a, np.float64) for a in (d_y, h, rstd))
    r = r[:, None]
    g = d_y if weight is None else d_y * np.asarray(weight, np.float64)
    d = r * (g - h * r * r * np.mean(g * h, axis=1, keepdims=True))
    if d_h is not None:
        d = d + np.asarray(d_h, np.float64)
    return d, np.sum(d_y * h * r, axis=0)


def quantize_int8(x):
    """-> (codes int8 [rows, K], scales float32 [rows])."""
    x = np.asarray(x, np.float32)
    s = np.maximum(np.max(np.abs(x), axis=1), F32_1E_12) * (np.float32(1.0) / np.float32(127.0))
    q = np.rint(x / s[:, None])
    return np.clip(q, -127, 127).astype(np.int8), s


def gemm_w8a8_int8(qa, sa, qb, sb):
    """float32 [M, N], rounded as the product's three steps are."""
    # float64 sums of 8-bit products are exact integers
    acc = np.asarray(qa, np.float64) @ np.asarray(qb, np.float64).T
    return (acc.astype(np.float32) * np.asarray(sa, np.float32)[:, None]) * np.asarray(sb, np.float32)[None, :]


def _softmax_rows(logits):
    x = np.asarray(logits, np.float64)
    p = np.zeros_like(x)
    there = np.zeros(x.shape[0], bool)
    for t in range(x.shape[0]):
        valid = x[t] > -np.inf
        if not valid.any():
            continue
        there[t] = True
        e = np.exp(x[t, valid] - x[t, valid].max())
        p[t, valid] = e / e.sum()
    return p, int(there.sum())


def _loads(counts, n: int, top_k: int):
    E = len(counts)
    return np.asarray(counts, np.float64) * E / (n * top_k) if n else np.zeros(E)


def balance_loss(logits, ids, coeff: float = 1.0):
    """-> (loss float64, counts int32 [E + 1], mean float64 [E])."""
    p, n = _softmax_rows(logits)
    E = p.shape[1]
    counts = np.zeros(E + 1, np.int32)
    for e in np.asarray(ids).reshape(-1):
        if 0 <= e < E:
            counts[e] += 1
    counts[E] = n
    mean = p.sum(axis=0) / n if n else np.zeros(E)
    f = _loads(counts[:E], n, np.asarray(ids).shape[1])
    return float(np.float32(coeff)) * float(f @ mean), counts, mean


def balance_loss_backward(logits, counts, top_k: int, d_loss: float, coeff: float = 1.0):
    """d_logits float64 [T, E]."""
    p, _ = _softmax_rows(logits)
    n = int(counts[-1])
    if not n:
        return np.zeros_like(p)
    f = _loads(counts[:-1], n, top_k)
    return d_loss * float(np.float32(coeff)) / n * p * (f - (p @ f)[:, None])
