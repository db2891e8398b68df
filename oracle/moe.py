"""Routing around the grouped expert products, and 8-bit activation checkpoints.

TEST INFRASTRUCTURE ONLY (see the package docstring): plain restatements in
float64 (the checkpoint's codes and scales: exact), one token, slot or expert
at a time, never called by the product path.

* Routing: V is a token's experts with a logit above -inf, C the first top_k of
  V by logit (ties to the lower index); slots without an expert get id -1 and
  weight 0.  Weights are the softmax over C ("topk") or over V ("all").
* Order: slots (t, j) by expert, then token, then j; an id outside [0, E) drops
  its slot, which takes one of the last rows and is marked by ~row.
* Checkpoint: E4M3 codes of x / s, one power-of-two scale per row and 128
  columns, the smallest s with max(amax, 1e-12) <= 448 s.  Where s = 2^120 (the
  largest), finite values stop at the code 240, so that code * s is finite.
* SwiGLU: h = silu(g) u; gradient at the restored g and u.
* Weight gradient: dW[e] = sum over the rows of expert e of d_y^T x_hat.
"""
from __future__ import annotations

import numpy as np

from .formats import E4M3_MAX, F32_1E_12, e4m3_decode
from .fp8 import e4m3_encode_signed


def route_topk(logits, top_k: int, normalize: str = "topk"):
    """-> (ids int32 [T, top_k], weights float64 [T, top_k])."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    ids = np.full((T, top_k), -1, np.int32)
    w = np.zeros((T, top_k))
    for t in range(T):
        valid = [e for e in range(E) if x[t, e] > -np.inf]
        chosen = sorted(valid, key=lambda e: (-x[t, e], e))[:top_k]
        if not chosen:
            continue
        m = x[t, chosen[0]]
        total = sum(np.exp(x[t, e] - m) for e in (chosen if normalize == "topk" else valid))
        ids[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = [np.exp(x[t, e] - m) / total for e in chosen]
    return ids, w


def route_topk_backward(logits, ids, d_weights, normalize: str = "topk"):
    """d_logits float64 [T, E]."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    d = np.zeros((T, E))
    for t in range(T):
        slots = [j for j, e in enumerate(ids[t]) if 0 <= e < E and x[t, e] > -np.inf]
        chosen = [int(ids[t, j]) for j in slots]
        over = chosen if normalize == "topk" else [e for e in range(E) if x[t, e] > -np.inf]
        if not over:
            continue
        m = max(x[t, e] for e in over)
        total = sum(np.exp(x[t, e] - m) for e in over)
        p = {e: np.exp(x[t, e] - m) / total for e in over}
        g = {e: 0.0 for e in over}
        for j, e in zip(slots, chosen):
            g[e] += float(d_weights[t, j])
        dot = sum(p[e] * g[e] for e in over)
        for e in over:
            d[t, e] = p[e] * (g[e] - dot)
    return d


def sort_tokens(ids, E: int):
    """-> (expert_offsets [E+1], row_token [T*k], slot_row [T, k]), int32."""
    ids = np.asarray(ids)
    T, k = ids.shape
    offsets = np.zeros(E + 1, np.int32)
    row_token, slot_row = np.zeros(T * k, np.int32), np.zeros((T, k), np.int32)
    row = 0
    for e in list(range(E)) + [None]:
        for t in range(T):
            for j in range(k):
                dropped = not 0 <= ids[t, j] < E
                if dropped if e is None else ids[t, j] == e:
                    row_token[row] = t
                    slot_row[t, j] = ~row if dropped else row
                    row += 1
        if e is not None:
            offsets[e + 1] = row
    return offsets, row_token, slot_row


def dispatch(x, slot_row):
    x = np.asarray(x)
    T, k = slot_row.shape
    rows = np.zeros((T * k, x.shape[1]), x.dtype)
    for t in range(T):
        for s in slot_row[t]:
            if s >= 0:
                rows[s] = x[t]
    return rows


def combine(rows, slot_row, weights=None):
    """-> (out [T, H], sum of the absolute terms [T, H]), float64."""
    rows = np.asarray(rows, np.float64)
    T, k = slot_row.shape
    out, size = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j, s in enumerate(slot_row[t]):
            if s >= 0:
                term = (1.0 if weights is None else float(weights[t, j])) * rows[s]
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def combine_backward(d_out, rows, slot_row, weights):
    """-> (d_rows [T*k, H], d_weights [T, k], absolute terms of d_weights)."""
    d_out, rows = np.asarray(d_out, np.float64), np.asarray(rows, np.float64)
    T, k = slot_row.shape
    d_rows = np.zeros((T * k, d_out.shape[1]))
    dw, size = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j, s in enumerate(slot_row[t]):
            if s >= 0:
                d_rows[s] = float(weights[t, j]) * d_out[t]
                dw[t, j] = np.sum(d_out[t] * rows[s])
                size[t, j] = np.sum(np.abs(d_out[t] * rows[s]))
    return d_rows, dw, size


def quantize_fp8_checkpoint(x):
    """-> (codes u8 [rows, K], scales float32 [rows, ceil(K / 128)])."""
    x = np.asarray(x, np.float32)
    rows, K = x.shape
    codes = np.zeros((rows, K), np.uint8)
    scales = np.zeros((rows, -(-K // 128)), np.float32)
    for b in range(scales.shape[1]):
        v = x[:, 128 * b:128 * b + 128].astype(np.float64)
        amax = np.maximum(np.max(np.abs(v), axis=1), float(F32_1E_12))
        e = np.floor(np.log2(amax)).astype(int) - 10      # certainly too small
        for _ in range(8):
            e = np.where(amax > E4M3_MAX * np.exp2(e.astype(float)), e + 1, e)
        s = np.exp2(e.astype(float))
        q = v / s[:, None]
        # 256 * 2^120 would be beyond float32: finite values stop at the code before
        q = np.where(np.isfinite(q) & (e == 120)[:, None], np.clip(q, -240.0, 240.0), q)
        codes[:, 128 * b:128 * b + 128] = e4m3_encode_signed(q.astype(np.float32))
        scales[:, b] = s
    return codes, scales


def restore_fp8_checkpoint(codes, scales):
    """code * scale, float64 (exact)."""
    v = e4m3_decode(codes)
    return v * np.repeat(np.asarray(scales, np.float64), 128, axis=1)[:, :v.shape[1]]


def swiglu(gate_up):
    x = np.asarray(gate_up, np.float64)
    g, u = x[:, :x.shape[1] // 2], x[:, x.shape[1] // 2:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def swiglu_backward(d_h, gate_up):
    """-> (d_gate_up, size of its terms)."""
    d, x = np.asarray(d_h, np.float64), np.asarray(gate_up, np.float64)
    g, u = x[:, :d.shape[1]], x[:, d.shape[1]:]
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    dg, du = d * u * s * (1.0 + g * (1.0 - s)), d * g * s
    return (np.concatenate([dg, du], axis=1),
            np.concatenate([np.abs(d * u * s) * (1.0 + np.abs(g) * (1.0 - s)), np.abs(du)], axis=1))


def grouped_wgrad(d_y, x_hat, row_token, offsets):
    """-> (dW [E, N, K], sum of the absolute terms), float64."""
    d_y, x_hat = np.asarray(d_y, np.float64), np.asarray(x_hat, np.float64)
    E = len(offsets) - 1
    out = np.zeros((E, d_y.shape[1], x_hat.shape[1]))
    size = np.zeros_like(out)
    for e in range(E):
        r = np.arange(offsets[e], offsets[e + 1])
        x = x_hat[r if row_token is None else np.asarray(row_token)[r]]
        out[e] = d_y[r].T @ x
        size[e] = np.abs(d_y[r]).T @ np.abs(x)
    return out, size
