"""The oracle's norm, 8-bit integers and balance loss against plain loops,
closed forms and differences."""
import json
import os

import numpy as np
import pytest

from oracle import norm


def _x(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("residual", [False, True])
def test_norm_by_loops(residual):
    x, r, w = _x(1, 3, 7), _x(2, 3, 7) if residual else None, _x(3, 7)
    y, h, rstd = norm.rms_norm(x, w, r, eps=0.25)
    for t in range(3):
        row = [x[t, i] + (r[t, i] if residual else 0.0) for i in range(7)]
        s = 1.0 / (sum(v * v for v in row) / 7 + 0.25) ** 0.5
        assert abs(rstd[t] - s) < 1e-14
        for i in range(7):
            assert abs(h[t, i] - row[i]) < 1e-15 and abs(y[t, i] - row[i] * s * w[i]) < 1e-14


def test_norm_gradient_against_differences():
    x, w, d_y, d_h = _x(4, 4, 9), _x(5, 9), _x(6, 4, 9), _x(7, 4, 9)
    _, h, rstd = norm.rms_norm(x, w, eps=0.1)
    d_x, d_w = norm.rms_norm_backward(d_y, h, rstd, w, d_h)

    def loss(x, w):
        return float(np.sum(norm.rms_norm(x, w, eps=0.1)[0] * d_y) + np.sum(x * d_h))
    step = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = step
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * step) - d_x[i]) < 1e-8
    for i in range(9):
        e = np.zeros_like(w)
        e[i] = step
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * step) - d_w[i]) < 1e-8


def test_int8_worked_row():
    """The eight-weight worked example: the printed INT8 scale."""
    gold = json.load(open(os.path.join(os.path.dirname(__file__), "golden", "pages_values.json")))["worked_row"]
    row = np.array([gold["weights"]], np.float32)
    q, s = norm.quantize_int8(row)
    assert s[0] == np.float32(0.88) * (np.float32(1) / np.float32(127)) and abs(s[0] - gold["scale_int8"]) < 5e-6
    assert q[0, 3] == 127 and np.all(np.abs(q * s[:, None] - row) <= s[0] / 2 * (1 + 1e-6))


def test_int8_ties_and_edges():
    x = np.array([[127.0, 0.5, 1.5, -2.5, -0.5, 126.5], [0, 0, 0, 0, 0, 0], [1e-20, 0, 0, 0, 0, -1e-20]], np.float32)
    q, s = norm.quantize_int8(x)
    assert s[0] == 1.0 and q[0].tolist() == [127, 0, 2, -2, 0, 126]
    assert not q[1].any() and not q[2].any() and s[1] == np.float32(1e-12) * (np.float32(1) / np.float32(127))


def test_int8_product_by_loops():
    r = np.random.default_rng(8)
    qa, qb = r.integers(-128, 128, (3, 5)).astype(np.int8), r.integers(-128, 128, (4, 5)).astype(np.int8)
    sa, sb = r.random(3).astype(np.float32), r.random(4).astype(np.float32)
    C = norm.gemm_w8a8_int8(qa, sa, qb, sb)
    for m in range(3):
        for n in range(4):
            acc = sum(int(qa[m, k]) * int(qb[n, k]) for k in range(5))
            assert C[m, n] == np.float32(acc) * sa[m] * sb[n]


def test_balance_by_loops_and_uniform_load():
    x = _x(9, 6, 4)
    x[1, 2], x[5] = -np.inf, -np.inf
    ids = np.array([[0, 1], [3, 0], [1, 2], [-1, 2], [0, 7], [-1, -1]], np.int32)
    loss, counts, mean = norm.balance_loss(x, ids, 0.5)
    assert counts.tolist() == [3, 2, 2, 1, 5]
    want = 0.0
    for e in range(4):
        p = 0.0
        for t in range(5):
            z = [np.exp(v) for v in x[t]]
            p += z[e] / sum(z)
        assert abs(mean[e] - p / 5) < 1e-14
        want += 0.5 * counts[e] * 4 / (5 * 2) * p / 5
    assert abs(loss - want) < 1e-14
    ids = np.arange(8, dtype=np.int32).reshape(8, 1)
    assert abs(norm.balance_loss(np.zeros((8, 8)), ids, 0.25)[0] - 0.25) < 1e-15
    assert norm.balance_loss(np.full((2, 3), -np.inf), np.full((2, 1), -1), 1.0)[0] == 0.0


def test_balance_gradient_against_differences():
    x = _x(10, 5, 6)
    x[2, 1] = -np.inf
    ids = np.array([[0, 1], [1, 2], [0, 3], [1, 5], [1, -1]], np.int32)
    _, counts, _ = norm.balance_loss(x, ids, 0.3)
    d = norm.balance_loss_backward(x, counts, 2, 1.7, 0.3)
    step = 1e-6
    for i in np.ndindex(x.shape):
        if x[i] == -np.inf:
            assert d[i] == 0.0
            continue
        e = np.zeros_like(x)
        e[i] = step
        diff = 1.7 * (norm.balance_loss(x + e, ids, 0.3)[0] - norm.balance_loss(x - e, ids, 0.3)[0]) / (2 * step)
        assert abs(diff - d[i]) < 1e-8
