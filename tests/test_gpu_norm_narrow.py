"""Many rows shorter than a 16-byte word or little longer, off 16-byte boundaries: the
norm and its gradient through the ring.  Bounds as in test_gpu_norm."""
import numpy as np
import pytest
import torch

from test_gpu_norm import DTYPES, _call, _check, _check_gradient, _dev, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["none", "fp8", "int8"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H,pitch,offset", [(9003, 1, 0, 0), (9003, 3, 0, 1), (9003, 7, 0, 3), (9001, 5, 2, 1), (8000, 2, 0, 0),
                                                 (8001, 9, 0, 1), (8001, 17, 0, 7)])
def test_norm(lib, rows, H, pitch, offset, dtype, form):
    x, xv = _dev(_rows(rows + H, rows, H), dtype, pitch, offset)
    r, rv = _dev(np.random.default_rng(H).standard_normal((rows, H)), dtype, 2 * pitch, 1)
    w, wv = _dev(1.0 + 0.3 * np.random.default_rng(H).standard_normal((1, H)), dtype)
    _check(lib, form, _call(lib, form, x, w[0], residual=r), xv, wv[0], rv, dtype, 1e-6)
    _check(lib, form, _call(lib, form, x), xv, None, None, dtype, 1e-6)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H,pitch,offset", [(9003, 1, 0, 0), (9003, 3, 0, 1), (9003, 7, 0, 3), (6001, 5, 2, 1), (8001, 9, 0, 1)])
def test_gradient(lib, rows, H, pitch, offset, dtype):
    h, hv = _dev(np.random.default_rng(rows).standard_normal((rows, H)), dtype, pitch, offset)
    dy, dyv = _dev(np.random.default_rng(H).standard_normal((rows, H)) * 0.02, dtype, 2 * pitch, 1)
    dh, dhv = _dev(np.random.default_rng(H + 1).standard_normal((rows, H)) * 0.03, dtype)
    w, wv = _dev(1.0 + 0.3 * np.random.default_rng(H).standard_normal((1, H)), dtype)
    _, _, rstd = lib.rms_norm(h)
    rv = rstd.double().cpu().numpy()
    d_x, d_w = lib.rms_norm_backward(dy, h, rstd, w[0], d_h=dh)
    _check_gradient(d_x, d_w, dyv, hv, rv, wv[0], dhv, dtype)
    over, again = lib.rms_norm_backward(dy, h, rstd, w[0], d_h=dh, out=dh)
    assert torch.equal(over, d_x) and torch.equal(again, d_w) and lib.sync_status() == 0


@pytest.mark.parametrize("form", ["none", "fp8", "int8"])
def test_residual_stream_in_place(lib, form):
    x, _ = _dev(_rows(3, 9003, 7), torch.bfloat16)
    r, _ = _dev(_rows(4, 9003, 7), torch.bfloat16)
    want = _call(lib, form, x, residual=r)
    keep = r.clone()
    got = _call(lib, form, x, residual=keep, h_out=keep)
    assert got[-2] is keep and lib.sync_status() == 0
    for a, b in zip(got, want):
        assert a is b is None or torch.equal(a, b)
