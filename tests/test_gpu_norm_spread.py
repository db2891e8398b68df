"""The norm and its gradient over the ways in which rows are spread over blocks: one
row at a time or several side by side, by groups within a warp or of several, through
shared memory or straight, rows too long to be held; pitched rows and FP32 weights on
16-bit rows on each of them.  Bounds as in test_gpu_norm."""
import numpy as np
import pytest
import torch

from test_gpu_norm import DTYPES, _call, _check, _check_gradient, _dev, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H", [(153, 64), (400, 1000), (608, 4096), (1000, 1024), (1200, 4100), (305, 20000),
                                    (160, 32768), (310, 7001), (2500, 260), (5000, 48), (5000, 2048), (153, 129)])
def test_gradient(lib, rows, H, dtype):
    h, hv = _dev(_rows(rows + H, rows, H), dtype)
    dy, dyv = _dev(np.random.default_rng(rows).standard_normal((rows, H)) * 0.02, dtype)
    dh, dhv = _dev(np.random.default_rng(H).standard_normal((rows, H)) * 0.03, dtype)
    w = torch.randn(H, generator=torch.Generator().manual_seed(2))
    _, _, rstd = lib.rms_norm(h)
    rv, wv = rstd.double().cpu().numpy(), w.double().numpy()
    d_x, d_w = lib.rms_norm_backward(dy, h, rstd, w.cuda(), d_h=dh)
    _check_gradient(d_x, d_w, dyv, hv, rv, wv, dhv, dtype)
    over, again = lib.rms_norm_backward(dy, h, rstd, w.cuda(), d_h=dh, out=dh)
    assert torch.equal(over, d_x) and torch.equal(again, d_w)
    d_x, d_w = lib.rms_norm_backward(dy, h, rstd)
    _check_gradient(d_x, d_w, dyv, hv, rv, np.ones(H), None, dtype)
    assert lib.sync_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H,pitch", [(5000, 520, 8), (5000, 513, 3), (2500, 2048, 1), (9000, 72, 0), (1300, 8192, 16)])
def test_pitched_gradient_of_many_rows(lib, rows, H, pitch, dtype):
    h, hv = _dev(_rows(rows + H, rows, H), dtype, pitch)
    dy, dyv = _dev(np.random.default_rng(rows).standard_normal((rows, H)) * 0.02, dtype, 2 * pitch)
    w, wv = _dev(1.0 + 0.3 * np.random.default_rng(H).standard_normal((1, H)), dtype)
    _, _, rstd = lib.rms_norm(h)
    d_x, d_w = lib.rms_norm_backward(dy, h, rstd, w[0])
    _check_gradient(d_x, d_w, dyv, hv, rstd.double().cpu().numpy(), wv[0], None, dtype)
    assert lib.sync_status() == 0


@pytest.mark.parametrize("form", ["none", "fp8", "int8"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H,pitch", [(5000, 520, 8), (5000, 513, 3), (2500, 2048, 0), (9000, 72, 0), (1300, 8192, 16), (310, 7001, 0),
                                          (160, 32768, 0)])
def test_norm_with_weights_in_float32(lib, rows, H, pitch, dtype, form):
    x, xv = _dev(_rows(rows * 3 + H, rows, H), dtype, pitch)
    r, rv = _dev(np.random.default_rng(H + 1).standard_normal((rows, H)), dtype, 2 * pitch)
    w = torch.randn(H, generator=torch.Generator().manual_seed(3))
    _check(lib, form, _call(lib, form, x, w.cuda(), residual=r), xv, w.double().numpy(), rv, dtype, 1e-6)
    assert lib.sync_status() == 0
