"""The norm and its gradient at the ends of the number range."""
import numpy as np
import pytest
import torch

from oracle import norm as o

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,H", [(5, 512), (4000, 512), (4000, 2048), (4000, 501)])
@pytest.mark.parametrize("power", [-30, 44, 50])
def test_gradient_scales_with_its_input(lib, rows, H, power):
    """h 2^p has rstd 2^-p, d_weight as before and d_x 2^-p: all powers of two, so
    that every bit is the same (eps is beside nothing)."""
    g = torch.Generator("cuda").manual_seed(H + rows)
    h, d_y = (torch.randn((rows, H), device="cuda", generator=g) for _ in range(2))
    w = torch.randn(H, device="cuda", generator=g)
    rstd = torch.rsqrt(h.square().mean(dim=1))
    want, want_w = lib.rms_norm_backward(d_y, h, rstd, w)
    got, got_w = lib.rms_norm_backward(d_y, h * 2.0 ** power, rstd * 2.0 ** -power, w)
    assert torch.equal(got * 2.0 ** power, want) and torch.equal(got_w, want_w) and lib.sync_status() == 0


@pytest.mark.parametrize("rows", [5, 4000])
def test_gradient_of_zero_rows_with_the_least_eps(lib, rows):
    """d_x = rstd g, whatever rstd is: no power of it overflows by itself."""
    x = torch.zeros((rows, 512), device="cuda")
    _, h, rstd = lib.rms_norm(x, eps=1e-30)
    d_y = torch.randn((rows, 512), device="cuda")
    d_x, d_w = lib.rms_norm_backward(d_y, x, rstd)
    assert torch.equal(d_x, d_y * rstd.reshape(-1, 1)) and not d_w.any() and lib.sync_status() == 0


@pytest.mark.parametrize("rows", [5, 4000])
@pytest.mark.parametrize("form", ["rms_norm_fp8", "rms_norm_int8"])
def test_codes_of_the_largest_magnitudes(lib, rows, form):
    """|h w| up to 2^127.  Half a step of E4M3 (2^-4 relative, 2^-10 steps of its
    subnormals) or of the integers, and FP32 roundings."""
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.rand((rows, 512), device="cuda", generator=g) + 0.5
    w = torch.full((512,), 2.0 ** 126, device="cuda")
    codes, s, _, _, _ = getattr(lib, form)(x, w)
    y, _, _ = o.rms_norm(x.cpu().numpy(), w.cpu().numpy())
    if form == "rms_norm_fp8":
        s = s.repeat_interleave(128, dim=1).double().cpu().numpy()
        got = codes.view(torch.float8_e4m3fn).double().cpu().numpy() * s
        bound = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s)
    else:
        s = s.reshape(-1, 1).double().cpu().numpy()
        got, bound = codes.double().cpu().numpy() * s, 0.5 * s
    assert np.all(np.abs(got - y) <= bound + 2.0 ** -19 * np.abs(y)) and lib.sync_status() == 0
