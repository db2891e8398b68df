"""What is not finite stays visible in the 8-bit forms: a NaN among h * weight, from
the weight alone, makes the scale of its row (INT8) or of its block of 128 columns
(FP8) NaN and is reported; an infinity likewise.  Over the ways in which rows are
spread."""
import pytest
import torch

pytestmark = pytest.mark.gpu

NONFINITE = -5
SIZES = [(3, 40), (5, 512), (4, 7168), (3, 20000), (400, 513), (4000, 512), (4000, 2048), (4000, 501), (3000, 72)]


def _inputs(rows, H, dtype):
    g = torch.Generator("cuda").manual_seed(rows + H)
    return torch.randn((rows, H), device="cuda", generator=g).to(dtype), torch.randn(H, device="cuda", generator=g)


@pytest.mark.parametrize("w_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", ["rms_norm_fp8", "rms_norm_int8"])
@pytest.mark.parametrize("rows,H", SIZES)
def test_a_weight_that_is_nan(lib, rows, H, form, w_dtype):
    x, w = _inputs(rows, H, torch.bfloat16)
    w = w.to(w_dtype)
    call = getattr(lib, form)
    want_codes, want_scales, _, _, want_r = call(x, w)
    at = H - 3
    w[at] = float("nan")
    codes, scales, y, _, rstd = call(x, w, need_y=True)
    assert lib.sync_status() == NONFINITE and lib.sync_status() == 0
    assert torch.equal(rstd, want_r) and torch.isnan(y[:, at]).all() and torch.isfinite(y[:, :at]).all()
    if form == "rms_norm_int8":
        assert torch.isnan(scales).all()
    else:  # the other blocks are as ever
        b = at // 128
        assert torch.isnan(scales[:, b]).all()
        assert torch.equal(scales[:, :b], want_scales[:, :b]) and torch.equal(codes[:, :128 * b], want_codes[:, :128 * b])


@pytest.mark.parametrize("form", ["rms_norm_fp8", "rms_norm_int8"])
@pytest.mark.parametrize("rows,H", SIZES)
def test_a_weight_that_is_infinite(lib, rows, H, form):
    """On h = 0 (NaN) in the second row, on other values (an infinity) in the rest."""
    x, w = _inputs(rows, H, torch.float32)
    at = H // 2
    w[at] = float("inf")
    x[1, at] = 0.0
    _, scales, _, _, rstd = getattr(lib, form)(x, w)
    assert lib.sync_status() == NONFINITE and torch.isfinite(rstd).all()
    s = scales if form == "rms_norm_int8" else scales[:, at // 128]
    assert torch.isnan(s[1]) and torch.isinf(s[0]) and torch.isinf(s[2:]).all()
    if form == "rms_norm_fp8":
        assert torch.isfinite(scales).sum() == scales.numel() - rows
    # by itself, too: a row of zeros
    getattr(lib, form)(torch.zeros_like(x[:1]), w)
    assert lib.sync_status() == NONFINITE


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,H", [(3, 40), (4, 7168), (4, 501), (3, 20000), (2000, 2048)])
def test_quantizer(lib, rows, H, dtype):
    """The scale of a row with a NaN is NaN, of one with an infinity infinite."""
    x, _ = _inputs(rows, H, dtype)
    want, want_s = lib.quantize_int8(x)
    x[0, H - 2], x[1, 1] = float("nan"), -float("inf")
    codes, s = lib.quantize_int8(x)
    assert lib.sync_status() == NONFINITE
    assert torch.isnan(s[0]) and torch.isinf(s[1]) and torch.equal(s[2:], want_s[2:]) and torch.equal(codes[2:], want[2:])
