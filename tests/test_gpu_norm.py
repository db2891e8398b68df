"""Root-mean-square norm, its 8-bit forms and its gradient on the GPU against the
oracle in float64.

Tolerances.  U: rounding unit of the type.  eps32 = 2^-24.
 * h: rounded to FP32, then to the type: |h| (U + eps32).
 * rstd: a sum of H squares of rounded h, all positive: a thread adds at most
   64 one after another, then at most 10 levels of pairs, each rounding within
   eps32 of the sum, 2 eps32 for the squares of rounded h; division, sum with eps
   and root add 3: below 80 eps32 / 2 + 3 eps32 < 2^-18 relative.
 * y: rstd's error and two products: 2^-17 |y|, then U |y|.
 * 8-bit scales: y's error: 2^-17.  A code lies between the codes of y / s moved
   by 2^-15 both ways (encoding is monotone).
 * d_x = rstd (g - h c) + d_h, c = rstd^2 mean(g h): c is off by 80 eps32 of
   rstd^2 mean|g h|, and every product and sum by eps32 of its terms.
 * d_w: a sum of `rows` terms in some order: (rows + 8) eps32 of the sum of
   |terms|, each term off by 2 eps32.
"""
import numpy as np
import pytest
import torch

from oracle import norm
from oracle.fp8 import e4m3_encode_signed
from oracle.formats import e4m3_decode

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-40, torch.bfloat16: 1e-40, torch.float16: 2.0 ** -25}
E32 = 2.0 ** -24
# rows, H: one element, one row, odd widths, a lane group, a warp, blocks of threads, the widest
SHAPES = [(1, 1), (3, 7), (5, 64), (37, 128), (9, 129), (700, 200), (2, 1411), (301, 1024), (13, 2047), (310, 2048), (400, 2056),
          (4, 7168), (650, 4104), (2, 8200), (320, 16384), (3, 32768), (2, 32761)]


def _dev(x, dtype, pitch=0, offset=0):
    """(device tensor, its values): pitched with NaN between the rows where asked."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dtype)
    if pitch or offset:
        big = torch.full((x.shape[0] * (x.shape[1] + pitch) + offset + 8,), float("nan"), dtype=dtype)
        view = big.as_strided(x.shape, (x.shape[1] + pitch, 1), offset)
        view.copy_(t)
        return big.cuda().as_strided(x.shape, (x.shape[1] + pitch, 1), offset), t.double().numpy()
    return t.cuda(), t.double().numpy()


def _rows(seed, rows, H):
    """Ordinary rows, an outlier column, a zero row, a tiny one and a large one."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, H))
    x[:, H // 2] *= 20.0
    if rows > 2:
        x[1] = 0.0
        x[2] *= 1e-4
    if rows > 4:
        x[4] *= 1e2
    return x


def _near(got, want, bound):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape and np.all(np.isfinite(got))
    off = np.abs(got - want) - bound
    assert np.all(off <= 0), float(off.max())


def _check_codes_fp8(codes, scales, y):
    rows, H = y.shape
    s = scales.double().cpu().numpy()
    amax = np.stack([np.abs(y[:, c:c + 128]).max(axis=1) for c in range(0, H, 128)], axis=1)
    want = np.maximum(amax, 1e-12) / 448.0
    assert s.shape == want.shape and np.all(np.abs(s - want) <= 2.0 ** -17 * want)
    v = e4m3_decode(codes.cpu().numpy()).astype(np.float64)
    q = y / np.repeat(s, 128, axis=1)[:, :H]

    def encode(x):
        return e4m3_decode(e4m3_encode_signed(np.clip(x, -448, 448).astype(np.float32))).astype(np.float64)
    a, b = encode(q * (1 - 2.0 ** -15)), encode(q * (1 + 2.0 ** -15))
    assert np.all(np.minimum(a, b) <= v) and np.all(v <= np.maximum(a, b))


def _check_codes_int8(codes, scales, y):
    s = scales.double().cpu().numpy()
    want = np.maximum(np.abs(y).max(axis=1), 1e-12) / 127.0
    assert np.all(np.abs(s - want) <= 2.0 ** -17 * want)
    v, q = codes.cpu().numpy().astype(np.float64), y / s[:, None]
    a, b = np.rint(q * (1 - 2.0 ** -15)), np.rint(q * (1 + 2.0 ** -15))
    assert np.all(np.minimum(a, b) <= v) and np.all(v <= np.maximum(a, b)) and np.abs(v).max() <= 127


def _check(lib, form, out, x, w, r, dtype, eps):
    y, h, rstd = norm.rms_norm(x, w, r, eps)
    got_h, got_rstd = out[-2], out[-1]
    if r is None:
        assert got_h is None
    else:
        _near(got_h, h, np.abs(h) * (U[dtype] + E32) + TINY[dtype])
    _near(got_rstd, rstd, rstd * 2.0 ** -18)
    if form == "fp8":
        _check_codes_fp8(out[0], out[1], y)
    elif form == "int8":
        _check_codes_int8(out[0], out[1], y)
    got_y = out[0] if form == "none" else out[2]
    if got_y is not None:
        _near(got_y, y, np.abs(y) * (U[dtype] + 2.0 ** -17) + TINY[dtype])
    assert lib.sync_status() == 0


def _call(lib, form, *args, **kw):
    if form == "none":
        kw.pop("need_y", None)
        return lib.rms_norm(*args, **kw)
    return (lib.rms_norm_fp8 if form == "fp8" else lib.rms_norm_int8)(*args, **kw)


@pytest.mark.parametrize("form", ["none", "fp8", "int8"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_norm(lib, shape, dtype, form):
    rows, H = shape
    x, xv = _dev(_rows(rows + H, rows, H), dtype)
    r, rv = _dev(_rows(rows * H, rows, H) * 3.0, dtype)
    w, wv = _dev(1.0 + 0.3 * np.random.default_rng(H).standard_normal((1, H)), dtype)
    _check(lib, form, _call(lib, form, x, w[0], residual=r, need_y=True), xv, wv[0], rv, dtype, 1e-6)
    _check(lib, form, _call(lib, form, x), xv, None, None, dtype, 1e-6)


@pytest.mark.parametrize("form", ["none", "fp8", "int8"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,pitch,offset", [((33, 256), 8, 0), ((33, 256), 8, 1), ((20, 2048), 3, 0), ((7, 130), 6, 2)])
def test_pitches_and_weights_in_float32(lib, shape, pitch, offset, dtype, form):
    rows, H = shape
    x, xv = _dev(_rows(1, rows, H), dtype, pitch, offset)
    r, rv = _dev(_rows(2, rows, H), dtype, 2 * pitch, offset)
    w = torch.randn(H + 1, generator=torch.Generator().manual_seed(H))[1:]
    wd = torch.cat([w[:1], w])[1:].cuda()
    _check(lib, form, _call(lib, form, x, wd, residual=r, eps=0.5, need_y=True), xv, w.double().numpy(), rv, dtype, 0.5)


@pytest.mark.parametrize("form", ["none", "fp8", "int8"])
@pytest.mark.parametrize("H", [64, 1411, 7168])
def test_residual_stream_in_place(lib, form, H):
    """h over the residual, through two norms one after another."""
    x, xv = _dev(_rows(3, 6, H), torch.bfloat16)
    r, _ = _dev(_rows(4, 6, H), torch.bfloat16)
    want = _call(lib, form, x, residual=r)
    keep = r.clone()
    got = _call(lib, form, x, residual=keep, h_out=keep)
    assert got[-2] is keep
    for a, b in zip(got, want):
        assert a is b is None or torch.equal(a, b)
    # and the next block's: the stream goes on
    again = _call(lib, form, x, residual=keep, h_out=keep)
    _check(lib, form, again, xv, None, want[-2].double().cpu().numpy(), torch.bfloat16, 1e-6)


def test_zero_and_tiny_rows(lib):
    for dtype in DTYPES:
        x = torch.zeros((4, 256), dtype=dtype, device="cuda")
        x[1] = 6e-5
        for form in ("none", "fp8", "int8"):
            out = _call(lib, form, x, eps=1e-6)
            _check(lib, form, out, x.double().cpu().numpy(), None, None, dtype, 1e-6)
            if form != "none":
                assert not out[0][0].any() and torch.all(out[1] > 0)


@pytest.mark.parametrize("form", ["none", "fp8", "int8"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_non_finite_rows_are_reported(lib, form, bad):
    """The row's status is latched, the other rows are as ever."""
    x = torch.randn((5, 1024), generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    want = _call(lib, form, x)
    x[3, 77] = bad
    got = _call(lib, form, x)
    assert lib.sync_status() == -5 and lib.sync_status() == 0
    for a, b in zip(got, want):
        if a is not None:
            assert torch.equal(a[[0, 1, 2, 4]].view(torch.uint8), b[[0, 1, 2, 4]].view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES + [(9973, 72), (3000, 1411)])
@pytest.mark.parametrize("joined", [False, True])
def test_gradient(lib, shape, dtype, joined):
    rows, H = shape
    seed = rows * 3 + H
    h, hv = _dev(_rows(seed, rows, H), dtype)
    dy, dyv = _dev(np.random.default_rng(seed + 1).standard_normal((rows, H)) * 0.02, dtype)
    dh, dhv = _dev(np.random.default_rng(seed + 2).standard_normal((rows, H)) * 0.03, dtype)
    w, wv = _dev(1.0 + 0.3 * np.random.default_rng(H).standard_normal((1, H)), dtype)
    rstd = torch.from_numpy(norm.rms_norm(hv, None)[2].astype(np.float32)).cuda()
    rv = rstd.double().cpu().numpy()
    d_x, d_w = lib.rms_norm_backward(dy, h, rstd, w[0], d_h=dh if joined else None)
    _check_gradient(d_x, d_w, dyv, hv, rv, wv[0], dhv if joined else None, dtype)
    assert lib.sync_status() == 0


def _check_gradient(d_x, d_w, dy, h, r, w, dh, dtype):
    rows = dy.shape[0]
    want_x, want_w = norm.rms_norm_backward(dy, h, r, w, dh)
    g = dy * w
    r = r[:, None]
    c = r * r * np.mean(np.abs(g * h), axis=1, keepdims=True)
    terms = np.abs(r * g) + np.abs(r * h) * c + (0 if dh is None else np.abs(dh))
    _near(d_x, want_x, 96 * E32 * np.abs(r * h) * c + 6 * E32 * terms + U[dtype] * np.abs(want_x) + TINY[dtype])
    if d_w is not None:
        _near(d_w, want_w, (rows + 12) * E32 * np.sum(np.abs(dy * h * r), axis=0) + 1e-40)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_forms(lib, dtype):
    """Pitches, FP32 weights, no weights, no d_weight, d_x over d_h, a given workspace."""
    rows, H = 130, 520
    h, hv = _dev(_rows(11, rows, H), dtype, 8)
    dy, dyv = _dev(np.random.default_rng(12).standard_normal((rows, H)), dtype, 16, 8)
    dh, dhv = _dev(np.random.default_rng(13).standard_normal((rows, H)), dtype)
    w = torch.randn(H, generator=torch.Generator().manual_seed(2))
    _, _, rstd = lib.rms_norm(h, w.cuda())
    rv = rstd.double().cpu().numpy()
    ws = lib.workspace(lib.OP_RMS_NORM_BACKWARD, rows, 0, H, "cuda")
    d_x, d_w = lib.rms_norm_backward(dy, h, rstd, w.cuda(), d_h=dh.clone(), ws=ws)
    _check_gradient(d_x, d_w, dyv, hv, rv, w.double().numpy(), dhv, dtype)
    keep = dh.clone()
    over, _ = lib.rms_norm_backward(dy, h, rstd, w.cuda(), d_h=keep, out=keep)
    assert over is keep and torch.equal(over, d_x)
    alone, none = lib.rms_norm_backward(dy, h, rstd, w.cuda(), need_d_weight=False)
    assert none is None
    _check_gradient(alone, None, dyv, hv, rv, w.double().numpy(), None, dtype)
    d_x, d_w = lib.rms_norm_backward(dy, h, rstd)
    _check_gradient(d_x, d_w, dyv, hv, rv, np.ones(H), None, dtype)
    for t in (h[:0], h[:1]):  # no row, a single one
        n = t.shape[0]
        d_x, d_w = lib.rms_norm_backward(dy[:n], t, rstd[:n], w.cuda())
        assert d_x.shape == (n, H) and (n or not d_w.any())


def test_gradient_against_differences(lib):
    """The FP32 forward differentiated numerically along random directions: central
    differences of a sum of 6 x 96 terms of order 1 at step 2^-6 are off by about
    2^-12 (third derivative) and 2^-24 * 600 / 2^-5 (roundings)."""
    g = torch.Generator("cuda").manual_seed(5)
    x, d_y = (torch.randn((6, 96), device="cuda", generator=g) for _ in range(2))
    w = torch.randn(96, device="cuda", generator=g)
    _, _, rstd = lib.rms_norm(x, w, eps=0.1)
    d_x, d_w = lib.rms_norm_backward(d_y, x, rstd, w)
    step = 2.0 ** -6

    def loss(x, w):
        return float((lib.rms_norm(x, w, eps=0.1)[0].double() * d_y.double()).sum())
    for seed in range(4):
        v = torch.randn((6, 96), device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
        v /= v.norm()
        assert abs((loss(x + step * v, w) - loss(x - step * v, w)) / (2 * step) - float((d_x.double() * v.double()).sum())) < 2e-3
        u = v[0] / v[0].norm()
        assert abs((loss(x, w + step * u) - loss(x, w - step * u)) / (2 * step) - float((d_w.double() * u.double()).sum())) < 2e-3


def test_results_do_not_change_from_call_to_call(lib):
    g = torch.Generator("cuda").manual_seed(6)
    h, dy = (torch.randn((4000, 1543), device="cuda", generator=g).bfloat16() for _ in range(2))
    _, _, rstd = lib.rms_norm(h)
    first = lib.rms_norm_backward(dy, h, rstd)
    for _ in range(5):
        again = lib.rms_norm_backward(dy, h, rstd)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_refusals(lib):
    x = torch.zeros((4, 64), device="cuda", dtype=torch.bfloat16)
    r, rstd = x.clone(), torch.ones(4, device="cuda")
    for call in (lambda: lib.rms_norm(x.cpu()), lambda: lib.rms_norm(x, torch.ones(63, device="cuda")),
                 lambda: lib.rms_norm(x, torch.ones(64, device="cuda", dtype=torch.float16)),
                 lambda: lib.rms_norm(x, residual=r.float()), lambda: lib.rms_norm(x, residual=r[:3]),
                 lambda: lib.rms_norm(x, h_out=r), lambda: lib.rms_norm(x, out=r.float()), lambda: lib.rms_norm(x.t()),
                 lambda: lib.rms_norm_int8(x[0]), lambda: lib.rms_norm_fp8(x.to(torch.float64)),
                 lambda: lib.rms_norm_backward(x, r, rstd.double()), lambda: lib.rms_norm_backward(x, r[:2], rstd),
                 lambda: lib.rms_norm_backward(x, r, rstd, d_h=r.float()), lambda: lib.rms_norm_backward(x, r, rstd[:3])):
        with pytest.raises((ValueError, IndexError)):
            call()
    for call in (lambda: lib.rms_norm(x, eps=0.0), lambda: lib.rms_norm(x, eps=-1e-6), lambda: lib.rms_norm(x, out=x),
                 lambda: lib.rms_norm(x, residual=r, out=r), lambda: lib.rms_norm(x, residual=r, h_out=x),
                 lambda: lib.rms_norm_backward(x, r, rstd, out=x), lambda: lib.rms_norm_backward(x, r, rstd, out=r),
                 lambda: lib.rms_norm_backward(x, r, rstd, ws=torch.empty(16, device="cuda", dtype=torch.uint8)),
                 lambda: lib.rms_norm(torch.zeros((2, 32769), device="cuda"))):
        with pytest.raises(lib.Q4Error):
            call()
    y, _, rstd = lib.rms_norm(x[:0])
    assert y.shape == (0, 64) and rstd.shape == (0,) and lib.sync_status() == 0
