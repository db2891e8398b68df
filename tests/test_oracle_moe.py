"""The oracle of the routed-expert operators against brute force, closed forms
and finite differences (float64)."""
import numpy as np
import pytest

from oracle import moe
from oracle.formats import e4m3_decode

EPS = 1e-6


def _differences(f, x):
    """Central differences of the scalar f at x."""
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += EPS
        lo[i] -= EPS
        d[i] = (f(hi) - f(lo)) / (2 * EPS)
    return d


def test_route_ties_masks_and_empty_rows():
    inf = np.inf
    x = np.array([[1.0, 3.0, 3.0, 3.0], [-inf, 0.0, -inf, -0.0], [-inf] * 4, [-3e38, -3e38, -inf, -3e38]])
    for normalize in ("topk", "all"):
        ids, w = moe.route_topk(x, 3, normalize)
        assert ids.tolist() == [[1, 2, 3], [1, 3, -1], [-1, -1, -1], [0, 1, 3]]
        assert np.allclose(w[1], [0.5, 0.5, 0.0]) and not w[2].any() and np.allclose(w[3], 1 / 3)
    _, w = moe.route_topk(x[:1], 3, "topk")
    assert np.allclose(w, 1 / 3)
    _, w = moe.route_topk(x[:1], 3, "all")
    assert np.allclose(w, 1 / (3 + np.exp(-2.0)))


@pytest.mark.parametrize("normalize", ["topk", "all"])
def test_route_gradient_is_the_difference_quotient(normalize):
    r = np.random.default_rng(3)
    x, g = r.standard_normal((4, 6)), r.standard_normal((4, 3))
    x[1, 2] = -np.inf
    x[2, 1:] = -np.inf                      # one expert left, two slots empty
    ids, _ = moe.route_topk(x, 3, normalize)
    got = moe.route_topk_backward(x, ids, np.where(ids < 0, np.nan, g), normalize)

    def loss(y):
        return float(np.sum(moe.route_topk(y, 3, normalize)[1] * np.where(ids < 0, 0.0, g)))
    live = np.isfinite(x)
    want = _differences(lambda y: loss(np.where(live, y, -np.inf)), np.where(live, x, 0.0))
    assert np.allclose(got, np.where(live, want, 0.0), atol=1e-8)


def test_sort_is_stable_and_parks_dropped_slots():
    ids = np.array([[2, 0], [0, -1], [7, 2], [0, 2]], np.int32)
    offsets, row_token, slot_row = moe.sort_tokens(ids, 3)
    assert offsets.tolist() == [0, 3, 3, 6]
    assert row_token.tolist() == [0, 1, 3, 0, 2, 3, 1, 2]
    assert slot_row.tolist() == [[3, 0], [1, ~6], [~7, 4], [2, 5]]


def test_dispatch_and_combine_are_adjoint():
    r = np.random.default_rng(4)
    ids = r.integers(-1, 5, (7, 3)).astype(np.int32)
    _, row_token, slot_row = moe.sort_tokens(ids, 5)
    x, y = r.standard_normal((7, 11)), r.standard_normal((21, 11))
    rows = moe.dispatch(x, slot_row)
    live = np.sort(slot_row[slot_row >= 0])
    assert np.array_equal(rows[live], x[row_token[live]])
    assert not rows[len(live):].any()
    back, _ = moe.combine(y, slot_row)
    assert np.isclose(np.sum(rows * y), np.sum(x * back))


def test_combine_gradient_is_the_difference_quotient():
    r = np.random.default_rng(5)
    ids = r.integers(-1, 4, (3, 2)).astype(np.int32)
    _, _, slot_row = moe.sort_tokens(ids, 4)
    y, w, d = r.standard_normal((6, 4)), r.standard_normal((3, 2)), r.standard_normal((3, 4))
    d_rows, dw, _ = moe.combine_backward(d, y, slot_row, w)
    assert np.allclose(d_rows, _differences(lambda v: np.sum(d * moe.combine(v, slot_row, w)[0]), y), atol=1e-8)
    assert np.allclose(dw, _differences(lambda v: np.sum(d * moe.combine(y, slot_row, v)[0]), w), atol=1e-8)


def test_checkpoint_scale_is_the_smallest_power_of_two():
    for amax, s in ((448.0, 1.0), (np.nextafter(np.float32(448), np.float32(1e9)), 2.0), (224.0, 0.5),
                    (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7), (1.0, 2.0 ** -8), (0.0, 2.0 ** -48), (1e-20, 2.0 ** -48)):
        codes, scales = moe.quantize_fp8_checkpoint(np.array([[amax, 0.0]], np.float32))
        assert scales[0, 0] == s, amax
        assert s == 2.0 ** -48 or abs(e4m3_decode(codes)[0, 0]) > 208.0


def test_checkpoint_values_are_bf16_and_near():
    torch = pytest.importorskip("torch")
    r = np.random.default_rng(6)
    x = (r.standard_normal((9, 300)) * np.exp2(r.integers(-20, 20, (9, 1)))).astype(np.float32)
    codes, scales = moe.quantize_fp8_checkpoint(x)
    v = moe.restore_fp8_checkpoint(codes, scales)
    assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)
    step = np.repeat(scales, 128, axis=1)[:, :300].astype(np.float64)
    # half a unit of four significant bits, or half the smallest code step
    assert np.all(np.abs(v - x) <= np.maximum(np.abs(x) / 16.0, step * 2.0 ** -10))
    want = torch.from_numpy((x / step).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)


def test_swiglu_gradient_is_the_difference_quotient():
    r = np.random.default_rng(7)
    x, d = 3 * r.standard_normal((3, 10)), r.standard_normal((3, 5))
    got, _ = moe.swiglu_backward(d, x)
    assert np.allclose(got, _differences(lambda v: np.sum(d * moe.swiglu(v)), x), atol=1e-7)


def test_wgrad_is_the_difference_quotient():
    r = np.random.default_rng(8)
    offsets, row_token = np.array([0, 3, 3, 5]), np.array([1, 0, 3, 3, 2])
    d, x, w = r.standard_normal((5, 2)), r.standard_normal((4, 3)), r.standard_normal((3, 2, 3))

    def loss(v):
        return sum(float(d[i] @ v[e] @ x[row_token[i]]) for e in range(3) for i in range(offsets[e], offsets[e + 1]))
    got, _ = moe.grouped_wgrad(d, x, row_token, offsets)
    assert np.allclose(got, _differences(loss, w), atol=1e-7)


def test_checkpoint_of_the_largest_values_restores_as_finite():
    top = np.finfo(np.float32).max
    x = np.array([[top, -top, 248 * 2.0 ** 120, 247 * 2.0 ** 120, 1.0]], np.float32)
    codes, scales = moe.quantize_fp8_checkpoint(x)
    assert scales[0, 0] == 2.0 ** 120
    v = moe.restore_fp8_checkpoint(codes, scales)
    assert np.all(np.isfinite(v.astype(np.float32)))
    assert np.array_equal(v[0], np.array([240, -240, 240, 240, 0]) * 2.0 ** 120)
