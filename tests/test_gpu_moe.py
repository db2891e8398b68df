"""Routing, sort by expert, dispatch and combine with their gradients on the GPU
against the float64 oracle.

Tolerances.  U is the rounding unit of a type (half of its spacing at 1):
2^-24, 2^-8, 2^-11 for float32, bfloat16, float16; results rounded to a type
may differ by U of their size (and by half the smallest subnormal, 2^-25, in
float16).
 * weights: expf is within 2 ulp, the difference l - m it takes is rounded once
   (|l - m| * 2^-24 in the exponent, at most 2^-18 where the weight is above
   2^-90), and a sum of at most 1024 positive terms over 32 lanes adds fewer
   than 64 roundings: below 2^-16 of the weight;
 * their gradient: as many roundings of p (g - S): 2^-15 of p (|g| + |S|);
 * combine: one fused multiply-add per slot: k 2^-24 of the sum of |terms|;
 * d_weights: H products over at least 128 partial sums: fewer than
   H / 128 + 32 roundings of the sum of |terms|.
"""
import numpy as np
import pytest
import torch

from oracle import moe

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-38, torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25}


def _dev(x, dtype):
    """(the device tensor, the float64 values it holds)"""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dtype)
    return t.cuda(), t.double().numpy()


def _pitched(x, dtype, extra, offset=0):
    """A view with row pitch cols + extra and first element at `offset`; NaN around it."""
    big = torch.full((x.shape[0] * (x.shape[1] + extra) + offset + 8,), float("nan"), dtype=dtype)
    view = big.as_strided(x.shape, (x.shape[1] + extra, 1), offset)
    view.copy_(torch.from_numpy(np.ascontiguousarray(x, np.float32)))
    return big.cuda().as_strided(x.shape, (x.shape[1] + extra, 1), offset), view.double().numpy()


def _near(got, want, bound, dtype=torch.float32):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    worst = np.abs(got - want) - (bound + U[dtype] * np.abs(want) + TINY[dtype])
    assert np.all(worst <= 0.0), float(worst.max())


def _logits(T, E, seed, ties=True):
    r = np.random.default_rng(seed)
    x = r.standard_normal((T, E)) * 3.0
    if ties:
        x = np.round(x * 4.0) / 4.0            # many equal logits in every type
    x[r.random((T, E)) < 0.1] = -np.inf
    return x


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("normalize", ["topk", "all"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 8, 2), (5, 32, 32), (9, 33, 8), (130, 64, 8), (67, 100, 5),
                                   (33, 256, 10), (6, 513, 6), (7, 1024, 32)])
def test_route(lib, dtype, normalize, shape):
    T, E, k = shape
    x, xh = _dev(_logits(T, E, T + E), dtype)
    ids, w = lib.moe_route_topk(x, k, normalize=normalize)
    want_ids, want = moe.route_topk(xh, k, normalize)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    _near(w, want, 2.0 ** -16 * want)
    g = np.random.default_rng(T).standard_normal((T, k)).astype(np.float32)
    gd = torch.from_numpy(np.where(want_ids < 0, np.nan, g).astype(np.float32)).cuda()
    d = lib.moe_route_topk_backward(x, ids, gd, normalize=normalize)
    want_d = moe.route_topk_backward(xh, want_ids, g, normalize)
    p = moe.route_topk(xh, E, "all" if normalize == "all" else "topk")
    size = np.zeros((T, E))
    for t in range(T):
        live = p[0][t] >= 0 if normalize == "all" else np.isin(p[0][t], want_ids[t][want_ids[t] >= 0])
        of = {int(e): v for e, v in zip(want_ids[t], g[t]) if e >= 0}
        wt = {int(e): v for e, v in zip(want_ids[t], want[t]) if e >= 0}
        S = sum(abs(of[e]) * wt[e] for e in of)
        for e, v in zip(p[0][t][live], p[1][t][live]):
            pe = v if normalize == "all" else wt[int(e)]
            size[t, e] = pe * (abs(of.get(int(e), 0.0)) + S)
    _near(d, want_d, 2.0 ** -15 * size, dtype)
    assert lib.sync_status() == 0


def test_route_lowest_values_signed_zeros_and_empty_rows(lib):
    low = torch.finfo(torch.float32).min
    x = torch.tensor([[low, low, low, low], [0.0, -0.0, 0.0, -0.0], [-np.inf] * 4, [low, 1.0, -np.inf, low],
                      [3e38, -3e38, 3e38, low], [-np.inf, -np.inf, 2.0, -np.inf]], dtype=torch.float32)
    for normalize in ("topk", "all"):
        ids, w = lib.moe_route_topk(x.cuda(), 2, normalize=normalize)
        want_ids, want = moe.route_topk(x.double().numpy(), 2, normalize)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        _near(w, want, 2.0 ** -16 * want)
        d = lib.moe_route_topk_backward(x.cuda(), ids, torch.full((6, 2), 2.0, device="cuda"), normalize=normalize)
        _near(d, moe.route_topk_backward(x.double().numpy(), want_ids, np.full((6, 2), 2.0), normalize), 2.0 ** -14)
    assert lib.sync_status() == 0


def test_route_reports_and_masks_non_finite_logits(lib):
    for bad in (np.nan, np.inf):
        x = np.tile(np.arange(40, dtype=np.float32), (3, 1))
        x[1, 39] = bad
        ids, w = lib.moe_route_topk(torch.from_numpy(x).cuda(), 2)
        assert ids.tolist() == [[39, 38], [38, 37], [39, 38]]
        assert torch.isfinite(w).all()
        assert lib.sync_status() == -5 and lib.sync_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_route_row_pitch(lib, dtype):
    x, xh = _pitched(_logits(19, 37, 3), dtype, 5, 1)
    ids, w = lib.moe_route_topk(x, 4)
    want_ids, want = moe.route_topk(xh, 4)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    _near(w, want, 2.0 ** -16 * want)
    g = torch.ones((19, 4), device="cuda")
    a = lib.moe_route_topk_backward(x, ids, g, normalize="all")
    b = lib.moe_route_topk_backward(x.contiguous(), ids, g, normalize="all")
    assert torch.equal(a, b)
    assert lib.sync_status() == 0


def test_route_gradient_is_the_difference_quotient(lib):
    """The kernel's own forward: float32 weights, central differences of 2^-6
    (error of order h^2 of the third derivative and 2^-24 / h)."""
    r = np.random.default_rng(12)
    T, E, k, h = 2, 12, 3, 2.0 ** -6
    x = np.stack([r.permutation(E) for _ in range(T)]).astype(np.float32)   # gaps of 1: the choice is stable
    g = r.standard_normal((T, k)).astype(np.float32)
    for normalize in ("topk", "all"):
        ids, _ = lib.moe_route_topk(torch.from_numpy(x).cuda(), k, normalize=normalize)
        d = lib.moe_route_topk_backward(torch.from_numpy(x).cuda(), ids, torch.from_numpy(g).cuda(),
                                        normalize=normalize).cpu().numpy()
        for t in range(T):
            for e in range(E):
                y = np.stack([x, x])
                y[0, t, e] += h
                y[1, t, e] -= h
                w = [lib.moe_route_topk(torch.from_numpy(v).cuda(), k, normalize=normalize)[1].double().cpu().numpy()
                     for v in y]
                q = np.sum((w[0] - w[1]) * g) / (2 * h)
                assert abs(q - d[t, e]) <= np.abs(g).sum() * (h * h + 2.0 ** -22 / h)


def _ids(T, k, E, seed, drop=0.0):
    r = np.random.default_rng(seed)
    ids = np.stack([r.permutation(max(E, k))[:k] for _ in range(T)]) if T else np.zeros((0, k))
    ids = np.where(ids < E, ids, -1).astype(np.int32)
    ids[r.random((T, k)) < drop] = r.choice([-1, E, -2 ** 31, 2 ** 31 - 1])
    return ids


@pytest.mark.parametrize("shape", [(1, 1, 1, 0.0), (1, 8, 64, 0.0), (16, 8, 64, 0.2), (255, 3, 7, 0.1),
                                   (256, 8, 1024, 0.0), (257, 8, 5, 0.5), (2049, 1, 33, 0.02), (700, 6, 256, 1.0),
                                   (4099, 4, 300, 0.03)])
def test_sort(lib, shape):
    T, k, E, drop = shape
    ids = _ids(T, k, E, T, drop)
    got = lib.moe_sort_tokens(torch.from_numpy(ids).cuda(), E)
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    row = np.empty_like(order)
    row[order] = np.arange(order.size)
    assert np.array_equal(got[0].cpu().numpy(), np.searchsorted(key[order], np.arange(E + 1)))
    assert np.array_equal(got[1].cpu().numpy(), order // k)
    assert np.array_equal(got[2].cpu().numpy(), np.where(key < E, row, ~row).reshape(T, k))
    if T * k <= 4000:
        for a, b in zip(got, moe.sort_tokens(ids, E)):
            assert np.array_equal(a.cpu().numpy(), b)
    assert lib.sync_status() == 0


@pytest.mark.parametrize("shape", [(65536, 8, 256), (100003, 5, 1000), (40000, 32, 3)])
def test_sort_large(lib, shape):
    T, k, E = shape
    ids = torch.randint(-1, E, (T, k), dtype=torch.int32, device="cuda", generator=torch.Generator("cuda").manual_seed(T))
    offsets, row_token, slot_row = lib.moe_sort_tokens(ids, E)
    key = torch.where(ids < 0, E, ids).reshape(-1).long()
    order = torch.sort(key, stable=True).indices
    assert torch.equal(row_token.long(), order // k)
    assert torch.equal(offsets.long(), torch.searchsorted(key[order], torch.arange(E + 1, device="cuda")))
    slot = slot_row.reshape(-1).long()
    assert torch.equal(torch.where(slot < 0, -1 - slot, slot)[order], torch.arange(T * k, device="cuda"))
    assert torch.equal(slot < 0, ids.reshape(-1) < 0)


def test_sort_of_one_expert_and_of_no_tokens(lib):
    ids = torch.zeros((5000, 1), dtype=torch.int32, device="cuda")
    offsets, row_token, slot_row = lib.moe_sort_tokens(ids, 2)
    assert offsets.tolist() == [0, 5000, 5000]
    assert torch.equal(row_token, torch.arange(5000, device="cuda", dtype=torch.int32))
    assert torch.equal(slot_row.reshape(-1), row_token)
    offsets, row_token, slot_row = lib.moe_sort_tokens(ids[:0], 3)
    assert offsets.tolist() == [0, 0, 0, 0] and row_token.numel() == 0 and slot_row.shape == (0, 1)


WIDTHS = [(1, 1, 1), (1, 8, 7168), (3, 2, 8), (2, 1, 24), (5, 32, 40), (17, 3, 257), (40, 8, 1000), (9, 4, 4104), (64, 6, 511)]


def _problem(T, k, seed, drop=0.2):
    ids = _ids(T, k, 2 * k + 1, seed, drop)
    _, _, slot = moe.sort_tokens(ids, 2 * k + 1)
    return torch.from_numpy(slot).cuda(), slot


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", WIDTHS)
def test_dispatch(lib, dtype, shape):
    T, k, H = shape
    slot, sh = _problem(T, k, T + H)
    x, xh = _dev(np.random.default_rng(H).standard_normal((T, H)), dtype)
    want = moe.dispatch(xh, sh)
    out = torch.full((T * k, H), float("nan"), dtype=dtype, device="cuda")
    got = lib.moe_dispatch(x, slot, out=out)
    assert got is out and np.array_equal(got.double().cpu().numpy(), want)
    y, yh = _pitched(xh, dtype, 3, 1)
    assert torch.equal(lib.moe_dispatch(y, slot), got)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", WIDTHS)
def test_combine_and_dispatch_gradient(lib, dtype, shape):
    T, k, H = shape
    slot, sh = _problem(T, k, T + H)
    r = np.random.default_rng(H)
    x = r.standard_normal((T * k, H))
    w = r.standard_normal((T, k)).astype(np.float32)
    # nothing of a dropped slot may reach the result
    x[[~s for s in sh.reshape(-1) if s < 0]] = np.nan
    w[sh < 0] = np.nan
    rows, rh = _dev(x, dtype)
    wd = torch.from_numpy(w).cuda()
    want, size = moe.combine(rh, sh, w)
    _near(lib.moe_combine(rows, slot, wd), want, k * 2.0 ** -24 * size, dtype)
    want, size = moe.combine(rh, sh)
    got = lib.moe_dispatch_backward(rows, slot)
    _near(got, want, k * 2.0 ** -24 * size, dtype)
    assert torch.equal(lib.moe_combine(rows, slot), got)
    for extra, offset in ((8, 0), (1, 3)):
        p, _ = _pitched(x, dtype, extra, offset)
        assert torch.equal(lib.moe_dispatch_backward(p, slot), got)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", WIDTHS)
def test_combine_gradient(lib, dtype, shape):
    T, k, H = shape
    slot, sh = _problem(T, k, T + H)
    r = np.random.default_rng(H + 1)
    x, w = r.standard_normal((T * k, H)), r.standard_normal((T, k)).astype(np.float32)
    x[[~s for s in sh.reshape(-1) if s < 0]] = np.nan
    w[sh < 0] = np.nan
    rows, rh = _dev(x, dtype)
    d, dh = _dev(r.standard_normal((T, H)), dtype)
    wd = torch.from_numpy(w).cuda()
    out = torch.full((T * k, H), float("nan"), dtype=dtype, device="cuda")
    d_rows, d_w = lib.moe_combine_backward(d, rows, slot, wd, out=out)
    want, want_w, size = moe.combine_backward(dh, rh, sh, w)
    _near(d_rows, want, 2.0 ** -24 * np.abs(want), dtype)
    _near(d_w, want_w, (H / 128 + 32) * 2.0 ** -24 * size)
    assert not d_w.cpu().numpy()[sh < 0].any()
    only, none = lib.moe_combine_backward(d, rows, slot, wd, need_d_weights=False)
    assert none is None and torch.equal(only, d_rows)
    dp, _ = _pitched(dh, dtype, 8, 0)
    rp, _ = _pitched(x, dtype, 3, 2)
    a, b = lib.moe_combine_backward(dp, rp, slot, wd)
    assert torch.equal(a, d_rows)
    _near(b, want_w, (H / 128 + 32) * 2.0 ** -24 * size)


def test_slots_that_name_no_row_are_left_out(lib):
    x = torch.ones((2, 16), device="cuda")
    slot = torch.tensor([[1, 100], [2 ** 31 - 1, ~100]], dtype=torch.int32, device="cuda")
    rows = lib.moe_dispatch(x, slot, out=torch.full((4, 16), 7.0, device="cuda"))
    assert rows[:, 0].tolist() == [7.0, 1.0, 7.0, 7.0]
    w = torch.full((2, 2), 3.0, device="cuda")
    assert lib.moe_combine(rows, slot, w)[:, 5].tolist() == [3.0, 0.0]
    d_rows, d_w = lib.moe_combine_backward(x, rows, slot, w, out=torch.full((4, 16), 7.0, device="cuda"))
    assert d_rows[:, 3].tolist() == [7.0, 3.0, 7.0, 7.0]
    assert d_w.tolist() == [[16.0, 0.0], [0.0, 0.0]]


def test_empty_inputs(lib):
    f = dict(device="cuda")
    ids, w = lib.moe_route_topk(torch.empty((0, 8), **f), 2)
    assert ids.shape == w.shape == (0, 2)
    assert lib.moe_route_topk_backward(torch.empty((0, 8), **f), ids, w).shape == (0, 8)
    slot = torch.empty((0, 2), dtype=torch.int32, **f)
    assert lib.moe_dispatch(torch.empty((0, 16), **f), slot).shape == (0, 16)
    assert lib.moe_combine(torch.empty((0, 16), **f), slot, w).shape == (0, 16)
    d_rows, d_w = lib.moe_combine_backward(torch.empty((0, 16), **f), torch.empty((0, 16), **f), slot, w)
    assert d_rows.shape == (0, 16) and d_w.shape == (0, 2)
    _, one = lib.moe_combine_backward(torch.empty((1, 0), **f), torch.empty((2, 0), **f),
                                      torch.tensor([[0, 1]], dtype=torch.int32, **f), torch.ones((1, 2), **f))
    assert one.tolist() == [[0.0, 0.0]]


def test_another_stream_and_repeats(lib):
    """Given stream: results follow its work; the same call gives the same bits."""
    T, k, E, H = 512, 4, 32, 384
    g = torch.Generator("cuda").manual_seed(5)
    logits = torch.randn((T, E), device="cuda", generator=g)
    x = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    ids, w = lib.moe_route_topk(logits, k)
    _, _, slot = lib.moe_sort_tokens(ids, E)
    want = lib.moe_combine(lib.moe_dispatch(x, slot), slot, w)
    want_w = lib.moe_combine_backward(x, lib.moe_dispatch(x, slot), slot, w)[1]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        i2, w2 = lib.moe_route_topk(logits, k, stream=s)
        _, _, slot2 = lib.moe_sort_tokens(i2, E, stream=s)
        rows = lib.moe_dispatch(x, slot2, stream=s)
        got = lib.moe_combine(rows, slot2, w2, stream=s)
        got_w = lib.moe_combine_backward(x, rows, slot2, w2, stream=s)[1]
        s.synchronize()
        assert torch.equal(slot, slot2) and torch.equal(got, want) and torch.equal(got_w, want_w)


def test_refusals(lib):
    f, i = dict(device="cuda"), dict(device="cuda", dtype=torch.int32)
    x, slot = torch.zeros((4, 16), **f), torch.zeros((4, 2), **i)
    for bad in (lambda: lib.moe_route_topk(x.cpu(), 2), lambda: lib.moe_route_topk(x.double(), 2),
                lambda: lib.moe_route_topk(x.t(), 2), lambda: lib.moe_route_topk(x[:1].expand(4, 16), 2),
                lambda: lib.moe_route_topk_backward(x, slot, x[:, :2]),
                lambda: lib.moe_route_topk_backward(x, slot.long(), torch.zeros((4, 2), **f)),
                lambda: lib.moe_sort_tokens(slot.long(), 4), lambda: lib.moe_sort_tokens(slot, 0),
                lambda: lib.moe_dispatch(x, slot[:3]), lambda: lib.moe_dispatch(x, slot, out=x),
                lambda: lib.moe_combine(x, slot), lambda: lib.moe_dispatch_backward(x, slot),
                lambda: lib.moe_combine(torch.zeros((8, 16), **f), slot, torch.zeros((4, 2), **f).double()),
                lambda: lib.moe_combine_backward(x, x, slot, torch.zeros((4, 2), **f))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(KeyError):
        lib.moe_route_topk(x, 2, normalize="none")
    for k, status in ((0, -1), (17, -1)):
        with pytest.raises(lib.Q4Error) as e:
            lib.moe_route_topk(x, k)
        assert e.value.status == status
    with pytest.raises(lib.Q4Error) as e:
        lib.moe_route_topk(torch.zeros((1, 1025), **f), 2)
    assert e.value.status == -2
    with pytest.raises(lib.Q4Error) as e:
        lib.moe_sort_tokens(torch.zeros((20000, 2), **i), 4, ws=torch.empty(0, dtype=torch.uint8, **f))
    assert e.value.status == -6
