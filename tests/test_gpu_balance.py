"""The router's balance loss and its gradient on the GPU against the oracle in
float64.

Tolerances.  eps32 = 2^-24, U: rounding unit of the type.
 * p: the fast exponential is documented within 2 + floor(1.173 |x|) ulp (an ulp
   is at most 2^-23 of the value), x the distance from the top, at most 25 here
   where p matters (beyond, p < 1e-10 is covered by an absolute 1e-12): 31 ulp;
   the sum of positive terms and a division add less than 20 more eps32: 2^-17.
 * mean, loss: sums of positive terms, in all at most 400 additions one after
   another: 2^-17 + 404 eps32 < 2^-15.
 * d_logits = g p (f - dot): 2^-16 of g p f and g p dot, then U.
"""
import numpy as np
import pytest
import torch

from oracle import norm

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-40, torch.bfloat16: 1e-40, torch.float16: 2.0 ** -25}


def _case(seed, T, E, k, dtype, pad=0.1, masked=0.1):
    r = np.random.default_rng(seed)
    x = r.standard_normal((T, E)) * 2.0
    x[r.random((T, E)) < masked] = -np.inf
    ids = np.argsort(-x, axis=1, kind="stable")[:, :k].astype(np.int32)
    gone = r.random(T) < pad
    x[gone] = -np.inf
    ids[gone] = -1
    ids[r.random((T, k)) < 0.05] = -1
    if T > 3:
        ids[3, 0] = E  # outside: dropped
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    return t, t.double().numpy(), ids


def _check(loss, counts, mean, x, ids, coeff):
    want, n, m = norm.balance_loss(x, ids, coeff)
    assert np.array_equal(counts.cpu().numpy(), n)
    assert abs(float(loss) - want) <= 2.0 ** -15 * abs(want) + 1e-12
    assert np.all(np.abs(mean.double().cpu().numpy() - m) <= 2.0 ** -15 * m + 1e-12)


def _check_gradient(d, x, counts, k, d_loss, coeff, dtype, before=0.0):
    n = counts.cpu().numpy()
    want = norm.balance_loss_backward(x, n, k, d_loss, coeff) + before
    p, _ = norm._softmax_rows(x)
    f = norm._loads(n[:-1], int(n[-1]), k)
    g = abs(d_loss * coeff) / max(int(n[-1]), 1)
    bound = 2.0 ** -16 * g * p * (f + (p @ f)[:, None]) + U[dtype] * np.abs(want) + TINY[dtype]
    off = np.abs(d.double().cpu().numpy() - want) - bound - 1e-12 * g
    assert np.all(off <= 0), float(off.max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (17, 33, 3), (100, 64, 8), (64, 32, 1), (700, 96, 4), (65, 160, 8),
                                  (2000, 256, 8), (300, 257, 8), (4099, 8, 2), (257, 512, 10), (90, 1000, 32), (40, 1024, 8),
                                  (9001, 48, 6)])
def test_loss_and_gradient(lib, size, dtype):
    T, E, k = size
    t, x, ids = _case(sum(size), T, E, k, dtype)
    logits, i = t.cuda(), torch.from_numpy(ids).cuda()
    loss, counts, mean = lib.moe_balance_loss(logits, i, 0.3)
    _check(loss, counts, mean, x, ids, 0.3)
    d = lib.moe_balance_loss_backward(logits, counts, k, torch.full((1,), 1.7, device="cuda"), 0.3)
    _check_gradient(d, x, counts, k, float(np.float32(1.7)), 0.3, dtype)
    assert lib.sync_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,pitch", [(64, 8), (50, 3), (256, 0)])
def test_pitch_and_accumulation(lib, dtype, E, pitch):
    """Logits with NaN between the rows; the gradient added to the router's."""
    T, k = 210, 4
    t, x, ids = _case(E, T, E, k, dtype)
    big = torch.full((T, E + pitch), float("nan"), dtype=dtype)
    big[:, :E] = t
    logits, i = big.cuda()[:, :E], torch.from_numpy(ids).cuda()
    loss, counts, mean = lib.moe_balance_loss(logits, i, 1.0)
    _check(loss, counts, mean, x, ids, 1.0)
    one = torch.ones(1, device="cuda")
    before = (torch.randn((T, E), generator=torch.Generator().manual_seed(1)) * 0.01).to(dtype)
    d = before.cuda()
    assert lib.moe_balance_loss_backward(logits, counts, k, one, 1.0, out=d, accumulate=True) is d
    _check_gradient(d, x, counts, k, 1.0, 1.0, dtype, before.double().numpy())
    assert lib.sync_status() == 0


def test_beside_the_router(lib):
    """With moe_route_topk's ids: a uniform load costs coeff, a collapsed router E / k times it."""
    T, E, k = 512, 64, 8
    logits = torch.full((T, E), -30.0, device="cuda")
    for t in range(T):
        logits[t, (torch.arange(k) + t * k) % E] = 0.0
    ids, _ = lib.moe_route_topk(logits, k)
    loss, counts, _ = lib.moe_balance_loss(logits, ids, 0.01)
    assert torch.all(counts[:E] == T * k // E) and int(counts[E]) == T and abs(float(loss) / 0.01 - 1) < 1e-5
    logits[:] = -30.0
    logits[:, :k] = 0.0
    ids, _ = lib.moe_route_topk(logits, k)
    loss, counts, _ = lib.moe_balance_loss(logits, ids, 0.01)
    assert torch.all(counts[:k] == T) and not counts[k:E].any() and abs(float(loss) / 0.01 - E / k) < 1e-4


def test_no_token_takes_part(lib):
    logits = torch.full((5, 16), -float("inf"), device="cuda")
    ids = torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    loss, counts, mean = lib.moe_balance_loss(logits, ids)
    d = lib.moe_balance_loss_backward(logits, counts, 2, torch.ones(1, device="cuda"))
    assert float(loss) == 0 and not counts.any() and not mean.any() and not d.any()
    loss, counts, mean = lib.moe_balance_loss(logits[:0], ids[:0])
    d = lib.moe_balance_loss_backward(logits[:0], counts, 2, torch.ones(1, device="cuda"))
    assert float(loss) == 0 and not counts.any() and not mean.any() and d.shape == (0, 16) and lib.sync_status() == 0


def test_lowest_value_masks_like_minus_infinity(lib):
    """A mask of the type's lowest value leaves p = 0, and a row of nothing else is uniform."""
    for dtype in DTYPES:
        low = torch.finfo(dtype).min
        x = torch.randn((8, 24), generator=torch.Generator().manual_seed(3)).to(dtype)
        x[:, ::2] = low
        x[5] = low
        ids = torch.arange(8, dtype=torch.int32).reshape(8, 1)
        loss, counts, mean = lib.moe_balance_loss(x.cuda(), ids.cuda(), 1.0)
        _check(loss, counts, mean, x.double().numpy(), ids.numpy(), 1.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_logits_mask_their_expert(lib, bad):
    x = torch.randn((9, 40), generator=torch.Generator().manual_seed(4))
    ids = torch.zeros((9, 1), dtype=torch.int32)
    y = x.clone()
    y[2, 3], x[2, 3] = bad, -float("inf")
    got = lib.moe_balance_loss(y.cuda(), ids.cuda())
    assert lib.sync_status() == -5
    want = lib.moe_balance_loss(x.cuda(), ids.cuda())
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and lib.sync_status() == 0
    one = torch.ones(1, device="cuda")
    assert torch.equal(lib.moe_balance_loss_backward(y.cuda(), got[1], 1, one),
                       lib.moe_balance_loss_backward(x.cuda(), got[1], 1, one))


def test_results_do_not_change_from_call_to_call(lib):
    g = torch.Generator("cuda").manual_seed(7)
    logits = torch.randn((30000, 200), device="cuda", generator=g).bfloat16()
    ids, _ = lib.moe_route_topk(logits, 8)
    first = lib.moe_balance_loss(logits, ids)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, lib.moe_balance_loss(logits, ids)))


def test_refusals(lib):
    x = torch.zeros((4, 8), device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    _, counts, _ = lib.moe_balance_loss(x, ids)
    one = torch.ones(1, device="cuda")
    for call in (lambda: lib.moe_balance_loss(x.cpu(), ids), lambda: lib.moe_balance_loss(x, ids.long()),
                 lambda: lib.moe_balance_loss(x, ids[:3]), lambda: lib.moe_balance_loss(x, ids[:, 0]),
                 lambda: lib.moe_balance_loss(x.double(), ids),
                 lambda: lib.moe_balance_loss_backward(x, counts[:8], 2, one),
                 lambda: lib.moe_balance_loss_backward(x, counts, 2, one.double()),
                 lambda: lib.moe_balance_loss_backward(x, counts, 2, torch.ones(2, device="cuda")),
                 lambda: lib.moe_balance_loss_backward(x, counts, 1 << 40, one),
                 lambda: lib.moe_balance_loss_backward(x, counts, 2, one, accumulate=True),
                 lambda: lib.moe_balance_loss_backward(x, counts, 2, one, out=x.half())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lib.moe_balance_loss(x, ids, float("nan")), lambda: lib.moe_balance_loss_backward(x, counts, 9, one),
                 lambda: lib.moe_balance_loss_backward(x, counts, 2, one, out=x),
                 lambda: lib.moe_balance_loss(x.repeat(1 << 17, 1), ids.repeat(1 << 17, 1),
                                              ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
                 lambda: lib.moe_balance_loss(torch.zeros((2, 1025), device="cuda"), ids[:2])):
        with pytest.raises(lib.Q4Error):
            call()
