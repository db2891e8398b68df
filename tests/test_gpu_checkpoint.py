"""8-bit activation checkpoints, the gated activation that writes and reads
them, and the experts' weight gradient from them, on the GPU against the
oracle.

Tolerances.  U: rounding unit of the output type.  Codes and scales are exact.
 * swiglu: the fast exponential is documented within 2 + floor(1.173 |x|) ulp,
   below 2^-17 for |x| <= 88, and a handful of roundings follow: 2^-16 of the
   result; beyond |g| = 88 the factor is below 1e-37: absolute 1e-34;
 * its gradient: the same, of |d u s| (1 + |g| (1 - s)), where 1 - s costs
   |g| 2^-24 more: 2^-15;
 * the weight gradient: products of bf16 numbers are exact in FP32 and a sum
   of n terms, each addition truncated or rounded, is within n 2^-23 of the
   sum of |terms|.
"""
import numpy as np
import pytest
import torch

from oracle import moe

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-34, torch.bfloat16: 1e-34, torch.float16: 2.0 ** -25}


def _dev(x, dtype):
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dtype)
    return t.cuda(), t.float().numpy()


def _pitched(x, dtype, extra, offset):
    big = torch.full((x.shape[0] * (x.shape[1] + extra) + offset + 8,), float("nan"), dtype=dtype)
    view = big.as_strided(x.shape, (x.shape[1] + extra, 1), offset)
    view.copy_(torch.from_numpy(np.ascontiguousarray(x, np.float32)))
    return big.cuda().as_strided(x.shape, (x.shape[1] + extra, 1), offset), view.float().numpy()


def _near(got, want, bound, dtype=torch.float32):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    worst = np.abs(got - want) - (bound + U[dtype] * np.abs(want) + TINY[dtype])
    assert np.all(worst <= 0.0), float(worst.max())


def _acts(rows, K, seed):
    """Ordinary activations, an outlier column, zero and tiny blocks, E4M3 ties, a wide range."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, K)).astype(np.float32)
    x[:, K // 2] *= 20.0
    if rows > 2:
        x[1] = 0.0
        x[2] *= np.float32(1e-7)
    if rows > 3:
        x[3] = np.round(x[3] * 16) / 16 * (448.0 / 16)
    if rows > 4:
        x[4, 0] = 448.0
    return x


SHAPES = [(1, 1), (3, 7), (2, 128), (5, 129), (9, 200), (257, 256), (6, 1000), (33, 2048), (130, 1411)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_checkpoint_bit_exact(lib, dtype, shape):
    x, xh = _dev(_acts(*shape, seed=shape[1]), dtype)
    codes, scales = lib.quantize_fp8_checkpoint(x)
    want = moe.quantize_fp8_checkpoint(xh)
    assert np.array_equal(codes.cpu().numpy(), want[0])
    assert np.array_equal(scales.cpu().numpy(), want[1])
    for extra, offset in ((8, 0), (3, 1)):
        c, s = lib.quantize_fp8_checkpoint(_pitched(xh, dtype, extra, offset)[0])
        assert torch.equal(c, codes) and torch.equal(s, scales)
    assert lib.sync_status() == 0


def test_checkpoint_range(lib):
    """Largest and smallest float32 blocks, the 448 boundary on every binade."""
    top = float(torch.finfo(torch.float32).max)
    x = np.array([[top, -top, 1.0], [1e-45, -1e-45, 0.0], [1e-12, 2e-12, -0.0]], np.float32)
    e = np.arange(-60, 100)
    edge = np.stack([np.float32(1.75) * np.exp2(e), np.nextafter(np.float32(1.75), np.float32(2)) * np.exp2(e),
                     -np.exp2(e)], axis=1).astype(np.float32)
    x = np.concatenate([x, edge])
    codes, scales = lib.quantize_fp8_checkpoint(torch.from_numpy(x).cuda())
    want = moe.quantize_fp8_checkpoint(x)
    assert np.array_equal(scales.cpu().numpy(), want[1]) and np.array_equal(codes.cpu().numpy(), want[0])
    assert lib.sync_status() == 0


def test_non_finite_input_is_reported(lib):
    x = torch.ones((3, 300), device="cuda")
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[2, 299] = bad
        lib.quantize_fp8_checkpoint(y)
        assert lib.sync_status() == -5 and lib.sync_status() == 0
        lib.swiglu_fp8(y)
        assert lib.sync_status() == -5 and lib.sync_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_swiglu(lib, dtype, shape):
    rows, inner = shape
    x = np.concatenate([_acts(rows, inner, 3), _acts(rows, inner, 4)], axis=1)
    x[0, 0] = -90.0
    x[-1, inner - 1] = 200.0
    if dtype == torch.float16:                   # products of two values stay finite
        x = np.clip(x, -200.0, 200.0)
    x, xh = _dev(x, dtype)
    h, codes, scales = lib.swiglu_fp8(x)
    want = moe.swiglu(xh)
    _near(h, want, 2.0 ** -16 * np.abs(want), dtype)
    halves = [moe.quantize_fp8_checkpoint(v) for v in (xh[:, :inner], xh[:, inner:])]
    assert np.array_equal(codes.cpu().numpy(), np.concatenate([c for c, _ in halves], axis=1))
    assert np.array_equal(scales.cpu().numpy(), np.concatenate([s for _, s in halves], axis=1))
    for extra, offset in ((8, 0), (1, 3)):
        again = lib.swiglu_fp8(_pitched(xh, dtype, extra, offset)[0])
        assert torch.equal(again[1], codes) and torch.equal(again[2], scales)
        _near(again[0], want, 2.0 ** -16 * np.abs(want), dtype)

    d, dh = _dev(np.random.default_rng(inner).standard_normal((rows, inner)), dtype)
    got = lib.swiglu_fp8_backward(d, codes, scales)
    restored = np.concatenate([moe.restore_fp8_checkpoint(c, s) for c, s in halves], axis=1)
    want, size = moe.swiglu_backward(dh, restored)
    _near(got, want, 2.0 ** -15 * size, dtype)
    assert torch.equal(lib.swiglu_fp8_backward(_pitched(dh, dtype, 8, 0)[0], codes, scales), got)
    assert lib.sync_status() == 0


def test_swiglu_gradient_is_the_difference_quotient(lib):
    """On values the checkpoint holds exactly, against the kernel's forward
    (float32, differences of 2^-5: error of order h^2 and 2^-21 / h)."""
    r = np.random.default_rng(9)
    x = (r.integers(-14, 15, (2, 8)) / 8.0).astype(np.float32)
    d = r.standard_normal((2, 4)).astype(np.float32)
    h, codes, scales = lib.swiglu_fp8(torch.from_numpy(x).cuda())
    got = lib.swiglu_fp8_backward(torch.from_numpy(d).cuda(), codes, scales).cpu().numpy()
    step = 2.0 ** -5
    for i in np.ndindex(*x.shape):
        y = np.stack([x, x])
        y[0][i] += step
        y[1][i] -= step
        f = [lib.swiglu_fp8(torch.from_numpy(v).cuda())[0].double().cpu().numpy() for v in y]
        q = np.sum((f[0] - f[1]) * d) / (2 * step)
        assert abs(q - got[i]) <= 4.0 * np.abs(d).sum() * (step * step + 2.0 ** -21 / step)


def _groups(sizes, tail=0):
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    return offsets, int(offsets[-1]) + tail


WGRAD = [([1], 8, 16), ([0, 3, 0], 24, 48), ([64, 128, 65], 136, 272), ([1, 63, 2, 200], 256, 256),
         ([300], 520, 144), ([17, 0, 31, 5, 90, 1], 264, 528), ([70] * 9, 128, 1024)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", WGRAD)
@pytest.mark.parametrize("gather", [True, False])
def test_wgrad(lib, dtype, case, gather):
    sizes, N, K = case
    offsets, R = _groups(sizes, tail=5)
    r = np.random.default_rng(R + K)
    T = max(1, R // 2) if gather else R
    token = r.integers(0, T, R).astype(np.int32) if gather else None
    x = _acts(T, K, 5)
    codes, scales = lib.quantize_fp8_checkpoint(torch.from_numpy(x).cuda())
    xh = moe.restore_fp8_checkpoint(codes.cpu().numpy(), scales.cpu().numpy())
    y = r.standard_normal((R, N))
    y[offsets[-1]:] = np.nan                     # rows behind the last expert take no part
    d, dh = _dev(y, torch.bfloat16)
    td = None if token is None else torch.from_numpy(token).cuda()
    off = torch.from_numpy(offsets).cuda()
    out = torch.full((len(sizes), N, K), float("nan"), dtype=dtype, device="cuda")
    got = lib.grouped_wgrad_fp8(d, codes, scales, off, row_token=td, out=out)
    want, size = moe.grouped_wgrad(dh, xh, token, offsets)
    _near(got, want, max(sizes) * 2.0 ** -23 * size, dtype)
    assert lib.sync_status() == 0


def test_wgrad_keeps_experts_apart(lib):
    """Non-finite rows of one expert stay in its gradient."""
    offsets, R = _groups([40, 30, 50])
    d = torch.ones((R, 128), dtype=torch.bfloat16, device="cuda")
    d[40:70] = float("nan")
    d[30, 7] = float("inf")
    codes, scales = lib.quantize_fp8_checkpoint(torch.ones((R, 128), device="cuda"))
    got = lib.grouped_wgrad_fp8(d, codes, scales, torch.from_numpy(offsets).cuda())
    assert torch.isnan(got[1]).all()
    assert torch.equal(got[2], torch.full((128, 128), 50.0, device="cuda"))
    assert torch.isinf(got[0][7]).all()
    assert torch.equal(got[0][:7], torch.full((7, 128), 40.0, device="cuda"))


def test_wgrad_accumulates_and_takes_pitched_rows(lib):
    offsets, R = _groups([10, 0, 150])
    r = np.random.default_rng(1)
    codes, scales = lib.quantize_fp8_checkpoint(torch.from_numpy(_acts(R, 144, 6)).cuda())
    xh = moe.restore_fp8_checkpoint(codes.cpu().numpy(), scales.cpu().numpy())
    d, dh = _pitched(r.standard_normal((R, 72)), torch.bfloat16, 24, 8)
    off = torch.from_numpy(offsets).cuda()
    start = r.standard_normal((3, 72, 144)).astype(np.float32)
    out = torch.from_numpy(start).cuda()
    lib.grouped_wgrad_fp8(d, codes, scales, off, out=out, accumulate=True)
    want, size = moe.grouped_wgrad(dh, xh, None, offsets)
    _near(out, want + start, 151 * 2.0 ** -23 * (size + np.abs(start)))
    assert torch.equal(out[1], torch.from_numpy(start[1]).cuda())


def test_wgrad_of_scales_that_are_no_powers_of_two(lib):
    """x_hat is rounded to bf16: quantize_fp8_blockwise's codes and scales."""
    offsets, R = _groups([90, 38])
    r = np.random.default_rng(2)
    codes, scales = lib.quantize_fp8_blockwise(torch.from_numpy(_acts(R, 256, 7)).cuda(), 1)
    exact = moe.restore_fp8_checkpoint(codes.cpu().numpy(), scales.cpu().numpy())
    xh = torch.from_numpy(exact.astype(np.float32)).bfloat16().double().numpy()
    d, dh = _dev(r.standard_normal((R, 128)), torch.bfloat16)
    got = lib.grouped_wgrad_fp8(d, codes, scales, torch.from_numpy(offsets).cuda())
    want, size = moe.grouped_wgrad(dh, xh, None, offsets)
    _near(got, want, 90 * 2.0 ** -23 * size)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[6000], [5000, 0, 2900], [1, 9000]])
def test_wgrad_few_outputs_of_many_rows(lib, dtype, sizes):
    """Rows split over the GPU and joined (float64 on the GPU)."""
    g = torch.Generator("cuda").manual_seed(len(sizes))
    N, K, E = 264, 272, len(sizes)
    offsets, R = _groups(sizes, tail=3)
    codes, scales = lib.quantize_fp8_checkpoint(torch.randn((700, K), device="cuda", generator=g))
    token = torch.randint(0, 700, (R,), device="cuda", generator=g, dtype=torch.int32)
    d = torch.randn((R, N), device="cuda", generator=g).bfloat16()
    off = torch.from_numpy(offsets).cuda()
    x = codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, 1)[:, :K]
    start = torch.randn((E, N, K), device="cuda", generator=g)
    added = lib.grouped_wgrad_fp8(d, codes, scales, off, row_token=token, out=start.clone(), accumulate=True)
    got = lib.grouped_wgrad_fp8(d, codes, scales, off, row_token=token, out_dtype=dtype)
    assert torch.equal(got, lib.grouped_wgrad_fp8(d, codes, scales, off, row_token=token, out_dtype=dtype))
    for e in range(E):
        dd, xx = d[offsets[e]:offsets[e + 1]].double(), x[token[offsets[e]:offsets[e + 1]].long()]
        want, size = dd.t() @ xx, dd.abs().t() @ xx.abs()
        bound = (sizes[e] + 64) * 2.0 ** -23 * size
        assert bool(((got[e].double() - want).abs() <= bound + U[dtype] * want.abs()).all())
        want = want + start[e].double()
        bound = bound + 2.0 ** -23 * start[e].double().abs()
        assert bool(((added[e].double() - want).abs() <= bound + U[torch.float32] * want.abs()).all())
    assert lib.sync_status() == 0


def test_offsets_beyond_32_bits(lib):
    """More than 2^31 elements in the rows, the checkpoint and the gradient."""
    T, k, H = 40000, 8, 7168
    x = torch.randn((T, H), device="cuda").bfloat16()
    ids = torch.arange(T * k, device="cuda", dtype=torch.int32).reshape(T, k) % 97
    _, token, slot = lib.moe_sort_tokens(ids, 97)
    rows = lib.moe_dispatch(x, slot)
    assert rows.numel() > 2 ** 31
    assert torch.equal(rows[-1000:], x[token[-1000:].long()])
    back = lib.moe_combine(rows, slot, torch.full((T, k), 0.125, device="cuda"))
    assert torch.equal(back, x)
    d_rows, dw = lib.moe_combine_backward(x, rows, slot, torch.ones((T, k), device="cuda"), out=rows)
    assert torch.equal(d_rows[-1000:], x[token[-1000:].long()])
    want = x[-100:].double().square().sum(1, keepdim=True).expand(100, k)
    assert bool(((dw[-100:].double() - want).abs() <= 100 * 2.0 ** -24 * want).all())
    codes, scales = lib.quantize_fp8_checkpoint(rows)
    tail = moe.quantize_fp8_checkpoint(rows[-3:].float().cpu().numpy())
    assert np.array_equal(codes[-3:].cpu().numpy(), tail[0]) and np.array_equal(scales[-3:].cpu().numpy(), tail[1])
    del rows, d_rows, back
    h, c2, s2 = lib.swiglu_fp8(x.reshape(-1, 2 * 3584).repeat(8, 1))
    assert c2.numel() > 2 ** 31 and torch.equal(h[-40000:], h[:40000])
    g = lib.swiglu_fp8_backward(h, c2, s2)
    assert torch.equal(g[-40000:], g[:40000])
    del h, c2, s2, g
    E, N, K = 160, 2048, 7168
    off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * 3
    d = torch.randn((3 * E, N), device="cuda").bfloat16()
    dw = lib.grouped_wgrad_fp8(d, codes[:3 * E].contiguous(), scales[:3 * E].contiguous(), off, out_dtype=torch.bfloat16)
    assert dw.numel() > 2 ** 31
    xx = moe.restore_fp8_checkpoint(codes[3 * E - 3:3 * E].cpu().numpy(), scales[3 * E - 3:3 * E].cpu().numpy())
    want = d[-3:].double().cpu().numpy().T @ xx
    size = np.abs(d[-3:].double().cpu().numpy()).T @ np.abs(xx)
    _near(dw[-1], want, 3 * 2.0 ** -23 * size, torch.bfloat16)


def test_wgrad_large_groups(lib):
    """More tiles than SMs, groups of hundreds of rows, gathered tokens (float64 on the GPU)."""
    g = torch.Generator("cuda").manual_seed(4)
    T, E, N, K, k = 900, 12, 1288, 1552, 4
    ids = torch.stack([torch.randperm(E, device="cuda", generator=g)[:k] for _ in range(T)]).int()
    offsets, token, _ = lib.moe_sort_tokens(ids, E)
    codes, scales = lib.quantize_fp8_checkpoint(torch.randn((T, K), device="cuda", generator=g))
    d = torch.randn((T * k, N), device="cuda", generator=g).bfloat16()
    x = codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, 1)[:, :K]
    for dtype in (torch.float32, torch.bfloat16):
        got = lib.grouped_wgrad_fp8(d, codes, scales, offsets, row_token=token, out_dtype=dtype)
        again = lib.grouped_wgrad_fp8(d, codes, scales, offsets, row_token=token, out_dtype=dtype)
        assert torch.equal(got, again)
        b = offsets.tolist()
        for e in range(E):
            dd, xx = d[b[e]:b[e + 1]].double(), x[token[b[e]:b[e + 1]].long()]
            want, size = dd.t() @ xx, dd.abs().t() @ xx.abs()
            bound = (b[e + 1] - b[e]) * 2.0 ** -23 * size + U[dtype] * want.abs()
            assert bool(((got[e].double() - want).abs() <= bound).all())
    assert lib.sync_status() == 0


def test_empty_inputs(lib):
    f = dict(device="cuda")
    codes, scales = lib.quantize_fp8_checkpoint(torch.empty((0, 256), **f))
    assert codes.shape == (0, 256) and scales.shape == (0, 2)
    h, c, s = lib.swiglu_fp8(torch.empty((0, 512), **f))
    assert h.shape == (0, 256) and lib.swiglu_fp8_backward(h, c, s).shape == (0, 512)
    d = torch.empty((0, 16), dtype=torch.bfloat16, **f)
    out = lib.grouped_wgrad_fp8(d, codes, scales, torch.zeros(3, dtype=torch.int32, **f))
    assert out.shape == (2, 16, 256) and not out.any()


def test_refusals(lib):
    f = dict(device="cuda")
    d = torch.zeros((6, 16), dtype=torch.bfloat16, **f)
    codes, scales = torch.zeros((6, 32), dtype=torch.uint8, **f), torch.ones((6, 1), **f)
    off = torch.tensor([0, 6], dtype=torch.int32, **f)
    for bad in (lambda: lib.quantize_fp8_checkpoint(d.t()), lambda: lib.quantize_fp8_checkpoint(d.cpu()),
                lambda: lib.swiglu_fp8(torch.zeros((2, 5), **f)),
                lambda: lib.swiglu_fp8_backward(d, codes, scales),
                lambda: lib.swiglu_fp8_backward(d, codes.int(), torch.ones((6, 2), **f)),
                lambda: lib.grouped_wgrad_fp8(d.float(), codes, scales, off),
                lambda: lib.grouped_wgrad_fp8(d, codes, scales[:, :0], off),
                lambda: lib.grouped_wgrad_fp8(d, codes, scales, off.long()),
                lambda: lib.grouped_wgrad_fp8(d, codes, scales, off, row_token=off),
                lambda: lib.grouped_wgrad_fp8(d, codes, scales, off, accumulate=True),
                lambda: lib.grouped_wgrad_fp8(d, codes, scales, off, out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    for args, status in (((d[:, :12], codes, scales, off), -2), ((d, codes[:, :24].contiguous(), scales, off), -2),
                         ((d[:4], codes, scales, off), -1)):
        with pytest.raises(lib.Q4Error) as e:
            lib.grouped_wgrad_fp8(*args)
        assert e.value.status == status
    with pytest.raises(lib.Q4Error) as e:
        lib.grouped_wgrad_fp8(d, codes, scales, off, out=torch.empty((1, 16, 32), dtype=torch.bfloat16, **f),
                              accumulate=True)
    assert e.value.status == -1
