"""8-bit checkpoints of the largest float32 and bfloat16 numbers: what is finite
restores as a finite number, wherever it is restored.

Tolerances: half a unit of four significant bits, 1/16 of the value (248 and more
times 2^120 go to 240 times 2^120: at most 16/256), or half the smallest code's
step; the gated activation's
gradient as in its other tests, 2^-15 of its terms.
"""
import numpy as np
import pytest
import torch

from oracle import moe

pytestmark = pytest.mark.gpu

TOP = 2.0 ** 120


def _rows():
    edge = np.float32(248 * TOP)
    return np.array([[np.finfo(np.float32).max, -np.finfo(np.float32).max, 1.0],
                     [edge, -np.nextafter(edge, np.float32(0)), 0.0],
                     [np.nextafter(edge, np.float32(np.inf)), 240 * TOP, -250 * TOP],
                     [3.3895314e38, -3.3e38, 2e38],                      # the largest bfloat16
                     [224 * TOP, 223 * TOP, 2.0 ** 127]], np.float32)    # below: the scale is 2^119


@pytest.mark.parametrize("width", [3, 16, 131])
def test_largest_values_restore_as_finite(lib, width):
    x = np.tile(_rows(), (1, width // 3 + 1))[:, :width].copy()
    for dtype in (torch.float32, torch.bfloat16):
        t = torch.from_numpy(x).to(dtype)
        t = torch.where(torch.isinf(t), torch.sign(t) * torch.finfo(dtype).max, t)
        codes, scales = lib.quantize_fp8_checkpoint(t.cuda())
        want = moe.quantize_fp8_checkpoint(t.float().numpy())
        assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])
        v = moe.restore_fp8_checkpoint(codes.cpu().numpy(), scales.cpu().numpy())
        assert np.all(np.isfinite(v.astype(np.float32))) and np.all(np.abs(v) <= 240 * TOP)
        assert np.all(np.isfinite(torch.from_numpy(v).bfloat16().float().numpy()))
        step = np.repeat(scales.double().cpu().numpy(), 128, axis=1)[:, :width]
        assert np.all(np.abs(v - t.double().numpy()) <= np.maximum(np.abs(t.double().numpy()) / 16, step * 2.0 ** -10))
    assert lib.sync_status() == 0


def test_weight_gradient_of_the_largest_values(lib):
    x = torch.from_numpy(np.tile(_rows(), (1, 6))[:, :16].copy()).cuda()
    codes, scales = lib.quantize_fp8_checkpoint(x)
    v = moe.restore_fp8_checkpoint(codes.cpu().numpy(), scales.cpu().numpy())
    R = x.shape[0]
    off = torch.arange(R + 1, dtype=torch.int32, device="cuda")           # one row per expert
    d = torch.full((R, 8), 0.5, dtype=torch.bfloat16, device="cuda")
    got = lib.grouped_wgrad_fp8(d, codes, scales, off).double().cpu().numpy()
    assert np.array_equal(got, np.repeat(0.5 * v[:, None, :], 8, axis=1))
    assert lib.sync_status() == 0


@pytest.mark.parametrize("inner", [6, 16])
def test_gated_activation_of_the_largest_values(lib, inner):
    up = np.tile(_rows(), (1, 6))[:, :inner]
    gate = np.random.default_rng(0).standard_normal(up.shape).astype(np.float32)
    _, codes, scales = lib.swiglu_fp8(torch.from_numpy(np.concatenate([gate, up], axis=1)).cuda())
    halves = [moe.quantize_fp8_checkpoint(np.ascontiguousarray(h)) for h in (gate, up)]
    assert np.array_equal(codes.cpu().numpy(), np.concatenate([c for c, _ in halves], axis=1))
    d = np.full(up.shape, 2.0 ** -20, np.float32)
    got = lib.swiglu_fp8_backward(torch.from_numpy(d).cuda(), codes, scales).double().cpu().numpy()
    restored = np.concatenate([moe.restore_fp8_checkpoint(c, s) for c, s in halves], axis=1)
    want, size = moe.swiglu_backward(d, restored)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= 2.0 ** -15 * size + 1e-34)
    assert lib.sync_status() == 0


def test_what_is_not_finite_stays_so(lib):
    x = torch.tensor([[np.inf, 1.0, -np.inf, np.nan]], device="cuda")
    codes, scales = lib.quantize_fp8_checkpoint(x)
    assert lib.sync_status() == -5
    v = codes.view(torch.float8_e4m3fn).float() * scales
    assert v[0, 0] == np.inf and v[0, 2] == -np.inf and torch.isnan(v[0, 3])
