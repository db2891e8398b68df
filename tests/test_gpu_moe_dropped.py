"""Dropped slots through the grouped products: rows behind the last expert's
end are nobody's product, whatever the memory that the products' outputs get
held before.

Tolerances.  The grouped product: a BF16 rounding, 2^-8, and FP32 sums of K
terms, K 2^-23 of the sum of their magnitudes.  The layer's step in different
memory: none.
"""
import numpy as np
import pytest
import torch

import oracle
from examples import moe_training_step as ex

pytestmark = pytest.mark.gpu


def _weights(lib, E, N, K, seed):
    w = np.random.default_rng(seed).standard_normal((E, N, K)).astype(np.float32) * K ** -0.5
    parts = [lib.quantize_nvfp4(torch.from_numpy(e).cuda(), scale_layout="mma") for e in w]
    form = (torch.stack([c for c, _, _ in parts]), torch.cat([s for _, s, _ in parts]), torch.cat([g for _, _, g in parts]))
    return form, [oracle.quantize_nvfp4(e) for e in w]


@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("case", [(33, 4, 2, 256, 256), (200, 5, 3, 37, 512), (1, 3, 8, 320, 256)])
def test_rows_of_dropped_slots_are_zero(lib, case, drop):
    T, E, k, N, K = case
    r = np.random.default_rng(T)
    ids = r.integers(0, E, (T, k)).astype(np.int32)
    ids[r.random((T, k)) < drop] = -1
    offsets, token, slot = lib.moe_sort_tokens(torch.from_numpy(ids).cuda(), E)
    x = torch.from_numpy(r.standard_normal((T, K)).astype(np.float32)).bfloat16()
    form, experts = _weights(lib, E, N, K, 3)
    guard = torch.full((T * k + 2, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    C = lib.grouped_gemm_moe(x.cuda(), offsets, token, *form, N, out=guard[:T * k]).float().cpu().numpy()
    live = int(offsets[-1])
    assert not C[live:].any()
    assert torch.isnan(guard[T * k:]).all()
    tok = token.cpu().numpy()
    want = oracle.grouped_gemm_moe(x.float().numpy(), offsets.cpu().numpy(), tok, experts)
    assert want.shape == (T * k, N) and not want[live:].any()
    a_hat = np.abs(oracle.dequantize_nvfp4(*oracle.quantize_nvfp4(x.float().numpy())))
    size = np.zeros_like(want)
    for e in range(E):
        rows = slice(int(offsets[e]), int(offsets[e + 1]))
        size[rows] = a_hat[tok[rows]] @ np.abs(oracle.dequantize_nvfp4(*experts[e])).T
    assert np.all(np.abs(C - want) <= 2.0 ** -8 * np.abs(want) + K * 2.0 ** -23 * size)
    assert lib.sync_status() == 0


def test_rows_without_any_expert_are_zero(lib):
    f = dict(device="cuda")
    out = torch.full((6, 256), float("nan"), dtype=torch.bfloat16, **f)
    lib.grouped_gemm_moe(torch.ones((3, 256), dtype=torch.bfloat16, **f), torch.zeros(1, dtype=torch.int32, **f),
                         torch.zeros(6, dtype=torch.int32, **f), torch.empty((0, 256, 128), dtype=torch.uint8, **f),
                         torch.empty(0, dtype=torch.uint8, **f), torch.empty(0, **f), 256, out=out)
    assert not out.any()


def _poison(monkeypatch, value, byte):
    """New memory holds ``value`` (``byte`` in bytes), as recycled memory may."""
    plain = torch.empty

    def empty(*args, **kwargs):
        t = plain(*args, **kwargs)
        if t.is_floating_point():
            t.fill_(value)
        elif t.dtype == torch.uint8:
            t.fill_(byte)
        return t
    monkeypatch.setattr(torch, "empty", empty)


@pytest.mark.parametrize("masked,dropped", [(False, True), (True, False), (True, True)])
def test_layer_does_not_depend_on_what_memory_held(lib, monkeypatch, masked, dropped):
    """A layer's step with masked experts and dropped slots in zeroed memory, in
    memory of NaN and in memory of huge numbers: the same bits, all finite, and
    no error reported."""
    torch.manual_seed(2)
    T, H, I, E, k = 384, 512, 256, 8, 2
    layer = ex.MoeLayer(H, I, E, k)
    x = torch.randn((T, H), device="cuda").bfloat16()
    d_out = torch.randn((T, H), device="cuda").bfloat16()
    allowed = torch.ones((T, E), dtype=torch.bool, device="cuda")
    if masked:
        allowed = torch.rand((T, E), device="cuda") < 0.7
        allowed[::7] = False
        allowed[::7, 3] = True          # one expert left
        allowed[::11] = False           # none
    drop = torch.zeros((T, k), dtype=torch.bool, device="cuda")
    if dropped:
        drop = torch.rand((T, k), device="cuda") < 0.25
        drop[5] = True
    sort = lib.moe_sort_tokens
    results = []
    for value, byte in ((0.0, 0), (float("nan"), 0x7f), (3e38, 0x7e)):
        monkeypatch.setattr(lib, "moe_sort_tokens", lambda ids, E: sort(ids.masked_fill(drop, -1), E))
        _poison(monkeypatch, value, byte)
        out, kept = layer.forward(x, allowed=allowed)
        got = layer.backward(d_out, kept)
        monkeypatch.undo()
        assert lib.sync_status() == 0
        live = (kept["ids"] >= 0) & ~drop
        assert int(kept["offsets"][-1]) == int(live.sum()) < T * k
        assert torch.equal((kept["ids"] >= 0).sum(1), allowed.sum(1).clamp(max=k))
        assert not out[~live.any(1)].any() and out[live.any(1)].any(1).all()
        assert all(bool(torch.isfinite(t).all()) for t in (out,) + got)
        results.append((out,) + got)
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a, b)
