"""Both forms of the combine gradient (one warp per slot, and eight where the
slots are few), and the routed-expert calls inside a CUDA graph.

Tolerances of the combine gradient: d_rows is one rounding of a float32 product,
2^-24 and the output type's unit U; d_weights sums H products in at least 128
partial sums, which 32 more additions at most join: (H / 128 + 32) 2^-24 of the
sum of |terms|.  A replayed graph gives the eager calls' bits.
"""
import numpy as np
import pytest
import torch

from oracle import moe

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-38, torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25}


def _near(got, want, bound, dtype=torch.float32):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    worst = np.abs(got - want) - (bound + U[dtype] * np.abs(want) + TINY[dtype])
    assert np.all(worst <= 0.0), float(worst.max())


def _shape(slots):
    """(T, k) by name: the last count with eight warps per slot, the first with one."""
    few = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    return {"few": (few // 4, 4), "many": (few + 1, 1), "odd": (301, 3)}[slots]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [1, 67, 520, 1002, 2056, 3333])
@pytest.mark.parametrize("slots", ["few", "many", "odd"])
def test_combine_gradient_of_few_and_many_slots(lib, dtype, H, slots):
    """Units of 16 and 4 bytes and single elements, real weights, dropped slots
    whose rows and weights hold NaN, whole and partial last blocks."""
    T, k = _shape(slots)
    r = np.random.default_rng(T + H)
    ids = r.integers(0, 9, (T, k)).astype(np.int32)
    ids[r.random((T, k)) < 0.2] = -1
    sd = lib.moe_sort_tokens(torch.from_numpy(ids).cuda(), 9)[2]
    sh = sd.cpu().numpy()
    x, w = r.standard_normal((T * k, H)).astype(np.float32), r.standard_normal((T, k)).astype(np.float32)
    x[~sh[sh < 0]] = np.nan
    w[sh < 0] = np.nan
    rows = torch.from_numpy(x).to(dtype)
    d = torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(dtype)
    out = torch.full((T * k, H), float("nan"), dtype=dtype, device="cuda")
    d_rows, d_w = lib.moe_combine_backward(d.cuda(), rows.cuda(), sd, torch.from_numpy(w).cuda(), out=out)
    want, want_w, size = moe.combine_backward(d.double().numpy(), rows.double().numpy(), sh, w)
    _near(d_rows, want, 2.0 ** -24 * np.abs(want), dtype)
    _near(d_w, want_w, (H / 128 + 32) * 2.0 ** -24 * size)
    assert not d_w.cpu().numpy()[sh < 0].any()
    only, _ = lib.moe_combine_backward(d.cuda(), rows.cuda(), sd, torch.from_numpy(w).cuda(), need_d_weights=False)
    assert torch.equal(only, d_rows)
    assert lib.sync_status() == 0


@pytest.mark.parametrize("T", [3, 500, 6000])
def test_calls_in_a_cuda_graph(lib, T):
    """A layer's calls captured once and replayed on new inputs in the same buffers."""
    E, k, H, I = 8, 3, 256, 256
    g = torch.Generator("cuda").manual_seed(T)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    def form(N, K):
        q = [lib.quantize_nvfp4(normal(N, K) * K ** -0.5, scale_layout="mma") for _ in range(E)]
        return torch.stack([c for c, _, _ in q]), torch.cat([s for _, s, _ in q]), torch.cat([t for _, _, t in q])
    w1, w2 = form(2 * I, H), form(H, I)
    rows = torch.arange(T * k, dtype=torch.int32, device="cuda")
    x, logits, d_out = normal(T, H).bfloat16(), normal(T, E), normal(T, H).bfloat16()

    def step():
        ids, weights = lib.moe_route_topk(logits, k)
        offsets, token, slot = lib.moe_sort_tokens(ids, E)
        gate_up = lib.grouped_gemm_moe(x, offsets, token, *w1, 2 * I)
        h, codes, scales = lib.swiglu_fp8(gate_up)
        y = lib.grouped_gemm_moe(h, offsets, rows, *w2, H)
        out = lib.moe_combine(y, slot, weights)
        d_y, d_weights = lib.moe_combine_backward(d_out, y, slot, weights)
        dw2 = lib.grouped_wgrad_fp8(d_y, *lib.quantize_fp8_checkpoint(h), offsets)
        d_gate_up = lib.swiglu_fp8_backward(torch.ones_like(h), codes, scales)
        dw1 = lib.grouped_wgrad_fp8(d_gate_up, *lib.quantize_fp8_checkpoint(x), offsets, row_token=token,
                                    out_dtype=torch.bfloat16)
        d_rows = lib.moe_dispatch(x, slot)
        d_x = lib.moe_dispatch_backward(d_rows, slot)
        return ids, out, d_weights, dw2, dw1, d_x, lib.moe_route_topk_backward(logits, ids, d_weights)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(3):
        x.copy_(normal(T, H)), logits.copy_(normal(T, E)), d_out.copy_(normal(T, H))
        if seed == 2:                # a token without any expert, and one with a single one
            logits[0] = -float("inf")
            logits[1, 1:] = -float("inf")
        graph.replay()
        want = step()
        for a, b in zip(captured, want):
            assert torch.equal(a, b)
    assert lib.sync_status() == 0
