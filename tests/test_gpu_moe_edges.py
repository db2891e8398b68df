"""Edges of the routed-expert calls' arguments: matrices of one row and of no
columns, counts beyond 32 bits.

Tolerance of the weight gradient of one row: the product of two bf16 numbers is
exact in float32: none.
"""
import numpy as np
import pytest
import torch

from oracle import moe

pytestmark = pytest.mark.gpu


def test_pitch_of_one_row_does_not_matter(lib):
    """The pitch of a single row names nothing: any is taken, and the result is
    that of the contiguous row."""
    g = torch.Generator("cuda").manual_seed(1)
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    codes, scales = lib.quantize_fp8_checkpoint(torch.randn((1, 32), device="cuda", generator=g))
    buf = torch.randn(64, device="cuda", generator=g).bfloat16()
    x = moe.restore_fp8_checkpoint(codes.cpu().numpy(), scales.cpu().numpy())
    slot = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    for pitch in (1, 9, 17, 16, 24):
        d = buf.as_strided((1, 16), (pitch, 1))
        got = lib.grouped_wgrad_fp8(d, codes, scales, off)
        want = d.double().cpu().numpy().T @ x
        assert np.array_equal(got[0].double().cpu().numpy(), want)
        assert torch.equal(lib.moe_dispatch(d, slot), d)
        assert torch.equal(lib.quantize_fp8_checkpoint(d)[0], lib.quantize_fp8_checkpoint(d.contiguous())[0])
    assert lib.sync_status() == 0


def test_weight_gradient_of_no_outputs(lib):
    codes, scales = lib.quantize_fp8_checkpoint(torch.ones((5, 32), device="cuda"))
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    for d in (torch.empty((5, 0), dtype=torch.bfloat16, device="cuda"),
              torch.ones((5, 16), dtype=torch.bfloat16, device="cuda")[:, :0]):
        assert lib.grouped_wgrad_fp8(d, codes, scales, off).shape == (2, 0, 32)


def test_refused_top_k_allocates_nothing(lib):
    x = torch.zeros((1 << 20, 8), device="cuda")
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    with pytest.raises(lib.Q4Error) as e:
        lib.moe_route_topk(x, 1 << 10)
    assert e.value.status == -1
    assert torch.cuda.max_memory_allocated() - before < 1 << 20


def test_counts_beyond_32_bits_are_refused(lib):
    """2^32 + n is not n."""
    x = torch.zeros((1, 8), device="cuda")
    ids = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    for call in (lambda: lib.moe_route_topk(x, (1 << 32) + 2), lambda: lib.moe_sort_tokens(ids, (1 << 32) + 4),
                 lambda: lib.moe_route_topk(x, 2 - (1 << 32))):
        with pytest.raises(ValueError):
            call()
