"""Tensors of a device that is not the current one are refused before any launch
(kernels, the status word and the stream are the current device's).  There is one
device here, so the current one is made to look like another."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture
def calls(lib):
    x = torch.zeros((4, 64), device="cuda", dtype=torch.bfloat16)
    rstd, one = torch.ones(4, device="cuda"), torch.ones(1, device="cuda")
    logits, ids = torch.zeros((4, 8), device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    counts = torch.zeros(9, dtype=torch.int32, device="cuda")
    q, s = torch.zeros((4, 64), dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    return {
        "rms_norm": lambda: lib.rms_norm(x), "rms_norm_fp8": lambda: lib.rms_norm_fp8(x, residual=x),
        "rms_norm_int8": lambda: lib.rms_norm_int8(x), "rms_norm_backward": lambda: lib.rms_norm_backward(x, x, rstd),
        "quantize_int8": lambda: lib.quantize_int8(x), "gemm_w8a8_int8": lambda: lib.gemm_w8a8_int8(q, s, q, s),
        "moe_sort_tokens": lambda: lib.moe_sort_tokens(ids, 8), "moe_route_topk": lambda: lib.moe_route_topk(logits, 2),
        "moe_balance_loss": lambda: lib.moe_balance_loss(logits, ids),
        "moe_balance_loss_backward": lambda: lib.moe_balance_loss_backward(logits, counts, 2, one),
    }


def test_refused(lib, calls, monkeypatch):
    for call in calls.values():
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(lib, "_device", lambda: torch.cuda.device_count())
    # a call that is not refused would go on to the library: there is none
    monkeypatch.setattr(lib, "_lib", object())
    for name, call in calls.items():
        with pytest.raises(ValueError, match="current device"):
            call()
