"""Workspaces that the caller gives: one that is not the device's memory is refused
before any launch, one of another type counts by its bytes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _calls(lib):
    g = torch.Generator("cuda").manual_seed(1)
    x, dy = (torch.randn((700, 256), device="cuda", generator=g) for _ in range(2))
    _, _, rstd = lib.rms_norm(x)
    logits = torch.randn((20000, 16), device="cuda", generator=g)
    ids, _ = lib.moe_route_topk(logits, 2)
    size = lib.lib().q4_workspace_size
    return {
        "rms_norm_backward": (lambda ws: lib.rms_norm_backward(dy, x, rstd, ws=ws), size(lib.OP_RMS_NORM_BACKWARD, 700, 0, 256)),
        "moe_balance_loss": (lambda ws: lib.moe_balance_loss(logits, ids, ws=ws), size(lib.OP_MOE_BALANCE_LOSS, 20000, 16, 0)),
        "moe_sort_tokens": (lambda ws: lib.moe_sort_tokens(ids, 16, ws=ws), size(lib.OP_MOE_SORT, 40000, 16, 0)),
    }


def test_host_memory_and_strided_ones_are_refused(lib, monkeypatch):
    calls = _calls(lib)
    torch.cuda.synchronize()
    # the library is out of reach: a call that is not refused before fails otherwise
    monkeypatch.setattr(lib, "_lib", object())
    for call, n in calls.values():
        for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(ValueError, match="ws must"):
                call(ws)


def test_other_types_count_by_their_bytes(lib):
    for call, n in _calls(lib).values():
        want = call(None)
        got = call(torch.full((-(-n // 4),), float("nan"), device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and lib.sync_status() == 0
