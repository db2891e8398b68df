"""Outputs that share memory with inputs: refused where a call would read what it
has written, and the in-place form of moe_combine_backward."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def _slots(lib, T, k, seed, drop=0.2):
    r = np.random.default_rng(seed)
    ids = r.integers(0, 7, (T, k)).astype(np.int32)
    ids[r.random((T, k)) < drop] = -1
    return lib.moe_sort_tokens(torch.from_numpy(ids).cuda(), 7)[2]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(5, 3, 1000), (301, 3, 520), (301, 3, 67), (301, 3, 1), (64, 2, 4098), (400, 2, 4098)])
def test_combine_gradient_in_place(lib, dtype, shape):
    T, k, H = shape
    slot = _slots(lib, T, k, T)
    g = torch.Generator("cuda").manual_seed(H)
    rows = torch.randn((T * k, H), device="cuda", generator=g).to(dtype)
    d = torch.randn((T, H), device="cuda", generator=g).to(dtype)
    w = torch.randn((T, k), device="cuda", generator=g)
    want = lib.moe_combine_backward(d, rows, slot, w)
    got = lib.moe_combine_backward(d, rows, slot, w, out=rows)
    assert got[0] is rows and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert lib.sync_status() == 0


def test_overlapping_memory_is_refused(lib):
    f = dict(device="cuda")
    slot = torch.tensor([[1], [0], [3], [2]], dtype=torch.int32, **f)
    buf = torch.zeros(4096, **f)
    x, w = buf[:32].view(4, 8), torch.ones((4, 1), **f)
    near = buf[8:40].view(4, 8)                  # shares three rows with x
    pitched = buf.as_strided((4, 8), (24, 1))    # columns 0 to 7 of 24
    offsets = torch.tensor([0, 4], dtype=torch.int32, **f)
    d_y = torch.zeros((4, 8), dtype=torch.bfloat16, **f)
    codes, scales = torch.zeros((4, 16), dtype=torch.uint8, **f), torch.ones((4, 1), **f)
    calls = [lambda: lib.moe_dispatch(x, slot, out=x), lambda: lib.moe_dispatch(x, slot, out=near),
             lambda: lib.moe_dispatch(pitched, slot, out=buf[20:52].view(4, 8)),
             lambda: lib.moe_combine(x, slot, w, out=x), lambda: lib.moe_dispatch_backward(x, slot, out=near),
             lambda: lib.moe_combine(x, slot, buf[40:44].view(4, 1), out=buf[16:48].view(4, 8)),
             lambda: lib.moe_combine_backward(x, torch.zeros((4, 8), **f), slot, w, out=x),
             lambda: lib.moe_combine_backward(torch.zeros((4, 8), **f), x, slot, w, out=near),
             lambda: lib.moe_combine_backward(torch.zeros((4, 8), **f), pitched, slot, w, out=x),
             lambda: lib.swiglu_fp8(x, out=buf[16:32].view(4, 4)),
             lambda: lib.swiglu_fp8_backward(x[:, :4], torch.zeros((4, 8), dtype=torch.uint8, **f), torch.ones((4, 2), **f),
                                             out=x),
             lambda: lib.grouped_wgrad_fp8(d_y, codes, scales, offsets, out=buf[:128].view(1, 8, 16),
                                           ws=buf.view(torch.uint8)),
             lambda: lib.grouped_wgrad_fp8(buf.view(torch.bfloat16)[:32].view(4, 8), codes, scales, offsets,
                                           out=buf[:128].view(1, 8, 16))]
    for call in calls:
        with pytest.raises(lib.Q4Error) as e:
            call()
        assert e.value.status == -1
    assert not buf.any() and lib.sync_status() == 0


def test_neighbouring_memory_is_taken(lib):
    """Outputs right before, right behind and between the rows of an input."""
    f = dict(device="cuda")
    slot = torch.tensor([[1], [0]], dtype=torch.int32, **f)
    buf = torch.arange(256, dtype=torch.float32, **f)
    x = buf.as_strided((2, 8), (64, 1), 32)      # 32..39 and 96..103
    for at in (16, 40, 80, 104):
        want = x[[1, 0]].clone()
        got = lib.moe_dispatch(x, slot, out=buf[at:at + 16].view(2, 8))
        assert torch.equal(got, want)
    # rows is not read without d_weights
    d, rows = torch.ones((2, 8), **f), torch.ones((2, 8), **f)
    got, _ = lib.moe_combine_backward(d, rows, slot, torch.ones((2, 1), **f), need_d_weights=False, out=rows)
    assert torch.equal(got, d)
