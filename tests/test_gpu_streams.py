"""Calls on a stream that is given, while the current stream still has work
pending on memory that it has let go."""
import pytest
import torch

pytestmark = pytest.mark.gpu

# Cycles that the current stream is kept busy for: far longer than a call takes
# to come back to the host and to run.
BUSY = 200_000_000


def _calls(q4):
    """name -> call(stream) -> its outputs; inputs made beforehand."""
    g = torch.Generator("cuda").manual_seed(3)
    T, k, E, H = 640, 4, 16, 512

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)
    logits, x = normal(T, E), normal(T, H).bfloat16()
    ids, w = q4.moe_route_topk(logits, k)
    big_ids = torch.randint(-1, E, (20000, 2), device="cuda", dtype=torch.int32, generator=g)
    offsets, token, slot = q4.moe_sort_tokens(ids, E)
    rows, dw, d_h = normal(T * k, H).bfloat16(), normal(T, k), normal(T, H // 2).bfloat16()
    _, codes, scales = q4.swiglu_fp8(x)
    xc, xs = q4.quantize_fp8_checkpoint(x)
    d_y = normal(T * k, 256).bfloat16()
    wq = [q4.quantize_nvfp4(normal(256, H), scale_layout="mma") for _ in range(E)]
    form = (torch.stack([c for c, _, _ in wq]), torch.cat([s for _, s, _ in wq]), torch.cat([t for _, _, t in wq]))
    a, b = normal(256, H).bfloat16(), q4.Fp4Operand(*q4.quantize_mxfp4(normal(256, H), scale_layout="mma"), "mma")
    return {
        "route": lambda s: q4.moe_route_topk(logits, k, stream=s),
        "route_backward": lambda s: q4.moe_route_topk_backward(logits, ids, dw, stream=s),
        "sort": lambda s: q4.moe_sort_tokens(ids, E, stream=s),
        "sort_long": lambda s: q4.moe_sort_tokens(big_ids, E, stream=s),
        "dispatch": lambda s: q4.moe_dispatch(x, slot, stream=s),
        "dispatch_backward": lambda s: q4.moe_dispatch_backward(rows, slot, stream=s),
        "combine": lambda s: q4.moe_combine(rows, slot, w, stream=s),
        "combine_backward": lambda s: q4.moe_combine_backward(x, rows, slot, w, stream=s),
        "checkpoint": lambda s: q4.quantize_fp8_checkpoint(x, stream=s),
        "swiglu": lambda s: q4.swiglu_fp8(x, stream=s),
        "swiglu_backward": lambda s: q4.swiglu_fp8_backward(d_h, codes, scales, stream=s),
        "wgrad": lambda s: q4.grouped_wgrad_fp8(d_y, xc, xs, offsets, row_token=token, stream=s),
        "grouped_gemm": lambda s: q4.grouped_gemm_moe(x, offsets, token, *form, 256, stream=s),
        "quantize_nvfp4": lambda s: q4.quantize_nvfp4(x, scale_layout="mma", stream=s),
        "gemm_mxfp4": lambda s: q4.gemm_w4a4_mxfp4(a, b, H, stream=s),
        "gemm_mxfp4_fused": lambda s: q4.gemm_w4a4_mxfp4_fused(a, b, H, stream=s),
    }


NAMES = ["route", "route_backward", "sort", "sort_long", "dispatch", "dispatch_backward", "combine", "combine_backward",
         "checkpoint", "swiglu", "swiglu_backward", "wgrad", "grouped_gemm", "quantize_nvfp4", "gemm_mxfp4",
         "gemm_mxfp4_fused"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_with_work_pending_is_not_taken(lib, name):
    """The current stream lets go of blocks of every size that the call allocates
    while it is about to write them; the call on another stream keeps clear of them."""
    call = _calls(lib)[name]

    def tensors(r):
        return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]
    want = [t.clone() for t in tensors(call(None))]
    sizes = [t.numel() * t.element_size() for t in want] + [1 << n for n in range(9, 26)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)                          # the stream's own memory, so that nothing is allocated from the device below
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    held = {t.untyped_storage().data_ptr(): t.numel() for t in blocks}
    blocks[0].fill_(0)               # loads the kernels
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for t in blocks:
        t.fill_(0x7f)                # runs once the sleep is over
    del t, blocks
    got = tensors(call(s))
    busy = not torch.cuda.current_stream().query()
    for t in got:
        p = t.untyped_storage().data_ptr()
        assert not any(a < p + t.numel() * t.element_size() and p < a + n for a, n in held.items())
    torch.cuda.synchronize()
    assert busy                      # the call came back before the current stream's work was done
    for t, w in zip(got, want):
        assert torch.equal(t.contiguous().view(torch.uint8), w.view(torch.uint8))
    assert lib.sync_status() == 0


def test_results_outlive_their_readers(lib):
    """A result that the current stream still reads is not given to the next call
    on the stream that made it."""
    s = torch.cuda.Stream()
    x = torch.randn((512, 1024), device="cuda")
    y = -x
    codes, scales = lib.quantize_fp8_checkpoint(x)
    want = codes.clone()
    s.wait_stream(torch.cuda.current_stream())
    codes, scales = lib.quantize_fp8_checkpoint(x, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(BUSY)
    read = codes.clone()             # pending
    del codes, scales
    for _ in range(4):
        lib.quantize_fp8_checkpoint(y, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(read, want)
