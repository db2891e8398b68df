"""The norm, the 8-bit integers and the balance loss on a stream that is given, in
CUDA graphs, and beyond 32-bit offsets."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BUSY = 200_000_000  # cycles that the current stream is kept busy for


def _calls(q4):
    """name -> (call(stream), its inputs)."""
    g = torch.Generator("cuda").manual_seed(5)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)
    x, r, dy = (normal(640, 1024).bfloat16() for _ in range(3))
    few = normal(3, 1024).bfloat16()
    w, (qw, sw) = normal(1024), q4.quantize_int8(normal(300, 1024))
    _, h, rstd = q4.rms_norm(x, w, residual=r)
    qa, sa = q4.quantize_int8(x)
    qf, sf = q4.quantize_int8(few)
    logits, long_logits = normal(640, 32), normal(70000, 32)
    ids, _ = q4.moe_route_topk(logits, 4)
    long_ids, _ = q4.moe_route_topk(long_logits, 4)
    _, counts, _ = q4.moe_balance_loss(logits, ids)
    one = torch.ones(1, device="cuda")
    return {
        "norm": (lambda s: q4.rms_norm(x, w, residual=r, stream=s), (x, w, r)),
        "norm_few": (lambda s: q4.rms_norm(few, w, stream=s), (few, w)),
        "norm_fp8": (lambda s: q4.rms_norm_fp8(x, w, residual=r, need_y=True, stream=s), (x, w, r)),
        "norm_int8": (lambda s: q4.rms_norm_int8(x, w, stream=s), (x, w)),
        "norm_backward": (lambda s: q4.rms_norm_backward(dy, h, rstd, w, d_h=r, stream=s), (dy, h, rstd, w, r)),
        "quantize": (lambda s: q4.quantize_int8(x, stream=s), (x,)),
        "product": (lambda s: q4.gemm_w8a8_int8(qa, sa, qw, sw, stream=s), (qa, sa, qw, sw)),
        "product_few": (lambda s: q4.gemm_w8a8_int8(qf, sf, qw, sw, stream=s), (qf, sf, qw, sw)),
        "balance": (lambda s: q4.moe_balance_loss(logits, ids, 0.1, stream=s), (logits, ids)),
        "balance_long": (lambda s: q4.moe_balance_loss(long_logits, long_ids, 0.1, stream=s), (long_logits, long_ids)),
        "balance_backward": (lambda s: q4.moe_balance_loss_backward(logits, counts, 4, one, 0.1, stream=s), (logits, counts, one)),
    }


NAMES = ["norm", "norm_few", "norm_fp8", "norm_int8", "norm_backward", "quantize", "product", "product_few", "balance",
         "balance_long", "balance_backward"]


def _tensors(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_memory_with_work_pending_is_not_taken(lib, name):
    """The current stream lets go of blocks of every size that the call allocates
    while it is about to write them; the call on another stream keeps clear of them."""
    call, _ = _calls(lib)[name]
    want = [t.clone() for t in _tensors(call(None))]
    sizes = [t.numel() * t.element_size() for t in want] + [1 << n for n in range(9, 26)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    held = {t.untyped_storage().data_ptr(): t.numel() for t in blocks}
    blocks[0].fill_(0)
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for t in blocks:
        t.fill_(0x7f)
    del t, blocks
    got = _tensors(call(s))
    busy = not torch.cuda.current_stream().query()
    for t in got:
        p = t.untyped_storage().data_ptr()
        assert not any(a < p + t.numel() * t.element_size() and p < a + n for a, n in held.items())
    torch.cuda.synchronize()
    assert busy
    for t, w in zip(got, want):
        assert torch.equal(t.contiguous().view(torch.uint8), w.view(torch.uint8))
    assert lib.sync_status() == 0


def test_graphs(lib):
    """All of them captured, each into a graph of its own that shares nothing with
    the others; replayed on new inputs and compared with calls outside."""
    calls = _calls(lib)
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for call, _ in calls.values():
            call(None)
    torch.cuda.current_stream().wait_stream(side)
    for name, (call, inputs) in calls.items():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = _tensors(call(None))
        graphs.append((name, graph, call, out))
    moved = set()
    for _, inputs in calls.values():  # other values, in place
        for t in inputs:
            if t.data_ptr() not in moved and t.is_floating_point() and t.numel() > 1:
                moved.add(t.data_ptr())
                t.copy_(t.flip(0) * 0.5)
    for turn in range(2):
        for _, graph, _, out in graphs:
            for t in out:
                t.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for name, _, call, out in graphs:
            for a, b in zip(out, _tensors(call(None))):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
    assert lib.sync_status() == 0


def test_two_graphs_with_one_workspace(lib):
    """Captured with the same workspace and replayed in turn: a call leaves nothing
    in it that the next one needs."""
    g = torch.Generator("cuda").manual_seed(9)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)
    sizes = ((700, 1024), (5000, 512))
    n = max(lib.lib().q4_workspace_size(lib.OP_RMS_NORM_BACKWARD, r, 0, H) for r, H in sizes)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    logits = [normal(40000, 64), normal(9000, 256)]
    ids = [lib.moe_route_topk(t, 4)[0] for t in logits]
    m = max(lib.lib().q4_workspace_size(lib.OP_MOE_BALANCE_LOSS, *t.shape, 0) for t in logits)
    assert m
    ws_balance = torch.full((m,), 0xff, dtype=torch.uint8, device="cuda")
    calls = []
    for r, H in sizes:
        d_y, h, w = normal(r, H), normal(r, H), normal(H)
        _, _, rstd = lib.rms_norm(h)
        calls.append(lambda ws, a=(d_y, h, rstd, w): lib.rms_norm_backward(*a, ws=ws))
    for t, i in zip(logits, ids):
        calls.append(lambda ws, a=(t, i): lib.moe_balance_loss(*a, ws=ws))
    want = [[t.clone() for t in call(None)] for call in calls]
    graphs = []
    for k, call in enumerate(calls):
        shared = ws if k < 2 else ws_balance
        call(shared)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, call(shared)))
    for order in ((0, 1, 2, 3), (3, 2, 1, 0), (1, 1, 0, 3, 3, 2)):
        for k in order:
            for t in graphs[k][1]:
                t.zero_()
            graphs[k][0].replay()
            for t, u in zip(graphs[k][1], want[k]):
                assert torch.equal(t, u)
    assert lib.sync_status() == 0


def test_two_streams_at_once(lib):
    """The same call on two streams at the same time, with outputs and workspaces of
    their own."""
    calls = _calls(lib)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for name, (call, _) in calls.items():
        want = [t.clone() for t in _tensors(call(None))]
        for s in (a, b):
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            first, second = _tensors(call(a)), _tensors(call(b))
            torch.cuda.synchronize()
            for t, u, w in zip(first, second, want):
                assert torch.equal(t.view(torch.uint8), w.view(torch.uint8)), name
                assert torch.equal(u.view(torch.uint8), w.view(torch.uint8)), name
    assert lib.sync_status() == 0


def test_norm_beyond_32_bit_offsets(lib):
    """More than 2^31 elements: the last rows are those of a small call.  Few rows and
    many are summed in different orders.  No term of a row's sum goes through more
    than 128 additions (64 in its thread, 5 in its warp, 32 across warps), so two sums
    of squares differ by 2 * 128 * 2^-24 at most, and their roots by half of that: r.
    Results of fewer bits may then fall to two sides of a tie: a whole step."""
    rows, H, r = 270000, 8192, 128 * 2.0 ** -24
    x = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((64, H), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    x[-64:] = tail
    y, h, rstd = lib.rms_norm(x, residual=x)
    wy, wh, wr = lib.rms_norm(tail, residual=tail)

    def near(a, b, step, least=0.0):
        a, b = a.double(), b.double()
        return bool(torch.all((a - b).abs() <= step * b.abs() + least))
    assert torch.equal(h[-64:], wh) and near(rstd[-64:], wr, r) and near(y[-64:], wy, 2.0 ** -7)
    assert not y[:-64].any()
    del y
    codes, scales, _, _, _ = lib.rms_norm_fp8(h)
    wc, ws, _, _, _ = lib.rms_norm_fp8(wh)

    def value(c, s):
        return c.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, dim=1)
    # the largest magnitude's root, its division and rounding: 4 roundings more
    assert near(scales[-64:], ws, r + 4 * 2.0 ** -24)
    assert near(value(codes[-64:], scales[-64:]), value(wc, ws), 2.0 ** -3 + 2 * r, 2.0 ** -9 * float(ws.max()))
    del codes, scales
    # d_y that is not h's multiple, which would leave nothing of d_x
    x[-64:] = tail.flip(1)
    d_x, d_w = lib.rms_norm_backward(x, h, rstd)
    wd, ww = lib.rms_norm_backward(x[-64:].contiguous(), wh, wr)
    # d_x = r (g - h c): r and c in other orders, both terms with the errors of their factors
    size = float(wr.max()) * (tail.abs().max().double() * 2 + wh.abs().max().double())
    assert near(d_x[-64:], wd, 2.0 ** -7, 8 * r * float(size)) and wd.abs().max() > 1 and not d_x[:-64].any()
    # 64 terms in any order, zeros beside them
    terms = (x[-64:].double() * wh.double() * wr.double().reshape(-1, 1)).abs().sum(0)
    assert torch.all((d_w - ww).double().abs() <= (r + 2 * 68 * 2.0 ** -24) * terms)
    del d_x
    q, s = lib.quantize_int8(h)
    wq, wsq = lib.quantize_int8(wh)
    assert torch.equal(q[-64:], wq) and torch.equal(s[-64:], wsq) and lib.sync_status() == 0


def test_product_beyond_32_bit_offsets(lib):
    """More than 2^31 outputs, then more than 2^31 weights."""
    g = torch.Generator("cuda").manual_seed(2)
    qa = torch.randint(-128, 128, (70000, 64), dtype=torch.int8, device="cuda", generator=g)
    qb = torch.randint(-128, 128, (32768, 64), dtype=torch.int8, device="cuda", generator=g)
    sa, sb = torch.rand(70000, device="cuda", generator=g), torch.rand(32768, device="cuda", generator=g)

    def want(qa, sa, qb, sb):
        acc = (qa.double() @ qb.double().t()).float()
        return ((acc * sa.unsqueeze(1)) * sb).bfloat16()
    C = lib.gemm_w8a8_int8(qa, sa, qb, sb)
    assert torch.equal(C[-300:], want(qa[-300:], sa[-300:], qb, sb)) and torch.equal(C[:, -40:], want(qa, sa, qb[-40:], sb[-40:]))
    del C
    qb = torch.randint(-128, 128, (270000, 8192), dtype=torch.int8, device="cuda", generator=g)
    sb = torch.rand(270000, device="cuda", generator=g)
    for M in (5, 300):
        qa = torch.randint(-128, 128, (M, 8192), dtype=torch.int8, device="cuda", generator=g)
        C = lib.gemm_w8a8_int8(qa, sa[:M].contiguous(), qb, sb)
        assert torch.equal(C[:, -500:], want(qa, sa[:M], qb[-500:], sb[-500:]))
        assert torch.equal(C[:, :500], want(qa, sa[:M], qb[:500], sb[:500]))
    assert lib.sync_status() == 0


def test_balance_beyond_32_bit_offsets(lib):
    T, E = 2200000, 1024
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    logits[-1, 5] = 8.0
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    ids[-1] = 5
    loss, counts, mean = lib.moe_balance_loss(logits, ids)
    assert int(counts[0]) == T - 1 and int(counts[5]) == 1 and int(counts[E]) == T
    # E^2 / T sum of counts / E: every token puts 1 / E on each expert
    assert abs(float(loss) - 1.0) < 1e-4 and abs(float(mean.sum()) - 1.0) < 1e-4
    d = lib.moe_balance_loss_backward(logits, counts, 1, torch.full((1,), float(T), device="cuda"))
    p = torch.softmax(logits[-1:].float(), dim=1)[0]
    f = counts[:E].float() * E / T
    want = p * (f - (p * f).sum())
    assert torch.all((d[-1].float() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4) and lib.sync_status() == 0
