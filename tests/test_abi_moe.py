"""Host-side argument checks of the routed-expert and checkpoint calls (they
return before any launch) and their workspace sizes."""
import pytest

FAKE = 0x10000  # never dereferenced: every call below returns first


@pytest.fixture(scope="module")
def clib():
    from int4_gemm_gb300 import build
    import int4_gemm_gb300 as q4
    build.build()
    return q4.load()


def test_route(clib):
    def fwd(p=FAKE, dt=0, T=4, E=8, ld=8, k=2, norm=0, ids=FAKE, w=FAKE):
        return clib.moe_route_topk(p, dt, T, E, ld, k, norm, ids, w, None)

    def bwd(p=FAKE, dt=0, T=4, E=8, ld=8, k=2, norm=0, ids=FAKE, dw=FAKE, d=FAKE):
        return clib.moe_route_topk_backward(p, dt, T, E, ld, k, norm, ids, dw, d, None)
    for f in (fwd, bwd):
        for bad in (dict(dt=3), dict(T=-1), dict(E=0), dict(ld=7), dict(k=0), dict(k=9), dict(norm=2), dict(p=None),
                    dict(p=FAKE + 2), dict(ids=None), dict(ids=FAKE + 2)):
            assert f(**bad) == -1, bad
        assert f(E=1025, ld=1025) == -2 and f(E=64, ld=64, k=33) == -2 and f(T=1 << 40) == -2
        assert f(T=0, p=None, ids=None) == 0
    assert fwd(w=None) == -1 and bwd(dw=None) == -1 and bwd(d=None) == -1 and bwd(dt=1, d=FAKE + 1) == -1


def test_sort(clib):
    def sort(ids=FAKE, T=4, k=2, E=8, off=FAKE, tok=FAKE, slot=FAKE, ws=FAKE, nb=1 << 20):
        return clib.moe_sort_tokens(ids, T, k, E, off, tok, slot, ws, nb, None)
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(ids=None), dict(off=None), dict(tok=None), dict(slot=None),
                dict(slot=FAKE + 1)):
        assert sort(**bad) == -1, bad
    assert sort(k=33) == -2 and sort(E=1025) == -2 and sort(T=1 << 30) == -2
    big = clib.q4_workspace_size(10, 1 << 20, 1024, 0)
    assert big > 0 and clib.q4_workspace_size(10, -1, 8, 0) == 0
    for ws, nb in ((None, big), (FAKE + 16, big), (FAKE, big - 1)):
        assert sort(T=1 << 17, k=8, E=1024, ws=ws, nb=nb) == -6


def test_rows(clib):
    def dispatch(x=FAKE, dt=1, T=4, H=8, ld=8, slot=FAKE, k=2, out=FAKE):
        return clib.moe_dispatch(x, dt, T, H, ld, slot, k, out, None)

    def back(x=FAKE, dt=1, T=4, H=8, ld=8, slot=FAKE, k=2, out=FAKE):
        return clib.moe_dispatch_backward(x, dt, T, H, ld, slot, k, out, None)

    def combine(x=FAKE, dt=1, T=4, H=8, ld=8, slot=FAKE, k=2, out=FAKE, w=FAKE):
        return clib.moe_combine(x, dt, T, H, ld, slot, w, k, out, None)

    def grad(x=FAKE, dt=1, T=4, H=8, ld=8, slot=FAKE, k=2, out=FAKE, rows=FAKE, ldr=8, w=FAKE, dw=FAKE):
        return clib.moe_combine_backward(x, dt, T, H, ld, rows, ldr, slot, w, k, out, dw, None)
    for f in (dispatch, back, combine, grad):
        for bad in (dict(dt=5), dict(T=-1), dict(H=-1), dict(k=0), dict(ld=7), dict(x=None), dict(x=FAKE + 1),
                    dict(slot=None), dict(slot=FAKE + 2), dict(out=None)):
            assert f(**bad) == -1, bad
        assert f(k=33) == -2 and f(T=1 << 30) == -2 and f(H=1 << 40, ld=1 << 40) == -2
        assert f(T=0, x=None, slot=None, out=None) == 0
    for f in (dispatch, back, combine):
        assert f(H=0, x=None, out=None) == 0
    assert combine(w=FAKE + 2) == -1
    for bad in (dict(rows=None), dict(ldr=7), dict(w=None), dict(dw=FAKE + 2)):
        assert grad(**bad) == -1, bad


def test_checkpoint(clib):
    def quant(x=FAKE, dt=1, rows=4, K=8, ld=8, codes=FAKE, scales=FAKE):
        return clib.quantize_fp8_checkpoint(x, dt, rows, K, ld, codes, scales, None)

    def fwd(x=FAKE, dt=1, rows=4, K=8, ld=16, codes=FAKE, scales=FAKE, h=FAKE):
        return clib.swiglu_fp8(x, dt, rows, K, ld, h, codes, scales, None)

    def bwd(x=FAKE, dt=1, rows=4, K=8, ld=8, codes=FAKE, scales=FAKE, d=FAKE):
        return clib.swiglu_fp8_backward(x, dt, rows, K, ld, codes, scales, d, None)
    for f in (quant, fwd, bwd):
        for bad in (dict(dt=-1), dict(rows=-1), dict(K=0), dict(ld=7), dict(x=None), dict(x=FAKE + 1),
                    dict(codes=None), dict(scales=None), dict(scales=FAKE + 2)):
            assert f(**bad) == -1, bad
        assert f(rows=1 << 40, K=1024, ld=2048) == -2
        assert f(rows=0, x=None, codes=None) == 0
    assert fwd(ld=15) == -1 and fwd(h=None) == -1 and bwd(d=None) == -1


def test_wgrad(clib):
    def wgrad(y=FAKE, R=64, N=16, ldy=16, codes=FAKE, scales=FAKE, T=64, K=32, tok=None, off=FAKE, E=2, w=FAKE, dt=0,
              acc=0, ws=FAKE, nb=1 << 30):
        return clib.grouped_wgrad_fp8(y, R, N, ldy, codes, scales, T, K, tok, off, E, w, dt, acc, ws, nb, None)
    for bad in (dict(R=-1), dict(N=-8), dict(K=-16), dict(T=-1), dict(E=-1), dict(ldy=8), dict(dt=2), dict(dt=1, acc=1),
                dict(w=None), dict(w=FAKE + 8), dict(T=63), dict(y=None), dict(y=FAKE + 8), dict(codes=None),
                dict(codes=FAKE + 8), dict(scales=None), dict(tok=FAKE + 2), dict(off=None), dict(T=0, tok=FAKE)):
        assert wgrad(**bad) == -1, bad
    for bad in (dict(N=12), dict(ldy=20), dict(K=40), dict(E=1025), dict(R=1 << 30, T=1 << 30)):
        assert wgrad(**bad) == -2, bad
    for none in (dict(E=0), dict(N=0, ldy=0), dict(K=0)):
        assert wgrad(w=None, **none) == 0, none
    need = clib.q4_workspace_size_wgrad(64, 16, 32, 2)
    assert need >= 64 * 32 * 2 and clib.q4_workspace_size_wgrad(-1, 16, 32, 2) == 0
    for ws, nb in ((None, need), (FAKE + 16, need), (FAKE, need - 1)):
        assert wgrad(ws=ws, nb=nb) == -6


def test_overlapping_memory(clib):
    """Outputs that share memory with an input, with one another or with the
    workspace (otherwise valid calls)."""
    far = [FAKE + (i << 24) for i in range(8)]

    def calls(x, y, z, u, v, ws):
        return [("route", clib.moe_route_topk(x, 0, 4, 8, 8, 2, 0, y, z, None)),
                ("route_backward", clib.moe_route_topk_backward(x, 0, 4, 8, 8, 2, 0, u, v, y, None)),
                ("sort", clib.moe_sort_tokens(x, 4, 2, 8, y, z, u, None, 0, None)),
                ("sort_long", clib.moe_sort_tokens(far[6], 1 << 15, 2, 8, y, far[5], far[7], x, 1 << 20, None)),
                ("checkpoint", clib.quantize_fp8_checkpoint(x, 1, 4, 8, 8, y, z, None)),
                ("swiglu", clib.swiglu_fp8(x, 1, 4, 8, 16, y, z, u, None)),
                ("swiglu_backward", clib.swiglu_fp8_backward(x, 1, 4, 8, 8, z, u, y, None)),
                ("dispatch", clib.moe_dispatch(x, 1, 4, 8, 8, z, 2, y, None)),
                ("combine", clib.moe_combine(x, 1, 4, 8, 8, z, u, 2, y, None)),
                ("combine_backward", clib.moe_combine_backward(x, 1, 4, 8, 8, z, 8, u, v, 2, y, far[7], None)),
                ("wgrad", clib.grouped_wgrad_fp8(x, 4, 8, 8, z, u, 4, 16, None, v, 1, y, 0, 0, ws, 1 << 20, None))]
    for name, status in calls(far[0], far[0] + 16, far[1], far[2], far[3], far[4]):
        assert status == -1, name
    # two outputs of one call
    assert clib.moe_route_topk(far[0], 0, 4, 8, 8, 2, 0, far[1], far[1] + 16, None) == -1
    assert clib.moe_sort_tokens(far[0], 4, 2, 8, far[1], far[2], far[2] + 4, None, 0, None) == -1
    assert clib.swiglu_fp8(far[0], 1, 4, 8, 16, far[1], far[2], far[2] + 60, None) == -1
    assert clib.quantize_fp8_checkpoint(far[0], 1, 4, 8, 8, far[1], far[1] + 28, None) == -1
    assert clib.moe_combine_backward(far[0], 1, 4, 8, 8, far[1], 8, far[2], far[3], 2, far[4], far[4] + 124, None) == -1
    # d_rows over rows: only the same matrix
    assert clib.moe_combine_backward(far[0], 1, 4, 8, 8, far[1], 16, far[2], far[3], 2, far[1], far[4], None) == -1
    assert clib.moe_combine_backward(far[0], 1, 4, 8, 8, far[1], 8, far[2], far[3], 2, far[1] + 16, far[4], None) == -1
    # the workspace over an input, over dW
    assert clib.grouped_wgrad_fp8(far[0], 4, 8, 8, far[1], far[2], 4, 16, None, far[3], 1, far[4], 0, 0, far[0], 1 << 20, None) == -1
    assert clib.grouped_wgrad_fp8(far[0], 4, 8, 8, far[1], far[2], 4, 16, None, far[3], 1, far[4], 0, 0, far[4], 1 << 20, None) == -1
