"""Host-side argument checks of the norm, the 8-bit integers and the balance loss
(they return before any launch), and their workspace sizes."""
import pytest

FAKE = 0x10000  # never dereferenced: every call below returns first
FAR = [FAKE + (i << 24) for i in range(9)]


@pytest.fixture(scope="module")
def clib():
    from int4_gemm_gb300 import build
    import int4_gemm_gb300 as q4
    build.build()
    return q4.load()


def test_norm(clib):
    def plain(x=FAR[0], dt=1, rows=4, H=64, ldx=64, r=None, ldr=0, w=FAR[2], wd=1, eps=1e-6, codes=None, scales=None, y=FAR[5],
              h=None, rstd=FAR[7]):
        return clib.rms_norm(x, dt, rows, H, ldx, r, ldr, w, wd, eps, y, h, rstd, None)

    def eight(name):
        def f(x=FAR[0], dt=1, rows=4, H=64, ldx=64, r=None, ldr=0, w=FAR[2], wd=1, eps=1e-6, codes=FAR[3], scales=FAR[4], y=None,
              h=None, rstd=None):
            return getattr(clib, name)(x, dt, rows, H, ldx, r, ldr, w, wd, eps, codes, scales, y, h, rstd, None)
        return f
    fp8, int8 = eight("rms_norm_fp8"), eight("rms_norm_int8")
    for f in (plain, fp8, int8):
        for bad in (dict(dt=3), dict(rows=-1), dict(H=0), dict(ldx=63), dict(x=None), dict(x=FAR[0] + 1), dict(w=FAR[2] + 1),
                    dict(wd=2), dict(wd=0, w=FAR[2] + 2), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                    dict(eps=float("inf")), dict(r=FAR[1], ldr=63), dict(r=FAR[1] + 1, ldr=64), dict(h=FAR[6] + 1),
                    dict(y=FAR[5] + 1), dict(rstd=FAR[7] + 2)):
            assert f(**bad) == -1, bad
        assert f(H=32769, ldx=32769) == -2 and f(rows=1 << 40) == -2
        assert f(rows=0, x=None) == 0
        # outputs over an input or one another
        for bad in (dict(y=FAR[0]), dict(h=FAR[0]), dict(rstd=FAR[0] + 64), dict(y=FAR[5], h=FAR[5] + 128), dict(y=FAR[2]),
                    dict(r=FAR[1], ldr=64, h=FAR[1] + 128), dict(r=FAR[1], ldr=80, h=FAR[1]), dict(r=FAR[1], ldr=64, y=FAR[1])):
            assert f(**bad) == -1, bad
    assert plain(y=None) == -1
    for f in (fp8, int8):
        for bad in (dict(codes=None), dict(scales=None), dict(scales=FAR[4] + 2), dict(codes=FAR[0]), dict(scales=FAR[3]),
                    dict(codes=FAR[2] + 16), dict(r=FAR[1], ldr=64, codes=FAR[1] + 511)):
            assert f(**bad) == -1, bad


def test_norm_backward(clib):
    def back(dy=FAR[0], dt=1, rows=4, H=64, ldy=64, h=FAR[1], ldh=64, rstd=FAR[2], w=FAR[3], wd=1, dh=None, ldd=0, dx=FAR[5],
             dw=FAR[6], ws=FAR[7], nb=1 << 20):
        return clib.rms_norm_backward(dy, dt, rows, H, ldy, h, ldh, rstd, w, wd, dh, ldd, dx, dw, ws, nb, None)
    for bad in (dict(dt=-1), dict(rows=-1), dict(H=0), dict(ldy=63), dict(ldh=63), dict(dh=FAR[4], ldd=63), dict(dy=None),
                dict(h=None), dict(rstd=None), dict(dx=None), dict(dy=FAR[0] + 1), dict(rstd=FAR[2] + 2), dict(w=FAR[3] + 1),
                dict(wd=2), dict(dw=FAR[6] + 2), dict(dh=FAR[4] + 1, ldd=64), dict(dx=FAR[0]), dict(dx=FAR[1]),
                dict(dw=FAR[3]), dict(dw=FAR[5] + 4), dict(dh=FAR[4], ldd=64, dx=FAR[4] + 16), dict(dh=FAR[4], ldd=72, dx=FAR[4]),
                dict(ws=FAR[5]), dict(ws=FAR[0])):
        assert back(**bad) == -1, bad
    assert back(H=32769, ldy=32769, ldh=32769) == -2 and back(rows=1 << 40) == -2
    assert back(rows=0, dw=None) == 0
    need = clib.q4_workspace_size(13, 4, 0, 64)
    assert need >= 64 * 4 and clib.q4_workspace_size(13, -1, 0, 64) == 0 and clib.q4_workspace_size(13, 4, 0, 40000) == 0
    for ws, nb in ((None, need), (FAR[7] + 16, need), (FAR[7], need - 1)):
        assert back(ws=ws, nb=nb) == -6


def test_int8(clib):
    def quant(x=FAR[0], dt=1, rows=4, K=64, ld=64, codes=FAR[1], scales=FAR[2]):
        return clib.quantize_int8(x, dt, rows, K, ld, codes, scales, None)
    for bad in (dict(dt=3), dict(rows=-1), dict(K=0), dict(ld=63), dict(x=None), dict(x=FAR[0] + 1), dict(codes=None),
                dict(scales=None), dict(scales=FAR[2] + 1), dict(codes=FAR[0] + 100), dict(scales=FAR[1] + 4)):
        assert quant(**bad) == -1, bad
    assert quant(rows=1 << 40) == -2 and quant(K=1 << 30, ld=1 << 30) == -2 and quant(rows=0, x=None) == 0

    def gemm(qa=FAR[0], sa=FAR[1], qb=FAR[2], sb=FAR[3], M=4, N=8, K=64, C=FAR[4], dt=1, ws=None, nb=0):
        return clib.gemm_w8a8_int8(qa, sa, qb, sb, M, N, K, C, dt, ws, nb, None)
    for bad in (dict(M=-1), dict(N=-1), dict(K=0), dict(dt=2), dict(qa=None), dict(qb=None), dict(sa=None), dict(sb=None),
                dict(C=None), dict(qa=FAR[0] + 8), dict(qb=FAR[2] + 8), dict(sa=FAR[1] + 2), dict(C=FAR[4] + 8), dict(C=FAR[0]),
                dict(C=FAR[3])):
        assert gemm(**bad) == -1, bad
    for bad in (dict(K=40), dict(K=131072), dict(M=1 << 40), dict(N=1 << 40), dict(M=1 << 29, N=1 << 29)):
        assert gemm(**bad) == -2, bad
    assert gemm(M=0, qa=None) == 0 and gemm(N=0, C=None) == 0


def test_balance(clib):
    def fwd(x=FAR[0], dt=0, T=4, E=8, ld=8, ids=FAR[1], k=2, coeff=0.5, loss=FAR[2], counts=FAR[3], mean=FAR[4], ws=FAR[5],
            nb=1 << 20):
        return clib.moe_balance_loss(x, dt, T, E, ld, ids, k, coeff, loss, counts, mean, ws, nb, None)

    def bwd(x=FAR[0], dt=0, T=4, E=8, ld=8, counts=FAR[1], k=2, d=FAR[2], coeff=0.5, acc=0, out=FAR[3]):
        return clib.moe_balance_loss_backward(x, dt, T, E, ld, counts, k, d, coeff, acc, out, None)
    for f in (fwd, bwd):
        for bad in (dict(dt=3), dict(T=-1), dict(E=0), dict(ld=7), dict(k=0), dict(k=9), dict(x=None), dict(x=FAR[0] + 2),
                    dict(counts=None), dict(coeff=float("nan")), dict(coeff=float("inf"))):
            assert f(**bad) == -1, bad
        assert f(E=1025, ld=1025) == -2 and f(E=64, ld=64, k=33) == -2 and f(T=1 << 40) == -2
    for bad in (dict(ids=None), dict(loss=None), dict(mean=None), dict(loss=FAR[0]), dict(counts=FAR[1] + 4),
                dict(mean=FAR[3] + 32)):
        assert fwd(**bad) == -1, bad
    far = dict(T=1 << 20, x=FAR[8], ids=FAR[8] + (1 << 28))
    for bad in (dict(ws=FAR[8]), dict(ws=FAR[8] + (1 << 28)), dict(ws=FAR[3])):
        assert fwd(**far, **bad) == -1, bad
    need = clib.q4_workspace_size(14, 1 << 20, 8, 0)
    assert need > 0 and clib.q4_workspace_size(14, 4, 1025, 0) == 0 and clib.q4_workspace_size(14, -4, 8, 0) == 0
    for ws, nb in ((None, need), (FAR[5] + 16, need), (FAR[5], need - 1)):
        assert fwd(T=1 << 20, x=FAR[8], ids=FAR[8] + (1 << 28), ws=ws, nb=nb) == -6
    for bad in (dict(d=None), dict(out=None), dict(out=FAR[0] + 16), dict(out=FAR[2]), dict(out=FAR[1])):
        assert bwd(**bad) == -1, bad
    assert bwd(T=0, x=None) == 0
