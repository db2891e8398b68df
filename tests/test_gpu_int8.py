"""8-bit integers on the GPU: the quantizer bit for bit, the product bit for bit
(exact integer sums, then the documented roundings)."""
import numpy as np
import pytest
import torch

from oracle import norm

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def _rows(seed, rows, K):
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, K)).astype(np.float32)
    x[:, K // 2] *= 20.0
    if rows > 2:
        x[1] = 0.0
        x[2] *= np.float32(1e-4)
    if rows > 3:  # ties: multiples of s / 2 where s = 1
        x[3] = r.integers(-254, 255, K) / 2.0
        x[3, 0] = -127.0
    return x


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 1), (4, 7), (5, 64), (33, 128), (9, 1000), (4, 7168), (200, 2064), (6, 8192), (5, 20000),
                                   (4, 65537)])
def test_quantizer(lib, shape, dtype):
    x = torch.from_numpy(_rows(shape[0] + shape[1], *shape)).to(dtype)
    codes, scales = lib.quantize_int8(x.cuda())
    want, ws = norm.quantize_int8(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), ws) and np.array_equal(codes.cpu().numpy(), want)
    assert lib.sync_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pitch,offset", [(8, 0), (8, 3), (5, 0)])
def test_quantizer_pitched(lib, dtype, pitch, offset):
    x = torch.from_numpy(_rows(3, 21, 272)).to(dtype)
    big = torch.full((21 * (272 + pitch) + offset,), float("nan"), dtype=dtype)
    big.as_strided(x.shape, (272 + pitch, 1), offset).copy_(x)
    codes, scales = lib.quantize_int8(big.cuda().as_strided(x.shape, (272 + pitch, 1), offset))
    want, ws = norm.quantize_int8(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), ws) and np.array_equal(codes.cpu().numpy(), want)
    assert lib.sync_status() == 0


def test_quantizer_near_ties(lib):
    """x / s next to every half-integer: the float below, on and above it, for
    scales that are no powers of two."""
    half = (np.arange(-126, 127) + 0.5).astype(np.float32)
    rows = []
    for s in (0.37, 1.0, 0.0123, 3.3e5):
        s = np.float32(s) * np.float32(127) / np.float32(127)
        x = (half * s).astype(np.float32)
        rows.append(np.concatenate([[np.float32(127) * s], np.nextafter(x, -np.inf, dtype=np.float32), x,
                                    np.nextafter(x, np.inf, dtype=np.float32)]))
    x = np.stack(rows).astype(np.float32)
    codes, scales = lib.quantize_int8(torch.from_numpy(x).cuda())
    want, ws = norm.quantize_int8(x)
    assert np.array_equal(scales.cpu().numpy(), ws) and np.array_equal(codes.cpu().numpy(), want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_quantizer_reports_non_finite(lib, bad):
    x = torch.ones((3, 40), device="cuda")
    x[1, 39] = bad
    lib.quantize_int8(x)
    assert lib.sync_status() == -5 and lib.sync_status() == 0


def _operands(seed, M, N, K, lo=-128):
    g = torch.Generator("cuda").manual_seed(seed)
    qa = torch.randint(lo, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    qb = torch.randint(lo, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    sa = torch.rand(M, device="cuda", generator=g) * 0.1 + 1e-3
    sb = torch.rand(N, device="cuda", generator=g) * 0.01 + 1e-4
    return qa, sa, qb, sb


def _want(qa, sa, qb, sb, dtype):
    # float64 sums of 8-bit products are exact; the rest in float32, step by step
    acc = (qa.double() @ qb.double().t()).float()
    return ((acc * sa.unsqueeze(1)) * sb).to(dtype)


# tokens on both sides of every tile and form; N and K off them
SIZES = [(1, 1, 16), (1, 256, 4096), (2, 8192, 1024), (3, 70, 48), (5, 129, 1040), (8, 1000, 2064), (9, 512, 8192), (16, 4100, 7168),
         (17, 300, 160), (31, 640, 1024), (33, 2049, 3216), (64, 1024, 2048), (65, 256, 512), (100, 4100, 7168), (127, 130, 1008),
         (128, 128, 1024), (129, 257, 1056), (200, 2048, 4096), (255, 1030, 2080), (256, 256, 128), (257, 513, 4112),
         (400, 8192, 1024), (513, 64, 2048), (640, 7168, 2048), (1001, 2056, 2064), (1500, 3, 1024), (2048, 1552, 512),
         (2300, 4160, 1072)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
def test_product(lib, size, dtype):
    ops = _operands(sum(size), *size)
    C = lib.gemm_w8a8_int8(*ops, out_dtype=dtype)
    assert torch.equal(C, _want(*ops, dtype))
    assert lib.sync_status() == 0


@pytest.mark.parametrize("M", [1, 7, 40, 130, 300])
@pytest.mark.parametrize("K", [1024, 1040, 16384, 131056])
def test_product_of_largest_values(lib, M, K):
    """Sums up to 2^14 K: beyond 2^24 from K = 1024 on, 2^31 - 2^18 at the largest K."""
    N = 140
    qa = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    qb = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    qb[1::2] = 127
    qb[2, ::3] = 1
    qa[M // 2, 1::2] = 127
    one = torch.ones(max(M, N), device="cuda")
    C = lib.gemm_w8a8_int8(qa, one[:M], qb, one[:N], out_dtype=torch.float32)
    assert torch.equal(C, _want(qa, one[:M], qb, one[:N], torch.float32))
    # odd sums near 2^24 show any lost unit
    qa.random_(100, 128, generator=torch.Generator("cuda").manual_seed(1))
    qb.random_(100, 128, generator=torch.Generator("cuda").manual_seed(2))
    C = lib.gemm_w8a8_int8(qa, one[:M], qb, one[:N], out_dtype=torch.float32)
    assert torch.equal(C, _want(qa, one[:M], qb, one[:N], torch.float32))
    assert lib.sync_status() == 0


@pytest.mark.parametrize("M", [4, 50, 1000])
def test_quantized_product_of_a_norm(lib, M):
    """Norm, INT8 product, quantizer, product again: against the same steps in
    float64 on the codes that each call returned."""
    H, N = 1024, 1600
    g = torch.Generator("cuda").manual_seed(M)
    x, r = (torch.randn((M, H), device="cuda", generator=g).bfloat16() for _ in range(2))
    w1, s1 = lib.quantize_int8(torch.randn((N, H), device="cuda", generator=g) * 0.02)
    w2, s2 = lib.quantize_int8(torch.randn((H, N), device="cuda", generator=g) * 0.02)
    codes, scales, _, h, _ = lib.rms_norm_int8(x, residual=r)
    up = lib.gemm_w8a8_int8(codes, scales, w1, s1)
    assert torch.equal(up, _want(codes, scales, w1, s1, torch.bfloat16))
    q, s = lib.quantize_int8(up)
    want, ws = norm.quantize_int8(up.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), want) and np.array_equal(s.cpu().numpy(), ws)
    down = lib.gemm_w8a8_int8(q, s, w2, s2)
    assert torch.equal(down, _want(q, s, w2, s2, torch.bfloat16))
    # and near the unquantized layer: INT8 steps of both operands, twice
    y, _, _ = norm.rms_norm(x.double().cpu().numpy(), None, r.double().cpu().numpy())
    ref = (torch.from_numpy(y).cuda() @ (w1.double() * s1.double().unsqueeze(1)).t()) @ (w2.double() * s2.double().unsqueeze(1)).t()
    assert float((down.double() - ref).norm() / ref.norm()) < 0.03
    assert lib.sync_status() == 0


def test_norms_fp8_form_feeds_the_fp8_product(lib):
    M, H, N = 70, 512, 256
    g = torch.Generator("cuda").manual_seed(9)
    x = torch.randn((M, H), device="cuda", generator=g).bfloat16()
    qw, sw = lib.quantize_fp8_blockwise(torch.randn((N, H), device="cuda", generator=g) * 0.02, 128)
    codes, scales, _, _, _ = lib.rms_norm_fp8(x)
    C = lib.gemm_fp8_blockwise(codes, scales, qw, sw, out_dtype=torch.float32)
    a = codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, 1)
    b = qw.view(torch.float8_e4m3fn).double() * sw.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    ref = a @ b.t()
    assert float((C.double() - ref).norm() / ref.norm()) < 2e-3
    assert lib.sync_status() == 0


def test_product_in_a_graph(lib):
    """Captured once, replayed on new operands; two graphs alive at once."""
    graphs = []
    for M in (3, 300):
        ops = _operands(M, M, 520, 1040)
        out = torch.empty((M, 520), device="cuda")
        lib.gemm_w8a8_int8(*ops, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.gemm_w8a8_int8(*ops, out=out)
        graphs.append((graph, ops, out))
    for turn in range(2):
        for graph, ops, out in graphs:
            for t, new in zip(ops, _operands(turn + 50, ops[0].shape[0], 520, 1040)):
                t.copy_(new)
            out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, ops, out in graphs:
            assert torch.equal(out, _want(*ops, torch.float32))
    assert lib.sync_status() == 0


def test_refusals(lib):
    qa, sa, qb, sb = _operands(1, 4, 32, 64)
    for call in (lambda: lib.gemm_w8a8_int8(qa.cpu(), sa, qb, sb), lambda: lib.gemm_w8a8_int8(qa, sa, qb[:, :48], sb),
                 lambda: lib.gemm_w8a8_int8(qa.view(torch.uint8), sa, qb, sb), lambda: lib.gemm_w8a8_int8(qa, sa[:3], qb, sb),
                 lambda: lib.gemm_w8a8_int8(qa, sa, qb, sb.double()), lambda: lib.gemm_w8a8_int8(qa[0], sa, qb, sb),
                 lambda: lib.gemm_w8a8_int8(qa, sa, qb, sb, out_dtype=torch.float16),
                 lambda: lib.gemm_w8a8_int8(qa, sa, qb, sb, out=torch.empty((4, 31), device="cuda")),
                 lambda: lib.quantize_int8(qa), lambda: lib.quantize_int8(sa)):
        with pytest.raises(ValueError):
            call()
    flat = torch.zeros(8192, dtype=torch.int8, device="cuda")
    for call in (lambda: lib.gemm_w8a8_int8(qa[:, :40].contiguous(), sa, qb[:, :40].contiguous(), sb),
                 lambda: lib.gemm_w8a8_int8(flat[8:264].view(4, 64), sa, qb, sb),
                 lambda: lib.gemm_w8a8_int8(torch.zeros((1, 131072), dtype=torch.int8, device="cuda"), sa[:1],
                                            torch.zeros((1, 131072), dtype=torch.int8, device="cuda"), sb[:1]),
                 lambda: lib.gemm_w8a8_int8(flat[:256].view(4, 64), sa, qb, sb, out=flat[128:640].view(torch.float32).view(4, 32))):
        with pytest.raises(lib.Q4Error):
            call()
    assert lib.gemm_w8a8_int8(qa[:0], sa[:0], qb, sb).shape == (0, 32)
    assert lib.gemm_w8a8_int8(qa, sa, qb[:0], sb[:0]).shape == (4, 0) and lib.sync_status() == 0
