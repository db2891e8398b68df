"""The integer product in every form that a call can take: each width of tile with
the K range whole, in two and in four parts, and CTA pairs with several tiles each
and with every kind of last run.  Bit for bit, as in test_gpu_int8; which form a size
takes is checked in test_int8_plan."""
import pytest
import torch

from test_gpu_int8 import _operands, _want

pytestmark = pytest.mark.gpu

# (pair, tokens of a tile, K parts) on 152 SMs -> sizes; of two parts several, whose
# last group of tokens, round of groups and weight rows end in different places
SIZES = {
    (0, 16, 1): [(5, 30000, 272)],
    (0, 16, 2): [(1, 8192, 8192), (11, 7974, 3104), (16, 9000, 2640), (4, 4894, 2608)],
    (0, 16, 4): [(7, 1000, 4112)],
    (0, 32, 1): [(31, 20001, 528)],
    (0, 32, 2): [(56, 4742, 2800), (27, 8100, 6160), (1306, 1, 2672)],
    (0, 32, 4): [(29, 3500, 7184)],
    (0, 64, 1): [(60, 20001, 1040)],
    (0, 64, 2): [(505, 970, 4592), (64, 8192, 8192), (2504, 1, 4688)],
    (0, 64, 4): [(50, 3500, 8208)],
    (0, 128, 1): [(128, 16500, 2064)],
    (0, 128, 2): [(83, 7223, 7696), (128, 8193, 8192), (97, 8001, 7184), (5056, 1, 6848)],
    (0, 128, 4): [(100, 4100, 7168), (127, 3500, 8208)],
    # 1, 2, 3, 4, 5, 13 half runs of 512 columns, the last whole or not; weight rows
    # and tokens that are no multiple of 256; one tile and several per pair
    (1, 256, 1): [(5121, 9000, 80), (5121, 9000, 512), (4400, 4300, 1040), (4100, 4300, 1536), (3001, 9001, 1552), (2600, 6001, 1008),
                  (2305, 4700, 2064), (2162, 4659, 6368), (400, 8192, 1040), (500, 8000, 1552)],
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [s for sizes in SIZES.values() for s in sizes])
def test_product(lib, size, dtype):
    ops = _operands(sum(size), *size)
    C = lib.gemm_w8a8_int8(*ops, out_dtype=dtype)
    assert torch.equal(C, _want(*ops, dtype))
    assert lib.sync_status() == 0


def test_most_weight_rows(lib):
    """2^30 - 1 of them, the most that a call takes."""
    N, K = 2 ** 30 - 1, 16
    g = torch.Generator("cuda").manual_seed(8)
    qa = torch.randint(-128, 128, (1, K), dtype=torch.int8, device="cuda", generator=g)
    qb = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    parts = [slice(0, 1000), slice(N // 2, N // 2 + 1000), slice(N - 1000, N)]
    for at in parts:
        qb[at] = torch.randint(-128, 128, (1000, K), dtype=torch.int8, device="cuda", generator=g)
    sa, sb = torch.rand(1, device="cuda", generator=g), torch.ones(N, device="cuda")
    C = lib.gemm_w8a8_int8(qa, sa, qb, sb)
    for at in parts:
        assert torch.equal(C[:, at], _want(qa, sa, qb[at], sb[at], torch.bfloat16))
    assert int(torch.count_nonzero(C)) <= 3000 and lib.sync_status() == 0
