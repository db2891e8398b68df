"""Probabilities of the balance loss at every distance from the largest logit.

A single token's mean is its probability p = e^-d / Z, d = top - x, nothing added to
it but zeros.  With u = 2^-24:
 * e^-d is taken as 2^z, z = RN(RN(x - top) * RN(log2 e)): the roundings of the
   difference and the product are u each, the constant is off by less than u / 4, so
   z is off by 2.25 u |z| and the result by 2.25 u d (|z| ln 2 = d); 2^z itself is
   within 2^-22: e(d) = 2.25 u d + 4 u.
 * Z: the sum of p e(d) over the experts, where the sum of p d is the entropy less ln
   Z, at most ln E < 7: 2.25 u 7 + 4 u.  Positive terms, at most 32 one after another
   in a lane and 5 levels of pairs: 37 u.
 * 1 / Z: 2 ulp, 4 u.  The product and the division by one token: 2 u.
In all (2.25 d + 67) u.  At the distances of test_gpu_balance, 25 where p matters,
that is 124 u < 2^-17, the bound that it counts with.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offset", [0.0, 37.3, -1000.7])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E", [5, 8, 33, 60, 64, 256, 257, 512, 1000, 1024])
def test_probabilities(lib, E, dtype, offset):
    r = np.random.default_rng(E)
    x = offset - r.permutation(np.linspace(0.0, 80.0, E) ** 1.5 / 80.0 ** 0.5)
    logits = torch.from_numpy(x).to(dtype).reshape(1, E).cuda()
    ids = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    _, _, mean = lib.moe_balance_loss(logits, ids)
    v = logits.double().cpu().numpy()[0]
    d = v.max() - v
    p = np.exp(-d) / np.exp(-d).sum()
    off = np.abs(mean.double().cpu().numpy() - p)
    assert np.all(off <= (2.25 * d + 67) * 2.0 ** -24 * p), float((off / p / (2.25 * d + 67)).max() * 2 ** 24)
    assert lib.sync_status() == 0
