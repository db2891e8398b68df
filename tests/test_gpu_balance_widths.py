"""The balance loss where the experts are few or no multiple of eight."""
import numpy as np
import pytest
import torch

from oracle import norm as o

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,E", [(2048, 6), (2049, 6), (5000, 60), (80000, 6), (512, 60), (513, 60), (2048, 64), (2049, 64), (512, 1000), (513, 1000),
                                      (700, 1024), (512, 256), (513, 264)])
def test_balance_of_few_unaligned_experts(lib, tokens, E):
    g = torch.Generator("cuda").manual_seed(E)
    logits = torch.randn((tokens, E), device="cuda", generator=g)
    ids, _ = lib.moe_route_topk(logits, 2)
    loss, counts, mean = lib.moe_balance_loss(logits, ids)
    want, want_counts, want_mean = o.balance_loss(logits.cpu().numpy(), ids.cpu().numpy())
    assert np.array_equal(counts.cpu().numpy(), want_counts)
    # an exponential within 2^-20 of its value and fewer than 1024 additions in a row
    assert np.allclose(mean.cpu().numpy(), want_mean, rtol=2.0 ** -13, atol=0) and abs(loss.item() / want - 1) < 2.0 ** -12
