"""The routed-expert operators together: one layer's step, as the example runs it."""
import numpy as np
import pytest
import torch

from examples import moe_training_step as ex

pytestmark = pytest.mark.gpu


def test_loss_goes_down(lib):
    losses = ex.main(["--tokens", "512", "--hidden", "512", "--inner", "256", "--experts", "8", "--top-k", "2",
                      "--steps", "6"])
    assert np.all(np.isfinite(losses)) and losses[-1] < 0.9 * losses[0]


def test_gradients_against_autograd(lib):
    """The layer's gradients against autograd through the plain layer of the
    same quantized weights.  Bounds: every activation and gradient passes two
    NVFP4 quantizations (relative error of a value near 2^-3.5 each, of a sum
    of a hundred and more independent ones near 10%) and one E4M3 one (2^-4):
    relative Frobenius error 0.25 and a cosine of 0.97."""
    torch.manual_seed(1)
    T, H, I, E, k = 384, 512, 256, 8, 2
    layer = ex.MoeLayer(H, I, E, k)
    x = torch.randn((T, H), device="cuda").bfloat16()
    d_out = torch.randn((T, H), device="cuda").bfloat16()
    out, kept = layer.forward(x)
    got = layer.backward(d_out, kept)
    assert lib.sync_status() == 0

    xr = x.float().requires_grad_()
    router = layer.router.clone().requires_grad_()
    w1, w2 = layer.w1.master.clone().requires_grad_(), layer.w2.master.clone().requires_grad_()
    logits = xr @ router.t()
    value = torch.gather(logits, 1, kept["ids"].long())
    weights = torch.softmax(value, dim=1)
    ref = torch.zeros((T, H), device="cuda")
    for e in range(E):
        t, j = (kept["ids"] == e).nonzero(as_tuple=True)
        g, u = (xr[t] @ w1[e].t()).chunk(2, dim=1)
        ref = ref.index_add(0, t, weights[t, j].unsqueeze(1) * ((torch.nn.functional.silu(g) * u) @ w2[e].t()))
    want = torch.autograd.grad(ref, (xr, router, w1, w2), d_out.float())
    for a, b in zip((out,) + got, (ref.detach(),) + want):
        a, b = a.float().reshape(-1), b.reshape(-1)
        assert torch.linalg.norm(a - b) <= 0.25 * torch.linalg.norm(b)
        assert torch.dot(a, b) >= 0.97 * torch.linalg.norm(a) * torch.linalg.norm(b)
