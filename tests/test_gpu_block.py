"""The norm, the router with its balance loss and the experts together: a block of
the residual stream, as the example runs it."""
import numpy as np
import pytest
import torch

from examples import moe_training_step as ex

pytestmark = pytest.mark.gpu


def test_example_runs(lib):
    losses = ex.main(["--tokens", "256", "--hidden", "256", "--inner", "256", "--experts", "8", "--top-k", "2",
                      "--steps", "3", "--block"])
    assert len(losses) == 3 and np.all(np.isfinite(losses))


def test_gradients_against_autograd(lib):
    """Against autograd through the plain block.  The branch passes two NVFP4
    quantizations and one E4M3 one both ways, as the layer by itself does: relative
    Frobenius error r = 0.25.  |a - b| <= r |b| puts a inside a ball around b whose
    tangent from the origin has the cosine sqrt(1 - r^2) = 0.968, so that is what the
    cosine can be held to; 0.97 would ask for r = 0.243.  That much is the experts'
    four bits.  The norm's own gradient is held to 32-bit sums, from the d_y that it
    was given."""
    torch.manual_seed(2)
    T, H, I, E, k, coeff = 384, 512, 256, 8, 2, 0.5
    block = ex.MoeBlock(H, I, E, k, balance=coeff)
    block.norm += 0.2 * torch.randn(H, device="cuda")
    x, stream, d_out, d_stream = (torch.randn((T, H), device="cuda").bfloat16() for _ in range(4))
    out, after, kept = block.forward(x, stream)
    got = block.backward(d_out, d_stream, kept)
    d_y = block.layer.backward(d_out, kept)[0].double()
    assert lib.sync_status() == 0

    xhat = after.double() * kept["rstd"].double().reshape(-1, 1)
    # a sum of T terms in 32 bits, each with the roundings of two products and of rstd
    bound = (T + 4) * 2.0 ** -24 * (d_y * xhat).abs().sum(0)
    assert torch.all((got[1].double() - (d_y * xhat).sum(0)).abs() <= bound)

    xr = x.float().requires_grad_()
    norm, router = block.norm.clone().requires_grad_(), block.layer.router.clone().requires_grad_()
    w1, w2 = block.layer.w1.master.clone().requires_grad_(), block.layer.w2.master.clone().requires_grad_()
    h = xr + stream.float()
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + 1e-6) * norm
    logits = y @ router.t()
    ids = kept["ids"].long()
    weights = torch.softmax(torch.gather(logits, 1, ids), dim=1)
    ref = torch.zeros((T, H), device="cuda")
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        g, u = (y[t] @ w1[e].t()).chunk(2, dim=1)
        ref = ref.index_add(0, t, weights[t, j].unsqueeze(1) * ((torch.nn.functional.silu(g) * u) @ w2[e].t()))
    load = torch.bincount(ids.reshape(-1), minlength=E).float() * E / (T * k)
    balance = coeff * (load * torch.softmax(logits, dim=1).mean(dim=0)).sum()
    # the balance loss from rounded tokens: 2^-8 of each logit's terms, far below 1%
    assert abs(float(kept["balance_loss"]) / float(balance.detach()) - 1) < 0.01
    total = (ref * d_out.float()).sum() + (h * d_stream.float()).sum() + balance
    want = torch.autograd.grad(total, (xr, norm, router, w1, w2))
    for a, b in zip((out, after) + got, (ref.detach(), h.detach()) + want):
        a, b = a.float().reshape(-1), b.reshape(-1)
        assert torch.linalg.norm(a - b) <= 0.25 * torch.linalg.norm(b)
        assert torch.dot(a, b) >= (1 - 0.25 ** 2) ** 0.5 * torch.linalg.norm(a) * torch.linalg.norm(b)


def test_balance_gradient_reaches_the_router(lib):
    """d_logits of route and balance loss together, against the two by themselves."""
    torch.manual_seed(3)
    logits = torch.randn((200, 24), device="cuda")
    ids, weights = lib.moe_route_topk(logits, 4)
    d_weights, one = torch.randn_like(weights), torch.ones(1, device="cuda")
    _, counts, _ = lib.moe_balance_loss(logits, ids, 0.3)
    route = lib.moe_route_topk_backward(logits, ids, d_weights)
    balance = lib.moe_balance_loss_backward(logits, counts, 4, one, 0.3)
    both = lib.moe_balance_loss_backward(logits, counts, 4, one, 0.3, out=route.clone(), accumulate=True)
    # one rounding more or less of the sum
    assert torch.all((both - (route + balance)).abs() <= 2.0 ** -23 * (route.abs() + balance.abs()))
