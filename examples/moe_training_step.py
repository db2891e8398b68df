"""One training step of a routed-expert layer with quantized weights, on one GPU.

The experts' products run on NVFP4 weights (grouped_gemm_moe); the master
weights get straight-through gradients.  Everything between and behind the
products is this library's:

  forward   logits -> moe_route_topk -> moe_sort_tokens
            tokens -> grouped_gemm_moe (gate and up) -> swiglu_fp8
                   -> grouped_gemm_moe (down) -> moe_combine
            kept for the backward pass, in 8 bits: the tokens, gate and up, h
  backward  moe_combine_backward -> d_y, d_weights
            grouped_wgrad_fp8(d_y, h) -> dW2;  grouped_gemm_moe(d_y, W2^T) -> d_h
            swiglu_fp8_backward -> d_gate_up
            grouped_wgrad_fp8(d_gate_up, tokens) -> dW1
            grouped_gemm_moe(d_gate_up, W1^T) -> moe_dispatch_backward -> d_x
            moe_route_topk_backward -> d_logits -> d_router, d_x

``python examples/moe_training_step.py`` takes a few steps of gradient descent
towards a random target and prints the loss, the time of a step and the bytes
kept for the backward pass.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_gemm_gb300 as q4  # noqa: E402


class QuantizedExperts:
    """E float32 master weights [E, N, K] and their NVFP4 forms, as stored and transposed."""

    def __init__(self, E, N, K, device, std):
        self.master = torch.randn((E, N, K), device=device) * std
        self.refresh()

    def refresh(self):
        self.forward = self._quantize(self.master)
        self.transposed = self._quantize(self.master.transpose(1, 2))

    @staticmethod
    def _quantize(w):
        parts = [q4.quantize_nvfp4(e.contiguous(), scale_layout="mma") for e in w]
        return (torch.stack([c for c, _, _ in parts]), torch.cat([s for _, s, _ in parts]),
                torch.cat([g for _, _, g in parts]))

    @staticmethod
    def apply(form, x, offsets, row_token, N):
        return q4.grouped_gemm_moe(x, offsets, row_token, *form, N)


class MoeLayer:
    def __init__(self, hidden, inner, experts, top_k, device="cuda"):
        self.hidden, self.inner, self.E, self.k = hidden, inner, experts, top_k
        self.router = torch.randn((experts, hidden), device=device) * hidden ** -0.5
        self.w1 = QuantizedExperts(experts, 2 * inner, hidden, device, hidden ** -0.5)
        self.w2 = QuantizedExperts(experts, hidden, inner, device, inner ** -0.5)

    def forward(self, x, allowed=None):
        """x bf16 [T, hidden] -> (out bf16 [T, hidden], what backward needs).
        allowed: bool [T, experts], the experts that a token may go to."""
        logits = x.float() @ self.router.t()
        if allowed is not None:
            logits = logits.masked_fill(~allowed, -float("inf"))
        ids, weights = q4.moe_route_topk(logits, self.k)
        offsets, row_token, slot_row = q4.moe_sort_tokens(ids, self.E)
        rows = torch.arange(row_token.numel(), dtype=torch.int32, device=x.device)
        gate_up = QuantizedExperts.apply(self.w1.forward, x, offsets, row_token, 2 * self.inner)
        h, gu_codes, gu_scales = q4.swiglu_fp8(gate_up)
        y = QuantizedExperts.apply(self.w2.forward, h, offsets, rows, self.hidden)
        out = q4.moe_combine(y, slot_row, weights)
        kept = dict(x=x, logits=logits, ids=ids, weights=weights, offsets=offsets, row_token=row_token, rows=rows,
                    slot_row=slot_row, y=y, gate_up=(gu_codes, gu_scales), tokens=q4.quantize_fp8_checkpoint(x),
                    h=q4.quantize_fp8_checkpoint(h))
        return out, kept

    def backward(self, d_out, kept):
        """-> (d_x bf16, d_router, dW1, dW2), the weights' gradients float32."""
        offsets, rows = kept["offsets"], kept["rows"]
        d_y, d_weights = q4.moe_combine_backward(d_out, kept["y"], kept["slot_row"], kept["weights"])
        dw2 = q4.grouped_wgrad_fp8(d_y, *kept["h"], offsets)
        d_h = QuantizedExperts.apply(self.w2.transposed, d_y, offsets, rows, self.inner)
        d_gate_up = q4.swiglu_fp8_backward(d_h, *kept["gate_up"])
        dw1 = q4.grouped_wgrad_fp8(d_gate_up, *kept["tokens"], offsets, row_token=kept["row_token"])
        d_rows = QuantizedExperts.apply(self.w1.transposed, d_gate_up, offsets, rows, self.hidden)
        d_x = q4.moe_dispatch_backward(d_rows, kept["slot_row"])
        d_logits = q4.moe_route_topk_backward(kept["logits"], kept["ids"], d_weights)
        d_x = (d_x.float() + d_logits @ self.router).to(d_x.dtype)
        return d_x, d_logits.t() @ kept["x"].float(), dw1, dw2

    def step(self, x, target, lr):
        """One step of gradient descent on the square error per token; returns
        the mean square error of an element and what was kept."""
        out, kept = self.forward(x)
        error = out.float() - target.float()
        d_out = (error * (2.0 / error.shape[0])).to(torch.bfloat16)
        _, d_router, dw1, dw2 = self.backward(d_out, kept)
        self.router -= lr * d_router
        for w, d in ((self.w1, dw1), (self.w2, dw2)):
            w.master -= lr * d
            w.refresh()
        return error.square().mean(), kept


def bytes_kept(kept):
    eight = sum(t.numel() * t.element_size() for name in ("tokens", "gate_up", "h") for t in kept[name])
    sixteen = sum(2 * kept[name][0].numel() for name in ("tokens", "gate_up", "h"))
    return eight, sixteen


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=512)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--lr", type=float, default=0.1)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    layer = MoeLayer(a.hidden, a.inner, a.experts, a.top_k)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    target = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16) * 0.1
    losses = []
    for _ in range(a.steps):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        loss, kept = layer.step(x, target, a.lr)
        end.record()
        losses.append(float(loss))
        print(f"loss {losses[-1]:.5f}  step {begin.elapsed_time(end):.2f} ms")
    if q4.sync_status() != 0:
        raise RuntimeError("a kernel reported an error")
    eight, sixteen = bytes_kept(kept)
    print(f"kept for the backward pass: {eight / 1e6:.1f} MB in 8 bits ({sixteen / 1e6:.1f} MB in 16)")
    return losses


if __name__ == "__main__":
    main()
