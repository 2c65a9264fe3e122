"""A sandwich-normed expert block with microscaled 4-bit weights, put together
from the operators around the expert layer, and the same block around the
weight-only layer:

    h      = rms(x) * w_in                                   block_norm
    ids, w = top-k of softmax(h @ router)                    torch
    plan   = routes sorted by expert                         expert_sort
    a      = quantise(h, into expert order) @ W1[expert]     mx4_quantize, mx4_matmul
    y      = quantise(silu(gate) * up of a) @ W2[expert]     mx4_quantize, mx4_matmul
    o      = sum over a token's slots of w * y               combine
    r      = residual_scale * x + gate * rms(o) * w_out      block_norm (one pass with
    h_next = rms(r) * w_next                                 the next block's norm)

``train_step`` runs the block with 16-bit expert weights forward and backward
through dispatch, combine and block_norm.

    python examples/expert_block.py [--tokens 32] [--hidden 2048] [--inter 768] [--experts 128] [--top-k 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from weight_only_quantized_qmoe_gb300 import ops  # noqa: E402


class MX4ExpertBlock:
    """Weights of one block: drawn at random, the experts' quantised once."""

    def __init__(self, hidden, inter, experts, top_k, residual_scale=1.0, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0, shift=0.0):
            return (shift + scale * torch.randn(shape, generator=g, device="cuda")).to(dtype)

        self.hidden, self.inter, self.experts, self.top_k = hidden, inter, experts, top_k
        self.residual_scale = residual_scale
        self.router = normal(hidden, experts, scale=hidden ** -0.5)
        self.w_in, self.w_out, self.w_next = (normal(hidden, scale=0.1, shift=1.0) for _ in range(3))
        self.gate = normal(hidden, scale=0.1, shift=0.5)                       # of the block's output, per channel
        # [gate (inter rows) | up (inter rows)] and the way back
        self.w1 = ops.mx4_quantize(normal(experts, 2 * inter, hidden, scale=hidden ** -0.5))
        self.w2 = ops.mx4_quantize(normal(experts, hidden, inter, scale=inter ** -0.5))

    def route(self, h):
        top, ids = torch.topk(h @ self.router, self.top_k, dim=1)
        return ops.expert_sort(ids, self.experts), torch.softmax(top.float(), dim=1)

    def experts_forward(self, h, plan, weights):
        a = ops.mx4_matmul(ops.mx4_quantize(h, plan=plan), self.w1, plan=plan, out_dtype=h.dtype)
        y = ops.mx4_matmul(ops.mx4_quantize(a, activation="swiglu"), self.w2, plan=plan, out_dtype=h.dtype)
        return ops.combine(y, weights, plan)

    def forward(self, x):
        """(r, h_next) of x [T, hidden]."""
        _, h = ops.block_norm(x, w_pre=self.w_in)
        plan, weights = self.route(h)
        o = self.experts_forward(h, plan, weights)
        return ops.block_norm(x, o, gate=self.gate, w_post=self.w_out, w_pre=self.w_next, residual_scale=self.residual_scale)


def around_the_layer(block, layer, x):
    """The same block around a prepacked weight-only layer
    (:class:`weight_only_quantized_qmoe_gb300.QMoELayer`)."""
    _, h = ops.block_norm(x, w_pre=block.w_in)
    o = layer.forward(h, (h @ block.router).float())
    return ops.block_norm(x, o, gate=block.gate, w_post=block.w_out, w_pre=block.w_next, residual_scale=block.residual_scale)


def train_step(block, x, w1, w2, target):
    """One step's loss and gradients with 16-bit expert weights w1 [experts,
    hidden, inter], w2 [experts, inter, hidden] (leaves): (loss, gradients of x,
    w1, w2, the router, the norms' weights and the gate)."""
    leaves = [t.detach().requires_grad_() for t in (x, w1, w2, block.router, block.w_in, block.w_out, block.w_next, block.gate)]
    x, w1, w2, router, w_in, w_out, w_next, gate = leaves
    _, h = ops.block_norm(x, w_pre=w_in)
    top, ids = torch.topk(h @ router, block.top_k, dim=1)
    plan = ops.expert_sort(ids, block.experts)
    hs = ops.dispatch(h, plan)
    ends = plan.offsets.tolist()
    ys = [torch.nn.functional.silu(hs[b:e] @ w1[i]) @ w2[i] for i, (b, e) in enumerate(zip(ends, ends[1:]))]
    o = ops.combine(torch.cat(ys), torch.softmax(top.float(), dim=1), plan)
    r, h_next = ops.block_norm(x, o, gate=gate, w_post=w_out, w_pre=w_next, residual_scale=block.residual_scale)
    loss = ((h_next.float() - target.float()) ** 2).mean() + 1e-3 * (r.float() ** 2).mean()
    return loss.detach(), torch.autograd.grad(loss, leaves)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=768)
    ap.add_argument("--experts", type=int, default=128)
    ap.add_argument("--top-k", type=int, default=8)
    a = ap.parse_args()
    block = MX4ExpertBlock(a.hidden, a.inter, a.experts, a.top_k)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    for _ in range(3):
        r, h_next = block.forward(x)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        r, h_next = block.forward(x)
    end.record()
    torch.cuda.synchronize()
    if ops.poll_status():
        raise RuntimeError("a bounded wait ran out")
    print(f"{a.tokens} tokens, hidden {a.hidden}, inter {a.inter}, {a.experts} experts, top {a.top_k}: "
          f"{begin.elapsed_time(end) / 20 * 1e3:.1f} us a block, |r| {r.float().norm():.4g}, |h_next| {h_next.float().norm():.4g}")
    g = torch.Generator(device="cuda").manual_seed(1)
    w1, w2 = ((torch.randn(s, generator=g, device="cuda") * s[1] ** -0.5).to(torch.bfloat16)
              for s in ((a.experts, a.hidden, a.inter), (a.experts, a.inter, a.hidden)))
    loss, grads = train_step(block, x, w1, w2, torch.randn((a.tokens, a.hidden), device="cuda"))
    print(f"training step: loss {loss:.4f}, gradient norms " + ", ".join(f"{t.float().norm():.3g}" for t in grads))


if __name__ == "__main__":
    main()
