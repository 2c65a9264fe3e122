"""The operators together: the example block against a 64-bit evaluation of the
same steps, around the weight-only layer, in a CUDA graph, and its training
step against automatic differentiation in 64 bits."""
import os
import sys

import numpy as np
import pytest
import torch

import ops_reference as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    import expert_block
    return expert_block


def plain_block(block, x, ids, weights):
    """(r, h_next) in 64 bits for the routes the block took."""
    X = ref.f64(x)
    _, h, _ = ref.norm(X, None, None, None, ref.f64(block.w_in), 1.0, 1e-6)
    h = ref.quantize(h)[2]
    w1 = [ref.unpack(block.w1.codes[e].cpu().numpy(), block.w1.scales[e].cpu().numpy(), block.w1.cols) for e in range(block.experts)]
    w2 = [ref.unpack(block.w2.codes[e].cpu().numpy(), block.w2.scales[e].cpu().numpy(), block.w2.cols) for e in range(block.experts)]
    o = np.zeros_like(X)
    for t in range(X.shape[0]):
        for j, e in enumerate(ids[t]):
            a = w1[e] @ h[t]
            act = ref.quantize(ref.glu("swiglu", a[:block.inter], a[block.inter:])[None])[2][0]
            o[t] += weights[t, j] * (w2[e] @ act)
    r, hn, _ = ref.norm(X, o, ref.f64(block.gate), ref.f64(block.w_out), ref.f64(block.w_next), block.residual_scale, 1e-6)
    return r, hn


@pytest.mark.parametrize("T,H,inter,E,k", [(1, 256, 128, 4, 2), (37, 320, 96, 6, 3), (130, 256, 160, 3, 1)])
def test_block_against_64_bits(ex, T, H, inter, E, k):
    """Both quantisations see values that bf16 has rounded (2^-8): about one in
    twenty of them then takes a neighbouring E2M1 value, a third off, which
    moves the branch by sqrt(1/20) / 3 = 7 % of its size at most (two such
    steps: 10 %), and less the sum r."""
    block = ex.MX4ExpertBlock(H, inter, E, k, residual_scale=0.8, seed=T)
    x = torch.randn((T, H), generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
    r, hn = block.forward(x)
    _, h = ex.ops.block_norm(x, w_pre=block.w_in)
    top, ids = torch.topk(h @ block.router, k, dim=1)
    weights = torch.softmax(top.float(), dim=1)
    R, HN = plain_block(block, x, ids.cpu().numpy(), ref.f64(weights))
    for got, want in ((r, R), (hn, HN)):
        off = np.linalg.norm(ref.f64(got) - want) / np.linalg.norm(want)
        assert off <= 0.10, off
    assert ex.ops.poll_status() == 0


def test_block_in_a_graph(ex):
    block = ex.MX4ExpertBlock(512, 128, 8, 2)
    x = torch.randn((24, 512), device="cuda").to(torch.bfloat16)
    block.forward(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, hn = block.forward(x)
    x.copy_(torch.randn((24, 512), device="cuda"))
    graph.replay()
    want = block.forward(x)
    assert torch.equal(r, want[0]) and torch.equal(hn, want[1])


def test_around_the_weight_only_layer(ex):
    import weight_only_quantized_qmoe_gb300 as q
    from qmoe_inputs import CONFIGS, make_inputs
    cfg = CONFIGS["tiny"].with_(H=256, I=128, E=8, dtype="bf16", B=32, T=9)
    layer = q.QMoELayer.from_config(cfg)
    q.load_inputs(layer, make_inputs(cfg))
    block = ex.MX4ExpertBlock(256, 128, 8, 2, residual_scale=0.5)
    x = torch.randn((9, 256), device="cuda").to(torch.bfloat16)
    r, hn = ex.around_the_layer(block, layer, x)
    _, h = ex.ops.block_norm(x, w_pre=block.w_in)
    o = layer.forward(h, (h @ block.router).float())
    R, HN, mag = ref.norm(ref.f64(x), ref.f64(o), ref.f64(block.gate), ref.f64(block.w_out), ref.f64(block.w_next), 0.5, 1e-6)
    ref.within(r, R, mag, "bf16", 64 * 2.0 ** -24)
    assert np.linalg.norm(ref.f64(hn) - HN) <= 2.0 ** -8 * np.linalg.norm(HN)
    layer.close()


def test_training_step_against_64_bits(ex):
    """In fp32, so that the routes and every value agree with the 64-bit
    evaluation to fp32 rounding: a chain of some ten sums of up to 256 terms,
    256 2^-24 each, 2e-4 of a gradient's size."""
    T, H, inter, E, k = 45, 192, 64, 5, 2
    block = ex.MX4ExpertBlock(H, inter, E, k, residual_scale=0.7, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, target = (torch.randn((T, H), generator=g, device="cuda") for _ in range(2))
    w1 = torch.randn((E, H, inter), generator=g, device="cuda") * H ** -0.5
    w2 = torch.randn((E, inter, H), generator=g, device="cuda") * inter ** -0.5
    loss, grads = ex.train_step(block, x, w1, w2, target)

    leaves = [t.double().detach().requires_grad_() for t in
              (x, w1, w2, block.router, block.w_in, block.w_out, block.w_next, block.gate)]
    X, W1, W2, router, w_in, w_out, w_next, gate = leaves

    def rms(v):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)

    h = rms(X) * w_in
    top, ids = torch.topk(h @ router, k, dim=1)
    w = torch.softmax(top, dim=1)
    o = torch.zeros_like(X)
    for j in range(k):
        a = torch.nn.functional.silu(torch.einsum("th,thi->ti", h, W1[ids[:, j]]))
        o = o + w[:, j:j + 1] * torch.einsum("ti,tih->th", a, W2[ids[:, j]])
    r = 0.7 * X + gate * (rms(o) * w_out)
    hn = rms(r) * w_next
    want = ((hn - target.double()) ** 2).mean() + 1e-3 * (r ** 2).mean()
    assert abs(float(loss) - float(want.detach())) <= 1e-5 * abs(float(want.detach()))
    for got, exact in zip(grads, torch.autograd.grad(want, leaves)):
        assert float((got.double() - exact).norm()) <= 2e-4 * float(exact.norm())
