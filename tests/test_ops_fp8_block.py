"""The router, the 8-bit rows and products and their gradients together, as a
block uses them: the example's 8-bit block against a 64-bit evaluation of the
same steps, in a CUDA graph, with tokens that no expert takes, and its training
step against automatic differentiation in 64 bits.

Rounding: an E4M3 value is off by at most 2^-4 of itself.  Where both sides
quantise values that bf16 has rounded on one of them (2^-8), about one in eight
takes a neighbour, 2^-3 away at most: sqrt(1/8) / 8 = 4.5 % of the size of what is
quantised.  Two such steps forward: 6.5 %."""
import os
import sys

import numpy as np
import pytest
import torch

import ops_reference as ref
import ops_reference8 as ref8

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    import expert_block
    return expert_block


def weights(q):
    codes, scales = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    return [ref8.unpack(c, s, q.cols, True) for c, s in zip(codes, scales)]


@pytest.mark.parametrize("T,H,inter,E,k,groups,top", [(1, 256, 128, 4, 2, 1, 1), (37, 320, 96, 6, 3, 2, 1), (400, 512, 160, 16, 4, 4, 2)])
def test_block_against_64_bits(ex, T, H, inter, E, k, groups, top):
    block = ex.FP8ExpertBlock(H, inter, E, k, groups, top, residual_scale=0.8, seed=T)
    x = torch.randn((T, H), generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
    r, hn = block.forward(x)
    _, h = ex.ops.block_norm(x, w_pre=block.w_in)
    ids, w = block.choose(h)
    logits = (h @ block.router).float()
    want_ids, want_w = ref8.route(ref.f64(logits), k, "sigmoid", ref.f64(block.bias), groups, top, block.how["group_best"], True, 2.5)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    np.testing.assert_allclose(ref.f64(w), want_w, rtol=64 * 2.0 ** -24)
    X = ref.f64(x)
    H64 = ref8.quantize(ref.norm(X, None, None, None, ref.f64(block.w_in), 1.0, 1e-6)[1])[2]
    w1, w2 = weights(block.w1), weights(block.w2)
    o = np.zeros_like(X)
    for t in range(T):
        for j, e in enumerate(want_ids[t]):
            a = w1[e] @ H64[t]
            o[t] += want_w[t, j] * (w2[e] @ ref8.quantize(ref.glu("swiglu", a[:inter], a[inter:])[None])[2][0])
    R, HN, _ = ref.norm(X, o, ref.f64(block.gate), ref.f64(block.w_out), ref.f64(block.w_next), 0.8, 1e-6)
    for got, want in ((r, R), (hn, HN)):
        off = np.linalg.norm(ref.f64(got) - want) / np.linalg.norm(want)
        assert off <= 0.065, off
    assert ex.ops.poll_status() == 0


def test_block_in_a_graph(ex):
    block = ex.FP8ExpertBlock(512, 128, 8, 2, 2, 1)
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


def test_tokens_without_an_expert(ex):
    # a padded batch: the padding's logits are closed, it takes no row of any
    # expert, adds nothing and gets no gradient
    ops = ex.ops
    g = torch.Generator().manual_seed(2)
    logits = torch.randn((50, 8), generator=g).cuda()
    logits[30:] = -float("inf")
    leaf = logits.clone().requires_grad_()
    r = ops.expert_route(leaf, 3)
    assert (r.ids[30:] == -1).all() and (r.weights[30:] == 0).all()
    plan = ops.expert_sort(r.ids, 8)
    assert int(plan.offsets[-1]) == 90
    x = torch.randn((50, 96), generator=g).bfloat16()
    x[30:] = float("nan")      # what the padding holds reaches nothing
    x, w = x.cuda().requires_grad_(), (0.1 * torch.randn((8, 40, 96), generator=g)).cuda().requires_grad_()
    y = ops.fp8_linear(ops.dispatch(x, plan), w, plan=plan)
    out = ops.combine(y, r.weights, plan)
    assert (y[90:] == 0).all() and (out[30:] == 0).all()
    dl, dx, dw = torch.autograd.grad(out, (leaf, x, w), torch.ones_like(out))
    few = logits[:30].clone().requires_grad_()
    r2 = ops.expert_route(few, 3)
    plan2 = ops.expert_sort(r2.ids, 8)
    x2 = x.detach()[:30].clone().requires_grad_()
    out2 = ops.combine(ops.fp8_linear(ops.dispatch(x2, plan2), w, plan=plan2), r2.weights, plan2)
    dl2, dx2, dw2 = torch.autograd.grad(out2, (few, x2, w), torch.ones_like(out2))
    assert torch.equal(out[:30], out2) and torch.equal(dl[:30], dl2) and torch.equal(dx[:30], dx2) and torch.equal(dw, dw2)
    assert (dl[30:] == 0).all() and (dx[30:] == 0).all()


def test_training_step_against_64_bits(ex):
    """Besides the two quantisations forward, the gradients of two products'
    rows are quantised (2^-4 of each value at most, a third of that on average),
    which the 64-bit evaluation leaves out: 2 % each.  All together 10 %."""
    T, H, inter, E, k = 90, 192, 64, 6, 2
    block = ex.FP8ExpertBlock(H, inter, E, k, 3, 2, residual_scale=0.7)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    target = torch.randn((T, H), generator=g, device="cuda")
    w1 = torch.randn((E, 2 * inter, H), generator=g, device="cuda") * H ** -0.5
    w2 = torch.randn((E, H, inter), generator=g, device="cuda") * inter ** -0.5
    loss, grads = ex.fp8_train_step(block, x, w1, w2, target)
    assert ex.ops.poll_status() == 0
    ids = block.choose(ex.ops.block_norm(x, w_pre=block.w_in)[1]).ids.long()

    leaves = [t.double().detach().requires_grad_() for t in
              (x, w1, w2, block.router, block.w_in, block.w_out, block.w_next, block.gate)]
    X, W1, W2, router, w_in, w_out, w_next, gate = leaves

    def rms(v):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)

    def quantized(v, square=False):   # its gradient passes unchanged
        d = v.detach()
        q = torch.stack([torch.from_numpy(ref8.quantize(m.cpu().numpy(), True)[2]) for m in d]) if square else torch.from_numpy(ref8.quantize(d.cpu().numpy())[2])
        return v + (q.cuda() - d)

    h = rms(X) * w_in
    s = torch.sigmoid(h @ router).gather(1, ids)
    w = 2.5 * s / s.sum(1, keepdim=True)
    W1q, W2q, o = quantized(W1, True), quantized(W2, True), torch.zeros_like(X)
    for j in range(k):
        a = torch.einsum("th,tih->ti", quantized(h), W1q[ids[:, j]])
        act = torch.nn.functional.silu(a[:, :inter]) * a[:, inter:]
        o = o + w[:, j:j + 1] * torch.einsum("ti,thi->th", quantized(act), W2q[ids[:, j]])
    r = 0.7 * X + gate * (rms(o) * w_out)
    hn = rms(r) * w_next
    want = ((hn - target.double()) ** 2).mean() + 1e-3 * (r ** 2).mean()
    assert abs(float(loss) - float(want.detach())) <= 0.02 * abs(float(want.detach()))
    for got, exact in zip(grads, torch.autograd.grad(want, leaves)):
        off = float((got.double() - exact).norm()) / float(exact.norm())
        assert off <= 0.10, off


def test_a_plan_that_changes_in_between_is_refused(ex):
    ops = ex.ops
    g = torch.Generator().manual_seed(4)
    plan = ops.expert_sort(torch.randint(0, 3, (20, 2), generator=g).cuda(), 3)
    x, w = torch.randn((40, 64), generator=g).bfloat16().cuda().requires_grad_(), torch.randn((3, 32, 64), generator=g).cuda().requires_grad_()
    y = ops.fp8_linear(x, w, plan=plan)
    plan.offsets.add_(0)
    with pytest.raises(RuntimeError):
        y.backward(torch.ones_like(y))
    y = ops.fp8_linear(x, w, plan=ops.expert_sort(torch.zeros((20, 2), dtype=torch.int32, device="cuda"), 3))
    dx, = torch.autograd.grad(y, x, torch.ones_like(y), create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()      # a second derivative
