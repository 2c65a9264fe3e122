"""The gradient of the experts' weights and the 8-bit linear layer, against the
plain 64-bit forms.

A product of two 16-bit values is exact in fp32; a sum of R of them, in any
order and with every addition truncated instead of rounded, is off by at most R
2^-23 times the sum of their magnitudes, and its result rounded once."""
import numpy as np
import pytest
import torch

import ops_reference as ref
import ops_reference8 as ref8
from test_ops_routes import DT, routes

pytestmark = pytest.mark.gpu
HALF = ("bf16", "f16")


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    from weight_only_quantized_qmoe_gb300 import ops as o
    return o


def normal(g, *shape, dtype="bf16", scale=1.0):
    return (scale * torch.randn(shape, generator=g)).to(DT[dtype]).cuda()


# (R, N, K): one row, one column, tails, tiles without a neighbour, many rows
# shared by a cluster, many tiles
DENSE = [(1, 1, 1), (1, 64, 128), (15, 16, 8), (16, 256, 128), (17, 257, 129), (63, 100, 300), (64, 40, 40), (65, 8, 1000), (200, 513, 31),
         (1000, 130, 70), (5000, 96, 264), (300, 2880, 1111), (129, 2048, 4096)]


@pytest.mark.parametrize("R,N,K", DENSE)
@pytest.mark.parametrize("dtype", HALF)
def test_dense(ops, R, N, K, dtype):
    g = torch.Generator().manual_seed(R + N + K)
    dy, x = normal(g, R, N, dtype=dtype), normal(g, R, K, dtype=dtype)
    want, mag = ref8.weight_grad(ref.f64(dy), ref.f64(x), [0, R])
    for out in DT:
        got = ops.weight_grad(dy, x, out_dtype=DT[out])
        assert ops.poll_status() == 0
        ref.within(got, want[0], mag[0], out, R * 2.0 ** -23)
        assert torch.equal(ops.weight_grad(dy, x, out_dtype=DT[out]), got)
    assert ops.weight_grad(dy, x).dtype == DT[dtype]


# A sum in the tensor core is cut off towards zero: in one piece of 12800 rows it
# would be some 1.5e-5 off.  32-bit results are summed in pieces of 640 rows: off
# by some 8e-7 each, and the rounded sum of 20 pieces (20 2^-24) less than that.
@pytest.mark.parametrize("N,K", [(96, 130), (1100, 1500), (300, 264)])
@pytest.mark.parametrize("R", [640, 641, 1290, 12800])
@pytest.mark.parametrize("dtype", HALF)
def test_long_sums_keep_their_precision(ops, N, K, R, dtype):
    g = torch.Generator(device="cuda").manual_seed(R + N)
    dy, x = (torch.randn((R, n), generator=g, device="cuda").to(DT[dtype]) for n in (N, K))
    want = dy.double().T @ x.double()
    got = ops.weight_grad(dy, x, out_dtype=torch.float32)
    assert float((got.double() - want).norm()) <= 2e-6 * float(want.norm())
    # with experts: a short one before, a long one, one without rows
    if R > 700:
        plan = ops.expert_sort(torch.where(torch.arange(R, device="cuda") < 37, 0, 1).int().unsqueeze(1), 3)
        grouped = ops.weight_grad(dy, x, plan=plan, out_dtype=torch.float32)
        for e, rows in enumerate((slice(0, 37), slice(37, R), slice(0, 0))):
            want = dy[rows].double().T @ x[rows].double()
            assert float((grouped[e].double() - want).norm()) <= 2e-6 * float(want.norm())


# (T, E, k, N, K, drop)
GROUPED = [(1, 4, 1, 64, 64, 0.0), (32, 128, 8, 96, 256, 0.0), (50, 3, 2, 200, 160, 0.2), (700, 4, 2, 300, 288, 0.1),
           (33, 1024, 3, 40, 64, 0.0), (9, 2, 1, 128, 512, 1.0), (2000, 5, 2, 64, 64, 0.05), (301, 7, 3, 129, 77, 0.0),
           # many tiles: pairs of CTAs, with rows of every remainder of 64, no rows, odd widths
           (300, 12, 3, 600, 700, 0.0), (500, 9, 2, 1000, 1111, 0.1), (1500, 40, 4, 264, 384, 0.0), (7, 3, 1, 4096, 2048, 0.0)]


@pytest.mark.parametrize("T,E,k,N,K,drop", GROUPED)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32")])
def test_grouped(ops, T, E, k, N, K, drop, dtype, out):
    ids = routes(np.random.default_rng(T + E), T, E, k, drop, skew=3.0)
    plan = ops.expert_sort(torch.from_numpy(ids).cuda(), E)
    g = torch.Generator().manual_seed(N + K)
    dy, x = normal(g, T * k, N, dtype=dtype, scale=0.1), normal(g, T * k, K, dtype=dtype)
    offsets = ref.sort(ids, E)[2]
    # rows no route owns are not used
    dy[offsets[-1]:], x[offsets[-1]:] = float("nan"), float("inf")
    got = ops.weight_grad(dy, x, plan=plan, out_dtype=DT[out])
    assert ops.poll_status() == 0
    want, mag = ref8.weight_grad(ref.f64(dy), ref.f64(x), offsets)
    ref.within(got, want, mag, out, T * k * 2.0 ** -23)
    assert torch.equal(ops.weight_grad(dy, x, plan=plan, out_dtype=DT[out]), got)


@pytest.mark.parametrize("N,K", [(140, 200), (2000, 1500)])
def test_a_nan_stays_with_its_expert(ops, N, K):
    # rows of 3, 18, 64 and 5: tails beside rows that hold NaN
    ends = [0, 3, 21, 85, 90]
    ids = torch.repeat_interleave(torch.arange(4), torch.tensor([3, 18, 64, 5])).int().unsqueeze(1).cuda()
    plan = ops.expert_sort(ids, 4)
    g = torch.Generator().manual_seed(3)
    dy, x = normal(g, 90, N), normal(g, 90, K)
    clean = ops.weight_grad(dy, x, plan=plan, out_dtype=torch.float32)
    for e in range(4):
        for t, bad in ((dy, float("nan")), (x, float("inf"))):
            keep = t[ends[e]:ends[e + 1]].clone()
            t[ends[e]:ends[e + 1]] = bad
            got = ops.weight_grad(dy, x, plan=plan, out_dtype=torch.float32)
            others = torch.arange(4) != e
            assert torch.equal(got[others], clean[others]) and not torch.isfinite(got[e]).any()
            t[ends[e]:ends[e + 1]] = keep


def test_strides_streams_and_graphs(ops):
    g = torch.Generator().manual_seed(5)
    base, other = normal(g, 150, 400), normal(g, 150, 300)
    for dy in (base[:, 3:203], base[:, 8:72], base[:100].t()[:150, :64].contiguous(), base[:, :1], base[:1, :40].expand(150, 40), base.t()[:150]):
        for x in (other, other[:, 1:], other[:, 16:80], other[:, 5:6]):
            want, mag = ref8.weight_grad(ref.f64(dy), ref.f64(x), [0, 150])
            ref.within(ops.weight_grad(dy, x, out_dtype=torch.float32), want[0], mag[0], "f32", 150 * 2.0 ** -23)
    for every in (base[::2], base[::2, 1:]):
        want, mag = ref8.weight_grad(ref.f64(every), ref.f64(other[:75]), [0, 75])
        ref.within(ops.weight_grad(every, other[:75]), want[0], mag[0], "bf16", 75 * 2.0 ** -23)
    want = ops.weight_grad(base, other)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.weight_grad(base, other, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, odd = ops.weight_grad(base, other), ops.weight_grad(base[:, 1:], other[:, 1:])
    base.copy_(normal(g, 150, 400))
    graph.replay()
    assert torch.equal(out, ops.weight_grad(base, other)) and torch.equal(odd, ops.weight_grad(base[:, 1:], other[:, 1:]))


def test_no_rows(ops):
    e = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    assert (ops.weight_grad(e, e[:, :5]) == 0).all()
    plan = ops.expert_sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 3)
    d = ops.weight_grad(e, e, plan=plan)
    assert d.shape == (3, 24, 24) and (d == 0).all()


@pytest.mark.parametrize("R,N,K", [(300, 64, 64), (5000, 64, 64), (300, 4000, 4000)])
def test_a_wait_that_runs_out_is_reported(ops, R, N, K):
    # host-injected: the first copy's barrier is armed and its copy never issued
    from weight_only_quantized_qmoe_gb300 import binding
    g = torch.Generator().manual_seed(4)
    dy, x = normal(g, R, N), normal(g, R, K)
    want = ops.weight_grad(dy, x)
    assert ops.poll_status() == 0
    assert binding.qmoe_op_set_wait_limit(2000) == 0 and binding.qmoe_op_debug_inject_stall(1) == 0
    try:
        ops.weight_grad(dy, x)
        assert ops.poll_status() == binding.QMOE_ERR_TIMEOUT
    finally:
        binding.qmoe_op_debug_inject_stall(0)
        binding.qmoe_op_set_wait_limit(0)
    assert torch.equal(ops.weight_grad(dy, x), want) and ops.poll_status() == 0


# --- the linear layer ------------------------------------------------------------------
def linear(x, w, dy, offsets):
    """(y, dx, dw) with the magnitudes of their terms, from the definition."""
    xq, dyq = ref8.quantize(x)[2], ref8.quantize(dy)[2]
    y, ym = np.zeros(dy.shape), np.zeros(dy.shape)
    dx, dxm = np.zeros(x.shape), np.zeros(x.shape)
    for e, (b, c) in enumerate(zip(offsets, offsets[1:])):
        W = ref8.quantize(w[e], True)[2]
        y[b:c], ym[b:c] = xq[b:c] @ W.T, np.abs(xq[b:c]) @ np.abs(W.T)
        dx[b:c], dxm[b:c] = dyq[b:c] @ W, np.abs(dyq[b:c]) @ np.abs(W)
    return (y, ym), (dx, dxm), ref8.weight_grad(dy, x, offsets)


@pytest.mark.parametrize("T,E,k,N,K,drop", [(1, 1, 1, 40, 30, 0.0), (40, 1, 1, 513, 257, 0.0), (60, 6, 3, 160, 200, 0.1), (500, 4, 2, 136, 300, 0.0)])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
def test_linear_and_its_gradients(ops, T, E, k, N, K, drop, dtype, wdtype):
    g = torch.Generator().manual_seed(T + K)
    R = T * k
    x, w = normal(g, R, K, dtype=dtype).requires_grad_(), normal(g, E, N, K, dtype=wdtype, scale=K ** -0.5).requires_grad_()
    dy = normal(g, R, N, dtype=dtype, scale=0.1)
    ids = routes(np.random.default_rng(T), T, E, k, drop)
    plan = None if E == 1 else ops.expert_sort(torch.from_numpy(ids).cuda(), E)
    offsets = [0, R] if E == 1 else ref.sort(ids, E)[2]
    y = ops.fp8_linear(x, w, plan=plan)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert ops.poll_status() == 0 and y.dtype == dx.dtype == DT[dtype] and dw.dtype == DT[wdtype] and dw.shape == w.shape
    (wy, ym), (wdx, dxm), (wdw, dwm) = linear(ref.f64(x), ref.f64(w), ref.f64(dy), offsets)
    ref.within(y, wy, ym, dtype, K * 2.0 ** -23)
    ref.within(dx, wdx, dxm, dtype, N * 2.0 ** -23)
    ref.within(dw, wdw, dwm, wdtype, R * 2.0 ** -23)
    # one gradient alone, quantised weights, no gradient: the same bits
    q = ops.fp8_quantize(w.detach(), square=True)
    assert torch.equal(torch.autograd.grad(ops.fp8_linear(x, w.detach(), plan=plan), x, dy)[0], dx)
    assert torch.equal(torch.autograd.grad(ops.fp8_linear(x.detach(), w, plan=plan), w, dy)[0], dw)
    assert torch.equal(torch.autograd.grad(ops.fp8_linear(x, q, plan=plan), x, dy)[0], dx)
    assert torch.equal(ops.fp8_linear(x.detach(), q, plan=plan), y.detach()) and torch.equal(ops.fp8_linear(x.detach(), w.detach(), plan=plan), y.detach())


@pytest.mark.parametrize("grouped", [False, True])
def test_linear_without_rows(ops, grouped):
    x = torch.empty((0, 48), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    w = torch.randn((3, 20, 48) if grouped else (20, 48), device="cuda", requires_grad=True)
    plan = ops.expert_sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 3) if grouped else None
    y = ops.fp8_linear(x, w, plan=plan)
    dx, dw = torch.autograd.grad(y, (x, w), torch.empty_like(y))
    assert y.shape == (0, 20) and dx.shape == x.shape and dw.shape == w.shape and (dw == 0).all()


def test_gradients_by_differences(ops):
    # operands that quantise to themselves, and a dy that does: the layer is then
    # linear in both, and differences with steps on the grid are exact
    x = torch.tensor([[1.0, -2.0, 3.0, 0.5], [0.0, 4.0, -1.0, 2.0]], dtype=torch.bfloat16, device="cuda")
    w = torch.tensor([[1.0, 2.0, -1.0, 0.5], [-3.0, 1.0, 2.0, 4.0], [0.5, 0.0, 1.0, -2.0]], device="cuda")
    dy = torch.tensor([[1.0, -0.5, 2.0], [0.25, 3.0, -1.0]], dtype=torch.bfloat16, device="cuda")

    def loss(x, w):
        return (ops.fp8_linear(x, w).double() * dy.double()).sum().item()
    lx, lw = x.clone().requires_grad_(), w.clone().requires_grad_()
    dx, dw = torch.autograd.grad(ops.fp8_linear(lx, lw), (lx, lw), dy)
    for leaf, grad in ((x, dx), (w, dw)):
        for i in np.ndindex(tuple(leaf.shape)):
            keep = leaf[i].item()
            leaf[i] = keep + 1
            up = loss(x, w)
            leaf[i] = keep - 1
            down = loss(x, w)
            leaf[i] = keep
            assert (up - down) / 2 == grad[i].item()


def test_training_step_in_a_graph(ops):
    g = torch.Generator().manual_seed(8)
    x, w, dy = normal(g, 96, 160), normal(g, 3, 72, 160, scale=0.1), normal(g, 96, 72)
    plan = ops.expert_sort(torch.arange(96, device="cuda").remainder(3).int().unsqueeze(1), 3)

    def step():
        a, b = x.detach().requires_grad_(), w.detach().requires_grad_()
        y = ops.fp8_linear(a, b, plan=plan)
        return (y.detach(),) + torch.autograd.grad(y, (a, b), dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.copy_(normal(g, 96, 160))
    w.copy_(normal(g, 3, 72, 160))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_refusals(ops):
    from weight_only_quantized_qmoe_gb300 import QMoEError, binding
    h = torch.randn((8, 64), device="cuda").bfloat16()
    plan = ops.expert_sort(torch.zeros((4, 2), dtype=torch.int32, device="cuda"), 2)
    w = torch.randn((2, 16, 64), device="cuda")
    q = ops.fp8_quantize(w, square=True)
    bad = [lambda: ops.weight_grad(h.cpu(), h), lambda: ops.weight_grad(h, h.half()), lambda: ops.weight_grad(h, h[:4]),
           lambda: ops.weight_grad(h[0], h), lambda: ops.weight_grad(h, h[:, :0]), lambda: ops.weight_grad(h[:4], h[:4], plan=plan),
           lambda: ops.weight_grad(h, h, out_dtype=torch.int32), lambda: ops.weight_grad(h, h, plan=(1, 2)), lambda: ops.weight_grad(None, h),
           lambda: ops.fp8_linear(h, w), lambda: ops.fp8_linear(h, w[0], plan=plan), lambda: ops.fp8_linear(h[:, :32], w, plan=plan),
           lambda: ops.fp8_linear(h[:4], w, plan=plan), lambda: ops.fp8_linear(h, None), lambda: ops.fp8_linear(h, w.int(), plan=plan),
           lambda: ops.fp8_linear(h, q), lambda: ops.fp8_linear(h, ops.fp8_quantize(w[0])), lambda: ops.fp8_linear(h, w.cpu(), plan=plan)]
    for call in bad:
        with pytest.raises(QMoEError) as e:
            call()
        assert e.value.status == binding.QMOE_ERR_INVALID_ARG
    for call in (lambda: ops.weight_grad(h.float(), h.float()), lambda: ops.fp8_linear(h.float(), w, plan=plan)):
        with pytest.raises(QMoEError) as e:
            call()
        assert e.value.status == binding.QMOE_ERR_UNSUPPORTED
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(h, h)
        for call in (lambda: ops.fp8_linear(dual, q, plan=plan), lambda: ops.expert_route(torch.autograd.forward_ad.make_dual(h, h), 2)):
            with pytest.raises(QMoEError):
                call()
