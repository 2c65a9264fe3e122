"""Routes sorted by expert, rows taken there and back, and the gradients,
against the plain 64-bit forms.

Bounds: a sum of n products in fp32 is off by at most (n + 1) 2^-24 times the
sum of the products' magnitudes, however it is ordered, and its result is
rounded once to the type."""
import numpy as np
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    from weight_only_quantized_qmoe_gb300 import ops as o
    return o


def routes(rng, T, E, k, drop=0.0, skew=0.0):
    """ids [T, k], distinct experts of a token where there are enough."""
    p = np.exp(-skew * np.arange(E) / max(1, E))
    score = rng.gumbel(size=(T, E)) + np.log(p / p.sum())
    ids = np.argsort(-score, axis=1)[:, :k] if k <= E else rng.integers(0, E, (T, k))
    return np.where(rng.random((T, k)) < drop, -1, ids).astype(np.int64)


# (T, E, k, drop): one route, one cluster pass and more, all dropped, one
# expert, more slots than a group of eight, the most experts
SORTS = [(1, 1, 1, 0.0), (1, 4, 2, 0.0), (5, 3, 3, 0.3), (33, 7, 2, 0.0), (64, 128, 8, 0.1), (128, 8, 2, 0.0), (129, 8, 2, 0.0),
         (512, 8, 2, 0.0), (513, 8, 2, 0.0), (1000, 64, 8, 0.05), (4099, 256, 6, 0.0), (7, 2, 11, 0.0), (300, 1024, 4, 0.2),
         (40000, 32, 4, 0.0), (50, 5, 2, 1.0), (3000, 1, 1, 0.0)]


@pytest.mark.parametrize("T,E,k,drop", SORTS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(ops, T, E, k, drop, dtype):
    rng = np.random.default_rng(T * 31 + E)
    ids = routes(rng, T, E, k, drop, skew=2.0)
    plan = ops.expert_sort(torch.from_numpy(ids).to(dtype).cuda(), E)
    perm, pos, offsets = ref.sort(ids, E)
    np.testing.assert_array_equal(plan.offsets.cpu().numpy(), offsets)
    np.testing.assert_array_equal(plan.pos.cpu().numpy(), pos)
    np.testing.assert_array_equal(plan.perm.cpu().numpy(), perm)


def test_sort_drops_ids_out_of_range(ops):
    ids = torch.tensor([[0, 5], [-1, 2], [7, 1], [2 ** 40, -2 ** 40], [4, 0]])
    plan = ops.expert_sort(ids.cuda(), 5)
    want = ref.sort(np.where((ids.numpy() >= 0) & (ids.numpy() < 5), ids.numpy(), -1), 5)
    for got, w in zip((plan.perm, plan.pos, plan.offsets), want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)


def test_sort_takes_strided_ids(ops):
    rng = np.random.default_rng(3)
    wide = torch.from_numpy(routes(rng, 700, 16, 6)).cuda()
    for ids in (wide[:, 1:4], wide[::2, :2], wide.t().contiguous().t()[:, :3]):
        plan = ops.expert_sort(ids, 16)
        for got, w in zip((plan.perm, plan.pos, plan.offsets), ref.sort(ids.cpu().numpy(), 16)):
            np.testing.assert_array_equal(got.cpu().numpy(), w)


# (T, E, k, H, drop): vectors and odd lengths, rows shorter than a warp's
# vectors and longer than a CTA's, more than eight slots, tokens left empty
ROWS = [(1, 2, 1, 8, 0.0), (8, 8, 2, 2048, 0.0), (37, 5, 3, 1001, 0.2), (64, 16, 4, 2880, 0.0), (129, 4, 2, 64, 0.5),
        (20, 24, 17, 136, 0.1), (3, 2, 2, 1, 0.0), (11, 6, 2, 9000, 0.3), (257, 3, 1, 250, 1.0), (6, 4, 3, 4100, 0.0)]


@pytest.mark.parametrize("T,E,k,H,drop", ROWS)
@pytest.mark.parametrize("dtype", list(DT))
def test_rows_there_and_back(ops, T, E, k, H, drop, dtype):
    rng = np.random.default_rng(T * 1009 + H)
    ids = routes(rng, T, E, k, drop)
    g = torch.Generator().manual_seed(T + H)
    R = T * k
    x, dout = (torch.randn((T, H), generator=g).to(DT[dtype]).cuda() for _ in range(2))
    y, dxs = (torch.randn((R, H), generator=g).to(DT[dtype]).cuda() for _ in range(2))
    w = torch.rand((T, k), generator=g).cuda()
    plan = ops.expert_sort(torch.from_numpy(ids).cuda(), E)
    _, pos, offsets = ref.sort(ids, E)
    # rows no route owns hold what may not be read
    y[offsets[-1]:] = float("nan")
    dxs[offsets[-1]:] = float("inf")
    np.testing.assert_array_equal(ref.f64(ops.dispatch(x, plan)), ref.dispatch(ref.f64(x), pos, k))
    for weights in (w, None):
        want, mag = ref.combine(ref.f64(y), ref.f64(weights), pos, k)
        ref.within(ops.combine(y, weights, plan), want, mag, dtype, (k + 1) * 2.0 ** -24)
    want, mag = ref.combine(ref.f64(dxs), None, pos, k)
    ref.within(ops.dispatch_grad(dxs, plan), want, mag, dtype, (k + 1) * 2.0 ** -24)
    dy, dw = ops.combine_grad(dout, y, w, plan)
    wy, ww, mag = ref.combine_grad(ref.f64(dout), ref.f64(y), ref.f64(w), pos, k)
    ref.within(dy, wy, np.abs(wy), dtype, 2.0 ** -24)
    ref.within(dw, ww, mag, "f32", (H + 1) * 2.0 ** -24)
    only_dy, none = ops.combine_grad(dout, y, None, plan, need_dweights=False)
    assert none is None
    ref.within(only_dy, ref.combine_grad(ref.f64(dout), ref.f64(y), None, pos, k)[0], 0.0, dtype, 0.0)
    none, only_dw = ops.combine_grad(dout, y, w, plan, need_dy=False)
    assert none is None and torch.equal(only_dw, dw)


@pytest.mark.parametrize("dtype", list(DT))
def test_rows_with_strides(ops, dtype):
    rng = np.random.default_rng(8)
    T, E, k, H = 45, 6, 2, 96
    ids = routes(rng, T, E, k)
    g = torch.Generator().manual_seed(5)
    big = torch.randn((T * k, 3 * H + 5), generator=g).to(DT[dtype]).cuda()
    plan = ops.expert_sort(torch.from_numpy(ids).cuda(), E)
    _, pos, _ = ref.sort(ids, E)
    w = torch.rand((T, k), generator=g).cuda()
    for y in (big[:, 3:3 + H], big[:, H:2 * H], big[:, 0:2 * H:2], big.t()[:T * k, :H] if T * k <= 3 * H + 5 else None):
        if y is None or y.shape != (T * k, H):
            continue
        want, mag = ref.combine(ref.f64(y), ref.f64(w), pos, k)
        ref.within(ops.combine(y, w, plan), want, mag, dtype, (k + 1) * 2.0 ** -24)
        x = y[:T]
        np.testing.assert_array_equal(ref.f64(ops.dispatch(x, plan)), ref.dispatch(ref.f64(x), pos, k))
    one = big[:1, :1].expand(T, H)         # a broadcast row
    np.testing.assert_array_equal(ref.f64(ops.dispatch(one, plan)), ref.dispatch(ref.f64(one), pos, k))


def test_rows_carry_infinities_and_nan_of_their_own_token_only(ops):
    T, E, k, H = 12, 4, 2, 40
    ids = routes(np.random.default_rng(1), T, E, k)
    plan = ops.expert_sort(torch.from_numpy(ids).cuda(), E)
    x = torch.ones((T, H), device="cuda")
    x[5] = float("nan")
    xs = ops.dispatch(x, plan)
    out = ops.combine(xs, torch.full((T, k), 0.5, device="cuda"), plan)
    assert torch.isnan(out[5]).all() and torch.equal(out[torch.arange(T) != 5], x[torch.arange(T) != 5])


@pytest.mark.parametrize("T,k", [(0, 2), (0, 1)])
def test_no_tokens(ops, T, k):
    plan = ops.expert_sort(torch.empty((T, k), dtype=torch.int32, device="cuda"), 5)
    assert plan.offsets.tolist() == [0] * 6 and plan.perm.numel() == 0
    x = torch.empty((0, 16), device="cuda")
    assert ops.dispatch(x, plan).shape == (0, 16) and ops.combine(x, None, plan).shape == (0, 16)
    dy, dw = ops.combine_grad(x, x, None, plan)
    assert dy.shape == (0, 16) and dw.shape == (0, k)


def test_automatic_differentiation_and_differences(ops):
    """The gradients of a route there and back agree with the 64-bit formula's
    and with differences of the 64-bit forward."""
    rng = np.random.default_rng(21)
    T, E, k, H = 29, 5, 3, 77
    ids = routes(rng, T, E, k, 0.15)
    g = torch.Generator().manual_seed(2)
    x = torch.randn((T, H), generator=g).cuda().requires_grad_()
    w = torch.rand((T, k), generator=g).cuda().requires_grad_()
    m = torch.randn((T * k, H), generator=g).cuda()
    c = torch.randn((T, H), generator=g).cuda()
    plan = ops.expert_sort(torch.from_numpy(ids).cuda(), E)
    loss = (ops.combine(ops.dispatch(x, plan) * m, w, plan) * c).sum()
    dx, dw = torch.autograd.grad(loss, [x, w])
    _, pos, _ = ref.sort(ids, E)
    X, W, M, C = (ref.f64(t) for t in (x, w, m, c))

    def f(xv, wv):
        return (ref.combine(ref.dispatch(xv, pos, k) * M, wv, pos, k)[0] * C).sum()

    dy, ww, wmag = ref.combine_grad(C, ref.dispatch(X, pos, k) * M, W, pos, k)
    wx, xmag = ref.combine(dy * M, None, pos, k)
    ref.within(dx, wx, xmag, "f32", (k + 4) * 2.0 ** -24)
    ref.within(dw, ww, wmag, "f32", (H + 4) * 2.0 ** -24)
    vx, vw = rng.standard_normal(X.shape), rng.standard_normal(W.shape)
    for dvx, dvw, got in ((vx, 0 * vw, (ref.f64(dx) * vx).sum()), (0 * vx, vw, (ref.f64(dw) * vw).sum())):
        step = 1e-3    # the forward is linear in each: differences are exact but for 64-bit rounding
        diff = (f(X + step * dvx, W + step * dvw) - f(X - step * dvx, W - step * dvw)) / (2 * step)
        scale = (np.abs(ref.f64(dx) * dvx)).sum() + (np.abs(ref.f64(dw) * dvw)).sum()
        assert abs(got - diff) <= 1e-5 * scale


def test_a_second_derivative_is_refused(ops):
    # the gradients are kernels of their own: differentiating them again must
    # fail, not give zeros
    plan = ops.expert_sort(torch.zeros((3, 1), dtype=torch.int32, device="cuda"), 2)
    x = torch.randn((3, 8), device="cuda", requires_grad=True)
    (g,) = torch.autograd.grad((ops.dispatch(x, plan) ** 2).sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), [x])


def test_gradients_do_not_change_from_run_to_run(ops):
    rng = np.random.default_rng(4)
    T, E, k, H = 600, 16, 4, 1024
    plan = ops.expert_sort(torch.from_numpy(routes(rng, T, E, k)).cuda(), E)
    y, dout, w = torch.randn((T * k, H), device="cuda"), torch.randn((T, H), device="cuda"), torch.rand((T, k), device="cuda")
    a, b = ops.combine_grad(dout, y, w, plan), ops.combine_grad(dout, y, w, plan)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_on_another_stream_and_in_a_graph(ops):
    rng = np.random.default_rng(6)
    T, E, k, H = 64, 8, 2, 256
    ids = torch.from_numpy(routes(rng, T, E, k)).to(torch.int32).cuda()
    x, w = torch.randn((T, H), device="cuda"), torch.rand((T, k), device="cuda")

    def there_and_back(stream=None):
        plan = ops.expert_sort(ids, E, stream=stream)
        return ops.combine(ops.dispatch(x, plan, stream=stream), w, plan, stream=stream)

    want = there_and_back()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = there_and_back(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = there_and_back()
    x.copy_(torch.randn((T, H), device="cuda"))
    ids.copy_(torch.from_numpy(routes(rng, T, E, k)))
    graph.replay()
    assert torch.equal(out, there_and_back())


def test_refusals(ops):
    from weight_only_quantized_qmoe_gb300 import QMoEError, binding
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    plan = ops.expert_sort(ids, 3)
    x = torch.zeros((4, 16), device="cuda")
    bad = [lambda: ops.expert_sort(ids.cpu(), 3), lambda: ops.expert_sort(ids.float(), 3),
           lambda: ops.expert_sort(ids.reshape(-1), 3), lambda: ops.expert_sort(ids, 0), lambda: ops.expert_sort(ids, -2),
           lambda: ops.dispatch(x[:3], plan), lambda: ops.dispatch(x.double(), plan), lambda: ops.dispatch(x.cpu(), plan),
           lambda: ops.dispatch(x, plan[:3]), lambda: ops.dispatch(x, plan._replace(experts=4)),
           lambda: ops.combine(x, None, plan), lambda: ops.combine(torch.zeros((8, 16), device="cuda"), x, plan),
           lambda: ops.combine(torch.zeros((8, 16), device="cuda"), torch.zeros((4, 2), device="cuda").half(), plan),
           lambda: ops.combine_grad(x, torch.zeros((8, 17), device="cuda"), None, plan),
           lambda: ops.combine_grad(x, torch.zeros((8, 16), device="cuda").half(), None, plan)]
    for call in bad:
        with pytest.raises(QMoEError) as e:
            call()
        assert e.value.status == binding.QMOE_ERR_INVALID_ARG
    with pytest.raises(QMoEError) as e:
        ops.expert_sort(ids, 1025)
    assert e.value.status == binding.QMOE_ERR_UNSUPPORTED
