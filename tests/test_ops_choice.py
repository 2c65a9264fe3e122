"""The router against its plain 64-bit form: choices bit for bit, weights and
gradients within the rounding of fp32.

A weight is an exponential of a difference (2 steps of 2^-24, and half a step
of the difference, which is at most D), a sum of at most E such terms (at most 37
additions one after the other), a division and a product by the scale: with the
terms' own errors some 2 * (D / 2 + 2) + 37 + 3 < D + 45 steps."""
import numpy as np
import pytest
import torch

import ops_reference as ref
import ops_reference8 as ref8
from test_ops_routes import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    from weight_only_quantized_qmoe_gb300 import ops as o
    return o


def steps(logits):
    """The bound above, for these logits."""
    fine = logits[np.isfinite(logits)]
    return (45 + (np.ptp(fine) if fine.size else 0.0)) * 2.0 ** -24


def check(ops, logits, k, scoring="softmax", bias=None, groups=1, top_groups=None, group_best=1, renormalize=True, scale=1.0):
    how = dict(scoring=scoring, bias=bias, groups=groups, top_groups=top_groups, group_best=group_best, renormalize=renormalize, scale=scale)
    r = ops.expert_route(logits, k, **how)
    l = ref.f64(logits)
    ids, w = ref8.route(l, k, scoring, ref.f64(bias), groups, top_groups or groups, group_best, renormalize, scale)
    np.testing.assert_array_equal(r.ids.cpu().numpy(), ids)
    assert r.ids.dtype == torch.int32 and r.weights.dtype == torch.float32
    ref.within(r.weights, w, np.abs(w), "f32", steps(l))
    again = ops.expert_route(logits, k, **how)
    assert torch.equal(again.ids, r.ids) and torch.equal(again.weights, r.weights)
    return r


# (T, E, k): one token, one expert, lanes of one to 32 values, ragged counts
SIZES = [(1, 1, 1), (1, 128, 8), (5, 8, 8), (3, 31, 4), (17, 33, 5), (130, 60, 6), (64, 200, 32), (9, 257, 3), (33, 1024, 8), (4, 1000, 32)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_choice_and_weights(ops, T, E, k, dtype, scoring):
    g = torch.Generator().manual_seed(T * 7 + E + k)
    logits = (2.0 * torch.randn((T, E), generator=g)).to(DT[dtype]).cuda()
    bias = (0.1 * torch.randn(E, generator=g)).cuda()
    for renormalize in (True, False):
        check(ops, logits, k, scoring, None, renormalize=renormalize)
        check(ops, logits, k, scoring, bias, renormalize=renormalize, scale=2.5)


# (E, groups, top, best, k)
GROUPS = [(16, 4, 2, 1, 3), (256, 8, 4, 2, 8), (60, 3, 1, 2, 20), (96, 32, 5, 2, 10), (64, 16, 15, 1, 8), (1024, 2, 1, 2, 32), (12, 12, 7, 1, 7),
          (30, 5, 5, 2, 4)]


@pytest.mark.parametrize("E,groups,top,best,k", GROUPS)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(ops, E, groups, top, best, k, scoring, biased):
    g = torch.Generator().manual_seed(E + groups)
    for dtype in ("f32", "bf16"):
        logits = torch.randn((70, E), generator=g).to(DT[dtype]).cuda()
        bias = (0.2 * torch.randn(E, generator=g)).cuda() if biased else None
        check(ops, logits, k, scoring, bias, groups, top, best, renormalize=dtype == "f32")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top,best", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lower_index(ops, scoring, groups, top, best, biased):
    # few different values, so that most neighbours in the order are equal
    g = torch.Generator().manual_seed(2)
    logits = torch.randint(-2, 3, (200, 64), generator=g).float().cuda()
    bias = (torch.randint(0, 2, (64,), generator=g).float() * 0.25).cuda() if biased else None
    check(ops, logits, 9, scoring, bias, groups, top, best)
    check(ops, torch.zeros((3, 40), device="cuda"), 7, scoring, None, groups, top, best)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_neighbours_too_near_for_32_bits(ops, scoring):
    # bias takes from each expert what its score has over the first one's, rounded
    # to 32 bits: all choices are equal but for what 32 bits cannot hold
    g = torch.Generator().manual_seed(5)
    row = torch.randn(48, generator=g)
    s = ref8.scores(row.double().numpy(), scoring)
    bias = torch.from_numpy((s[0] + 0.5 - s).astype(np.float32)).cuda()
    logits = row.repeat(4, 1).cuda()
    r = check(ops, logits, 12, scoring, bias)
    assert (r.ids == r.ids[0]).all()
    for best in (1, 2):
        check(ops, logits, 12, scoring, bias, 8, 3, best)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased,groups,top,best", [(False, 1, 1, 1), (True, 1, 1, 1), (False, 4, 2, 2), (True, 4, 2, 1), (True, 4, 2, 2)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_closed_experts(ops, scoring, biased, groups, top, best, renormalize):
    # rows with all experts open, some, fewer than k, one, none
    g = torch.Generator().manual_seed(8)
    logits = torch.randn((40, 32), generator=g)
    open_ = torch.rand((40, 32), generator=g) < torch.linspace(0, 1, 40).unsqueeze(1)
    open_[1], open_[2] = False, torch.arange(32) == 17
    logits = torch.where(open_, logits, -float("inf")).cuda()
    bias = torch.randn(32, generator=g).cuda() if biased else None
    r = check(ops, logits, 6, scoring, bias, groups, top, best, renormalize)
    assert (r.ids[1] == -1).all() and (r.weights[1] == 0).all()
    if biased:
        bias[3] = -float("inf")
        assert not (check(ops, logits, 6, scoring, bias, groups, top, best, renormalize).ids == 3).any()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_nan_and_infinity(ops, scoring):
    g = torch.Generator().manual_seed(9)
    logits = torch.randn((6, 40), generator=g).cuda()
    clean = ops.expert_route(logits, 5, scoring=scoring)
    logits[2, 7], logits[4, 39] = float("nan"), -float("nan")
    for bias in (None, torch.zeros(40, device="cuda")):
        r = ops.expert_route(logits, 5, scoring=scoring, bias=bias)
        for t in range(6):
            if t in (2, 4):
                assert torch.isnan(r.weights[t]).all() and not (r.ids[t] == (7 if t == 2 else 39)).any() and (r.ids[t] >= 0).all()
            else:
                assert torch.equal(r.ids[t], clean.ids[t]) and torch.equal(r.weights[t], clean.weights[t])
    logits = torch.randn((2, 40), generator=g).cuda()
    bias = torch.zeros(40, device="cuda")
    bias[11] = float("nan")
    r = ops.expert_route(logits, 30, scoring=scoring, bias=bias)
    assert torch.isnan(r.weights).all() and not (r.ids == 11).any()
    logits[0, 3] = float("inf")
    r = ops.expert_route(logits, 4, scoring=scoring)
    assert r.ids[0, 0] == 3
    if scoring == "sigmoid":
        ref.within(r.weights[:1], ref8.route(ref.f64(logits[:1]), 4, scoring, None, 1, 1, 1, True, 1.0)[1], 1.0, "f32", 2.0 ** -18)
    else:
        assert torch.isnan(r.weights[0]).any()


def test_scores_that_are_small_keep_their_ratios(ops):
    # sigmoid scores below the smallest float32 number
    logits = torch.tensor([[-200.0, -201.0, -199.0, -300.0], [-3.0, 5.0, -120.0, 0.0]], device="cuda")
    for k in (2, 4):
        check(ops, logits, k, "sigmoid")
        check(ops, logits, k, "softmax")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 8), (40, 60, 6), (9, 257, 32), (33, 1024, 8)])
@pytest.mark.parametrize("dtype", list(DT))
def test_gradient(ops, scoring, renormalize, T, E, k, dtype):
    g = torch.Generator().manual_seed(T + E)
    logits = torch.randn((T, E), generator=g).to(DT[dtype])
    if T > 5:
        logits[T // 2, ::2] = -float("inf")
        logits[T // 3] = -float("inf")
    logits = logits.cuda()
    dw = torch.randn((T, k), generator=g).cuda()
    r = ops.expert_route(logits, k, scoring=scoring, renormalize=renormalize, scale=1.5)
    got = ops.expert_route_grad(dw, logits, r.ids, scoring=scoring, renormalize=renormalize, scale=1.5)
    want, mag = ref8.route_grad(ref.f64(dw), ref.f64(logits), r.ids.cpu().numpy(), scoring, renormalize, 1.5)
    assert got.dtype == logits.dtype
    # two weights' errors, and the sum of k products
    ref.within(got, want, mag, dtype, 2 * steps(ref.f64(logits)) + (k + 8) * 2.0 ** -24)
    # and by automatic differentiation
    leaf = logits.clone().requires_grad_()
    out = ops.expert_route(leaf, k, scoring=scoring, renormalize=renormalize, scale=1.5)
    assert torch.equal(out.weights.detach(), r.weights) and not out.ids.requires_grad
    assert torch.equal(torch.autograd.grad(out.weights, leaf, dw)[0], got)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_by_differences(ops, scoring, renormalize):
    # the formula's gradient against differences of the plain form in 64 bits,
    # the kernel's against the formula's above
    rng = np.random.default_rng(3)
    l, dw, h = rng.standard_normal((3, 12)), rng.standard_normal((3, 4)), 1e-5
    ids, _ = ref8.route(l, 4, scoring, None, 1, 1, 1, renormalize, 1.0)

    def loss(x):
        total = 0.0
        for t in range(3):
            s = ref8.scores(x[t], scoring)[ids[t]]
            total += (dw[t] * (s / s.sum() if renormalize else s)).sum()
        return total
    want = np.zeros_like(l)
    for i in np.ndindex(l.shape):
        up, down = l.copy(), l.copy()
        up[i] += h
        down[i] -= h
        want[i] = (loss(up) - loss(down)) / (2 * h)
    np.testing.assert_allclose(ref8.route_grad(dw, l, ids, scoring, renormalize, 1.0)[0], want, atol=1e-8)
    got = ops.expert_route_grad(torch.from_numpy(dw).float().cuda(), torch.from_numpy(l).float().cuda(),
                                torch.from_numpy(ids).int().cuda(), scoring=scoring, renormalize=renormalize)
    np.testing.assert_allclose(ref.f64(got), want, atol=2e-5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_an_expert_named_twice_and_slots_without_one(ops, scoring, renormalize):
    g = torch.Generator().manual_seed(4)
    logits, dw = torch.randn((4, 20), generator=g).cuda(), torch.randn((4, 5), generator=g).cuda()
    ids = torch.tensor([[3, 3, 7, 3, 19], [-1, 2, 20, 2, 0], [-1] * 5, [0, 1, 2, 3, 4]], dtype=torch.int32, device="cuda")
    got = ops.expert_route_grad(dw, logits, ids, scoring=scoring, renormalize=renormalize)
    want, mag = ref8.route_grad(ref.f64(dw), ref.f64(logits), ids.cpu().numpy(), scoring, renormalize, 1.0)
    ref.within(got, want, mag, "f32", 2 * steps(ref.f64(logits)) + 16 * 2.0 ** -24)


def test_strides_streams_and_graphs(ops):
    g = torch.Generator().manual_seed(6)
    base = torch.randn((50, 90), generator=g).cuda()
    for logits in (base[:, 3:67], base[::2, 1:41], base[:40, :32].t(), base[:1].expand(7, 90)):
        check(ops, logits, 4, "sigmoid", torch.zeros(logits.shape[1], device="cuda"))
    logits, bias = base[:, :64].contiguous(), torch.randn(64, generator=g).cuda()
    want = ops.expert_route(logits, 4, bias=bias, groups=8, top_groups=3, group_best=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.expert_route(logits, 4, bias=bias, groups=8, top_groups=3, group_best=2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got.ids, want.ids) and torch.equal(got.weights, want.weights)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.expert_route(logits, 4, scoring="sigmoid", bias=bias)
        plan = ops.expert_sort(out.ids, 64)
        d = ops.expert_route_grad(out.weights, logits, out.ids, scoring="sigmoid")
    logits.copy_(torch.randn((50, 64), generator=g))
    graph.replay()
    want = ops.expert_route(logits, 4, scoring="sigmoid", bias=bias)
    assert torch.equal(out.ids, want.ids) and torch.equal(out.weights, want.weights)
    assert torch.equal(plan.pos, ops.expert_sort(want.ids, 64).pos)
    assert torch.equal(d, ops.expert_route_grad(want.weights, logits, want.ids, scoring="sigmoid"))


def test_no_tokens(ops):
    empty = torch.empty((0, 16), device="cuda")
    r = ops.expert_route(empty, 3)
    assert r.ids.shape == r.weights.shape == (0, 3)
    assert ops.expert_route_grad(r.weights, empty, r.ids).shape == (0, 16)


def test_the_layers_own_choice(ops):
    # softmax, renormalised: what the weight-only layer's routing gives
    from weight_only_quantized_qmoe_gb300 import binding as b
    st, h = b.qmoe_create(64, 64, 32, 4, 4, 4, 32, b.QMOE_ZP_SYMMETRIC, b.QMOE_ACT_SWIGLU, b.QMOE_BF16)
    assert st == b.QMOE_OK
    try:
        g = torch.Generator().manual_seed(1)
        for fc, n, k in ((1, 128, 64), (2, 64, 64)):
            codes = torch.randint(0, 256, (32, n, k // 2), generator=g, dtype=torch.uint8).cuda()
            scales = torch.ones((32, n, k // 32), dtype=torch.bfloat16, device="cuda")
            assert b.qmoe_prepack(h, fc, codes.data_ptr(), scales.data_ptr(), None, 0) == b.QMOE_OK
        logits = torch.randn((20, 32), generator=g).cuda()
        x, out = torch.zeros((20, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((20, 64), dtype=torch.bfloat16, device="cuda")
        ids, w = torch.empty((20, 4), dtype=torch.int32, device="cuda"), torch.empty((20, 4), device="cuda")
        torch.cuda.synchronize()
        assert b.qmoe_forward(h, x.data_ptr(), logits.data_ptr(), out.data_ptr(), 20, 0) == b.QMOE_OK
        assert b.qmoe_get_routing(h, ids.data_ptr(), w.data_ptr(), None, None, 0) == b.QMOE_OK
        torch.cuda.synchronize()
    finally:
        b.qmoe_destroy(h)
    r = ops.expert_route(logits, 4)
    assert torch.equal(r.ids, ids)
    ref.within(r.weights, ref.f64(w), ref.f64(w), "f32", 2 * steps(ref.f64(logits)))


def test_refusals(ops):
    from weight_only_quantized_qmoe_gb300 import QMoEError, binding
    x = torch.randn((8, 64), device="cuda")
    r = ops.expert_route(x, 4)
    bad = [lambda: ops.expert_route(x.cpu(), 2), lambda: ops.expert_route(x.int(), 2), lambda: ops.expert_route(x[0], 2),
           lambda: ops.expert_route(x, 0), lambda: ops.expert_route(x, 65), lambda: ops.expert_route(x, 2, scoring="tanh"),
           lambda: ops.expert_route(x, 2, bias=x[0].half()), lambda: ops.expert_route(x, 2, bias=x[0, :63]),
           lambda: ops.expert_route(x, 2, bias=x[:1]), lambda: ops.expert_route(x, 2, groups=7), lambda: ops.expert_route(x, 2, groups=0),
           lambda: ops.expert_route(x, 2, groups=8, top_groups=9), lambda: ops.expert_route(x, 2, groups=8, top_groups=0),
           lambda: ops.expert_route(x, 9, groups=8, top_groups=1), lambda: ops.expert_route(x, 2, groups=8, top_groups=2, group_best=3),
           lambda: ops.expert_route(x[:, :32], 2, groups=32, top_groups=4, group_best=2), lambda: ops.expert_route(x, 2, scale=float("inf")),
           lambda: ops.expert_route(x, 2, scale=float("nan")), lambda: ops.expert_route(x[:, :0], 1),
           lambda: ops.expert_route_grad(r.weights, x, r.ids.long()), lambda: ops.expert_route_grad(r.weights[:, :3], x, r.ids),
           lambda: ops.expert_route_grad(r.weights.half(), x, r.ids), lambda: ops.expert_route_grad(r.weights, x[:4], r.ids),
           lambda: ops.expert_route_grad(r.weights, x, r.ids, scoring=None)]
    for call in bad:
        with pytest.raises(QMoEError) as e:
            call()
        assert e.value.status == binding.QMOE_ERR_INVALID_ARG
    wide = torch.randn((2, 1056), device="cuda")
    for call in (lambda: ops.expert_route(wide, 2), lambda: ops.expert_route(x, 33), lambda: ops.expert_route(x, 2, groups=64)):
        with pytest.raises(QMoEError) as e:
            call()
        assert e.value.status == binding.QMOE_ERR_UNSUPPORTED
