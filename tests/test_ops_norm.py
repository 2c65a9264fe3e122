"""The norms around a block and their gradients against the plain 64-bit forms.

Bounds: a row's sum of squares adds at most 64 values in a thread and then a
tree of 16 levels, so a statistic is off by at most 80 2^-24 / 2 + a few units;
with the handful of operations around it a value is off by 64 2^-24 of the
magnitudes it is made of, plus one rounding to the type.  In the gradients a
second mean of the same kind follows (128 2^-24), and the sums over the rows
add up to T / 304 + 50 terms one after another."""
import numpy as np
import pytest
import torch

import ops_reference as ref
from test_ops_routes import DT

pytestmark = pytest.mark.gpu
REL = 64 * 2.0 ** -24
GREL = 128 * 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    from weight_only_quantized_qmoe_gb300 import ops as o
    return o


def inputs(T, H, dtype, gate, seed=0):
    g = torch.Generator().manual_seed(seed + T * 3 + H)

    def normal(*shape, scale=1.0, shift=0.0):
        return (shift + scale * torch.randn(shape, generator=g)).to(DT[dtype]).cuda()

    shape = {"none": None, "token": (T, 1), "channel": (H,), "full": (T, H)}[gate]
    return dict(x=normal(T, H, scale=2.0), o=normal(T, H, scale=0.3), gate=None if shape is None else normal(*shape),
                w_post=normal(H, scale=0.2, shift=1.0), w_pre=normal(H, scale=0.2, shift=1.0),
                dr=normal(T, H), dh=normal(T, H))


def check_forward(ops, x, o, gate, w_post, w_pre, scale, dtype, eps=EPS):
    r, h, stats = ops.block_norm(x, o, gate=gate, w_post=w_post, w_pre=w_pre, residual_scale=scale, eps=eps,
                                 return_stats=True)
    R, Hh, mag = ref.norm(ref.f64(x), ref.f64(o), ref.f64(gate), ref.f64(w_post), ref.f64(w_pre), scale, eps)
    ref.within(r, R, mag, dtype, REL)
    if w_pre is None:
        assert h is None
    else:
        s2 = 1.0 / np.sqrt((R * R).mean(-1, keepdims=True) + eps)
        # rounding in r's terms moves its statistic by their share of the row
        lift = 1.0 + np.sqrt((mag * mag).mean(-1, keepdims=True)) * s2
        ref.within(h, Hh, mag * s2 * np.abs(ref.f64(w_pre)) * lift, dtype, REL)
    return r, h, stats


SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (8, 2048), (130, 96), (33, 1001), (17, 2880), (9, 4096), (4, 8200), (2, 16384),
          (2, 16383), (700, 40)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("dtype", list(DT))
def test_forward_and_gradients(ops, T, H, gate, dtype):
    v = inputs(T, H, dtype, gate)
    fwd = {n: v[n] for n in ("x", "o", "gate", "w_post", "w_pre")}
    _, _, stats = check_forward(ops, **fwd, scale=0.7, dtype=dtype)
    got = ops.block_norm_grad(v["dr"], v["dh"], v["x"], v["o"], stats, gate=v["gate"], w_post=v["w_post"],
                              w_pre=v["w_pre"], residual_scale=0.7)
    check_grads(got, v, 0.7, dtype)


def check_grads(got, v, scale, dtype, eps=EPS):
    a = {n: ref.f64(v.get(n)) for n in ("dr", "dh", "x", "o", "gate", "w_post", "w_pre")}
    want = ref.norm_grad(a["dr"], a["dh"], a["x"], a["o"], a["gate"], a["w_post"], a["w_pre"], scale, eps)
    T, H = v["x"].shape
    for name in ("x", "o", "gate", "w_post", "w_pre"):
        g = getattr(got, name)
        if name not in want:
            assert g is None, name
            continue
        w, mag = want[name]
        summed = name in ("w_post", "w_pre") or (name == "gate" and a["gate"].shape != (T, H))
        # values whose statistic is small beside the terms (short rows) carry
        # the statistic's error: one more factor of the row's own amplification
        rel = GREL + ((T / 304 + 50 + (H if name == "gate" else 0)) * 2.0 ** -24 if summed else 0.0)
        ref.within(g, w, mag, dtype, rel * amplification(a, scale, eps))


def amplification(a, scale, eps):
    """How much larger r's terms are than r, at the worst row: rounding errors
    of the terms reach the statistic and everything scaled by it."""
    r, _, mag = ref.norm(a["x"], a["o"], a["gate"], a["w_post"], None, scale, eps)
    s = np.sqrt((r * r).mean(-1) + eps)
    return 1.0 + float(np.max(np.sqrt((mag * mag).mean(-1)) / s))


@pytest.mark.parametrize("absent", ["w_post", "w_pre", "o", "dr", "dh", "w_post+w_pre", "o+w_pre"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_absent_arguments(ops, absent, dtype):
    v = inputs(40, 520, dtype, "channel")
    for n in absent.split("+"):
        v[n] = None
        if n == "o":
            v["gate"] = v["w_post"] = None
        if n == "w_pre":
            v["dh"] = None
    fwd = {n: v[n] for n in ("x", "o", "gate", "w_post", "w_pre")}
    _, _, stats = check_forward(ops, **fwd, scale=-1.3, dtype=dtype)
    got = ops.block_norm_grad(v["dr"], v["dh"], v["x"], v["o"], stats, gate=v["gate"], w_post=v["w_post"],
                              w_pre=v["w_pre"], residual_scale=-1.3)
    check_grads(got, v, -1.3, dtype)


@pytest.mark.parametrize("dtype", list(DT))
def test_strides_and_alignment(ops, dtype):
    T, H = 21, 128
    big = torch.randn((T, 3 * H + 7), generator=torch.Generator().manual_seed(1)).to(DT[dtype]).cuda()
    w = (1 + 0.1 * torch.randn(2 * H + 1, generator=torch.Generator().manual_seed(2))).to(DT[dtype]).cuda()
    for x, o in ((big[:, :H], big[:, H:2 * H]), (big[:, 1:H + 1], big[:, H + 3:2 * H + 3]), (big[:, 0:2 * H:2], big[:, 1:2 * H:2]),
                 (big[:1, :H].expand(T, H), big[:, :H])):
        check_forward(ops, x, o, big[:, 5:H + 5], w[1:H + 1], w[H:2 * H], 1.0, dtype)


def test_leading_dimensions(ops):
    g = torch.Generator().manual_seed(5)
    x, o = torch.randn((2, 3, 64), generator=g).cuda(), torch.randn((2, 3, 64), generator=g).cuda()
    w = torch.randn(64, generator=g).cuda()
    gate = torch.rand((2, 3, 1), generator=g).cuda()
    r, h = ops.block_norm(x, o, gate=gate, w_post=w, w_pre=w)
    r2, h2 = ops.block_norm(x.reshape(6, 64), o.reshape(6, 64), gate=gate.reshape(6, 1), w_post=w, w_pre=w)
    assert torch.equal(r.reshape(6, 64), r2) and torch.equal(h.reshape(6, 64), h2) and r.shape == x.shape


def test_rows_of_zeros_and_a_nan_row(ops):
    x = torch.randn((6, 200), device="cuda")
    o = torch.randn((6, 200), device="cuda")
    w = torch.ones(200, device="cuda")
    x[1] = 0
    o[1] = 0
    o[2] = 0
    x[4, 7] = float("nan")
    r, h = ops.block_norm(x, o, w_post=w, w_pre=w)
    assert (r[1] == 0).all() and (h[1] == 0).all() and torch.equal(r[2], x[2])
    assert torch.isnan(h[4]).all() and torch.isfinite(h[[0, 1, 2, 3, 5]]).all()


def test_no_rows(ops):
    x = torch.empty((0, 32), device="cuda")
    w = torch.ones(32, device="cuda")
    r, h, stats = ops.block_norm(x, x, w_post=w, w_pre=w, gate=w, return_stats=True)
    assert r.shape == h.shape == (0, 32)
    g = ops.block_norm_grad(x, x, x, x, stats, gate=w, w_post=w, w_pre=w)
    assert (g.w_post == 0).all() and (g.w_pre == 0).all() and (g.gate == 0).all() and g.x.shape == (0, 32)


@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
def test_automatic_differentiation_and_differences(ops, gate):
    T, H, scale = 13, 70, 0.6
    v = inputs(T, H, "f32", gate, seed=9)
    names = ["x", "o", "w_post", "w_pre"] + ([] if gate == "none" else ["gate"])
    leaf = {n: (v[n].clone().requires_grad_() if n in names else v.get(n)) for n in ("x", "o", "gate", "w_post", "w_pre")}
    r, h = ops.block_norm(leaf["x"], leaf["o"], gate=leaf["gate"], w_post=leaf["w_post"], w_pre=leaf["w_pre"],
                          residual_scale=scale)
    grads = torch.autograd.grad((r * v["dr"]).sum() + (h * v["dh"]).sum(), [leaf[n] for n in names])
    a = {n: ref.f64(v.get(n)) for n in ("dr", "dh", "x", "o", "gate", "w_post", "w_pre")}

    def f(p):
        rr, hh, _ = ref.norm(p["x"], p["o"], p["gate"], p["w_post"], p["w_pre"], scale, EPS)
        return (rr * a["dr"]).sum() + (hh * a["dh"]).sum()

    rng = np.random.default_rng(0)
    for n, g in zip(names, grads):
        d = rng.standard_normal(a[n].shape)
        step = 1e-5
        diff = (f({**a, n: a[n] + step * d}) - f({**a, n: a[n] - step * d})) / (2 * step)
        got = (ref.f64(g) * d).sum()
        # differences: third-order terms 1e-10 and 64-bit rounding 1e-11; fp32 gradients 1e-5 of their size
        assert abs(got - diff) <= 2e-5 * (np.abs(ref.f64(g) * d).sum() + 1.0), n
    # only one output used
    x = v["x"].clone().requires_grad_()
    r, h = ops.block_norm(x, v["o"], gate=v["gate"], w_post=v["w_post"], w_pre=v["w_pre"], residual_scale=scale)
    (gx,) = torch.autograd.grad((h * v["dh"]).sum(), [x])
    a1 = {n: ref.f64(v.get(n)) for n in ("dh", "x", "o", "gate", "w_post", "w_pre")}
    w, mag = ref.norm_grad(None, a1["dh"], a1["x"], a1["o"], a1["gate"], a1["w_post"], a1["w_pre"], scale, EPS)["x"]
    ref.within(gx, w, mag, "f32", GREL * amplification(a, scale, EPS))


def test_gradients_do_not_change_from_run_to_run(ops):
    v = inputs(900, 512, "bf16", "channel")
    _, _, stats = ops.block_norm(v["x"], v["o"], gate=v["gate"], w_post=v["w_post"], w_pre=v["w_pre"], return_stats=True)
    a, b = (ops.block_norm_grad(v["dr"], v["dh"], v["x"], v["o"], stats, gate=v["gate"], w_post=v["w_post"],
                                w_pre=v["w_pre"]) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_on_another_stream_and_in_a_graph(ops):
    v = inputs(64, 256, "bf16", "token")
    kw = dict(gate=v["gate"], w_post=v["w_post"], w_pre=v["w_pre"])
    want = ops.block_norm(v["x"], v["o"], **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.block_norm(v["x"], v["o"], stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, h = ops.block_norm(v["x"], v["o"], **kw)
    v["o"].mul_(3)
    graph.replay()
    want = ops.block_norm(v["x"], v["o"], **kw)
    assert torch.equal(r, want[0]) and torch.equal(h, want[1])


def test_refusals(ops):
    from weight_only_quantized_qmoe_gb300 import QMoEError, binding
    x, w = torch.zeros((4, 16), device="cuda"), torch.ones(16, device="cuda")
    s = ops.NormStats(torch.ones(4, device="cuda"), torch.ones(4, device="cuda"))
    bad = [lambda: ops.block_norm(x.cpu()), lambda: ops.block_norm(x.double()), lambda: ops.block_norm(x, x[:3]),
           lambda: ops.block_norm(x, x.half()), lambda: ops.block_norm(x, gate=w), lambda: ops.block_norm(x, w_post=w),
           lambda: ops.block_norm(x, x, gate=w[:5]), lambda: ops.block_norm(x, x, w_post=w[:5]),
           lambda: ops.block_norm(x, w_pre=w.half()), lambda: ops.block_norm(x, w_pre=w, eps=-1.0),
           lambda: ops.block_norm(x, w_pre=w, eps=float("nan")), lambda: ops.block_norm(x, residual_scale=float("inf")),
           lambda: ops.block_norm_grad(x, x, x, x, s, w_post=w), lambda: ops.block_norm_grad(x[:2], None, x, x, s, w_post=w),
           lambda: ops.block_norm_grad(x, None, x, x, ops.NormStats(s[0][:2], s[1]), w_post=w)]
    for call in bad:
        with pytest.raises(QMoEError) as e:
            call()
        assert e.value.status == binding.QMOE_ERR_INVALID_ARG
    with pytest.raises(QMoEError) as e:
        ops.block_norm(torch.zeros((2, 16385), device="cuda"))
    assert e.value.status == binding.QMOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("T,H", [(5, 4104), (3, 6000), (4, 8192), (160, 8192)])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_two_fragments_of_16_bit_rows(ops, T, H, gate, dtype):
    test_forward_and_gradients(ops, T, H, gate, dtype)
