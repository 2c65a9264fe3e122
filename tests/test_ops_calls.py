"""Calls of the operators that lie beside their ordinary arguments: padding that
is not used, empty and unusually shaped arguments, forward-mode derivatives."""
import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    from weight_only_quantized_qmoe_gb300 import ops as o
    return o


# --- microscaled rows ----------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("K", [1, 32, 65, 160, 257, 288, 1111, 2880])
@pytest.mark.parametrize("R,N", [(3, 40), (300, 400)])
def test_padding_scales_are_not_used(ops, R, N, K):
    # what follows the last block's scale in its word of four: 255 (NaN) must
    # not meet the padding codes
    g = torch.Generator().manual_seed(R + K)
    a, w = (ops.mx4_quantize(torch.randn((n, K), generator=g).cuda()) for n in (R, N))
    nb = -(-K // 32)

    def poisoned(q):
        s = q.scales.clone()
        if nb % 4:
            s[-1, :, nb % 4:] = 255
        return ops.MX4Tensor(q.codes, s, K)

    want = ops.mx4_matmul(a, w, out_dtype=torch.float32)
    assert torch.isfinite(want).all()
    assert torch.equal(ops.mx4_matmul(poisoned(a), poisoned(w), out_dtype=torch.float32), want)
    assert torch.equal(ops.mx4_dequantize(poisoned(a)), ops.mx4_dequantize(a))


# --- empty arguments -------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["token", "channel", "full"])
def test_no_rows_with_a_gate(ops, gate):
    x = torch.empty((0, 32), device="cuda")
    w = torch.ones(32, device="cuda")
    g = {"token": x[:, :1], "channel": w, "full": x}[gate]
    r, h, stats = ops.block_norm(x, x, w_post=w, w_pre=w, gate=g, return_stats=True)
    assert r.shape == h.shape == (0, 32)
    d = ops.block_norm_grad(x, x, x, x, stats, gate=g, w_post=w, w_pre=w)
    assert d.gate.shape == g.shape and (d.gate == 0).all()
    assert (d.w_post == 0).all() and (d.w_pre == 0).all() and d.x.shape == d.o.shape == (0, 32)


def test_no_rows_at_the_entry_point():
    from weight_only_quantized_qmoe_gb300 import binding as b, build
    build.build()
    P = 4096   # not used

    def call(gate, kind, T=0):
        return b.qmoe_block_norm(P, 32, P, 32, gate, kind, 32, P, P, 1.0, 1e-6, T, 32, b.QMOE_F32, P, P, 0, 0, None)
    for gate in (0, P):
        assert call(gate, b.QMOE_GATE_TOKEN) == call(gate, b.QMOE_GATE_FULL) == b.QMOE_OK
    for gate, kind, T in ((0, b.QMOE_GATE_CHANNEL, 0), (P, b.QMOE_GATE_NONE, 0), (0, b.QMOE_GATE_TOKEN, 4), (0, b.QMOE_GATE_FULL, 4)):
        assert call(gate, kind, T) == b.QMOE_ERR_INVALID_ARG


# --- shapes ------------------------------------------------------------------------
@pytest.mark.gpu
def test_route_weights_of_another_shape_are_refused(ops):
    from weight_only_quantized_qmoe_gb300 import QMoEError, binding
    T, k, H = 6, 2, 16
    plan = ops.expert_sort(torch.randint(0, 3, (T, k), device="cuda"), 3)
    y, dout = torch.randn((T * k, H), device="cuda"), torch.randn((T, H), device="cuda")
    w = torch.rand((T, k), device="cuda")
    for bad in (w.t(), w.t().contiguous(), w.reshape(-1)[:6], w[None], w.reshape(4, 3)):
        for call in (lambda: ops.combine(y, bad, plan), lambda: ops.combine_grad(dout, y, bad, plan)):
            with pytest.raises(QMoEError) as e:
                call()
            assert e.value.status == binding.QMOE_ERR_INVALID_ARG
    strided = torch.rand((T, 2 * k), device="cuda")[:, ::2]      # of the right shape: any strides, or flat
    want = ops.combine(y, strided.contiguous(), plan)
    assert torch.equal(ops.combine(y, strided, plan), want) and torch.equal(ops.combine(y, strided.reshape(-1), plan), want)
    flat = w.reshape(-1).clone().requires_grad_()
    (dw,) = torch.autograd.grad(ops.combine(y, flat, plan), [flat], [dout])
    assert torch.equal(dw.reshape(T, k), ops.combine_grad(dout, y, w, plan)[1])


@pytest.mark.gpu
def test_norm_weights_of_another_shape_are_refused(ops):
    from weight_only_quantized_qmoe_gb300 import QMoEError, binding
    x, w = torch.randn((4, 16), device="cuda"), torch.ones(16, device="cuda")
    for bad in (w.reshape(4, 4), w.reshape(16, 1), w[None, :, None], w[:8]):
        for kw in (dict(w_post=bad), dict(w_pre=bad)):
            with pytest.raises(QMoEError) as e:
                ops.block_norm(x, x, **kw)
            assert e.value.status == binding.QMOE_ERR_INVALID_ARG
    # axes of one before it say nothing, and the gradient has them too
    want = ops.block_norm(x, x, w_post=w, w_pre=w)
    row = torch.ones((1, 16), device="cuda", requires_grad=True)
    got = ops.block_norm(x, x, w_post=row, w_pre=row)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    (g,) = torch.autograd.grad(got[1].sum(), [row])
    assert g.shape == (1, 16)


# --- automatic differentiation ---------------------------------------------------------
def test_forward_mode_derivatives_are_refused(ops):
    # there is no tangent to give: an output without one would mean zero
    from torch.autograd import forward_ad
    from weight_only_quantized_qmoe_gb300 import QMoEError
    plan = ops.ExpertPlan(*(torch.zeros(4, dtype=torch.int32) for _ in range(3)), 2, 3)
    x, w = torch.randn(4, 8), torch.ones(8)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        dual_w = forward_ad.make_dual(w, torch.ones_like(w))
        weights = forward_ad.make_dual(torch.ones(2, 2), torch.ones(2, 2))
        for call in (lambda: ops.dispatch(dual, plan), lambda: ops.combine(dual, None, plan),
                     lambda: ops.combine(x, weights, plan), lambda: ops.block_norm(dual), lambda: ops.block_norm(x, dual),
                     lambda: ops.block_norm(x, x, w_post=dual_w), lambda: ops.block_norm(x, w_pre=dual_w),
                     lambda: ops.block_norm(x, x, gate=dual_w)):
            for enabled in (True, False):
                with torch.set_grad_enabled(enabled), pytest.raises(QMoEError, match="forward-mode"):
                    call()


@pytest.mark.gpu
def test_tensors_without_a_tangent_pass_inside_a_dual_level(ops):
    from torch.autograd import forward_ad
    x, w = torch.randn((4, 8), device="cuda"), torch.ones(8, device="cuda")
    want = ops.block_norm(x, w_pre=w)
    with forward_ad.dual_level():
        got = ops.block_norm(x, w_pre=w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_a_plan_changed_before_the_gradient_is_refused(ops):
    # as for any tensor that a gradient needs
    T, k, H = 5, 2, 16
    ids = torch.randint(0, 3, (T, k), device="cuda")

    def routed(what):
        plan = ops.expert_sort(ids, 3)
        if what == "dispatch":
            x = torch.randn((T, H), device="cuda", requires_grad=True)
            return plan, ops.dispatch(x, plan), x
        y = torch.randn((T * k, H), device="cuda", requires_grad=True)
        return plan, ops.combine(y, torch.rand((T, k), device="cuda"), plan), y

    for what in ("dispatch", "combine"):
        plan, out, leaf = routed(what)
        plan.pos.copy_(plan.pos.flip(0))
        with pytest.raises(RuntimeError, match="inplace"):
            torch.autograd.grad(out.sum(), [leaf])
        plan, out, leaf = routed(what)
        (g,) = torch.autograd.grad(out.sum(), [leaf])
        assert g.shape == leaf.shape


@pytest.mark.gpu
def test_a_plan_that_is_none_is_refused_where_a_gradient_is_needed_too(ops):
    from weight_only_quantized_qmoe_gb300 import QMoEError
    x = torch.randn((4, 16), device="cuda", requires_grad=True)
    for plan in (None, torch.zeros(4, device="cuda")):
        with pytest.raises(QMoEError):
            ops.dispatch(x, plan)
        with pytest.raises(QMoEError):
            ops.combine(x, None, plan)
