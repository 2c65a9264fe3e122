"""The router, the 8-bit rows and products and the weight gradient on tensors of
more than 2^31 elements: the last rows, whose offsets do not fit 32 bits, are
those of a call on these rows alone, or for the products (which add up few rows
in another order than many) within their bound of a 64-bit evaluation: a sum of K
exact products in fp32, in any order and with every addition truncated, is off by
at most K 2^-23 times the sum of their magnitudes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    from weight_only_quantized_qmoe_gb300 import ops as o
    return o


def check(ops, y, a, w, transpose=False):
    """y [n, ...] float32 of the rows a [n, K] of weights w."""
    A, W = (ops.fp8_dequantize(q, dtype=torch.float32).double() for q in (a, w))
    W = W if transpose else W.t()
    assert ((y.double() - A @ W).abs() <= (a.cols * 2.0 ** -23 + 2.0 ** -24) * (A.abs() @ W.abs())).all()


def test_router(ops):
    T, E = 2_200_000, 1000                      # 2.2e9 logits
    g = torch.Generator(device="cuda").manual_seed(0)
    logits = torch.randn((T, E), generator=g, device="cuda", dtype=torch.bfloat16)
    r = ops.expert_route(logits, 4, scoring="sigmoid")
    few = ops.expert_route(logits[-100:], 4, scoring="sigmoid")
    assert torch.equal(r.ids[-100:], few.ids) and torch.equal(r.weights[-100:], few.weights)
    d = ops.expert_route_grad(r.weights, logits, r.ids, renormalize=False)
    assert torch.equal(d[-100:], ops.expert_route_grad(few.weights, logits[-100:], few.ids, renormalize=False))


@pytest.mark.parametrize("transpose", [False, True])
def test_rows_and_product(ops, transpose):
    R, K, N = 1_200_000, 2048, 192              # 2.5e9 values and codes
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((R, K), generator=g, device="cuda", dtype=torch.bfloat16)
    w = ops.fp8_quantize(torch.randn((K, N) if transpose else (N, K), generator=g, device="cuda"), square=True)
    q = ops.fp8_quantize(x)
    assert q.codes.numel() > 2 ** 31
    y = ops.fp8_matmul(q, w, transpose=transpose, out_dtype=torch.float32)
    last = ops.fp8_quantize(x[-300:])
    assert torch.equal(q.codes[-300:], last.codes) and torch.equal(q.scales[:, -300:], last.scales)
    check(ops, y[-300:], last, w, transpose)
    assert torch.equal(ops.fp8_dequantize(q)[-300:], ops.fp8_dequantize(last))
    assert ops.poll_status() == 0


def test_weights_and_their_gradient(ops):
    E, N, K = 18, 16384, 8192                   # 2.4e9 values
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.empty((E, N, K), device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    q = ops.fp8_quantize(w, square=True)
    one = ops.fp8_quantize(w[-1], square=True)
    assert torch.equal(q.codes[-1], one.codes) and torch.equal(q.scales[-1], one.scales)
    plan = ops.expert_sort(torch.arange(E, device="cuda").repeat_interleave(20).int().unsqueeze(1), E)
    x = ops.fp8_quantize(torch.randn((20 * E, K), generator=g, device="cuda"))
    y = ops.fp8_matmul(x, q, plan=plan, out_dtype=torch.float32)
    alone = ops.FP8Tensor(x.codes[-20:], x.scales[:, -20:].contiguous(), K, False)
    check(ops, y[-20:], alone, one)
    dy, xs = (torch.randn((20 * E, n), generator=g, device="cuda").bfloat16() for n in (N, K))
    dw = ops.weight_grad(dy, xs, plan=plan)
    assert dw.numel() > 2 ** 31
    assert torch.equal(dw[-1], ops.weight_grad(dy[-20:], xs[-20:]))
    assert ops.poll_status() == 0


def test_a_wide_product(ops):
    R, K, N = 70_000, 64, 32_768                # 2.3e9 results
    g = torch.Generator(device="cuda").manual_seed(3)
    x = ops.fp8_quantize(torch.randn((R, K), generator=g, device="cuda"))
    w = ops.fp8_quantize(torch.randn((N, K), generator=g, device="cuda"), square=True)
    y = ops.fp8_matmul(x, w, out_dtype=torch.float32)
    check(ops, y[-300:], ops.FP8Tensor(x.codes[-300:], x.scales[:, -300:].contiguous(), K, False), w)
