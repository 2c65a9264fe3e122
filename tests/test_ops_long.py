"""The operators on tensors of more than 2^31 elements: the last rows, whose
offsets do not fit 32 bits, are those of a call on these rows alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    from weight_only_quantized_qmoe_gb300 import ops as o
    return o


def test_rows_there_and_back(ops):
    T, k, E, H = 280_000, 8, 16, 1024          # 2.3e9 elements in expert order
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.argsort(torch.rand((T, E), generator=g, device="cuda"), dim=1)[:, :k]
    plan = ops.expert_sort(ids, E)
    assert int(plan.offsets[-1]) == T * k
    xs = ops.dispatch(x, plan)
    assert xs.numel() > 2 ** 31
    w = torch.full((T, k), 0.125, device="cuda")
    assert torch.equal(ops.combine(xs, w, plan), x)      # eight eighths: exact
    dy, dw = ops.combine_grad(x, xs, w, plan)
    assert torch.equal(ops.dispatch_grad(dy, plan), x)
    norm2 = (x[-64:].float() ** 2).sum(1, keepdim=True).expand(64, k)
    assert torch.allclose(dw[-64:], norm2, rtol=1024 * 2.0 ** -24)


def test_microscaled_rows_and_product(ops):
    R, K, N = 2_200_000, 2048, 64               # 2.25 GB of codes, 4.5e9 values
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((R, K), generator=g, device="cuda", dtype=torch.bfloat16)
    w = ops.mx4_quantize(torch.randn((N, K), generator=g, device="cuda"))
    q = ops.mx4_quantize(x)
    assert q.codes.numel() > 2 ** 31
    y = ops.mx4_matmul(q, w, out_dtype=torch.float32)
    last = ops.mx4_quantize(x[-300:])
    assert torch.equal(q.codes[-300:], last.codes) and torch.equal(q.scales[:, -300:], last.scales)
    assert torch.equal(y[-300:], ops.mx4_matmul(last, w, out_dtype=torch.float32))
    assert torch.equal(ops.mx4_dequantize(q)[-300:], ops.mx4_dequantize(last))
    assert ops.poll_status() == 0


def test_norms(ops):
    T, H = 600_000, 4096                        # 2.5e9 elements
    g = torch.Generator(device="cuda").manual_seed(2)
    x, o = (torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = torch.ones(H, device="cuda", dtype=torch.bfloat16)
    kw = dict(gate=w * 0.5, w_post=w, w_pre=w, residual_scale=0.5)
    r, h, stats = ops.block_norm(x, o, return_stats=True, **kw)
    r2, h2, stats2 = ops.block_norm(x[-50:], o[-50:], return_stats=True, **kw)
    assert torch.equal(r[-50:], r2) and torch.equal(h[-50:], h2)
    grads = ops.block_norm_grad(r, h, x, o, stats, **kw)
    few = ops.block_norm_grad(r[-50:], h[-50:], x[-50:], o[-50:], stats2, **kw)
    assert torch.equal(grads.x[-50:], few.x) and torch.equal(grads.o[-50:], few.o)
