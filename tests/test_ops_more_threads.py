"""The products and the weight gradient from two host threads at once, each on a
stream of its own, at sizes that take different kernels: right statuses, and
right results from calls that overlap on the GPU."""
import pytest
import torch

import test_ops_threads as threads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    from weight_only_quantized_qmoe_gb300 import ops as o
    return o


def test_calls_that_overlap(ops, monkeypatch):
    monkeypatch.setattr(threads, "CALLS", 300)
    from weight_only_quantized_qmoe_gb300 import binding as b
    g = torch.Generator().manual_seed(0)
    held, wrong = [], []

    def product(R, N, K):
        a, w = ops.fp8_quantize(torch.randn((R, K), generator=g).cuda()), ops.fp8_quantize(torch.randn((N, K), generator=g).cuda(), square=True)
        out, want = torch.empty((R, N), device="cuda"), ops.fp8_matmul(a, w, out_dtype=torch.float32)
        held.extend((a, w, out, want))
        p = [t.data_ptr() for t in (a.codes, a.scales, w.codes, w.scales, out)]
        wrong.append(lambda: not torch.equal(out, want))
        return lambda s: b.qmoe_fp8_matmul(p[0], p[1], R, p[2], p[3], 0, 1, N, K, 0, b.QMOE_F32, p[4], N, s)

    def gradient(R, E, N, K):
        dy, x = torch.randn((R, N), generator=g).bfloat16().cuda(), torch.randn((R, K), generator=g).bfloat16().cuda()
        plan = ops.expert_sort(torch.randint(0, E, (R, 1), generator=g).cuda(), E)
        dw, want = torch.empty((E, N, K), device="cuda"), ops.weight_grad(dy, x, plan=plan, out_dtype=torch.float32)
        p = [t.data_ptr() for t in (dy, x, plan.offsets, dw)]
        n = b.qmoe_weight_grad_workspace(p[0], N, p[1], K, R, E, N, K)
        work = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        held.extend((dy, x, plan, dw, want, work))
        wrong.append(lambda: not torch.equal(dw, want))
        wp = work.data_ptr() if n else 0
        return lambda s: b.qmoe_weight_grad(p[0], N, p[1], K, p[2], R, E, N, K, b.QMOE_BF16, b.QMOE_F32, p[3], wp, n, s)

    for calls in ([product(16, 2048, 2048), product(700, 3000, 512)], [gradient(300, 9, 1000, 1111), gradient(2000, 1, 128, 128)],
                  [product(900, 2500, 640), gradient(500, 12, 600, 704)]):
        assert threads.both(calls) == [{b.QMOE_OK}] * 2
    assert not any(w() for w in wrong)
    assert ops.poll_status() == 0
