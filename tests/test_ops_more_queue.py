"""Ragged products and weight gradients queued behind one another with nothing in
between, every kernel after every other: each starts while the one before ends,
and gives what it gives alone."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    from weight_only_quantized_qmoe_gb300 import ops as o
    return o


# widths that leave a warp's last lanes without a column
def calls(ops):
    g = torch.Generator().manual_seed(7)

    def product(R, N, K, dtype, E=0, back=False):
        w = ops.fp8_quantize(torch.randn((E, N, K) if E else (N, K), generator=g).cuda(), square=True)
        x = torch.randn((R, N if back else K), generator=g).cuda()
        plan = ops.expert_sort(torch.randint(0, E, (R, 1), generator=g).cuda(), E) if E else None
        a = ops.fp8_quantize(x, plan)
        return lambda: ops.fp8_matmul(a, w, plan, transpose=back, out_dtype=dtype)

    def gradient(R, N, K, dtype, E=0):
        dy, x = torch.randn((R, N), generator=g).bfloat16().cuda(), torch.randn((R, K), generator=g).bfloat16().cuda()
        plan = ops.expert_sort(torch.randint(0, E, (R, 1), generator=g).cuda(), E) if E else None
        return lambda: ops.weight_grad(dy, x, plan=plan, out_dtype=dtype)

    f32, bf16 = torch.float32, torch.bfloat16
    return [product(3, 129, 1100, bf16),                 # in parts
            product(40, 1001, 300, f32, E=5),
            product(700, 3001, 500, bf16),               # pairs
            product(900, 2501, 400, f32, E=3, back=True),
            product(300, 130, 9000, f32, back=True),
            gradient(60, 129, 131, bf16, E=4),
            gradient(2000, 130, 100, f32),               # in parts
            gradient(500, 1001, 1111, bf16, E=9),        # pairs
            gradient(1500, 2500, 2005, f32)]


def test_queued(ops):
    todo = calls(ops)
    alone = []
    for call in todo:
        alone.append(call())
        torch.cuda.synchronize()
    rng = random.Random(3)
    for _ in range(20):
        order = [rng.randrange(len(todo)) for _ in range(40)]
        got = [todo[i]() for i in order]
        torch.cuda.synchronize()
        assert ops.poll_status() == 0
        for i, t in zip(order, got):
            assert torch.equal(t, alone[i]), i
