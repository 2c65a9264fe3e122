"""The C entry points from two host threads at once, each on a stream of its
own, at sizes that need different amounts of shared memory from the same
kernels: they keep nothing between calls that one could change for the other."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
CALLS = 4000


@pytest.fixture(scope="module")
def b():
    from weight_only_quantized_qmoe_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def both(calls):
    """The statuses of CALLS calls of each, made at the same time."""
    start = threading.Barrier(len(calls))
    got = [set() for _ in calls]

    def work(i, call, stream):
        torch.cuda.set_device(0)
        start.wait()
        for _ in range(CALLS):
            got[i].add(call(stream.cuda_stream))

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    threads = [threading.Thread(target=work, args=(i, c, s)) for i, (c, s) in enumerate(zip(calls, streams))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return got


def test_norms_of_two_widths(b):
    held = []

    def call(H, T=4):
        x, o, r, h = (torch.randn((T, H), device="cuda").to(torch.bfloat16) for _ in range(4))
        w = torch.ones(H, device="cuda", dtype=torch.bfloat16)
        held.extend((x, o, r, h, w))
        p = [t.data_ptr() for t in (x, o, w, r, h)]
        return lambda s: b.qmoe_block_norm(p[0], H, p[1], H, 0, 0, 0, p[2], p[2], 1.0, 1e-6, T, H, b.QMOE_BF16, p[3], p[4], 0, 0, s)

    assert both([call(3584), call(4096)]) == [{b.QMOE_OK}] * 2


def test_norm_gradients_of_two_widths(b):
    held = []

    def call(H, T=4):
        t = [torch.randn((T, H), device="cuda").to(torch.bfloat16) for _ in range(6)]
        w = [torch.ones(H, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
        s1 = torch.ones(T, device="cuda")
        n = b.qmoe_block_norm_grad_workspace(T, H, b.QMOE_BF16)
        work = torch.empty(n, dtype=torch.uint8, device="cuda")
        held.extend(t + w + [s1, work])
        p, q, v, wk = [x.data_ptr() for x in t], [x.data_ptr() for x in w], s1.data_ptr(), work.data_ptr()
        return lambda s: b.qmoe_block_norm_grad(p[0], H, p[1], H, p[2], H, p[3], H, 0, 0, 0, q[0], q[0], v, v, 1.0, T, H,
                                                b.QMOE_BF16, p[4], p[5], 0, q[1], q[2], wk, n, s)

    assert both([call(3584), call(4096)]) == [{b.QMOE_OK}] * 2


def test_sorts_of_two_expert_counts(b):
    held = []

    def call(E, T=8192, k=2):
        ids = torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32)
        out = [torch.empty(n, device="cuda", dtype=torch.int32) for n in (T * k, T * k, E + 1)]
        held.extend([ids] + out)
        p, q = ids.data_ptr(), [t.data_ptr() for t in out]
        return lambda s: b.qmoe_expert_sort(p, 4, k, T, k, E, q[0], q[1], q[2], s)

    assert both([call(500), call(1024)]) == [{b.QMOE_OK}] * 2
