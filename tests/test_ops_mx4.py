"""Microscaled 4-bit rows and their product against the plain 64-bit forms.

Quantisation has one rounding, of a value moved by a power of two, so codes and
scales are compared bit for bit.  The product of two elements is exact; a sum
of K of them in fp32, in any order and with every addition truncated instead
of rounded, is off by at most K 2^-23 times the sum of their magnitudes."""
import numpy as np
import pytest
import torch

import ops_reference as ref
from test_ops_routes import DT, routes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    from weight_only_quantized_qmoe_gb300 import ops as o
    return o


def spread(g, M, K, dtype):
    """Rows whose blocks differ widely in magnitude."""
    x = torch.randn((M, K), generator=g) * torch.exp2(torch.randint(-12, 10, (M, -(-K // 32)), generator=g).float()
                                                      ).repeat_interleave(32, 1)[:, :K]
    return x.to(DT[dtype]).cuda()


def check_stored(q, x):
    code, byte, _ = ref.quantize(x)
    codes, scales = ref.pack(code, byte)
    np.testing.assert_array_equal(q.scales.cpu().numpy().reshape(scales.shape), scales)
    np.testing.assert_array_equal(q.codes.cpu().numpy().reshape(codes.shape), codes)


QUANT = [(1, 1), (1, 32), (3, 31), (2, 33), (5, 128), (7, 129), (64, 2048), (33, 1111), (130, 2880), (2, 8200)]


@pytest.mark.parametrize("M,K", QUANT)
@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_and_back(ops, M, K, dtype):
    x = spread(torch.Generator().manual_seed(M * 7 + K), M, K, dtype)
    q = ops.mx4_quantize(x)
    check_stored(q, ref.f64(x))
    _, _, values = ref.quantize(ref.f64(x))
    for out in DT:
        got = ops.mx4_dequantize(q, dtype=DT[out])
        want = torch.from_numpy(values).to(DT[out])
        assert torch.equal(got.cpu(), want)


def test_every_tie_and_threshold(ops):
    # each midpoint of neighbouring values, the points beside it, and past the
    # largest; a 4 in every block fixes its scale at 1
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.96875]
    pts = [m * (1 + d) for m in mids[:8] for d in (-2.0 ** -9, 0.0, 2.0 ** -9)] + mids[8:]
    row = torch.tensor([4.0] + pts + [0.0] * (31 - len(pts)))
    x = torch.stack([row, -row, row * 2.0 ** 20, -row * 2.0 ** -30]).cuda()
    check_stored(ops.mx4_quantize(x), ref.f64(x))


def test_extreme_blocks(ops):
    x = torch.zeros((9, 96))
    x[1, 40] = 2.0 ** -149            # the smallest subnormal
    x[2, :32] = 2.0 ** -127
    x[3, 5] = 3.4e38                  # the largest scale
    x[4, 33] = float("inf")
    x[5, 64] = float("nan")
    x[6, 0] = -0.0
    x[7, :] = 1e-30
    x[8, 31], x[8, 32] = -float("inf"), 1.0
    q = ops.mx4_quantize(x.cuda())
    check_stored(q, ref.f64(x))
    got = ref.f64(ops.mx4_dequantize(q, dtype=torch.float32))
    np.testing.assert_array_equal(got, ref.quantize(ref.f64(x))[2])


def test_stack_of_matrices_and_strides(ops):
    g = torch.Generator().manual_seed(11)
    w = torch.randn((3, 20, 200), generator=g).cuda()
    q = ops.mx4_quantize(w)
    assert q.codes.shape == (3, 20, 112) and q.scales.shape == (3, 2, 20, 4)
    for e in range(3):
        check_stored(ops.MX4Tensor(q.codes[e], q.scales[e], 200), ref.f64(w[e]))
    assert torch.equal(ops.mx4_dequantize(q, dtype=torch.float32)[1],
                       ops.mx4_dequantize(ops.mx4_quantize(w[1]), dtype=torch.float32))
    for x in (w[0][:, 3:103], w[0][:, 8:72], w[0].t(), w[0][::2], w[0][:1].expand(20, 200)):
        check_stored(ops.mx4_quantize(x), ref.f64(x))


@pytest.mark.parametrize("T,E,k,K,drop", [(1, 4, 2, 64, 0.0), (37, 5, 3, 200, 0.3), (64, 128, 8, 2048, 0.0), (20, 3, 2, 33, 1.0)])
def test_quantize_into_expert_order(ops, T, E, k, K, drop):
    rng = np.random.default_rng(T + K)
    ids = routes(rng, T, E, k, drop)
    plan = ops.expert_sort(torch.from_numpy(ids).cuda(), E)
    x = spread(torch.Generator().manual_seed(K), T, K, "bf16")
    q = ops.mx4_quantize(x, plan=plan)
    check_stored(q, ref.dispatch(ref.f64(x), ref.sort(ids, E)[1], k))


@pytest.mark.parametrize("kind", ["swiglu", "geglu"])
@pytest.mark.parametrize("M,K,dtype", [(5, 64, "f32"), (33, 1111, "bf16"), (16, 768, "f16"), (2, 33, "f32")])
def test_quantize_after_an_activation(ops, kind, M, K, dtype):
    """The activation is a fp32 evaluation: a value may land on either side of
    a rounding point (or a block's largest of a power of two) that lies within
    its error, 2^-18 of its magnitude (some twenty fp32 operations), so every
    value is between the quantised ends of that interval."""
    g = torch.Generator().manual_seed(M + K)
    x = (2.0 * torch.randn((M, 2 * K), generator=g)).to(DT[dtype]).cuda()
    got = ref.f64(ops.mx4_dequantize(ops.mx4_quantize(x, activation=kind), dtype=torch.float32))
    X = ref.f64(x)
    h = ref.glu(kind, X[:, :K], X[:, K:])
    rel = 2.0 ** -18
    # gelu's 1 + tanh cancels for negative gates: the error is then of |gate u|
    err = rel * (np.abs(h) if kind == "swiglu" else np.abs(X[:, :K] * X[:, K:]))
    nb = -(-K // 32)
    pad = np.zeros((M, nb * 32))
    pad[:, :K] = np.abs(h) + err
    hi = pad.reshape(M, nb, 32).max(-1)
    pad[:, :K] = np.maximum(np.abs(h) - err, 0.0)
    lo = pad.reshape(M, nb, 32).max(-1)
    ok = np.zeros((M, K), bool)
    for big in (lo, hi):
        scale = np.ldexp(1.0, np.maximum(np.frexp(big)[1] - 3, -127)).repeat(32, 1)[:, :K]
        ends = []
        for v in (h - err, h + err):
            a = np.minimum(np.abs(v) / scale, 6.0)
            cand = ref.E2M1[np.argmin(np.abs(a[..., None] - ref.E2M1), -1)]
            ends.append(np.sign(v) * cand * scale)
        ok |= (got >= np.minimum(*ends) - 1e-300) & (got <= np.maximum(*ends) + 1e-300)
    assert ok.all()
    share = np.mean(got != ref.quantize(h)[2])
    assert share <= 0.01      # almost all of them are the plain form's


def operand(ops, g, shape, scale=1.0):
    return ops.mx4_quantize((scale * torch.randn(shape, generator=g)).cuda())


def check_product(got, a, w, offsets, dtype):
    """got [R, N] against the stored operands' values in 64 bits."""
    A = ref.unpack(a.codes.cpu().numpy(), a.scales.cpu().numpy(), a.cols)
    codes, scales = w.codes.cpu().numpy(), w.scales.cpu().numpy()
    want, mag = np.zeros(tuple(got.shape)), np.zeros(tuple(got.shape))
    for e in range(len(offsets) - 1):
        W = ref.unpack(codes[e], scales[e], w.cols)
        rows = slice(offsets[e], offsets[e + 1])
        want[rows] = A[rows] @ W.T
        mag[rows] = np.abs(A[rows]) @ np.abs(W.T)
    ref.within(got, want, mag, dtype, a.cols * 2.0 ** -23)


# (R, N, K): tails in every direction, one row, one column, many tiles
DENSE = [(1, 64, 64), (1, 2048, 2048), (3, 1, 32), (128, 192, 256), (129, 193, 257), (100, 65, 1), (300, 500, 544),
         (7, 333, 1111), (200, 31, 4097), (1000, 2000, 96), (2049, 3007, 160), (64, 2880, 2880)]


@pytest.mark.parametrize("R,N,K", DENSE)
@pytest.mark.parametrize("dtype", list(DT))
def test_dense_product(ops, R, N, K, dtype):
    g = torch.Generator().manual_seed(R + N + K)
    a, w = operand(ops, g, (R, K)), operand(ops, g, (N, K), K ** -0.5)
    got = ops.mx4_matmul(a, w, out_dtype=DT[dtype])
    assert ops.poll_status() == 0
    check_product(got, a, ops.MX4Tensor(w.codes[None], w.scales[None], K), [0, R], dtype)


# (T, E, k, N, K, drop): empty experts, one expert with everything, dropped
# rows, many experts with few rows, several row tiles an expert
GROUPED = [(1, 4, 1, 64, 64, 0.0), (32, 128, 8, 96, 256, 0.0), (50, 3, 2, 200, 160, 0.2), (700, 4, 2, 300, 288, 0.1),
           (33, 1024, 3, 40, 64, 0.0), (9, 2, 1, 128, 512, 1.0), (2000, 5, 2, 2000, 64, 0.05)]


@pytest.mark.parametrize("T,E,k,N,K,drop", GROUPED)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grouped_product(ops, T, E, k, N, K, drop, dtype):
    rng = np.random.default_rng(T + E)
    ids = routes(rng, T, E, k, drop, skew=3.0)
    plan = ops.expert_sort(torch.from_numpy(ids).cuda(), E)
    g = torch.Generator().manual_seed(N + K)
    w = operand(ops, g, (E, N, K), K ** -0.5)
    a = ops.mx4_quantize(torch.randn((T, K), generator=g).cuda(), plan=plan)
    got = ops.mx4_matmul(a, w, plan=plan, out_dtype=DT[dtype])
    assert ops.poll_status() == 0
    check_product(got, a, w, ref.sort(ids, E)[2], dtype)


def test_one_expert_takes_every_row(ops):
    T, E, N, K = 400, 6, 130, 96
    g = torch.Generator().manual_seed(1)
    w = operand(ops, g, (E, N, K))
    plan = ops.expert_sort(torch.full((T, 1), 4, dtype=torch.int32, device="cuda"), E)
    a = ops.mx4_quantize(torch.randn((T, K), generator=g).cuda(), plan=plan)
    check_product(ops.mx4_matmul(a, w, plan=plan, out_dtype=torch.float32), a, w, plan.offsets.tolist(), "f32")


def test_a_nan_stays_in_its_row_and_column(ops):
    g = torch.Generator().manual_seed(9)
    x, m = torch.randn((200, 300), generator=g).cuda(), torch.randn((250, 300), generator=g).cuda()
    clean = ops.mx4_matmul(ops.mx4_quantize(x), ops.mx4_quantize(m), out_dtype=torch.float32)
    x[17, 5] = float("nan")
    m[201, 299] = float("inf")
    got = ops.mx4_matmul(ops.mx4_quantize(x), ops.mx4_quantize(m), out_dtype=torch.float32)
    assert torch.isnan(got[17]).all() and torch.isnan(got[:, 201]).all()
    rows, cols = torch.arange(200) != 17, torch.arange(250) != 201
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols])


def test_product_does_not_read_past_the_rows(ops):
    # the same rows inside larger buffers filled with NaN scales and the
    # largest codes give the same bits
    g = torch.Generator().manual_seed(13)
    R, N, K = 70, 100, 320
    a, w = operand(ops, g, (R, K)), operand(ops, g, (N, K))
    want = ops.mx4_matmul(a, w, out_dtype=torch.float32)
    ca = torch.full((R + 60, a.codes.shape[1]), 0x77, dtype=torch.uint8, device="cuda")
    cw = torch.full((N + 300, w.codes.shape[1]), 0x77, dtype=torch.uint8, device="cuda")
    ca[:R], cw[:N] = a.codes, w.codes
    got = ops.mx4_matmul(ops.MX4Tensor(ca[:R], a.scales, K), ops.MX4Tensor(cw[:N], w.scales, K), out_dtype=torch.float32)
    assert torch.equal(got, want)


def test_no_rows(ops):
    q = ops.mx4_quantize(torch.empty((0, 64), device="cuda"))
    assert q.codes.shape == (0, 32) and ops.mx4_dequantize(q).shape == (0, 64)
    w = ops.mx4_quantize(torch.randn((40, 64), device="cuda"))
    assert ops.mx4_matmul(q, w).shape == (0, 40)


def test_on_another_stream_and_in_a_graph(ops):
    g = torch.Generator().manual_seed(3)
    x = torch.randn((150, 512), generator=g).cuda()
    w = operand(ops, g, (300, 512))
    want = ops.mx4_matmul(ops.mx4_quantize(x), w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.mx4_matmul(ops.mx4_quantize(x, stream=side), w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.mx4_matmul(ops.mx4_quantize(x), w)
    x.copy_(torch.randn((150, 512), generator=g))
    graph.replay()
    assert torch.equal(out, ops.mx4_matmul(ops.mx4_quantize(x), w))


def test_a_wait_that_runs_out_is_reported(ops):
    # host-injected: the first copy's barrier is armed and its copy never
    # issued, so the bounded waits on it end by themselves
    from weight_only_quantized_qmoe_gb300 import binding
    g = torch.Generator().manual_seed(4)
    a, w = operand(ops, g, (64, 512)), operand(ops, g, (128, 512))
    want = ops.mx4_matmul(a, w)
    assert ops.poll_status() == 0
    assert binding.qmoe_op_set_wait_limit(2000) == 0 and binding.qmoe_op_debug_inject_stall(1) == 0
    try:
        ops.mx4_matmul(a, w)
        assert ops.poll_status() == binding.QMOE_ERR_TIMEOUT
        assert ops.poll_status() == 0
    finally:
        binding.qmoe_op_debug_inject_stall(0)
        binding.qmoe_op_set_wait_limit(0)
    assert torch.equal(ops.mx4_matmul(a, w), want) and ops.poll_status() == 0


def test_refusals(ops):
    from weight_only_quantized_qmoe_gb300 import QMoEError, binding
    x = torch.randn((8, 64), device="cuda")
    a, w = ops.mx4_quantize(x), ops.mx4_quantize(torch.randn((2, 16, 64), device="cuda"))
    plan = ops.expert_sort(torch.zeros((4, 2), dtype=torch.int32, device="cuda"), 2)
    M = ops.MX4Tensor
    bad = [lambda: ops.mx4_quantize(x.cpu()), lambda: ops.mx4_quantize(x.int()), lambda: ops.mx4_quantize(x[0]),
           lambda: ops.mx4_quantize(x, activation="relu"), lambda: ops.mx4_quantize(x[:, :63], activation="swiglu"),
           lambda: ops.mx4_quantize(x, plan=plan), lambda: ops.mx4_quantize(x[:, :0]),
           lambda: ops.mx4_dequantize(x), lambda: ops.mx4_dequantize(a, dtype=torch.int8),
           lambda: ops.mx4_dequantize(M(a.codes, a.scales, 65)), lambda: ops.mx4_dequantize(M(a.codes, a.scales[:0], 64)),
           lambda: ops.mx4_matmul(a, w), lambda: ops.mx4_matmul(a, M(w.codes, w.scales, 60), plan=plan),
           lambda: ops.mx4_matmul(M(a.codes[:4], a.scales[:, :4], 64), w, plan=plan),
           lambda: ops.mx4_matmul(a, M(w.codes[0], w.scales[0], 64), plan=plan),
           lambda: ops.mx4_matmul(a, w, plan=plan, out_dtype=torch.int32),
           lambda: ops.mx4_matmul(a, w, plan=plan._replace(offsets=plan.offsets[:2]))]
    for call in bad:
        with pytest.raises(QMoEError) as e:
            call()
        assert e.value.status == binding.QMOE_ERR_INVALID_ARG
