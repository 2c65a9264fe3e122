"""8-bit rows, weights in square blocks and their products against the plain
64-bit forms.

Quantisation has one rounding, of a value moved by a power of two, so codes and
scales are compared bit for bit.  The product of two elements is exact; a sum
of K of them in fp32, in any order and with every addition truncated instead
of rounded, is off by at most K 2^-23 times the sum of their magnitudes."""
import numpy as np
import pytest
import torch

import ops_reference as ref
import ops_reference8 as ref8
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
    x = torch.randn((M, K), generator=g) * torch.exp2(torch.randint(-12, 10, (M, -(-K // 128)), generator=g).float()
                                                      ).repeat_interleave(128, 1)[:, :K]
    return x.to(DT[dtype]).cuda()


def check_stored(q, x, square=False):
    code, byte, _ = ref8.quantize(x, square)
    codes, scales = ref8.pack(code, byte)
    assert q.square is square
    np.testing.assert_array_equal(q.scales.cpu().numpy().reshape((byte if square else scales).shape), byte if square else scales)
    np.testing.assert_array_equal(q.codes.cpu().numpy().reshape(codes.shape), codes)


# --- rows and blocks ------------------------------------------------------------------
ROWS = [(1, 1), (1, 16), (3, 31), (2, 127), (5, 128), (7, 129), (64, 2048), (33, 1111), (130, 2880), (2, 8200), (9, 513), (4000, 130)]


@pytest.mark.parametrize("M,K", ROWS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("square", [False, True])
def test_quantize_and_back(ops, M, K, dtype, square):
    x = spread(torch.Generator().manual_seed(M * 7 + K), M, K, dtype)
    q = ops.fp8_quantize(x, square=square)
    check_stored(q, ref.f64(x), square)
    values = ref8.quantize(ref.f64(x), square)[2]
    for out in DT:
        assert torch.equal(ops.fp8_dequantize(q, dtype=DT[out]).cpu(), torch.from_numpy(values).to(DT[out]))


def test_every_tie_and_threshold(ops):
    # the largest value fixes the scale at 1; then each midpoint of neighbouring
    # values and the points beside it
    pts = [448.0]
    for lo, hi in zip(ref8.POSITIVE, ref8.POSITIVE[1:]):
        mid = (lo + hi) / 2
        pts += [mid, np.nextafter(np.float32(mid), np.float32(0)), np.nextafter(np.float32(mid), np.float32(1e9))]
    row = torch.zeros(128 * 4)
    for b in range(4):
        part = [448.0] + pts[1 + 127 * b:128 + 127 * b]
        row[128 * b:128 * b + len(part)] = torch.tensor(part)
    x = torch.stack([row, -row, row * 2.0 ** 20, -row * 2.0 ** -30]).cuda()
    check_stored(ops.fp8_quantize(x), ref.f64(x))


def test_scale_thresholds(ops):
    # 448 is the largest that keeps a scale, the next number takes the next one
    big = [448.0, np.nextafter(np.float32(448), np.float32(1e9)), np.nextafter(np.float32(448), np.float32(0)), 256.0, 511.9, 512.0, 895.9, 896.0]
    x = torch.zeros((len(big), 200))
    x[:, 3], x[:, 7] = torch.tensor(np.array(big, np.float32)), 1.0
    for t in (x, x * 2.0 ** -100, x * 2.0 ** 100):
        check_stored(ops.fp8_quantize(t.cuda()), ref.f64(t))


@pytest.mark.parametrize("square", [False, True])
def test_extreme_blocks(ops, square):
    x = torch.zeros((9 * 128 if square else 9, 300))
    n = 128 if square else 1
    x[1 * n, 140] = 2.0 ** -149          # the smallest subnormal
    x[2 * n, :32] = 2.0 ** -127
    x[3 * n, 5] = 3.2e38                 # near the largest scale
    x[4 * n, 133] = float("inf")
    x[5 * n, 256] = float("nan")
    x[6 * n, 0] = -0.0
    x[7 * n, :] = 1e-38
    x[8 * n, 127], x[8 * n, 128] = -float("inf"), 1.0
    q = ops.fp8_quantize(x.cuda(), square=square)
    check_stored(q, ref.f64(x), square)
    np.testing.assert_array_equal(ref.f64(ops.fp8_dequantize(q, dtype=torch.float32)), ref8.quantize(ref.f64(x), square)[2])


@pytest.mark.parametrize("square", [False, True])
def test_stack_of_matrices_and_strides(ops, square):
    g = torch.Generator().manual_seed(11)
    w = torch.randn((3, 140, 520), generator=g).cuda()
    q = ops.fp8_quantize(w, square=square)
    assert q.codes.shape == (3, 140, 528) and q.scales.shape == ((3, 2, 5) if square else (3, 2, 140, 4))
    for e in range(3):
        check_stored(ops.FP8Tensor(q.codes[e], q.scales[e], 520, square), ref.f64(w[e]), square)
    assert torch.equal(ops.fp8_dequantize(q, dtype=torch.float32)[1],
                       ops.fp8_dequantize(ops.fp8_quantize(w[1], square=square), dtype=torch.float32))
    h = w.bfloat16()
    for m in (w[0], h[0]):
        for x in (m[:, 3:403], m[:, 8:72], m[1:, 1:], m.t(), m[::2], m[:1].expand(20, 520), m[5:6, 7:]):
            check_stored(ops.fp8_quantize(x, square=square), ref.f64(x), square)


@pytest.mark.parametrize("T,E,k,K,drop", [(1, 4, 2, 64, 0.0), (37, 5, 3, 200, 0.3), (64, 128, 8, 2048, 0.0), (20, 3, 2, 33, 1.0), (9, 40, 36, 130, 0.1)])
def test_quantize_into_expert_order(ops, T, E, k, K, drop):
    rng = np.random.default_rng(T + K)
    ids = routes(rng, T, E, k, drop)
    plan = ops.expert_sort(torch.from_numpy(ids).cuda(), E)
    x = spread(torch.Generator().manual_seed(K), T, K, "bf16")
    check_stored(ops.fp8_quantize(x, plan=plan), ref.dispatch(ref.f64(x), ref.sort(ids, E)[1], k))


@pytest.mark.parametrize("kind", ["swiglu", "geglu"])
@pytest.mark.parametrize("M,K,dtype", [(5, 64, "f32"), (33, 1111, "bf16"), (16, 768, "f16"), (2, 33, "f32")])
def test_quantize_after_an_activation(ops, kind, M, K, dtype):
    """The activation is a fp32 evaluation, off by 2^-18 of its magnitude (some
    twenty fp32 operations): a value is between the quantised ends of that
    interval, with the scale of the block's lowest or highest possible largest."""
    g = torch.Generator().manual_seed(M + K)
    x = (2.0 * torch.randn((M, 2 * K), generator=g)).to(DT[dtype]).cuda()
    got = ref.f64(ops.fp8_dequantize(ops.fp8_quantize(x, activation=kind), dtype=torch.float32))
    X = ref.f64(x)
    h = ref.glu(kind, X[:, :K], X[:, K:])
    # gelu's 1 + tanh cancels for negative gates: the error is then of |gate u|
    err = 2.0 ** -18 * (np.abs(h) if kind == "swiglu" else np.abs(X[:, :K] * X[:, K:]))
    ok = np.zeros((M, K), bool)
    nb = -(-K // 128)
    for edge in (np.abs(h) + err, np.maximum(np.abs(h) - err, 0.0)):
        pad = np.zeros((M, nb * 128))
        pad[:, :K] = edge
        big = pad.reshape(M, nb, 128).max(-1)
        e = np.ceil(np.log2(np.maximum(big, 1e-30) / 448.0))
        scale = np.exp2(e).repeat(128, 1)[:, :K]
        ends = []
        for v in (h - err, h + err):
            a = np.minimum(np.abs(v) / scale, 448.0)
            up = np.clip(np.searchsorted(ref8.POSITIVE, a), 1, 126)
            near = np.where(ref8.POSITIVE[up] - a < a - ref8.POSITIVE[up - 1], ref8.POSITIVE[up], ref8.POSITIVE[up - 1])
            ends.append(np.sign(v) * near * scale)
        ok |= (got >= np.minimum(*ends)) & (got <= np.maximum(*ends))
    assert ok.all()
    assert np.mean(got != ref8.quantize(h)[2]) <= 0.01      # almost all of them are the plain form's


# --- products ------------------------------------------------------------------------
def operand(ops, g, shape, scale=1.0, square=False):
    return ops.fp8_quantize((scale * torch.randn(shape, generator=g)).cuda(), square=square)


def check_product(got, a, w, offsets, dtype, transpose=False):
    """got against the stored operands' values in 64 bits."""
    A = ref8.unpack(a.codes.cpu().numpy(), a.scales.cpu().numpy(), a.cols, False)
    codes, scales = w.codes.cpu().numpy(), w.scales.cpu().numpy()
    want, mag = np.zeros(tuple(got.shape)), np.zeros(tuple(got.shape))
    for e in range(len(offsets) - 1):
        W = ref8.unpack(codes[e], scales[e], w.cols, True)
        W = W if transpose else W.T
        rows = slice(offsets[e], offsets[e + 1])
        want[rows] = A[rows] @ W
        mag[rows] = np.abs(A[rows]) @ np.abs(W)
    ref.within(got, want, mag, dtype, a.cols * 2.0 ** -23)


# (R, N, K): tails in every direction, one row, one column, many tiles, few tiles
# whose reduction is shared
DENSE = [(1, 64, 64), (1, 2048, 2048), (3, 1, 32), (128, 192, 256), (129, 193, 257), (100, 65, 1), (300, 500, 544),
         (7, 333, 1111), (200, 31, 4097), (1000, 2000, 96), (2049, 3007, 160), (64, 2880, 2880), (33, 130, 8190), (16, 16, 127),
         (500, 5000, 129), (5000, 200, 640)]


@pytest.mark.parametrize("R,N,K", DENSE)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("transpose", [False, True])
def test_dense_product(ops, R, N, K, dtype, transpose):
    g = torch.Generator().manual_seed(R + N + K)
    a = operand(ops, g, (R, N if transpose else K))
    w = operand(ops, g, (N, K), (N if transpose else K) ** -0.5, True)
    got = ops.fp8_matmul(a, w, transpose=transpose, out_dtype=DT[dtype])
    assert ops.poll_status() == 0
    check_product(got, a, ops.FP8Tensor(w.codes[None], w.scales[None], K, True), [0, R], dtype, transpose)
    assert torch.equal(ops.fp8_matmul(a, w, transpose=transpose, out_dtype=DT[dtype]), got)


# A sum in the tensor core is cut off towards zero, by 2^-25.6 of it an MMA of 32
# values as measured: 1e-6 in one piece of 20000.  32-bit results are summed in
# pieces of 6144 values: off by some 4e-7.
@pytest.mark.parametrize("R", [16, 400, 1000])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("inner", [6144, 6145, 20000])
def test_long_sums_keep_their_precision(ops, R, transpose, inner):
    g = torch.Generator(device="cuda").manual_seed(R + inner)
    N, K = (inner, 1500) if transpose else (1500, inner)
    a = ops.fp8_quantize(torch.randn((R, inner), generator=g, device="cuda"))
    w = ops.fp8_quantize(torch.randn((N, K), generator=g, device="cuda"), square=True)
    A, W = (ops.fp8_dequantize(q, dtype=torch.float32).double() for q in (a, w))
    want = A @ (W if transpose else W.T)
    got = ops.fp8_matmul(a, w, transpose=transpose, out_dtype=torch.float32)
    assert float((got.double() - want).norm()) <= 1e-6 * float(want.norm())


# blocks and rows whose scales differ, from 2^-12 to 2^10 of one another
@pytest.mark.parametrize("R,N,K", [(5, 300, 700), (300, 700, 900), (400, 260, 3000)])
@pytest.mark.parametrize("transpose", [False, True])
def test_scales_of_every_block(ops, R, N, K, transpose):
    g = torch.Generator().manual_seed(R)
    a = ops.fp8_quantize(spread(g, R, N if transpose else K, "f32"))
    w = ops.fp8_quantize(spread(g, N, K, "f32") * torch.exp2(torch.randint(-8, 8, (N, 1), generator=g).float()).cuda(), square=True)
    got = ops.fp8_matmul(a, w, transpose=transpose, out_dtype=torch.float32)
    check_product(got, a, ops.FP8Tensor(w.codes[None], w.scales[None], K, True), [0, R], "f32", transpose)


# (T, E, k, N, K, drop): empty experts, one expert with everything, dropped
# rows, many experts with few rows, several row tiles an expert
GROUPED = [(1, 4, 1, 64, 64, 0.0), (32, 128, 8, 96, 256, 0.0), (50, 3, 2, 200, 160, 0.2), (700, 4, 2, 300, 288, 0.1),
           (33, 1024, 3, 40, 64, 0.0), (9, 2, 1, 128, 512, 1.0), (2000, 5, 2, 2000, 64, 0.05), (2, 8, 2, 640, 2000, 0.0),
           (1100, 6, 2, 1000, 700, 0.1), (3000, 3, 1, 400, 1300, 0.0), (900, 300, 32, 130, 1200, 0.0)]


@pytest.mark.parametrize("T,E,k,N,K,drop", GROUPED)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("transpose", [False, True])
def test_grouped_product(ops, T, E, k, N, K, drop, dtype, transpose):
    rng = np.random.default_rng(T + E)
    ids = routes(rng, T, E, k, drop, skew=3.0)
    plan = ops.expert_sort(torch.from_numpy(ids).cuda(), E)
    g = torch.Generator().manual_seed(N + K)
    inner = N if transpose else K
    w = operand(ops, g, (E, N, K), inner ** -0.5, True)
    a = ops.fp8_quantize(torch.randn((T, inner), generator=g).cuda(), plan=plan)
    got = ops.fp8_matmul(a, w, plan=plan, transpose=transpose, out_dtype=DT[dtype])
    assert ops.poll_status() == 0
    offsets = ref.sort(ids, E)[2]
    check_product(got, a, w, offsets, dtype, transpose)
    assert (got[offsets[-1]:] == 0).all()


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("R,N,K", [(200, 250, 300), (20, 250, 300), (700, 3000, 2500)])
def test_a_nan_stays_in_its_row_and_block(ops, transpose, R, N, K):
    g = torch.Generator().manual_seed(9)
    x, m = torch.randn((R, N if transpose else K), generator=g).cuda(), torch.randn((N, K), generator=g).cuda()
    clean = ops.fp8_matmul(ops.fp8_quantize(x), ops.fp8_quantize(m, square=True), transpose=transpose, out_dtype=torch.float32)
    x[17, 5] = float("nan")
    m[201, 299] = float("inf")      # the block of rows 128 .. 255, columns 256 .. 383
    got = ops.fp8_matmul(ops.fp8_quantize(x), ops.fp8_quantize(m, square=True), transpose=transpose, out_dtype=torch.float32)
    bad = slice(256, min(K, 384)) if transpose else slice(128, min(N, 256))
    assert torch.isnan(got[17]).all() and torch.isnan(got[:, bad]).all()
    rows = torch.arange(R) != 17
    for cols in (slice(0, bad.start), slice(bad.stop, None)):
        assert torch.equal(got[rows][:, cols], clean[rows][:, cols])


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("K", [1, 65, 130, 257, 513, 1111, 2880])
@pytest.mark.parametrize("R,N", [(3, 40), (300, 400), (1500, 2500)])
def test_padding_is_not_used(ops, R, N, K, transpose):
    # NaN codes past the columns and past the rows, NaN scales past the last block
    g = torch.Generator().manual_seed(R + K)
    inner = N if transpose else K
    a, w = operand(ops, g, (R, inner)), operand(ops, g, (N, K), 1.0, True)
    want = ops.fp8_matmul(a, w, transpose=transpose, out_dtype=torch.float32)
    assert torch.isfinite(want).all()

    def poisoned(q, rows):
        codes = torch.full((rows + 300, q.codes.shape[1]), 0x7f, dtype=torch.uint8, device="cuda")
        codes[:rows, :q.cols] = q.codes[:, :q.cols]
        s = q.scales.clone()
        nb = -(-q.cols // 128)
        if not q.square and nb % 4:
            s[-1, :, nb % 4:] = 255
        return ops.FP8Tensor(codes[:rows], s, q.cols, q.square)
    pa, pw = poisoned(a, R), poisoned(w, N)
    assert torch.equal(ops.fp8_matmul(pa, pw, transpose=transpose, out_dtype=torch.float32), want)
    assert torch.equal(ops.fp8_dequantize(pa), ops.fp8_dequantize(a)) and torch.equal(ops.fp8_dequantize(pw), ops.fp8_dequantize(w))


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("n,N,K", [(30, 200, 330), (200, 2500, 2330)])
def test_experts_do_not_read_one_another(ops, transpose, n, N, K):
    # every expert but one holds NaN codes; the rows of that one are as alone
    g = torch.Generator().manual_seed(3)
    w = operand(ops, g, (3, N, K), 1.0, True)
    codes = w.codes.clone()
    codes[0], codes[2] = 0x7f, 0x7f
    a = operand(ops, g, (3 * n, N if transpose else K))
    plan = ops.expert_sort(torch.arange(3, dtype=torch.int32, device="cuda").repeat_interleave(n).unsqueeze(1), 3)
    want = ops.fp8_matmul(a, w, plan=plan, transpose=transpose, out_dtype=torch.float32)
    got = ops.fp8_matmul(a, ops.FP8Tensor(codes, w.scales, K, True), plan=plan, transpose=transpose, out_dtype=torch.float32)
    assert torch.equal(got[n:2 * n], want[n:2 * n]) and torch.isnan(got[:n]).all() and torch.isnan(got[2 * n:]).all()


def test_no_rows(ops):
    q = ops.fp8_quantize(torch.empty((0, 64), device="cuda"))
    assert q.codes.shape == (0, 64) and ops.fp8_dequantize(q).shape == (0, 64)
    w = ops.fp8_quantize(torch.randn((40, 64), device="cuda"), square=True)
    assert ops.fp8_matmul(q, w).shape == (0, 40)
    e = ops.fp8_quantize(torch.empty((3, 0, 64), device="cuda"), square=True)
    assert e.codes.shape == (3, 0, 64) and e.scales.shape == (3, 0, 1) and ops.fp8_dequantize(e).shape == (3, 0, 64)


@pytest.mark.parametrize("R", [3, 300])
def test_on_another_stream_and_in_a_graph(ops, R):
    g = torch.Generator().manual_seed(3)
    x = torch.randn((R, 512), generator=g).cuda()
    w = operand(ops, g, (300, 512), 1.0, True)
    want = ops.fp8_matmul(ops.fp8_quantize(x), w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.fp8_matmul(ops.fp8_quantize(x, stream=side), w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.fp8_matmul(ops.fp8_quantize(x), w)
    x.copy_(torch.randn((R, 512), generator=g))
    graph.replay()
    assert torch.equal(out, ops.fp8_matmul(ops.fp8_quantize(x), w))


@pytest.mark.parametrize("R", [16, 128, 400])
def test_a_wait_that_runs_out_is_reported(ops, R):
    # host-injected: the first copy's barrier is armed and its copy never
    # issued, so the bounded waits on it end by themselves
    from weight_only_quantized_qmoe_gb300 import binding
    g = torch.Generator().manual_seed(4)
    a, w = operand(ops, g, (R, 2048)), operand(ops, g, (2048, 2048), 1.0, True)
    want = ops.fp8_matmul(a, w)
    assert ops.poll_status() == 0
    assert binding.qmoe_op_set_wait_limit(2000) == 0 and binding.qmoe_op_debug_inject_stall(1) == 0
    try:
        ops.fp8_matmul(a, w)
        assert ops.poll_status() == binding.QMOE_ERR_TIMEOUT
        assert ops.poll_status() == 0
    finally:
        binding.qmoe_op_debug_inject_stall(0)
        binding.qmoe_op_set_wait_limit(0)
    assert torch.equal(ops.fp8_matmul(a, w), want) and ops.poll_status() == 0


def test_refusals(ops):
    from weight_only_quantized_qmoe_gb300 import QMoEError, binding
    x = torch.randn((8, 64), device="cuda")
    a, w = ops.fp8_quantize(x), ops.fp8_quantize(torch.randn((2, 16, 64), device="cuda"), square=True)
    plan = ops.expert_sort(torch.zeros((4, 2), dtype=torch.int32, device="cuda"), 2)
    F = ops.FP8Tensor
    bad = [lambda: ops.fp8_quantize(x.cpu()), lambda: ops.fp8_quantize(x.int()), lambda: ops.fp8_quantize(x[0]),
           lambda: ops.fp8_quantize(x, activation="relu"), lambda: ops.fp8_quantize(x[:, :63], activation="swiglu"),
           lambda: ops.fp8_quantize(x, plan=plan), lambda: ops.fp8_quantize(x[:, :0]),
           lambda: ops.fp8_quantize(x, activation="swiglu", square=True), lambda: ops.fp8_quantize(x[:4], plan=plan, square=True),
           lambda: ops.fp8_dequantize(x), lambda: ops.fp8_dequantize(a, dtype=torch.int8),
           lambda: ops.fp8_dequantize(F(a.codes, a.scales, 65, False)), lambda: ops.fp8_dequantize(F(a.codes, a.scales[:0], 64, False)),
           lambda: ops.fp8_dequantize(F(a.codes, a.scales, 64, True)), lambda: ops.fp8_dequantize(F(a.codes, a.scales, 0, False)),
           lambda: ops.fp8_matmul(a, w), lambda: ops.fp8_matmul(a, a), lambda: ops.fp8_matmul(a, F(w.codes, w.scales, 60, True), plan=plan),
           lambda: ops.fp8_matmul(F(a.codes[:4], a.scales[:, :4], 64, False), w, plan=plan),
           lambda: ops.fp8_matmul(a, F(w.codes[0], w.scales[0], 64, True), plan=plan),
           lambda: ops.fp8_matmul(a, w, plan=plan, transpose=True), lambda: ops.fp8_matmul(a, w, plan=plan, out_dtype=torch.int32),
           lambda: ops.fp8_matmul(a, w, plan=plan._replace(offsets=plan.offsets[:2])),
           lambda: ops.fp8_matmul(a, F(w.codes.cpu(), w.scales, 64, True), plan=plan)]
    for call in bad:
        with pytest.raises(QMoEError) as e:
            call()
        assert e.value.status == binding.QMOE_ERR_INVALID_ARG
