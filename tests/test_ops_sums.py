"""Long sums of the 8-bit product and of the weight gradient.

An addition to the tensor core's accumulator cuts off towards zero, so that a sum
falls short by a share that grows with the number of its MMAs.  Sums are therefore
taken in pieces, which are added to nearest in float32."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    from weight_only_quantized_qmoe_gb300 import ops as o
    return o


def shortfall(got, want):
    """By how much `got` is nearer to zero, in parts of the whole: rounding, which
    goes either way, averages out."""
    got, want = got.double(), want.double()
    return float(((want - got) * want.sign()).sum() / want.abs().sum())


# Few rows: as many weight tiles as there are multiprocessors or more (no cluster
# shares a tile), half as many (its CTAs share one), few rows each of many experts.
# 32-bit results go in pieces of 6144 values: 4e-7 short each, and up to 6 roundings of
# 2^-24 of what is there.
@pytest.mark.parametrize("R,width,E", [(16, 9900, 0), (32, 30000, 0), (16, 4900, 0), (5, 3001, 8), (33, 2100, 16), (300, 2100, 16)])
@pytest.mark.parametrize("transpose", [False, True])
def test_long_products_of_few_rows(ops, R, width, E, transpose):
    inner = 36000 if E == 0 and width < 20000 else 20001
    g = torch.Generator(device="cuda").manual_seed(R + width)
    shape = (inner, width) if transpose else (width, inner)
    plan = ops.expert_sort(torch.randint(0, E, (R, 1), generator=g, device="cuda"), E) if E else None
    w = ops.fp8_quantize(torch.randn(((E,) if E else ()) + shape, generator=g, device="cuda", dtype=torch.bfloat16), square=True)
    a = ops.fp8_quantize(torch.randn((R, inner), generator=g, device="cuda"), plan)
    got = ops.fp8_matmul(a, w, plan, transpose=transpose, out_dtype=torch.float32)
    assert ops.poll_status() == 0
    A = ops.fp8_dequantize(a, dtype=torch.float32).double()
    ends = plan.offsets.tolist() if E else [0, R]
    for e, (b, c) in enumerate(zip(ends, ends[1:])):
        if b == c:
            continue
        one = ops.FP8Tensor(w.codes[e], w.scales[e], w.cols, True) if E else w
        W = ops.fp8_dequantize(one, dtype=torch.float32).double()
        want = A[b:c] @ (W if transpose else W.T)
        assert float((got[b:c].double() - want).norm()) <= 1e-6 * float(want.norm()), e
        assert abs(shortfall(got[b:c], want)) <= 6e-7, e
    assert torch.equal(ops.fp8_matmul(a, w, plan, transpose=transpose, out_dtype=torch.float32), got)


# Very many rows, 16-bit results: in pieces of 65536 rows, 4096 MMAs, 8e-5 short; the
# results' own rounding is up to 2^-11 or 2^-8 of each, either way, and is 2^-11 / 100
# or 2^-8 / 100 on the average of ten thousand.  (N, K): few tiles, shared by a
# cluster; more, not shared; pairs of CTAs.
@pytest.mark.parametrize("R,N,K", [(1 << 21, 96, 130), (400_000, 1000, 2500), (400_001, 2100, 2600), (65536, 2100, 2600), (65537, 1000, 2500),
                                   (131_200, 2100, 2600)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_weight_gradients_of_very_many_rows(ops, R, N, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(R + N)
    dy, x = ((0.25 * torch.randn((R, n), generator=g, device="cuda")).to(dtype) for n in (N, K))
    half, most = (2.0 ** -11, 1.3e-4) if dtype == torch.float16 else (2.0 ** -8, 2e-4)

    def close(got, want):
        assert abs(shortfall(got, want)) <= most
        # a value's own rounding, and some ten times what the pieces leave out
        scale = float(want.square().mean().sqrt())
        assert ((got.float() - want).abs() <= half * want.abs() + 1e-3 * scale).all()

    want = ops.weight_grad(dy, x, out_dtype=torch.float32)      # in pieces of 640 rows
    got = ops.weight_grad(dy, x)
    assert ops.poll_status() == 0
    close(got, want)
    assert torch.equal(ops.weight_grad(dy, x), got)
    # a short expert before the long one, one without rows, a short one behind
    rows = torch.arange(R, device="cuda")
    plan = ops.expert_sort((torch.where(rows < 37, 0, 1) + 2 * (rows >= R - 130)).int().unsqueeze(1), 4)
    got, want = (ops.weight_grad(dy, x, plan=plan, out_dtype=t) for t in (dtype, torch.float32))
    assert ops.poll_status() == 0
    assert (got[2] == 0).all()
    for e in (0, 1, 3):
        close(got[e], want[e])
