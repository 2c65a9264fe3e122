"""The C entry points of the router, the 8-bit rows and the weight gradient refuse
what they cannot run, before any device work (no GPU needed), and say why; and
what holds for their sources as text."""
import pytest

from test_ops_abi import P, refused
from test_ops_sources import code
from weight_only_quantized_qmoe_gb300 import binding as b


@pytest.fixture(scope="module", autouse=True)
def lib():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    return b.load()


def test_router():
    def fwd(l=P, ld=16, dt=b.QMOE_F32, bias=0, T=8, E=16, k=2, scoring=0, groups=1, top=1, best=1, scale=1.0, ids=P, w=P):
        return b.qmoe_expert_route(l, ld, dt, bias, T, E, k, scoring, groups, top, best, 1, scale, ids, w, None)

    def bwd(dw=P, l=P, ld=16, dt=b.QMOE_F32, ids=P, T=8, E=16, k=2, scoring=0, scale=1.0, dl=P):
        return b.qmoe_expert_route_grad(dw, l, ld, dt, ids, T, E, k, scoring, 1, scale, dl, None)
    for kw in (dict(l=0), dict(ld=15), dict(dt=3), dict(T=-1), dict(E=0), dict(k=0), dict(k=17), dict(scoring=2), dict(scoring=-1),
               dict(scale=float("inf")), dict(scale=float("nan")), dict(T=2 ** 30), dict(l=P + 2)):
        refused(fwd(**kw))
        refused(bwd(**kw))
    for kw in (dict(ids=0), dict(w=0), dict(groups=0), dict(groups=3), dict(groups=4, top=5), dict(groups=4, top=0), dict(best=0),
               dict(best=3), dict(groups=16, top=2, best=2), dict(groups=8, top=1, k=3), dict(bias=P + 1), dict(ids=P + 2), dict(w=P + 1)):
        refused(fwd(**kw))
    for kw in (dict(dw=0), dict(ids=0), dict(dl=0), dict(dl=P + 2), dict(dw=P + 2)):
        refused(bwd(**kw))
    for call in (fwd, bwd):
        refused(call(E=1025, ld=1025), b.QMOE_ERR_UNSUPPORTED, "1024")
        refused(call(E=64, ld=64, k=33), b.QMOE_ERR_UNSUPPORTED, "32")
        assert call(T=0) == b.QMOE_OK
    refused(fwd(E=64, ld=64, groups=64, top=64), b.QMOE_ERR_UNSUPPORTED, "32")


def test_8_bit_rows():
    def quant(x=P, ld=64, rows=8, cols=64, dt=b.QMOE_BF16, act=b.QMOE_ACT_NONE, pos=0, offsets=0, k=1, E=1, panel=8, square=0,
              codes=P, scales=P):
        return b.qmoe_fp8_quantize(x, ld, rows, cols, dt, act, pos, offsets, k, E, panel, square, codes, scales, None)

    def deq(codes=P, scales=P, rows=8, cols=64, panel=8, square=0, dt=b.QMOE_BF16, out=P, ld=64):
        return b.qmoe_fp8_dequantize(codes, scales, rows, cols, panel, square, dt, out, ld, None)

    def mm(ac=P, asc=P, rows=8, wc=P, ws=P, offsets=P, E=2, n=16, k=64, t=0, dt=b.QMOE_BF16, out=P, ld=64):
        return b.qmoe_fp8_matmul(ac, asc, rows, wc, ws, offsets, E, n, k, t, dt, out, ld, None)
    for kw in (dict(x=0), dict(ld=63), dict(rows=-1), dict(cols=0), dict(cols=2 ** 30, ld=2 ** 30), dict(dt=4), dict(act=b.QMOE_ACT_RELU),
               dict(act=b.QMOE_ACT_SWIGLU), dict(act=b.QMOE_ACT_SWIGLU, ld=128, square=1), dict(panel=3), dict(panel=0), dict(codes=0),
               dict(scales=0), dict(codes=P + 8), dict(scales=P + 2), dict(pos=P), dict(pos=P, offsets=P, k=0),
               dict(pos=P, offsets=P, k=2, panel=3), dict(pos=P, offsets=P, square=1), dict(x=P + 1)):
        refused(quant(**kw))
    for kw in (dict(codes=0), dict(scales=0), dict(out=0), dict(rows=-1), dict(cols=0), dict(panel=5), dict(panel=0), dict(dt=7),
               dict(ld=63), dict(codes=P + 8), dict(out=P + 1)):
        refused(deq(**kw))
    for kw in (dict(ac=0), dict(asc=0), dict(wc=0), dict(ws=0), dict(out=0), dict(rows=-1), dict(E=0), dict(offsets=0), dict(n=0),
               dict(k=0), dict(dt=5), dict(ld=15), dict(t=1, ld=63), dict(ac=P + 8), dict(wc=P + 4), dict(asc=P + 1), dict(offsets=P + 2),
               dict(n=2 ** 30, ld=2 ** 30), dict(rows=2 ** 31 - 256), dict(out=P + 1)):
        refused(mm(**kw))
    refused(mm(E=1025), b.QMOE_ERR_UNSUPPORTED, "1024")
    assert quant(rows=0) == deq(rows=0) == mm(rows=0) == quant(rows=0, square=1) == b.QMOE_OK


def test_weight_gradient():
    def call(dy=P, ldy=16, x=P, ldx=32, offsets=P, rows=8, E=2, n=16, k=32, dt=b.QMOE_BF16, odt=b.QMOE_F32, dw=P, work=0, nbytes=0):
        return b.qmoe_weight_grad(dy, ldy, x, ldx, offsets, rows, E, n, k, dt, odt, dw, work, nbytes, None)
    for kw in (dict(dy=0), dict(x=0), dict(dw=0), dict(ldy=15), dict(ldx=31), dict(offsets=0), dict(rows=-1), dict(E=0), dict(n=0), dict(k=0),
               dict(dt=4), dict(odt=3), dict(odt=-1), dict(ldx=33), dict(ldx=33, work=P, nbytes=8), dict(dy=P + 2), dict(dy=P + 1, work=P, nbytes=1 << 20),
               dict(ldx=33, work=P + 64, nbytes=1 << 20), dict(offsets=P + 1), dict(rows=2 ** 31 - 256), dict(n=2 ** 30, ldy=2 ** 30)):
        refused(call(**kw))
    refused(call(E=1025), b.QMOE_ERR_UNSUPPORTED, "1024")
    refused(call(dt=b.QMOE_F32), b.QMOE_ERR_UNSUPPORTED, "16-bit")
    need = b.qmoe_weight_grad_workspace
    assert need(P, 16, P, 32, 8, 2, 16, 32) == 0 and need(P, 2048, P, 2048, 8, 1, 2048, 2048) == 0
    assert need(P + 2, 16, P, 32, 8, 1, 16, 32) == 8 * 16 * 2 and need(P, 16, P, 33, 8, 1, 16, 31) == 8 * 32 * 2
    assert need(P, 17, P + 8, 32, 8, 1, 16, 30) == 8 * (16 + 32) * 2 and need(P, 17, P, 33, 0, 1, 16, 32) == 0
    assert need(P, 4096, P, 4096, 8, 16, 4096, 4096) == 16 * 256 and need(P, 17, P, 33, 8, 0, 16, 32) == 0


NEW = ["qmoe_choice.cu", "qmoe_fp8.cu", "qmoe_fp8_gemm.cu", "qmoe_wgrad.cu", "qmoe_tile.cuh", "qmoe_tma.cuh"]


@pytest.mark.parametrize("name", NEW)
def test_tensors_are_read_by_coherent_loads(name):
    import re
    found = re.findall(r"__ldg\w*|ld\.global\.nc|ld\.global[\w.:]*\.nc|ld_nc_\w+|ldu\.|__restrict__", code(name))
    assert not found, found


@pytest.mark.parametrize("name", [n for n in NEW if n.endswith(".cu")])
def test_every_kernel_waits_for_the_one_before(name):
    import re
    kernels = re.findall(r"__global__\s+void[\s\S]*?\n}\n", code(name))
    assert kernels
    for k in kernels:
        assert k.count("op_begin();") == 1, k.split("(", 1)[0]
