"""The operators' C entry points refuse what they cannot run, before any device
work (no GPU needed), and say why."""
import pytest

from weight_only_quantized_qmoe_gb300 import binding as b

P = 4096   # an aligned address that no call here gets to use


@pytest.fixture(scope="module", autouse=True)
def lib():
    from weight_only_quantized_qmoe_gb300 import build
    build.build()
    return b.load()


def refused(status, want=b.QMOE_ERR_INVALID_ARG, word=None):
    assert status == want, b.qmoe_op_last_error()
    assert b.qmoe_op_last_error()
    if word:
        assert word in b.qmoe_op_last_error()


def test_sort():
    def call(ids=P, nbytes=4, ld=2, T=8, k=2, E=4, perm=P, pos=P, offsets=P):
        return b.qmoe_expert_sort(ids, nbytes, ld, T, k, E, perm, pos, offsets, None)
    for kw in (dict(ids=0), dict(nbytes=2), dict(ld=1), dict(T=-1), dict(k=0), dict(E=0), dict(perm=0), dict(pos=0),
               dict(offsets=0), dict(T=2 ** 31, k=1, ld=1), dict(T=2 ** 30, k=2)):
        refused(call(**kw))
    refused(call(E=1025), b.QMOE_ERR_UNSUPPORTED, "1024")


def test_rows():
    def there(x=P, ld=16, pos=P, offsets=P, T=8, k=2, E=4, H=16, dt=b.QMOE_BF16, xs=P):
        return b.qmoe_dispatch(x, ld, pos, offsets, T, k, E, H, dt, xs, None)

    def back(y=P, ld=16, w=0, pos=P, T=8, k=2, H=16, dt=b.QMOE_BF16, out=P):
        return b.qmoe_combine(y, ld, w, pos, T, k, H, dt, out, None)

    def grad(dout=P, ld=16, y=P, ldy=16, w=0, pos=P, offsets=P, T=8, k=2, E=4, H=16, dt=b.QMOE_F32, dy=P, dw=P):
        return b.qmoe_combine_grad(dout, ld, y, ldy, w, pos, offsets, T, k, E, H, dt, dy, dw, None)
    for kw in (dict(x=0), dict(ld=15), dict(pos=0), dict(offsets=0), dict(T=-1), dict(k=0), dict(E=0), dict(H=0),
               dict(dt=3), dict(xs=0)):
        refused(there(**kw))
    for kw in (dict(y=0), dict(ld=15), dict(pos=0), dict(T=-1), dict(k=0), dict(H=0), dict(dt=-1), dict(out=0)):
        refused(back(**kw))
    refused(b.qmoe_dispatch_grad(0, 16, P, 8, 2, 16, b.QMOE_F32, P, None))
    for kw in (dict(dout=0), dict(ld=1), dict(y=0), dict(ldy=1), dict(pos=0), dict(offsets=0), dict(dt=9)):
        refused(grad(**kw))
    assert there(T=0) == back(T=0) == grad(T=0) == b.QMOE_OK           # nothing to do
    assert grad(dy=0, dw=0) == b.QMOE_OK


def test_microscaled_rows():
    def quant(x=P, ld=64, rows=8, cols=64, dt=b.QMOE_BF16, act=b.QMOE_ACT_NONE, pos=0, offsets=0, k=1, E=1, panel=8,
              codes=P, scales=P):
        return b.qmoe_mx4_quantize(x, ld, rows, cols, dt, act, pos, offsets, k, E, panel, codes, scales, None)

    def deq(codes=P, scales=P, rows=8, cols=64, panel=8, dt=b.QMOE_BF16, out=P, ld=64):
        return b.qmoe_mx4_dequantize(codes, scales, rows, cols, panel, dt, out, ld, None)

    def mm(ac=P, asc=P, rows=8, wc=P, ws=P, offsets=P, E=2, n=16, k=64, dt=b.QMOE_BF16, out=P, ld=16):
        return b.qmoe_mx4_matmul(ac, asc, rows, wc, ws, offsets, E, n, k, dt, out, ld, None)
    for kw in (dict(x=0), dict(ld=63), dict(rows=-1), dict(cols=0), dict(dt=4), dict(act=b.QMOE_ACT_RELU),
               dict(act=b.QMOE_ACT_SWIGLU), dict(panel=3), dict(panel=0), dict(codes=0), dict(scales=0), dict(codes=P + 8),
               dict(scales=P + 2), dict(pos=P), dict(pos=P, offsets=P, k=0, panel=8), dict(pos=P, offsets=P, k=2, panel=3)):
        refused(quant(**kw))
    for kw in (dict(codes=0), dict(scales=0), dict(out=0), dict(rows=-1), dict(cols=0), dict(panel=5), dict(dt=7),
               dict(ld=63), dict(codes=P + 2)):
        refused(deq(**kw))
    for kw in (dict(ac=0), dict(asc=0), dict(wc=0), dict(ws=0), dict(out=0), dict(rows=-1), dict(E=0), dict(offsets=0),
               dict(n=0), dict(k=0), dict(dt=5), dict(ld=15), dict(ac=P + 8), dict(wc=P + 4), dict(asc=P + 1), dict(ws=P + 2),
               dict(n=2 ** 30, ld=2 ** 30)):
        refused(mm(**kw))
    refused(mm(E=1025), b.QMOE_ERR_UNSUPPORTED, "1024")
    assert quant(rows=0) == deq(rows=0) == mm(rows=0) == b.QMOE_OK


def test_norms():
    def fwd(x=P, ldx=16, o=P, ldo=16, gate=0, kind=0, ldg=0, wq=P, wp=P, scale=1.0, eps=1e-6, T=8, H=16, dt=b.QMOE_F32, r=P,
            h=P):
        return b.qmoe_block_norm(x, ldx, o, ldo, gate, kind, ldg, wq, wp, scale, eps, T, H, dt, r, h, 0, 0, None)

    need = b.qmoe_block_norm_grad_workspace(8, 16, b.QMOE_F32)
    assert need > 0

    def bwd(dr=P, ldr=16, dh=P, ldh=16, x=P, o=P, gate=0, kind=0, wq=P, wp=P, s1=P, s2=P, T=8, H=16, dx=P, do=P, dg=0, dwq=P,
            dwp=P, work=P, nbytes=need):
        return b.qmoe_block_norm_grad(dr, ldr, dh, ldh, x, 16, o, 16, gate, kind, 16, wq, wp, s1, s2, 1.0, T, H, b.QMOE_F32,
                                      dx, do, dg, dwq, dwp, work, nbytes, None)
    for kw in (dict(x=0), dict(ldx=15), dict(o=0), dict(ldo=15), dict(gate=P), dict(kind=2), dict(kind=9, gate=P),
               dict(kind=3, gate=P, ldg=3), dict(scale=float("inf")), dict(eps=-1.0), dict(eps=float("nan")), dict(T=-1),
               dict(H=0), dict(dt=8), dict(h=0), dict(wp=0), dict(r=0, h=0, wp=0)):
        refused(fwd(**kw))
    refused(fwd(H=16385, ldx=16385, ldo=16385), b.QMOE_ERR_UNSUPPORTED, "16384")
    for kw in (dict(ldr=3), dict(ldh=3), dict(wp=0), dict(wq=0), dict(dg=P), dict(s1=0), dict(s2=0), dict(o=0),
               dict(work=0), dict(nbytes=need - 1)):
        refused(bwd(**kw))
    assert fwd(T=0) == b.QMOE_OK
    assert b.qmoe_block_norm_grad_workspace(8, 16385, b.QMOE_F32) == 0
    assert b.qmoe_block_norm_grad_workspace(-1, 16, b.QMOE_F32) == 0


def test_hooks():
    refused(b.qmoe_op_set_wait_limit(-1))
    assert b.qmoe_op_set_wait_limit(0) == b.qmoe_op_debug_inject_stall(0) == b.QMOE_OK
