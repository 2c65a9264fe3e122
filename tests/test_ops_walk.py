"""More rows than are under way at once: CTAs that walk their rows through a ring
or without one, several rows a CTA, sums kept from row to row, rows on any
boundary, in every kernel that does so, against the plain 64-bit forms.

Bounds of the norms as in test_ops_norm, but for the sums over the rows: a thread
adds the rows it walks one after another, at least 152 slices of rows side by
side (a slice is a row of a CTA; 512 threads a multiprocessor or more, 152 of
them), then 16 or 32 threads add every 16th or 32nd slice and their sums follow
in order.  At most 512 threads / 8 a row = 64 rows a multiprocessor are under way:
9728 slices, 304 a thread.  So a sum has at most T / 152 + 304 + 32 additions one
after another."""
import numpy as np
import pytest
import torch

import ops_reference as ref
from test_ops_mx4 import check_stored, spread
from test_ops_norm import EPS, GREL, amplification, check_forward, inputs, ops  # noqa: F401
from test_ops_routes import DT, routes

pytestmark = pytest.mark.gpu


def check_grads(got, v, scale, dtype):
    a = {n: ref.f64(v.get(n)) for n in ("dr", "dh", "x", "o", "gate", "w_post", "w_pre")}
    want = ref.norm_grad(a["dr"], a["dh"], a["x"], a["o"], a["gate"], a["w_post"], a["w_pre"], scale, EPS)
    T, H = v["x"].shape
    amp = amplification(a, scale, EPS)
    for name in ("x", "o", "gate", "w_post", "w_pre"):
        g = getattr(got, name)
        if name not in want:
            assert g is None, name
            continue
        w, mag = want[name]
        summed = name in ("w_post", "w_pre") or (name == "gate" and a["gate"].shape != (T, H))
        terms = T / 152 + 336 + (H if name == "gate" else 0) if summed else 0
        ref.within(g, w, mag, dtype, (GREL + terms * 2.0 ** -24) * amp)


def check(ops, v, scale, dtype):  # noqa: F811
    fwd = {n: v[n] for n in ("x", "o", "gate", "w_post", "w_pre")}
    _, _, stats = check_forward(ops, **fwd, scale=scale, dtype=dtype)
    got = ops.block_norm_grad(v["dr"], v["dh"], v["x"], v["o"], stats, gate=v["gate"], w_post=v["w_post"],
                              w_pre=v["w_pre"], residual_scale=scale)
    check_grads(got, v, scale, dtype)


# (rows, length, type): one to eight fragments a thread, aligned and not; sixteen
# rows a CTA at length 40.  The gradients have 152 CTAs of 512 threads or as many
# threads in smaller ones, the forward up to 2048 threads a multiprocessor.
WALKS = [(20000, 40, "f16"), (12000, 41, "f32"), (2600, 1001, "f32"), (2600, 1001, "bf16"), (2600, 2048, "bf16"),
         (1000, 2501, "f32"), (700, 2501, "f16"), (700, 4096, "bf16"), (400, 4099, "f32"), (400, 5001, "bf16"),
         (700, 8192, "bf16"), (330, 8191, "f32"), (330, 8192, "f32"), (310, 16383, "bf16"), (310, 16384, "f16"),
         (310, 16383, "f32"), (310, 16384, "f32")]


@pytest.mark.parametrize("T,H,dtype", WALKS)
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
def test_norms_and_gradients(ops, T, H, dtype, gate):  # noqa: F811
    check(ops, inputs(T, H, dtype, gate), 0.7, dtype)


@pytest.mark.parametrize("T,H,dtype", [(2600, 1001, "f32"), (2600, 2048, "bf16"), (700, 8192, "bf16"), (700, 4097, "f16")])
@pytest.mark.parametrize("absent", ["w_post", "w_pre", "dr", "dh", "o"])
def test_norms_with_an_argument_absent(ops, T, H, dtype, absent):  # noqa: F811
    v = inputs(T, H, dtype, "channel")
    v[absent] = None
    if absent == "o":
        v["gate"] = v["w_post"] = None
    if absent == "w_pre":
        v["dh"] = None
    check(ops, v, -1.3, dtype)


@pytest.mark.parametrize("T,H", [(30, 128), (1300, 1000)])
@pytest.mark.parametrize("dtype", list(DT))
def test_norm_gradients_of_strided_rows(ops, T, H, dtype):  # noqa: F811
    g = torch.Generator().manual_seed(T)
    wide = [torch.randn((T, 2 * H + 9), generator=g).to(DT[dtype]).cuda() for _ in range(5)]
    w = (1 + 0.1 * torch.randn(2 * H + 1, generator=g)).to(DT[dtype]).cuda()
    cuts = [slice(0, H), slice(1, H + 1), slice(3, H + 3), slice(0, 2 * H, 2), slice(H, 2 * H)]
    for turn in range(5):     # every tensor in every position
        x, o, gate, dr, dh = (wide[i][:, cuts[(i + turn) % 5]] for i in range(5))
        check(ops, dict(x=x, o=o, gate=gate, dr=dr, dh=dh, w_post=w[turn % 2:H + turn % 2], w_pre=w[H:2 * H]), 0.9, dtype)
    x, o, gate, dr, dh = (t[:, :H] for t in wide)
    one = wide[0][:1, :H].expand(T, H)      # a broadcast row
    check(ops, dict(x=one, o=o, gate=gate, dr=dr, dh=one, w_post=w[:H], w_pre=w[H:2 * H]), 0.9, dtype)


# a warp that takes two steps of its row: rows of more than 2048 values, or so
# many rows that each multiprocessor has its 32 warps
QUANT = [(40, 2881), (9, 4127), (2500, 1111), (3, 5003)]


@pytest.mark.parametrize("M,K", QUANT)
@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_and_back(ops, M, K, dtype):  # noqa: F811
    x = spread(torch.Generator().manual_seed(M * 7 + K), M, K, dtype)
    q = ops.mx4_quantize(x)
    check_stored(q, ref.f64(x))
    _, _, values = ref.quantize(ref.f64(x))
    for out in DT:
        assert torch.equal(ops.mx4_dequantize(q, dtype=DT[out]).cpu(), torch.from_numpy(values).to(DT[out]))


@pytest.mark.parametrize("T,E,k,K,drop", [(37, 5, 3, 2881, 0.3), (600, 16, 4, 1111, 0.1), (20, 40, 35, 2100, 0.2)])
def test_quantize_into_expert_order(ops, T, E, k, K, drop):  # noqa: F811
    ids = routes(np.random.default_rng(T + K), T, E, k, drop)
    plan = ops.expert_sort(torch.from_numpy(ids).cuda(), E)
    x = spread(torch.Generator().manual_seed(K), T, K, "f16")
    check_stored(ops.mx4_quantize(x, plan=plan), ref.dispatch(ref.f64(x), ref.sort(ids, E)[1], k))


@pytest.mark.parametrize("kind", ["swiglu", "geglu"])
@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_after_an_activation_by_rows(ops, kind, dtype):  # noqa: F811
    # a row quantised among many, in several steps, is the row quantised alone
    g = torch.Generator().manual_seed(4)
    x = (2.0 * torch.randn((33, 2 * 2881), generator=g)).to(DT[dtype]).cuda()
    q = ops.mx4_quantize(x, activation=kind)
    for i in (0, 1, 17, 32):
        one = ops.mx4_quantize(x[i:i + 1].clone(), activation=kind)
        assert torch.equal(q.codes[i], one.codes[0]) and torch.equal(q.scales[:, i], one.scales[:, 0])
    h = ops.mx4_dequantize(q, dtype=torch.float32)
    X = ref.f64(x)
    plain = ref.quantize(ref.glu(kind, X[:, :2881], X[:, 2881:]))[2]
    # a value beside a rounding point may take the neighbouring element: one in
    # a hundred at most, as the activation is off by 2^-18 of its size
    assert np.mean(ref.f64(h) != plain) <= 0.01


# --- the scales of a product, in place ---------------------------------------------
@pytest.mark.parametrize("E,R,N,K", [(1, 70, 100, 320), (1, 33, 65, 96), (3, 131, 193, 640), (5, 40, 31, 1111), (2, 257, 64, 160)])
def test_scales_inside_larger_buffers(ops, E, R, N, K):  # noqa: F811
    """R and N off the 32 rows of a copy, an odd number of 128-value panels and
    the last panel of the last expert, with NaN scales on either side: the same
    bits.  (That shows that no such byte reaches a result; a row past a matrix
    that is read and not used would not show.)"""
    g = torch.Generator().manual_seed(R + N)
    ids = torch.randint(0, E, (R, 1), generator=g).to(torch.int32).cuda()
    plan = ops.expert_sort(ids, E)
    a = ops.mx4_quantize(torch.randn((R, K), generator=g).cuda())
    w = ops.mx4_quantize(torch.randn((E, N, K), generator=g).cuda())
    want = ops.mx4_matmul(a, w, plan=plan, out_dtype=torch.float32)

    def inside(q):
        buf = torch.full((q.scales.numel() + 8192,), 255, dtype=torch.uint8, device="cuda")
        buf[4096:4096 + q.scales.numel()] = q.scales.reshape(-1)
        return ops.MX4Tensor(q.codes, buf[4096:4096 + q.scales.numel()].reshape(q.scales.shape), K)

    assert torch.equal(ops.mx4_matmul(inside(a), inside(w), plan=plan, out_dtype=torch.float32), want)
    assert ops.poll_status() == 0
    at = plan.offsets.tolist()
    A = ref.unpack(a.codes.cpu().numpy(), a.scales.cpu().numpy(), K)
    for e in range(E):
        W = ref.unpack(w.codes[e].cpu().numpy(), w.scales[e].cpu().numpy(), K)
        rows = slice(at[e], at[e + 1])
        ref.within(ref.f64(want)[rows], A[rows] @ W.T, np.abs(A[rows]) @ np.abs(W.T), "f32", K * 2.0 ** -23)
