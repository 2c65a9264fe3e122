"""Plain 64-bit forms of the operators around the expert layer (test
infrastructure: loops and definitions, none of the library's code)."""
import numpy as np

UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # half a unit in the last place, relative
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}  # the smallest subnormal
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def sort(ids, E):
    """(perm, pos, offsets) by walking the experts."""
    ids = np.asarray(ids).reshape(-1)
    R = len(ids)
    perm, pos, offsets = np.full(R, -1), np.full(R, -1), [0]
    n = 0
    for e in range(E):
        for r in np.flatnonzero(ids == e):
            perm[n], pos[r] = r, n
            n += 1
        offsets.append(n)
    return perm, pos, np.array(offsets)


def dispatch(x, pos, k):
    xs = np.zeros((len(pos), x.shape[1]))
    kept = np.flatnonzero(pos >= 0)
    xs[pos[kept]] = x[kept // k]
    return xs


def combine(y, w, pos, k):
    """(out, sum of the magnitudes of its terms)."""
    T = len(pos) // k
    w = np.ones(len(pos)) if w is None else w.reshape(-1)
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for r, p in enumerate(pos):
        if p >= 0:
            out[r // k] += w[r] * y[p]
            mag[r // k] += np.abs(w[r] * y[p])
    return out, mag


def combine_grad(dout, y, w, pos, k):
    """(dy, dw, magnitudes of dw's sums)."""
    w = np.ones(len(pos)) if w is None else w.reshape(-1)
    dy, dw, mag = np.zeros(y.shape), np.zeros(len(pos)), np.zeros(len(pos))
    for r, p in enumerate(pos):
        if p >= 0:
            dy[p] = w[r] * dout[r // k]
            dw[r] = np.dot(dout[r // k], y[p])
            mag[r] = np.dot(np.abs(dout[r // k]), np.abs(y[p]))
    return dy, dw.reshape(-1, k), mag.reshape(-1, k)


def quantize(x):
    """Codes (sign in bit 3) [M, 32 nb], scale bytes [M, nb] and values [M, K] of
    rows x [M, K]: every element compared with every E2M1 value."""
    M, K = x.shape
    nb = -(-K // 32)
    v = np.zeros((M, nb * 32))
    v[:, :K] = x
    v = v.reshape(M, nb, 32)
    big = np.max(np.abs(v), axis=2)
    bad = ~np.isfinite(big)
    exp = np.frexp(np.where(bad | (big == 0), 1.0, big))[1] - 1        # floor(log2), exactly
    byte = np.clip(exp - 2 + 127, 0, 254)
    byte = np.where(big == 0, 0, byte)
    scale = np.ldexp(1.0, byte - 127)
    a = np.abs(np.where(bad[..., None], 0.0, v)) / scale[..., None]
    dist = np.abs(np.minimum(a, 6.0)[..., None] - E2M1)
    # nearest, ties to the even code: odd codes lose a tie
    code = np.argmin(dist + np.where(np.arange(8) % 2, 1e-9, 0.0), axis=-1)
    sign = np.signbit(np.where(bad[..., None], 0.0, v)).astype(int)
    byte = np.where(bad, 255, byte)
    values = np.where(bad[..., None], np.nan, np.where(sign, -1.0, 1.0) * E2M1[code] * scale[..., None])
    return (code | sign << 3).reshape(M, -1), byte, values.reshape(M, -1)[:, :K]


def pack(code, byte):
    """The stored form of codes [M, 32 nb] and scale bytes [M, nb]: (codes,
    scales [ceil(nb / 4), M, 4])."""
    M, nb = byte.shape
    stored = (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8)
    nq = -(-nb // 4)
    sc = np.zeros((M, nq * 4), np.uint8)
    sc[:, :nb] = byte
    return stored, np.ascontiguousarray(sc.reshape(M, nq, 4).transpose(1, 0, 2))


def unpack(codes, scales, cols):
    """Values [M, cols] of stored codes [M, 16 nb] and scales [nq, M, 4]."""
    M, nb = codes.shape[0], codes.shape[1] // 16
    code = np.stack([codes & 15, codes >> 4], -1).reshape(M, nb, 32)
    byte = scales.transpose(1, 0, 2).reshape(M, -1)[:, :nb].astype(int)
    val = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7] * np.ldexp(1.0, byte - 127)[..., None]
    return np.where(byte[..., None] == 255, np.nan, val).reshape(M, -1)[:, :cols]


def sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


def glu(kind, g, u):
    if kind == "swiglu":
        return g * sigmoid(g) * u
    return 0.5 * g * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3))) * u


def norm(x, o, gate, wq, wp, scale, eps):
    """Forward in 64 bits: r, h, the magnitudes of r's two terms."""
    if o is None:
        n = np.zeros_like(x)
    elif wq is None:
        n = o
    else:
        n = o / np.sqrt((o * o).mean(-1, keepdims=True) + eps) * wq
    g = 1.0 if gate is None else gate
    r = scale * x + g * n
    h = None if wp is None else r / np.sqrt((r * r).mean(-1, keepdims=True) + eps) * wp
    return r, h, np.abs(scale * x) + np.abs(g * n)


def norm_grad(dr, dh, x, o, gate, wq, wp, scale, eps):
    """The gradients by the formula, each with the sum of the magnitudes of
    its terms: {name: (value, magnitude)}."""
    T, H = x.shape
    g = np.ones((1, 1)) if gate is None else gate.reshape((1, H) if gate.ndim == 1 else gate.shape)
    if o is None:
        s1, oh, n = 1.0, np.zeros_like(x), np.zeros_like(x)
    elif wq is None:
        s1, oh, n = 1.0, o, o
    else:
        s1 = 1.0 / np.sqrt((o * o).mean(1, keepdims=True) + eps)
        oh = o * s1
        n = oh * wq
    r = scale * x + g * n
    d, dm = (np.zeros_like(x), np.zeros_like(x)) if dr is None else (dr.copy(), np.abs(dr))
    out = {}
    if wp is not None and dh is not None:
        s2 = 1.0 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
        rm = (np.abs(scale * x) + np.abs(g * n)) * s2
        rh = r * s2
        dn = dh * wp
        d = d + s2 * (dn - rh * (dn * rh).mean(1, keepdims=True))
        dm = dm + s2 * (np.abs(dn) + rm * np.abs(dn * rm).mean(1, keepdims=True))
        out["w_pre"] = ((dh * rh).sum(0), np.abs(dh * rm).sum(0))
    elif wp is not None:
        out["w_pre"] = (np.zeros(H), np.zeros(H))
    out["x"] = (scale * d, np.abs(scale) * dm)
    if o is None:
        return out
    if gate is not None:
        dg, dgm = d * n, dm * np.abs(n)
        if gate.ndim == 1:
            dg, dgm = dg.sum(0), dgm.sum(0)
        elif gate.shape != x.shape:
            dg, dgm = dg.sum(1, keepdims=True), dgm.sum(1, keepdims=True)
        out["gate"] = (dg, dgm)
    d1, d1m = d * g, dm * np.abs(g)
    if wq is None:
        out["o"] = (d1, d1m)
        return out
    out["w_post"] = ((d1 * oh).sum(0), (d1m * np.abs(oh)).sum(0))
    d2, d2m = d1 * wq, d1m * np.abs(wq)
    out["o"] = (s1 * (d2 - oh * (d2 * oh).mean(1, keepdims=True)),
                s1 * (d2m + np.abs(oh) * (d2m * np.abs(oh)).mean(1, keepdims=True)))
    return out


def within(got, want, mag, dtype, rel):
    """Every element of got within the rounding of its type of want, plus rel
    times the magnitude of the terms it was summed from; the same infinities
    and NaN."""
    got, want = f64(got) if not isinstance(got, np.ndarray) else got, np.asarray(want)
    assert got.shape == want.shape, (got.shape, want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine)
    tol = UNIT[dtype] * np.abs(want) + TINY[dtype] + rel * (1 + UNIT[dtype]) * np.broadcast_to(mag, want.shape)
    err = np.abs(got - want)
    worst = np.max(np.where(fine, err - tol, -1.0), initial=-1.0)
    assert worst <= 0.0, f"past the bound by {worst:.3e}; largest error {np.max(err[fine], initial=0.0):.3e}"
