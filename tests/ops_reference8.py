"""Plain 64-bit forms of the router, the 8-bit rows and the gradient of the
experts' weights (test infrastructure: loops and definitions, none of the
library's code)."""
import numpy as np

# --- the router -------------------------------------------------------------------
def scores(l, scoring):
    """Scores of one token's logits; -inf gives 0."""
    if scoring == "sigmoid":
        return np.array([1.0 / (1.0 + np.exp(-v)) if v > -700 else np.exp(v) for v in l])
    if np.all(np.isneginf(l)):
        return np.zeros_like(l)
    e = np.exp(l - np.max(l))
    return e / e.sum()


def route(logits, k, scoring, bias, groups, top_groups, best, renorm, scale):
    """(ids, weights) token by token; no NaN among the logits."""
    T, E = logits.shape
    ids, weights = np.full((T, k), -1), np.zeros((T, k))
    n = E // groups
    for t in range(T):
        l = logits[t]
        s = scores(l, scoring)
        c = l if bias is None else np.where(np.isneginf(l), -np.inf, s + bias)
        may = ~np.isneginf(c)
        if top_groups < groups:
            by = np.where(may, s, -np.inf) if bias is None and best == 2 else c
            total = []
            for g in range(groups):
                at = sorted((by[e] for e in range(g * n, g * n + n) if may[e]), reverse=True)[:best]
                total.append(sum(at) if at else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-total[g], g))[:top_groups]
            may &= np.isin(np.arange(E) // n, kept)
        order = sorted(np.flatnonzero(may), key=lambda e: (-c[e], e))[:k]
        ids[t, :len(order)] = order
        w = log_weights(l[order], scoring) if renorm else s[order]
        weights[t, :len(order)] = scale * w
    return ids, weights


def log_weights(l, scoring):
    """The chosen scores divided by their sum, by their logarithms."""
    if len(l) == 0:
        return l
    a = l if scoring == "softmax" else -np.logaddexp(0.0, -l)
    e = np.exp(a - a.max())
    return e / e.sum()


def route_grad(dw, logits, ids, scoring, renorm, scale):
    """(dlogits, magnitude of its terms)."""
    out, mag = np.zeros(logits.shape), np.zeros(logits.shape)
    for t in range(len(logits)):
        l = logits[t]
        s = scores(l, scoring)
        slots = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < len(l)]
        if not slots:
            continue
        js, es = np.array(slots).T
        g = scale * dw[t, js]
        if renorm:
            u = log_weights(l[es], scoring)
            mean, amean = (g * u).sum(), (np.abs(g) * u).sum()
            f = u * (1.0 if scoring == "softmax" else 1.0 - s[es])
            d, m = f * (g - mean), f * (np.abs(g) + amean)
        elif scoring == "sigmoid":
            d = g * s[es] * (1.0 - s[es])
            m = np.abs(d)
        else:
            all_, aall = (g * s[es]).sum(), (np.abs(g) * s[es]).sum()
            out[t] -= s * all_
            mag[t] += s * aall
            d, m = g * s[es], np.abs(g) * s[es]
        for e, x, y in zip(es, d, m):
            out[t, e] += x
            mag[t, e] += y
    return out, mag


# --- 8-bit rows -------------------------------------------------------------------
# the value of every code; 0x7f and 0xff are NaN
E4M3 = np.array([(-1.0 if c & 128 else 1.0) * ((8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10) if c >> 3 & 15 else (c & 7) * 2.0 ** -9)
                 if c & 127 != 127 else np.nan for c in range(256)])
POSITIVE = E4M3[:127]


def blocks(x, square):
    """x [M, K] as [rows of blocks, columns of blocks, rows, 128], zeros outside."""
    M, K = x.shape
    r = 128 if square else 1
    v = np.zeros((-(-M // r) * r, -(-K // 128) * 128))
    v[:M, :K] = x
    return v.reshape(v.shape[0] // r, r, v.shape[1] // 128, 128).transpose(0, 2, 1, 3)


def quantize(x, square=False):
    """Codes [M, K], scale bytes [rows of blocks, columns of blocks] and values
    [M, K] of x [M, K]."""
    M, K = x.shape
    v = blocks(x, square)
    big = np.abs(v).max((2, 3))
    bad = ~np.isfinite(big)
    byte = np.zeros(big.shape, int)
    for i in np.ndindex(big.shape):
        if bad[i]:
            byte[i] = 255
            continue
        e = int(np.frexp(big[i] / 448.0)[1]) - 2 if big[i] > 0 else -127     # below the answer, or it
        while 448.0 * 2.0 ** e < big[i]:
            e += 1
        byte[i] = max(e, -127) + 127
    scale = np.ldexp(1.0, np.where(bad, 0, byte - 127))[..., None, None]
    a = np.where(bad[..., None, None], 0.0, v) / scale
    up = np.clip(np.searchsorted(POSITIVE, np.abs(a)), 1, 126)
    lo, hi = np.abs(a) - POSITIVE[up - 1], POSITIVE[up] - np.abs(a)
    code = np.where((hi < lo) | ((hi == lo) & (up % 2 == 0)), up, up - 1)    # ties to the even code
    code = code | np.where(np.signbit(a), 128, 0)
    value = np.where(bad[..., None, None], np.nan, E4M3[code] * scale)

    def rows(t):
        return t.transpose(0, 2, 1, 3).reshape(t.shape[0] * t.shape[2], -1)[:M, :K]
    return rows(code), byte, rows(value)


def pack(code, byte):
    """The stored form of codes [M, K] and the scale bytes of rows [M, nb]."""
    M, K = code.shape
    stored = np.zeros((M, -(-K // 16) * 16), np.uint8)
    stored[:, :K] = code
    return stored, pack_scales(byte)


def pack_scales(byte):
    M, nb = byte.shape
    sc = np.zeros((M, -(-nb // 4) * 4), np.uint8)
    sc[:, :nb] = byte
    return np.ascontiguousarray(sc.reshape(M, -1, 4).transpose(1, 0, 2))


def unpack(codes, scales, cols, square):
    """Values [M, cols] of stored codes and scales of one matrix."""
    M, nb = codes.shape[0], -(-cols // 128)
    byte = np.repeat(scales, 128, 0)[:M] if square else scales.transpose(1, 0, 2).reshape(M, -1)[:, :nb]
    scale = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(int) - 127))
    return E4M3[codes[:, :cols]] * np.repeat(scale, 128, 1)[:, :cols]


# --- weight gradient ----------------------------------------------------------------
def weight_grad(dy, x, offsets):
    """(dw, magnitude of its terms)."""
    dw = [dy[b:e].T @ x[b:e] for b, e in zip(offsets, offsets[1:])]
    mag = [np.abs(dy[b:e].T) @ np.abs(x[b:e]) for b, e in zip(offsets, offsets[1:])]
    return np.stack(dw), np.stack(mag)
