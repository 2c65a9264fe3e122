"""The router and the 8-bit expert products, as cases to be timed and compared.

* the router (``route``): softmax or sigmoid scores, a bias that balances the choice, groups of experts, the best k, renormalised weights,
  and in training the gradient of the logits;
* 8-bit floating point with a power-of-two scale for each block of 128 (``rows``: 128 values of a row, ``blocks``: 128 x 128 of a weight),
  quantised and read back;
* its product with expert weights (``product``), also with the weights transposed, which is the gradient of the rows;
* the gradient of the experts' weights (``wgrad``): for each expert the sum over its rows of the outer products;
* the linear layer made of them, forward and backward (``linear``).

``run`` computes a case with elementary torch operations in 32 bits (the router's choice in 64), or with the framework's kernels where
``own`` is true; ``exact`` computes it from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
LOWEST = float("-inf")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of a decode step chooses eight of the many-expert layer's 128: latency
        dict(name="route_token", kind="route", train=False, T=1, E=128, k=8, dtype="f32", scoring="softmax", bias=False, groups=1,
             top_groups=1, best=1, renorm=True, mask=0.0),
        # a training step's tokens, eight of 256 experts in four of eight groups, chosen with a balance bias; and the gradient
        dict(name="route_train", kind="route", train=True, T=8192, E=256, k=8, dtype="f32", scoring="sigmoid", bias=True, groups=8,
             top_groups=4, best=2, renorm=True, mask=0.0),
        # activations with rows of odd length quantised and read back
        dict(name="rows_odd", kind="rows", M=2880, K=4127, dtype="bf16"),
        # master weights of eight experts quantised at load, with a last block of one row and half a block of columns
        dict(name="blocks_weights", kind="blocks", E=8, N=1537, K=2880, dtype="f32"),
        # one token through a projection of the decode layer's size: weights streamed once, latency
        dict(name="product_token", kind="product", back=False, T=1, E=1, k=1, N=2048, K=2048, dtype="bf16", out="bf16"),
        # 32 tokens to eight of 128 experts: two rows an expert, every expert's weights read
        dict(name="product_decode", kind="product", back=False, T=32, E=128, k=8, N=1536, K=2048, dtype="bf16", out="bf16"),
        # the prefill layer's second projection: tokens quantised into expert order, then the grouped product
        dict(name="product_prefill", kind="product", back=False, T=4096, E=64, k=8, N=4096, K=1536, dtype="bf16", out="bf16"),
        # the gradient of the rows of one dense projection with ragged sizes on every side and a 32-bit result
        dict(name="product_back", kind="product", back=True, T=2001, E=1, k=1, N=5761, K=2880, dtype="f16", out="f32"),
        # the weight gradient of the prefill layer's second projection
        dict(name="wgrad_prefill", kind="wgrad", T=4096, E=64, k=8, N=4096, K=1536, dtype="bf16", out="bf16"),
        # few experts, odd lengths on every side, a 32-bit result
        dict(name="wgrad_odd", kind="wgrad", T=1001, E=7, k=3, N=1001, K=513, dtype="f16", out="f32"),
        # a training step of one projection of 16 experts, forward and backward, at the mixed-width layer's width
        dict(name="linear_train", kind="linear", T=2000, E=16, k=4, N=2880, K=2048, dtype="bf16", wdtype="bf16"),
        # a small dense layer with odd lengths and 32-bit master weights, forward and backward
        dict(name="linear_odd", kind="linear", T=777, E=1, k=1, N=1001, K=513, dtype="f16", wdtype="f32"),
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row length: often a multiple of 64 as weights have it, else any."""
    n = _between(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.6 else n


def draw(rng):
    while True:
        kind = rng.choice(["route", "route", "rows", "blocks", "product", "product", "wgrad", "linear"])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        half = rng.choice(["bf16", "bf16", "f16"])
        E = rng.choice([1, _between(rng, 2, 128)])
        k = rng.randint(1, min(E, 8))
        if kind == "route":
            groups = rng.choice([1, 1, 2, 4, 8])
            E = groups * _between(rng, 2, 512 // groups)
            top_groups = rng.randint(1, groups)
            case = dict(kind=kind, train=rng.random() < 0.5, T=_between(rng, 1, 8192), E=E, k=rng.randint(1, min(E // groups * top_groups, 16)),
                        dtype=dtype, scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                        top_groups=top_groups, best=rng.randint(1, 2), renorm=rng.random() < 0.6, mask=rng.choice([0.0, 0.0, 0.3]))
            fits = case["T"] * E <= 8192 * 256
        elif kind == "rows":
            case = dict(kind=kind, M=_between(rng, 1, 16384), K=_width(rng, 64, 8192), dtype=dtype)
            fits = case["M"] * case["K"] <= 3.0e7
        elif kind == "blocks":
            case = dict(kind=kind, E=rng.randint(1, 16), N=_width(rng, 64, 6144), K=_width(rng, 64, 6144), dtype=dtype)
            fits = case["E"] * case["N"] * case["K"] <= 3.5e7
        else:
            case = dict(kind=kind, T=_between(rng, 1, 4096), E=E, k=k, N=_width(rng, 64, 6144), K=_width(rng, 64, 6144),
                        dtype=dtype if kind == "product" else half)
            if kind == "product":
                case.update(back=rng.random() < 0.4, out=rng.choice(["bf16", "f16", "f32"]))
            elif kind == "wgrad":
                case.update(out=rng.choice([half, "f32"]))
            else:
                case.update(wdtype=rng.choice([half, "f32"]))
            w = work(case)
            fits = w["flops"] <= 4.0e11 and w["bytes"] <= 1.0e9 and E * case["N"] * case["K"] <= 4.0e8
        if fits:
            return case


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    kind = case["kind"]
    if kind == "route":
        T, E, k, d = case["T"], case["E"], case["k"], _size(case["dtype"])
        n = T * E * d + (4 * E if case["bias"] else 0) + 8 * T * k
        if case["train"]:
            n += T * E * d + 4 * T * k       # the gradient of the weights read, of the logits written
        return {"bytes": n, "flops": T * E * (10 if case["train"] else 5)}
    if kind in ("rows", "blocks"):
        n = case["M"] * case["K"] if kind == "rows" else case["E"] * case["N"] * case["K"]
        return {"bytes": n * (_size(case["dtype"]) + 2 + 2), "flops": 4 * n}     # read; codes written and read; 16-bit values written
    T, E, k, N, K, d = case["T"], case["E"], case["k"], case["N"], case["K"], _size(case["dtype"])
    R, used = T * k, min(E, T * k)
    if kind == "product":
        into, out = (N, K) if case["back"] else (K, N)
        return {"bytes": T * into * d + used * N * K + R * out * _size(case["out"]), "flops": 2 * R * N * K}
    if kind == "wgrad":
        return {"bytes": R * (N + K) * d + E * N * K * _size(case["out"]), "flops": 2 * R * N * K}
    return {"bytes": R * (2 * N + 2 * K) * d + (used + E) * N * K * _size(case["wdtype"]), "flops": 6 * R * N * K}


def _size(dtype):
    return 4 if dtype == "f32" else 2


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    kind, dt = case["kind"], DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def wide(*shape):
        """A wide spread of magnitudes from row to row, as weights and activations have it."""
        spread = torch.exp2(torch.randn(shape[:-1] + (1,), generator=g, device="cuda") * 2.0)
        return (normal(*shape, dtype=torch.float32) * spread * 0.02).to(dt)

    s = dict(case)
    if kind == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # router logits with a mild preference for the lower experts
        lean = 0.3 * torch.log(1.0 / (1.0 + torch.arange(E, device="cuda")))
        s["logits"] = (1.5 * torch.randn((T, E), generator=g, device="cuda") + lean).to(dt)
        if case["mask"]:   # experts that a token may not use; some tokens (padding) none at all
            closed = torch.rand((T, E), generator=g, device="cuda") < case["mask"]
            closed |= (torch.arange(T, device="cuda") % 97 == 5).unsqueeze(1)
            s["logits"] = torch.where(closed, LOWEST, s["logits"]).to(dt)
        s["b"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        s["dw"] = normal(T, k, dtype=torch.float32, scale=0.1) if case["train"] else None
        return s
    if kind == "rows":
        s["x"] = wide(case["M"], case["K"])
        return s
    if kind == "blocks":
        s["x"] = wide(case["E"], case["N"], case["K"])
        return s
    T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
    choice = torch.randn((T, E), generator=g, device="cuda") + 0.3 * torch.log(1.0 / (1.0 + torch.arange(E, device="cuda")))
    s["perm"], s["pos"], s["offsets"] = _sort(torch.topk(choice, k, dim=1).indices, E)
    s["most_rows"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())   # the capacity a padded batch needs
    if kind == "wgrad":
        s["x"], s["dy"] = normal(T * k, K), normal(T * k, N, scale=0.1)
        return s
    if kind == "linear":
        s["x"] = normal(T * k, K).requires_grad_()
        s["w"] = normal(E, N, K, dtype=DTYPES[case["wdtype"]], scale=K ** -0.5).requires_grad_()
        s["dy"] = normal(T * k, N, scale=0.1)
        return s
    s["x"] = normal(T, N if case["back"] else K)
    codes, scales = [], []
    for _ in range(E):   # an expert at a time: the 32-bit weights need not fit at once
        c, e = _codes(normal(N, K, dtype=torch.float32, scale=K ** -0.5), True)
        codes.append(torch.nn.functional.pad(c.view(torch.uint8), (0, -K % 16)))
        scales.append((e + 127).to(torch.uint8))
    s["w_codes"], s["w_scales"] = torch.stack(codes), torch.stack(scales)
    return s


# ---------------------------------------------------------------------------
# Plain forms: elementary operations in 32 bits, the router's choice in 64
# ---------------------------------------------------------------------------
def _sort(ids, E):
    key = ids.reshape(-1).long()
    order = torch.sort(key, stable=True).indices
    pos = torch.empty_like(key)
    pos[order] = torch.arange(key.numel(), device=key.device)
    offsets = torch.zeros(E + 1, dtype=torch.long, device=key.device)
    offsets[1:] = torch.cumsum(torch.zeros(E, dtype=torch.long, device=key.device).index_add_(0, key, torch.ones_like(key)), 0)
    return order.to(torch.int32), pos.to(torch.int32), offsets.to(torch.int32)


def _plain_route(s):
    T, E, k, G, dt = s["T"], s["E"], s["k"], s["groups"], s["logits"].dtype
    l = s["logits"].double()
    closed = l == LOWEST
    if s["scoring"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True).clamp(min=-1e300))
        score = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    c = l if s["b"] is None else torch.where(closed, LOWEST, score + s["b"].double())
    if G > 1 and s["top_groups"] < G:
        by = (torch.where(closed, LOWEST, score) if s["b"] is None and s["best"] == 2 else c).reshape(T, G, -1)
        two = torch.sort(by, dim=2, descending=True).values[:, :, :s["best"]]
        more = two[:, :, 1:]
        group = two[:, :, 0] + torch.where(more == LOWEST, 0.0, more).sum(2)
        kept = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        open_ = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        c = torch.where(open_.repeat_interleave(E // G, 1), c, LOWEST)
    order = torch.sort(c, dim=1, descending=True, stable=True)
    chosen, none = order.indices[:, :k], order.values[:, :k] == LOWEST
    sj = torch.where(none, 0.0, score.gather(1, chosen))
    total = sj.sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0)
    ids = torch.where(none, -1, chosen).to(torch.int32)
    if not s["train"]:
        return ids, (2.5 * (sj / total if s["renorm"] else sj)).float()
    g = 2.5 * torch.where(none, 0.0, s["dw"].double())
    if s["renorm"]:
        u = sj / total
        g = (g - (g * u).sum(1, keepdim=True)) / total     # gradient of the chosen scores
        w = 2.5 * u
    else:
        w = 2.5 * sj
    ds = torch.zeros_like(l).scatter_add_(1, chosen, torch.where(none, 0.0, g))
    dl = score * (ds - (ds * score).sum(1, keepdim=True)) if s["scoring"] == "softmax" else ds * score * (1.0 - score)
    return ids, w.float(), dl.to(dt)


def _codes(x, square):
    """E4M3 codes of x [..., N, K] and the exponents of their scales: of 128 values of a row, or of 128 x 128."""
    N, K = x.shape[-2:]
    v = torch.nn.functional.pad(x.float(), (0, -K % 128, 0, -N % 128 if square else 0))
    v = v.unflatten(-1, (-1, 128))
    amax = v.abs().amax(-1)
    if square:
        amax = amax.unflatten(-2, (-1, 128)).amax(-2)
    m, p = torch.frexp(amax)                                   # amax = m 2^p, m in [0.5, 1): 448 = 0.875 2^9
    e = torch.where(amax > 0, torch.clamp(p - 9 + (m > 0.875).int(), -127, 127), -127)
    each = e.repeat_interleave(128, -2)[..., :v.shape[-3], :] if square else e
    q = (v * ((127 - each) << 23).view(torch.float32).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.flatten(-2)[..., :N, :K], e


def _values(q, e, square):
    """The 32-bit values of E4M3 codes and the exponents of their scales."""
    N, K = q.shape[-2:]
    scale = torch.where(e <= -127, 1 << 22, (e.to(torch.int32) + 127) << 23).to(torch.int32).view(torch.float32)
    if square:
        scale = scale.repeat_interleave(128, -2)[..., :N, :]
    return q.float() * scale.repeat_interleave(128, -1)[..., :K]


def _fake(x, square=False):
    return _values(*_codes(x, square), square)


def _padded(s, rows):
    """Rows in expert order [R, ...] as a padded batch [E, most_rows, ...], and the place of each."""
    at = torch.arange(rows.shape[0], device=rows.device)
    e = torch.searchsorted(s["offsets"][1:], at.to(torch.int32), right=True)
    place = e * s["most_rows"] + at - s["offsets"].long()[e]
    batch = torch.zeros((s["E"] * s["most_rows"], rows.shape[1]), device=rows.device)
    batch[place] = rows
    return batch.reshape(s["E"], s["most_rows"], -1), place


def _grouped(s, rows, w):
    """Each expert's rows times its own matrix w [E, in, out]."""
    if s["E"] == 1:
        return rows @ w[0]
    batch, place = _padded(s, rows)
    return torch.bmm(batch, w).flatten(0, 1)[place]


def _outer(s, dy, x):
    """For each expert the sum over its rows of dy outer x."""
    if s["E"] == 1:
        return (dy.t() @ x).unsqueeze(0)
    return torch.bmm(_padded(s, dy)[0].transpose(1, 2), _padded(s, x)[0])


def _plain_linear(s):
    x, w, dy = s["x"].detach(), _fake(s["w"].detach(), True), s["dy"]
    y = _grouped(s, _fake(x), w.transpose(1, 2))
    dx = _grouped(s, _fake(dy), w)
    return y.to(x.dtype), dx.to(x.dtype), _outer(s, dy.float(), x.float()).to(s["w"].dtype)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    if s["kind"] == "route":
        return _plain_route(s)
    if s["kind"] in ("rows", "blocks"):
        return _fake(s["x"], s["kind"] == "blocks").to(torch.bfloat16)
    if s["kind"] == "wgrad":
        return _outer(s, s["dy"].float(), s["x"].float()).to(DTYPES[s["out"]])
    if s["kind"] == "linear":
        return _plain_linear(s)
    w = _values(s["w_codes"].view(torch.float8_e4m3fn)[..., :s["K"]], s["w_scales"].int() - 127, True)
    rows = _fake(s["x"])[s["perm"].long() // s["k"]]
    return _grouped(s, rows, w if s["back"] else w.transpose(1, 2)).to(DTYPES[s["out"]])


def _own(s):
    from weight_only_quantized_qmoe_gb300 import ops
    if s["kind"] == "route":
        how = dict(scoring=s["scoring"], renormalize=s["renorm"], scale=2.5)
        r = ops.expert_route(s["logits"], s["k"], bias=s["b"], groups=s["groups"], top_groups=s["top_groups"], group_best=s["best"], **how)
        if not s["train"]:
            return r.ids, r.weights
        return r.ids, r.weights, ops.expert_route_grad(s["dw"], s["logits"], r.ids, **how)
    if s["kind"] in ("rows", "blocks"):
        return ops.fp8_dequantize(ops.fp8_quantize(s["x"], square=s["kind"] == "blocks"), dtype=torch.bfloat16)
    plan = None if s["E"] == 1 else ops.ExpertPlan(s["perm"], s["pos"], s["offsets"], s["k"], s["E"])
    if s["kind"] == "wgrad":
        dw = ops.weight_grad(s["dy"], s["x"], plan=plan, out_dtype=DTYPES[s["out"]])
        return dw.reshape(s["E"], s["N"], s["K"])
    if s["kind"] == "linear":
        y = ops.fp8_linear(s["x"], s["w"], plan=plan)
        return (y.detach(),) + torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
    w = ops.FP8Tensor(s["w_codes"], s["w_scales"], s["K"], True)
    return ops.fp8_matmul(ops.fp8_quantize(s["x"], plan=plan), w, plan=plan, transpose=s["back"], out_dtype=DTYPES[s["out"]])


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "route":
        return _route64(s)
    if case["kind"] in ("rows", "blocks"):
        return _fake64(s["x"], case["kind"] == "blocks")
    E, N, K, k = s["E"], s["N"], s["K"], s["k"]
    ends = s["offsets"].tolist()
    spans = [slice(b, e) for b, e in zip(ends, ends[1:])]

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.float64, device="cuda")

    if case["kind"] == "product":
        x = _fake64(s["x"], False)
        out = zeros(s["T"] * k, K if s["back"] else N)
        for e, rows in enumerate(spans):
            code = s["w_codes"][e][:, :K].long()
            frac, p = (code & 7).double(), code >> 3 & 15
            w = torch.where(p > 0, (8 + frac) * torch.exp2(p.double() - 10), frac * 2.0 ** -9) * torch.where(code > 127, -1.0, 1.0).double()
            scale = torch.exp2(s["w_scales"][e].double() - 127)
            w = w * scale[torch.arange(N, device="cuda") // 128][:, torch.arange(K, device="cuda") // 128]
            out[rows] = x[s["perm"][rows].long() // k] @ (w if s["back"] else w.T)
        return out
    dy, x = s["dy"].double(), s["x"].detach().double()
    dw = torch.stack([dy[rows].T @ x[rows] for rows in spans])
    if case["kind"] == "wgrad":
        return dw
    xq, dyq = _fake64(x, False), _fake64(dy, False)
    y, dx = zeros(s["T"] * k, N), zeros(s["T"] * k, K)
    for e, rows in enumerate(spans):
        w = _fake64(s["w"].detach()[e].double(), True)
        y[rows], dx[rows] = xq[rows] @ w.T, dyq[rows] @ w
    return y, dx, dw


def _fake64(x, square):
    """x quantised and read back: the smallest power-of-two scale that leaves the largest of a block at most 448, elements to the nearest
    E4M3 value (steps of 1/8 of the leading power of two, at least 2^-9), ties to even."""
    N, K = x.shape[-2:]
    v = torch.nn.functional.pad(x.double(), (0, -K % 128, 0, -N % 128 if square else 0))
    v = v.unflatten(-1, (-1, 128))
    big = v.abs().amax(-1, keepdim=True)
    if square:
        big = big.unflatten(-3, (-1, 128)).amax(-3).repeat_interleave(128, -3)
    e = torch.ceil(torch.log2(big.clamp(min=2.0 ** -160) / 448.0))
    e = torch.where(448.0 * torch.exp2(e) < big, e + 1, torch.where(448.0 * torch.exp2(e - 1) >= big, e - 1, e))
    scale = torch.exp2(e.clamp(min=-127.0))
    a = v.abs() / scale
    lead = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    lead = torch.where(torch.exp2(lead) > a.clamp(min=2.0 ** -6), lead - 1, torch.where(torch.exp2(lead + 1) <= a, lead + 1, lead))
    step = torch.exp2(lead - 3)
    return (torch.sign(v) * torch.round(a / step) * step * scale).flatten(-2)[..., :N, :K]


def _route64(s):
    """The choice row by row on the host, weights and gradient by automatic differentiation in 64 bits."""
    l = s["logits"].double().cpu()
    T, E, k, G, best = s["T"], s["E"], s["k"], s["groups"], s["best"]
    logits = l.numpy()
    none = np.all(np.isneginf(logits), axis=1)
    safe = torch.where(torch.from_numpy(none).unsqueeze(1), 0.0, l).requires_grad_()
    score = torch.softmax(safe, 1) if s["scoring"] == "softmax" else torch.sigmoid(safe)
    val = score.detach().numpy()
    choice = logits if s["b"] is None else val + s["b"].double().cpu().numpy()
    ids = np.full((T, k), -1)
    for t in range(T):
        may = np.isfinite(logits[t])
        c = choice[t]
        by = val[t] if s["b"] is None and best == 2 else c
        if G > 1 and s["top_groups"] < G:
            n = E // G
            total = [sum(sorted(by[i * n:(i + 1) * n][may[i * n:(i + 1) * n]])[-best:]) if may[i * n:(i + 1) * n].any() else LOWEST
                     for i in range(G)]
            kept = sorted(range(G), key=lambda i: (-total[i], i))[:s["top_groups"]]
            may = may & np.isin(np.arange(E) // n, kept)
        at = np.flatnonzero(may)
        at = at[np.argsort(-c[at], kind="stable")][:k]
        ids[t, :len(at)] = at
    ids = torch.from_numpy(ids)
    sj = torch.where(ids >= 0, score.gather(1, ids.clamp(min=0)), 0.0)
    if s["renorm"]:
        total = sj.sum(1, keepdim=True)
        sj = sj / torch.where(total > 0, total, 1.0)
    w = 2.5 * sj
    if not s["train"]:
        return ids.to(torch.int32), w.detach()
    dl, = torch.autograd.grad(w, safe, s["dw"].double().cpu())
    return ids.to(torch.int32), w.detach(), dl
