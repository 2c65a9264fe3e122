"""Operators around the expert layer, on torch CUDA tensors.

Thin calls of the C entry points of the same names (include/qmoe.h, the
operators' part), which define what each computes:

* :func:`expert_sort`, :func:`dispatch`, :func:`combine` and the gradients
  :func:`dispatch_grad`, :func:`combine_grad`: routes sorted by expert, token
  rows taken into expert order and summed back with their weights;
* :func:`mx4_quantize`, :func:`mx4_dequantize`, :func:`mx4_matmul`:
  microscaled 4-bit floating point rows and their product, dense or grouped by
  expert;
* :func:`block_norm`, :func:`block_norm_grad`: the norms on either side of a
  block with the gate of its output and the residual scale.

``dispatch``, ``combine`` and ``block_norm`` take part in automatic
differentiation where an input requires a gradient.  Refused arguments raise
:class:`~weight_only_quantized_qmoe_gb300.QMoEError`.  Every call runs on the
current stream, or on ``stream=``: its outputs then belong to that stream (a
reader on another stream has to wait for it), and its inputs have to be ready
there.  Tensors whose last axis is not contiguous are copied first.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import QMoEError, binding

_DTYPES = {torch.float32: binding.QMOE_F32, torch.float16: binding.QMOE_F16, torch.bfloat16: binding.QMOE_BF16}
_ACTIVATIONS = {None: binding.QMOE_ACT_NONE, "swiglu": binding.QMOE_ACT_SWIGLU, "geglu": binding.QMOE_ACT_GEGLU_TANH}


class ExpertPlan(NamedTuple):
    """The routes of T tokens sorted by expert (int32 tensors): ``perm`` [T * k]
    routes by expert, ``pos`` [T * k] row of each route (-1: dropped),
    ``offsets`` [experts + 1] first row of each expert."""

    perm: torch.Tensor
    pos: torch.Tensor
    offsets: torch.Tensor
    k: int
    experts: int

    @property
    def tokens(self) -> int:
        return self.pos.numel() // self.k


class MX4Tensor(NamedTuple):
    """Microscaled 4-bit rows [..., N, cols]: ``codes`` uint8 [..., N, 16 * nb]
    and ``scales`` uint8 [..., ceil(nb / 4), N, 4], nb = ceil(cols / 32)."""

    codes: torch.Tensor
    scales: torch.Tensor
    cols: int


class NormStats(NamedTuple):
    """Per-row statistics of :func:`block_norm` its gradient needs."""

    rstd_post: Optional[torch.Tensor]
    rstd_pre: Optional[torch.Tensor]


class NormGrads(NamedTuple):
    """Gradients of :func:`block_norm` (None for an absent argument)."""

    x: torch.Tensor
    o: Optional[torch.Tensor]
    gate: Optional[torch.Tensor]
    w_post: Optional[torch.Tensor]
    w_pre: Optional[torch.Tensor]


# --- argument handling --------------------------------------------------------
def _refuse(msg):
    raise QMoEError(binding.QMOE_ERR_INVALID_ARG, msg)


def _check(status):
    if status != binding.QMOE_OK:
        raise QMoEError(status, binding.qmoe_op_last_error())


def _need(cond, msg):
    if not cond:
        _refuse(msg)


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _refuse(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        _refuse(f"{name} is on {t.device}, not on the current device")


def _dtype(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        _refuse(f"{name} is {t.dtype}: float32, float16 or bfloat16")
    return code


def _rows(t, name, dtype=None):
    """A 2-D tensor with a contiguous last axis and rows at least its length
    apart, and that row stride."""
    _cuda(t, name)
    if t.dim() != 2:
        _refuse(f"{name} must be two-dimensional, not {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        _refuse(f"{name} is {t.dtype}, not {dtype}")
    n, width = t.shape
    if (t.stride(1) != 1 and width > 1) or (t.stride(0) < width and n > 1):
        t = t.contiguous()
    return t, (t.stride(0) if n > 1 else max(width, 1))


def _flat(t, name, dtype, numel=None):
    _cuda(t, name)
    if t.dtype != dtype:
        _refuse(f"{name} is {t.dtype}, not {dtype}")
    if numel is not None and t.numel() != numel:
        _refuse(f"{name} has {t.numel()} elements, not {numel}")
    return t if t.is_contiguous() else t.contiguous()


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _elsewhere(stream, call, *args, **kw):
    """call(...) on `stream`; the inputs' memory is kept until it is done there."""
    with torch.cuda.stream(stream):
        out = call(*args, **kw)
    for a in list(args) + list(kw.values()):
        for t in a if isinstance(a, tuple) else (a,):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
    return out


def _plan(plan, tokens=None):
    """(pos, offsets) of a plan, checked."""
    if not isinstance(plan, ExpertPlan):
        _refuse("plan must be an ExpertPlan")
    _need(plan.k >= 1 and plan.pos.numel() % plan.k == 0, "plan.pos does not hold whole tokens")
    if tokens is not None and plan.tokens != tokens:
        _refuse(f"the plan is of {plan.tokens} tokens, not {tokens}")
    return (_flat(plan.pos, "plan.pos", torch.int32),
            _flat(plan.offsets, "plan.offsets", torch.int32, plan.experts + 1))


def _weights(weights, plan):
    return None if weights is None else _flat(weights, "weights", torch.float32, plan.pos.numel())


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def poll_status() -> int:
    """QMOE_OK, or QMOE_ERR_TIMEOUT if a bounded wait of an operator ran out
    since the last call (read and cleared; synchronises the device)."""
    return binding.qmoe_op_poll_status()


# --- tokens sorted by expert and back -----------------------------------------
def expert_sort(ids, experts, stream=None) -> ExpertPlan:
    """Sort the routes ids [T, k] (int32 or int64) by expert, stably.  Ids
    outside [0, experts) drop their route."""
    if stream is not None:
        return _elsewhere(stream, expert_sort, ids, experts)
    _cuda(ids, "ids")
    _need(ids.dtype in (torch.int32, torch.int64), f"ids is {ids.dtype}: int32 or int64")
    ids, ld = _rows(ids, "ids")
    T, k = ids.shape
    perm = torch.empty(T * k, dtype=torch.int32, device=ids.device)
    pos = torch.empty_like(perm)
    offsets = torch.empty(max(int(experts), 0) + 1, dtype=torch.int32, device=ids.device)
    _check(binding.qmoe_expert_sort(ids.data_ptr(), ids.element_size(), ld, T, k, experts, perm.data_ptr(),
                                    pos.data_ptr(), offsets.data_ptr(), _stream()))
    return ExpertPlan(perm, pos, offsets, k, int(experts))


def _dispatch(x, plan):
    dt = _dtype(x, "x")
    x, ld = _rows(x, "x")
    T, H = x.shape
    pos, offsets = _plan(plan, T)
    xs = torch.empty((T * plan.k, H), dtype=x.dtype, device=x.device)
    _check(binding.qmoe_dispatch(x.data_ptr(), ld, pos.data_ptr(), offsets.data_ptr(), T, plan.k, plan.experts, H, dt,
                                 xs.data_ptr(), _stream()))
    return xs


def dispatch_grad(dxs, plan, stream=None):
    """The gradient of :func:`dispatch`: dx [T, H] of dxs [T * k, H]."""
    if stream is not None:
        return _elsewhere(stream, dispatch_grad, dxs, plan)
    return _combine(dxs, None, plan, "dxs")


def _combine(y, weights, plan, name="y"):
    dt = _dtype(y, name)
    y, ld = _rows(y, name)
    pos, _ = _plan(plan)
    T, H = plan.tokens, y.shape[1]
    _need(y.shape[0] == pos.numel(), f"{name} has {y.shape[0]} rows, the plan {pos.numel()}")
    weights = _weights(weights, plan)
    out = torch.empty((T, H), dtype=y.dtype, device=y.device)
    _check(binding.qmoe_combine(y.data_ptr(), ld, _ptr(weights), pos.data_ptr(), T, plan.k, H, dt, out.data_ptr(),
                                _stream()))
    return out


def combine_grad(dout, y, weights, plan, need_dy=True, need_dweights=True, stream=None):
    """The gradients of :func:`combine`: (dy [T * k, H], dweights float32 [T, k])
    of dout [T, H]; one that is not needed is None."""
    if stream is not None:
        return _elsewhere(stream, combine_grad, dout, y, weights, plan, need_dy, need_dweights)
    dt = _dtype(dout, "dout")
    dout, ld = _rows(dout, "dout")
    T, H = dout.shape
    pos, offsets = _plan(plan, T)
    weights = _weights(weights, plan)
    ld_y = H
    if need_dweights:
        y, ld_y = _rows(y, "y", dout.dtype)
        _need(tuple(y.shape) == (pos.numel(), H), f"y is {tuple(y.shape)}, not {(pos.numel(), H)}")
    dy = torch.empty((T * plan.k, H), dtype=dout.dtype, device=dout.device) if need_dy else None
    dw = torch.empty((T, plan.k), dtype=torch.float32, device=dout.device) if need_dweights else None
    _check(binding.qmoe_combine_grad(dout.data_ptr(), ld, y.data_ptr() if need_dweights else 0, ld_y, _ptr(weights),
                                     pos.data_ptr(), offsets.data_ptr(), T, plan.k, plan.experts, H, dt, _ptr(dy),
                                     _ptr(dw), _stream()))
    return dy, dw


class _DispatchFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.plan = plan
        return _dispatch(x, plan)

    @staticmethod
    def backward(ctx, dxs):
        return dispatch_grad(dxs, ctx.plan), None


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, plan):
        ctx.save_for_backward(y, weights)
        ctx.plan = plan
        return _combine(y, weights, plan)

    @staticmethod
    def backward(ctx, dout):
        y, weights = ctx.saved_tensors
        dy, dw = combine_grad(dout, y, weights, ctx.plan, ctx.needs_input_grad[0],
                              weights is not None and ctx.needs_input_grad[1])
        return dy, None if dw is None else dw.reshape(weights.shape), None


def _differentiable(*tensors):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def dispatch(x, plan, stream=None):
    """Token rows x [T, H] into expert order [T * k, H] (zeros past the rows in
    use)."""
    if stream is not None:
        return _elsewhere(stream, dispatch, x, plan)
    return _DispatchFn.apply(x, plan) if _differentiable(x) else _dispatch(x, plan)


def combine(y, weights, plan, stream=None):
    """Expert rows y [T * k, H] back to token order [T, H], weighted with
    ``weights`` (float32 [T, k], or None for ones)."""
    if stream is not None:
        return _elsewhere(stream, combine, y, weights, plan)
    return _CombineFn.apply(y, weights, plan) if _differentiable(y, weights) else _combine(y, weights, plan)


# --- microscaled 4-bit floating point -----------------------------------------
def mx4_quantize(x, plan=None, activation=None, stream=None) -> MX4Tensor:
    """Quantise the rows of x [..., N, K].  With ``plan`` the rows x [T, K] are
    written in expert order [T * k, K].  With ``activation`` "swiglu" or
    "geglu" a row holds gate | up (2 K values) and act(gate) * up is quantised."""
    if stream is not None:
        return _elsewhere(stream, mx4_quantize, x, plan, activation)
    _cuda(x, "x")
    dt = _dtype(x, "x")
    _need(activation in _ACTIVATIONS, f"activation {activation!r}: None, 'swiglu' or 'geglu'")
    _need(x.dim() >= 2, "x must have rows: two dimensions at least")
    lead, n, width = x.shape[:-2], x.shape[-2], x.shape[-1]
    if activation is not None:
        _need(width % 2 == 0, f"gate | up needs an even row length, not {width}")
    cols = width if activation is None else width // 2
    flat, ld = _rows(x if x.dim() == 2 else x.reshape(-1, width), "x")
    rows = flat.shape[0]
    pos = offsets = None
    k = experts = 1
    if plan is not None:
        _need(x.dim() == 2, "with a plan x is [T, K]")
        pos, offsets = _plan(plan, rows)
        k, experts, n = plan.k, plan.experts, rows * plan.k
    nb = -(-cols // 32)
    codes = torch.empty((*lead, n, nb * 16), dtype=torch.uint8, device=x.device)
    scales = torch.empty((*lead, -(-nb // 4), n, 4), dtype=torch.uint8, device=x.device)
    _check(binding.qmoe_mx4_quantize(flat.data_ptr(), ld, rows, cols, dt, _ACTIVATIONS[activation], _ptr(pos),
                                     _ptr(offsets), k, experts, n, codes.data_ptr(), scales.data_ptr(), _stream()))
    return MX4Tensor(codes, scales, cols)


def _mx4(q, name):
    """(codes, scales) of an MX4Tensor, checked and contiguous."""
    if not isinstance(q, MX4Tensor):
        _refuse(f"{name} must be an MX4Tensor")
    codes, scales = _flat(q.codes, name + ".codes", torch.uint8), _flat(q.scales, name + ".scales", torch.uint8)
    nb = -(-q.cols // 32)
    if codes.dim() < 2 or codes.shape[-1] != nb * 16 or q.cols < 1:
        _refuse(f"{name}.codes {tuple(codes.shape)} does not hold rows of {q.cols} values")
    if tuple(scales.shape) != (*codes.shape[:-2], -(-nb // 4), codes.shape[-2], 4):
        _refuse(f"{name}.scales {tuple(scales.shape)} does not belong to codes {tuple(codes.shape)}")
    return codes, scales


def mx4_dequantize(q, dtype=torch.bfloat16, stream=None):
    """The values [..., N, cols] of an :class:`MX4Tensor`."""
    if stream is not None:
        return _elsewhere(stream, mx4_dequantize, q, dtype)
    codes, scales = _mx4(q, "q")
    _need(dtype in _DTYPES, f"dtype {dtype}: float32, float16 or bfloat16")
    n = codes.shape[-2]
    out = torch.empty((*codes.shape[:-1], q.cols), dtype=dtype, device=codes.device)
    rows = out.numel() // q.cols
    _check(binding.qmoe_mx4_dequantize(codes.data_ptr(), scales.data_ptr(), rows, q.cols, n, _DTYPES[dtype],
                                       out.data_ptr(), q.cols, _stream()))
    return out


def mx4_matmul(a, w, plan=None, out_dtype=torch.bfloat16, stream=None):
    """a [R, K] times the transpose of w: [N, K] for all rows, or with ``plan``
    [experts, N, K], each expert's rows with its own (zeros past the rows in
    use).  Returns [R, N]."""
    if stream is not None:
        return _elsewhere(stream, mx4_matmul, a, w, plan, out_dtype)
    a_codes, a_scales = _mx4(a, "a")
    w_codes, w_scales = _mx4(w, "w")
    _need(out_dtype in _DTYPES, f"out_dtype {out_dtype}: float32, float16 or bfloat16")
    _need(a_codes.dim() == 2, "a must be [R, K]")
    _need(a.cols == w.cols, f"a has rows of {a.cols} values, w of {w.cols}")
    R, N = a_codes.shape[0], w_codes.shape[-2]
    experts, offsets = 1, None
    if plan is not None:
        pos, offsets = _plan(plan)
        experts = plan.experts
        _need(pos.numel() == R, f"a has {R} rows, the plan {pos.numel()}")
    if experts != w_codes.numel() // max(1, w_codes.shape[-2] * w_codes.shape[-1]) or w_codes.dim() > 3:
        _refuse(f"w.codes {tuple(w_codes.shape)} does not hold {experts} expert(s)")
    out = torch.empty((R, N), dtype=out_dtype, device=a_codes.device)
    _check(binding.qmoe_mx4_matmul(a_codes.data_ptr(), a_scales.data_ptr(), R, w_codes.data_ptr(), w_scales.data_ptr(),
                                   _ptr(offsets), experts, N, a.cols, _DTYPES[out_dtype], out.data_ptr(), N, _stream()))
    return out


# --- norms around a block ------------------------------------------------------
class _Norm(NamedTuple):
    """Checked arguments of a block norm, flattened to rows."""

    shape: tuple
    T: int
    H: int
    dt: int
    x: torch.Tensor
    ld_x: int
    o: Optional[torch.Tensor]
    ld_o: int
    gate: Optional[torch.Tensor]
    kind: int
    ld_gate: int
    w_post: Optional[torch.Tensor]
    w_pre: Optional[torch.Tensor]


def _flat_rows(t, name, H, shape, dtype):
    _need(isinstance(t, torch.Tensor) and tuple(t.shape) == tuple(shape), f"{name} must have the shape {tuple(shape)}")
    return _rows(t if t.dim() == 2 else t.reshape(-1, H), name, dtype)


def _norm_args(x, o, gate, w_post, w_pre):
    _cuda(x, "x")
    dt = _dtype(x, "x")
    _need(x.dim() >= 1 and x.shape[-1] >= 1, "x must have rows of at least one value")
    shape, H = tuple(x.shape), x.shape[-1]
    fx, ld_x = _flat_rows(x, "x", H, shape, x.dtype)
    T = fx.shape[0]
    fo, ld_o = (None, 0) if o is None else _flat_rows(o, "o", H, shape, x.dtype)
    fg, kind, ld_g = None, binding.QMOE_GATE_NONE, 0
    if gate is not None:
        _need(o is not None, "gate needs o")
        g = tuple(gate.shape)
        if g == shape:
            kind = binding.QMOE_GATE_FULL
            fg, ld_g = _flat_rows(gate, "gate", H, shape, x.dtype)
        elif g == (H,):
            kind = binding.QMOE_GATE_CHANNEL
            fg = _flat(gate, "gate", x.dtype)
        elif g == shape[:-1] + (1,):
            kind = binding.QMOE_GATE_TOKEN
            fg = _flat(gate, "gate", x.dtype)
        else:
            _refuse(f"gate {g} is not {shape}, {(H,)} or {shape[:-1] + (1,)}")
    wq = None if w_post is None else _flat(w_post, "w_post", x.dtype, H)
    wp = None if w_pre is None else _flat(w_pre, "w_pre", x.dtype, H)
    return _Norm(shape, T, H, dt, fx, ld_x, fo, ld_o, fg, kind, ld_g, wq, wp)


def _block_norm(x, o, gate, w_post, w_pre, residual_scale, eps, stats):
    a = _norm_args(x, o, gate, w_post, w_pre)
    r = torch.empty(a.shape, dtype=x.dtype, device=x.device)
    h = None if w_pre is None else torch.empty_like(r)
    s1 = torch.empty(a.T, dtype=torch.float32, device=x.device) if stats and w_post is not None else None
    s2 = torch.empty(a.T, dtype=torch.float32, device=x.device) if stats and w_pre is not None else None
    _check(binding.qmoe_block_norm(a.x.data_ptr(), a.ld_x, _ptr(a.o), a.ld_o, _ptr(a.gate), a.kind, a.ld_gate,
                                   _ptr(a.w_post), _ptr(a.w_pre), residual_scale, eps, a.T, a.H, a.dt, r.data_ptr(),
                                   _ptr(h), _ptr(s1), _ptr(s2), _stream()))
    return r, h, NormStats(s1, s2)


def block_norm_grad(dr, dh, x, o, stats, gate=None, w_post=None, w_pre=None, residual_scale=1.0, eps=None,
                    stream=None) -> NormGrads:
    """The gradients of :func:`block_norm` for the gradients ``dr`` and ``dh``
    of its outputs (None: zero) and its own arguments; ``stats`` are the
    forward's (they hold ``eps``, taken here only so that the forward's keywords
    can be passed on)."""
    if stream is not None:
        return _elsewhere(stream, block_norm_grad, dr, dh, x, o, stats, gate, w_post, w_pre, residual_scale)
    a = _norm_args(x, o, gate, w_post, w_pre)
    _need(dh is None or w_pre is not None, "dh needs w_pre")
    fr, ld_r = (None, 0) if dr is None else _flat_rows(dr, "dr", a.H, a.shape, x.dtype)
    fh, ld_h = (None, 0) if dh is None else _flat_rows(dh, "dh", a.H, a.shape, x.dtype)
    s1 = _flat(stats.rstd_post, "stats.rstd_post", torch.float32, a.T) if w_post is not None else None
    s2 = _flat(stats.rstd_pre, "stats.rstd_pre", torch.float32, a.T) if w_pre is not None else None

    def like(t):
        return None if t is None else torch.empty(t.shape, dtype=x.dtype, device=x.device)

    dx, do, dgate, dwq, dwp = like(x), like(o), like(gate), like(w_post), like(w_pre)
    nbytes = binding.qmoe_block_norm_grad_workspace(a.T, a.H, a.dt)
    work = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    _check(binding.qmoe_block_norm_grad(_ptr(fr), ld_r, _ptr(fh), ld_h, a.x.data_ptr(), a.ld_x, _ptr(a.o), a.ld_o,
                                        _ptr(a.gate), a.kind, a.ld_gate, _ptr(a.w_post), _ptr(a.w_pre), _ptr(s1),
                                        _ptr(s2), residual_scale, a.T, a.H, a.dt, _ptr(dx), _ptr(do), _ptr(dgate),
                                        _ptr(dwq), _ptr(dwp), work.data_ptr(), nbytes, _stream()))
    return NormGrads(dx, do, dgate, dwq, dwp)


class _BlockNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, o, gate, w_post, w_pre, residual_scale, eps):
        r, h, stats = _block_norm(x, o, gate, w_post, w_pre, residual_scale, eps, True)
        ctx.save_for_backward(x, o, gate, w_post, w_pre, *stats)
        ctx.residual_scale = residual_scale
        ctx.set_materialize_grads(False)
        return r, h

    @staticmethod
    def backward(ctx, dr, dh):
        x, o, gate, w_post, w_pre, s1, s2 = ctx.saved_tensors
        g = block_norm_grad(dr, dh, x, o, NormStats(s1, s2), gate, w_post, w_pre, ctx.residual_scale)
        return g.x, g.o, g.gate, g.w_post, g.w_pre, None, None


def block_norm(x, o=None, gate=None, w_post=None, w_pre=None, residual_scale=1.0, eps=1e-6, return_stats=False,
               stream=None):
    """r = residual_scale * x + gate * rms(o) * w_post and h = rms(r) * w_pre.

    ``x`` and ``o`` are [..., H]; ``gate`` is [..., 1], [H] or [..., H] (None:
    1); without ``w_post`` the branch is not normalised, without ``o`` there is
    none, without ``w_pre`` h is None.  Returns (r, h), or (r, h, stats) with
    ``return_stats`` (not differentiated then)."""
    if stream is not None:
        return _elsewhere(stream, block_norm, x, o, gate, w_post, w_pre, residual_scale, eps, return_stats)
    if return_stats:
        return _block_norm(x, o, gate, w_post, w_pre, residual_scale, eps, True)
    if _differentiable(x, o, gate, w_post, w_pre):
        return _BlockNormFn.apply(x, o, gate, w_post, w_pre, residual_scale, eps)
    return _block_norm(x, o, gate, w_post, w_pre, residual_scale, eps, False)[:2]


__all__ = ["ExpertPlan", "MX4Tensor", "NormStats", "NormGrads", "expert_sort", "dispatch", "dispatch_grad", "combine",
           "combine_grad", "mx4_quantize", "mx4_dequantize", "mx4_matmul", "block_norm", "block_norm_grad",
           "poll_status"]
