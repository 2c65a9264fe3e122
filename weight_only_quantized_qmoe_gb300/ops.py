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
# A call on small tensors is bound by this code, so every argument is looked at
# once and the common case (contiguous tensors) takes the shortest way.
_empty, _f32, _i32, _u8 = torch.empty, torch.float32, torch.int32, torch.uint8
_raw_stream, _device = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device


def _refuse(msg):
    raise QMoEError(binding.QMOE_ERR_INVALID_ARG, msg)


def _failed(status):
    raise QMoEError(status, binding.qmoe_op_last_error())


def _first(t, name):
    """(device index, dtype code) of the tensor that decides both."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _refuse(f"{name} must be a CUDA tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        _refuse(f"{name} is {t.dtype}: float32, float16 or bfloat16")
    return _here(t, name), code


def _here(t, name):
    dev = t.get_device()
    if dev != _device():
        _refuse(f"{name} is on {t.device}, not on the current device")
    return dev


def _not(t, name, dtype, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _refuse(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        _refuse(f"{name} is {t.dtype}, not {dtype}")
    _refuse(f"{name} is on {t.device}, not on the current device")


def _rows(t, name, dtype, dev):
    """A 2-D tensor with a contiguous last axis and rows at least its length
    apart, and that row stride."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev:
        _not(t, name, dtype, dev)
    if t.dim() != 2:
        _refuse(f"{name} must be two-dimensional, not {tuple(t.shape)}")
    n, width = t.shape
    if t.is_contiguous():
        return t, width or 1
    if (t.stride(1) != 1 and width > 1) or (t.stride(0) < width and n > 1):
        return t.contiguous(), width
    return t, (t.stride(0) if n > 1 else max(width, 1))


def _flat(t, name, dtype, numel, dev):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev:
        _not(t, name, dtype, dev)
    if t.numel() != numel:
        _refuse(f"{name} has {t.numel()} elements, not {numel}")
    return t if t.is_contiguous() else t.contiguous()


def _elsewhere(stream, call, *args, **kw):
    """call(...) on `stream`; the inputs' memory is kept until it is done there."""
    with torch.cuda.stream(stream):
        out = call(*args, **kw)
    for a in list(args) + list(kw.values()):
        for t in a if isinstance(a, tuple) else (a,):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
    return out


def _plan(plan, dev, tokens=None):
    """(pos, offsets, tokens, k, experts) of a plan, checked."""
    if not isinstance(plan, ExpertPlan):
        _refuse("plan must be an ExpertPlan")
    _, pos, offsets, k, experts = plan
    if k < 1 or pos.numel() % k:
        _refuse("plan.pos does not hold whole tokens")
    n = pos.numel() // k
    if tokens is not None and n != tokens:
        _refuse(f"the plan is of {n} tokens, not {tokens}")
    return _flat(pos, "plan.pos", _i32, n * k, dev), _flat(offsets, "plan.offsets", _i32, experts + 1, dev), n, k, experts


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
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda:
        _refuse("ids must be a CUDA tensor")
    dt = ids.dtype
    if dt is not _i32 and dt is not torch.int64:
        _refuse(f"ids is {dt}: int32 or int64")
    dev = _here(ids, "ids")
    ids, ld = _rows(ids, "ids", dt, dev)
    T, k = ids.shape
    R, device = T * k, ids.device
    perm, pos = _empty(R, dtype=_i32, device=device), _empty(R, dtype=_i32, device=device)
    offsets = _empty(max(experts, 0) + 1, dtype=_i32, device=device)
    st = binding.qmoe_expert_sort(ids.data_ptr(), 4 if dt is _i32 else 8, ld, T, k, experts, perm.data_ptr(),
                                  pos.data_ptr(), offsets.data_ptr(), _raw_stream(dev))
    if st:
        _failed(st)
    return ExpertPlan(perm, pos, offsets, k, experts)


def _dispatch(x, plan):
    dev, dt = _first(x, "x")
    x, ld = _rows(x, "x", x.dtype, dev)
    T, H = x.shape
    pos, offsets, _, k, experts = _plan(plan, dev, T)
    xs = _empty((T * k, H), dtype=x.dtype, device=x.device)
    st = binding.qmoe_dispatch(x.data_ptr(), ld, pos.data_ptr(), offsets.data_ptr(), T, k, experts, H, dt,
                               xs.data_ptr(), _raw_stream(dev))
    if st:
        _failed(st)
    return xs


def dispatch_grad(dxs, plan, stream=None):
    """The gradient of :func:`dispatch`: dx [T, H] of dxs [T * k, H]."""
    if stream is not None:
        return _elsewhere(stream, dispatch_grad, dxs, plan)
    return _combine(dxs, None, plan, "dxs")


def _combine(y, weights, plan, name="y"):
    dev, dt = _first(y, name)
    y, ld = _rows(y, name, y.dtype, dev)
    pos, _, T, k, _ = _plan(plan, dev)
    R, H = y.shape
    if R != T * k:
        _refuse(f"{name} has {R} rows, the plan {T * k}")
    w = 0
    if weights is not None:
        weights = _flat(weights, "weights", _f32, R, dev)
        w = weights.data_ptr()
    out = _empty((T, H), dtype=y.dtype, device=y.device)
    st = binding.qmoe_combine(y.data_ptr(), ld, w, pos.data_ptr(), T, k, H, dt, out.data_ptr(), _raw_stream(dev))
    if st:
        _failed(st)
    return out


def combine_grad(dout, y, weights, plan, need_dy=True, need_dweights=True, stream=None):
    """The gradients of :func:`combine`: (dy [T * k, H], dweights float32 [T, k])
    of dout [T, H]; one that is not needed is None."""
    if stream is not None:
        return _elsewhere(stream, combine_grad, dout, y, weights, plan, need_dy, need_dweights)
    dev, dt = _first(dout, "dout")
    dout, ld = _rows(dout, "dout", dout.dtype, dev)
    T, H = dout.shape
    pos, offsets, _, k, experts = _plan(plan, dev, T)
    if weights is not None:
        weights = _flat(weights, "weights", _f32, T * k, dev)
    ld_y = H
    if need_dweights:
        y, ld_y = _rows(y, "y", dout.dtype, dev)
        if y.shape[0] != T * k or y.shape[1] != H:
            _refuse(f"y is {tuple(y.shape)}, not {(T * k, H)}")
    dy = _empty((T * k, H), dtype=dout.dtype, device=dout.device) if need_dy else None
    dw = _empty((T, k), dtype=_f32, device=dout.device) if need_dweights else None
    st = binding.qmoe_combine_grad(dout.data_ptr(), ld, y.data_ptr() if need_dweights else 0, ld_y, _ptr(weights),
                                   pos.data_ptr(), offsets.data_ptr(), T, k, experts, H, dt, _ptr(dy), _ptr(dw),
                                   _raw_stream(dev))
    if st:
        _failed(st)
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
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


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
    dev, dt = _first(x, "x")
    if x.dim() < 2:
        _refuse("x must have rows: two dimensions at least")
    *lead, n, width = x.shape
    act, cols = binding.QMOE_ACT_NONE, width
    if activation is not None:
        act = _ACTIVATIONS.get(activation)
        if act is None:
            _refuse(f"activation {activation!r}: None, 'swiglu' or 'geglu'")
        if width % 2:
            _refuse(f"gate | up needs an even row length, not {width}")
        cols = width // 2
    flat, ld = _rows(x if not lead else x.reshape(-1, width), "x", x.dtype, dev)
    rows = flat.shape[0]
    pos = offsets = 0
    k = experts = 1
    if plan is not None:
        if lead:
            _refuse("with a plan x is [T, K]")
        tpos, toffsets, _, k, experts = _plan(plan, dev, rows)
        pos, offsets, n = tpos.data_ptr(), toffsets.data_ptr(), rows * k
    nb = (cols + 31) // 32
    codes = _empty((*lead, n, nb * 16), dtype=_u8, device=x.device)
    scales = _empty((*lead, (nb + 3) // 4, n, 4), dtype=_u8, device=x.device)
    st = binding.qmoe_mx4_quantize(flat.data_ptr(), ld, rows, cols, dt, act, pos, offsets, k, experts, n,
                                   codes.data_ptr(), scales.data_ptr(), _raw_stream(dev))
    if st:
        _failed(st)
    return MX4Tensor(codes, scales, cols)


def _mx4(q, name):
    """(codes, scales, shape of codes, device index) of an MX4Tensor, checked
    and contiguous."""
    if not isinstance(q, MX4Tensor):
        _refuse(f"{name} must be an MX4Tensor")
    codes, scales, cols = q
    if not isinstance(codes, torch.Tensor) or not codes.is_cuda:
        _refuse(f"{name}.codes must be a CUDA tensor")
    dev = _here(codes, name + ".codes")
    if codes.dtype is not _u8:
        _refuse(f"{name}.codes is {codes.dtype}, not uint8")
    nb, shape = (cols + 31) // 32, codes.shape
    if len(shape) < 2 or shape[-1] != nb * 16 or cols < 1:
        _refuse(f"{name}.codes {tuple(shape)} does not hold rows of {cols} values")
    scales = _flat(scales, name + ".scales", _u8, codes.numel() // max(1, nb * 16) * ((nb + 3) // 4) * 4, dev)
    if scales.shape != (*shape[:-2], (nb + 3) // 4, shape[-2], 4):
        _refuse(f"{name}.scales {tuple(scales.shape)} does not belong to codes {tuple(shape)}")
    return codes if codes.is_contiguous() else codes.contiguous(), scales, shape, dev


def mx4_dequantize(q, dtype=torch.bfloat16, stream=None):
    """The values [..., N, cols] of an :class:`MX4Tensor`."""
    if stream is not None:
        return _elsewhere(stream, mx4_dequantize, q, dtype)
    codes, scales, shape, dev = _mx4(q, "q")
    dt = _DTYPES.get(dtype)
    if dt is None:
        _refuse(f"dtype {dtype}: float32, float16 or bfloat16")
    cols, n = q.cols, shape[-2]
    out = _empty((*shape[:-1], cols), dtype=dtype, device=codes.device)
    st = binding.qmoe_mx4_dequantize(codes.data_ptr(), scales.data_ptr(), out.numel() // cols, cols, n, dt,
                                     out.data_ptr(), cols, _raw_stream(dev))
    if st:
        _failed(st)
    return out


def mx4_matmul(a, w, plan=None, out_dtype=torch.bfloat16, stream=None):
    """a [R, K] times the transpose of w: [N, K] for all rows, or with ``plan``
    [experts, N, K], each expert's rows with its own (zeros past the rows in
    use).  Returns [R, N]."""
    if stream is not None:
        return _elsewhere(stream, mx4_matmul, a, w, plan, out_dtype)
    a_codes, a_scales, a_shape, dev = _mx4(a, "a")
    w_codes, w_scales, w_shape, _ = _mx4(w, "w")
    dt = _DTYPES.get(out_dtype)
    if dt is None:
        _refuse(f"out_dtype {out_dtype}: float32, float16 or bfloat16")
    if len(a_shape) != 2:
        _refuse("a must be [R, K]")
    if a.cols != w.cols:
        _refuse(f"a has rows of {a.cols} values, w of {w.cols}")
    R, N = a_shape[0], w_shape[-2]
    experts, offsets = 1, 0
    if plan is not None:
        _, toffsets, T, k, experts = _plan(plan, dev)
        offsets = toffsets.data_ptr()
        if T * k != R:
            _refuse(f"a has {R} rows, the plan {T * k}")
    if (w_shape[0] if len(w_shape) == 3 else 1) != experts or len(w_shape) > 3:
        _refuse(f"w.codes {tuple(w_shape)} does not hold {experts} expert(s)")
    out = _empty((R, N), dtype=out_dtype, device=a_codes.device)
    st = binding.qmoe_mx4_matmul(a_codes.data_ptr(), a_scales.data_ptr(), R, w_codes.data_ptr(), w_scales.data_ptr(),
                                 offsets, experts, N, a.cols, dt, out.data_ptr(), N, _raw_stream(dev))
    if st:
        _failed(st)
    return out


# --- norms around a block ------------------------------------------------------
def _norm_rows(t, name, shape, dtype, dev):
    if t.shape != shape:
        _refuse(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    return _rows(t if len(shape) == 2 else t.reshape(-1, shape[-1]), name, dtype, dev)


def _norm_args(x, o, gate, w_post, w_pre):
    """The checked tensors of a block norm as rows (kept alive by the caller),
    the device index, and the leading arguments of its C calls from x on."""
    dev, dt = _first(x, "x")
    shape, dtype = x.shape, x.dtype
    if not shape or shape[-1] < 1:
        _refuse("x must have rows of at least one value")
    H = shape[-1]
    x, ld_x = _norm_rows(x, "x", shape, dtype, dev)
    po = ld_o = pg = kind = ld_g = pq = pp = 0
    if o is not None:
        o, ld_o = _norm_rows(o, "o", shape, dtype, dev)
        po = o.data_ptr()
    if gate is not None:
        if o is None:
            _refuse("gate needs o")
        g = gate.shape
        if g == shape:
            kind = binding.QMOE_GATE_FULL
            gate, ld_g = _norm_rows(gate, "gate", shape, dtype, dev)
        elif g == (H,):
            kind = binding.QMOE_GATE_CHANNEL
            gate = _flat(gate, "gate", dtype, H, dev)
        elif g == (*shape[:-1], 1):
            kind = binding.QMOE_GATE_TOKEN
            gate = _flat(gate, "gate", dtype, x.shape[0], dev)
        else:
            _refuse(f"gate {tuple(g)} is not {tuple(shape)}, {(H,)} or {(*shape[:-1], 1)}")
        pg = gate.data_ptr()
    if w_post is not None:
        w_post = _flat(w_post, "w_post", dtype, H, dev)
        pq = w_post.data_ptr()
    if w_pre is not None:
        w_pre = _flat(w_pre, "w_pre", dtype, H, dev)
        pp = w_pre.data_ptr()
    return (x, o, gate, w_post, w_pre), dev, (x.data_ptr(), ld_x, po, ld_o, pg, kind, ld_g, pq, pp), x.shape[0], H, dt


def _block_norm(x, o, gate, w_post, w_pre, residual_scale, eps, stats):
    keep, dev, args, T, H, dt = _norm_args(x, o, gate, w_post, w_pre)
    r = _empty(x.shape, dtype=x.dtype, device=x.device)
    h = s1 = s2 = None
    ph = p1 = p2 = 0
    if w_pre is not None:
        h = _empty(x.shape, dtype=x.dtype, device=x.device)
        ph = h.data_ptr()
    if stats:
        if w_post is not None:
            s1 = _empty(T, dtype=_f32, device=x.device)
            p1 = s1.data_ptr()
        if w_pre is not None:
            s2 = _empty(T, dtype=_f32, device=x.device)
            p2 = s2.data_ptr()
    st = binding.qmoe_block_norm(*args, residual_scale, eps, T, H, dt, r.data_ptr(), ph, p1, p2, _raw_stream(dev))
    if st:
        _failed(st)
    return r, h, NormStats(s1, s2)


def block_norm_grad(dr, dh, x, o, stats, gate=None, w_post=None, w_pre=None, residual_scale=1.0, eps=None,
                    stream=None) -> NormGrads:
    """The gradients of :func:`block_norm` for the gradients ``dr`` and ``dh``
    of its outputs (None: zero) and its own arguments; ``stats`` are the
    forward's (they hold ``eps``, taken here only so that the forward's keywords
    can be passed on)."""
    if stream is not None:
        return _elsewhere(stream, block_norm_grad, dr, dh, x, o, stats, gate, w_post, w_pre, residual_scale)
    keep, dev, args, T, H, dt = _norm_args(x, o, gate, w_post, w_pre)
    dtype, device = x.dtype, x.device
    pr = ld_r = ph = ld_h = p1 = p2 = 0
    if dr is not None:
        dr, ld_r = _norm_rows(dr, "dr", x.shape, dtype, dev)
        pr = dr.data_ptr()
    if dh is not None:
        if w_pre is None:
            _refuse("dh needs w_pre")
        dh, ld_h = _norm_rows(dh, "dh", x.shape, dtype, dev)
        ph = dh.data_ptr()
    if w_post is not None:
        s1 = _flat(stats.rstd_post, "stats.rstd_post", _f32, T, dev)
        p1 = s1.data_ptr()
    if w_pre is not None:
        s2 = _flat(stats.rstd_pre, "stats.rstd_pre", _f32, T, dev)
        p2 = s2.data_ptr()

    def like(t):
        return None if t is None else _empty(t.shape, dtype=dtype, device=device)

    dx, do, dgate, dwq, dwp = like(x), like(o), like(gate), like(w_post), like(w_pre)
    nbytes = binding.qmoe_block_norm_grad_workspace(T, H, dt)
    work = _empty(nbytes, dtype=_u8, device=device)
    st = binding.qmoe_block_norm_grad(pr, ld_r, ph, ld_h, *args, p1, p2, residual_scale, T, H, dt, dx.data_ptr(),
                                      _ptr(do), _ptr(dgate), _ptr(dwq), _ptr(dwp), work.data_ptr(), nbytes,
                                      _raw_stream(dev))
    if st:
        _failed(st)
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
