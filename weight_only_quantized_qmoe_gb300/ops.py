"""Operators around the expert layer, on torch CUDA tensors.

Calls of the C entry points of the same names (include/qmoe.h, the operators'
part), which define what each computes:

* :func:`expert_route` and its gradient :func:`expert_route_grad`: the experts
  of every token by softmax or sigmoid scores, and their weights;
* :func:`expert_sort`, :func:`dispatch`, :func:`combine` and the gradients
  :func:`dispatch_grad`, :func:`combine_grad`: routes sorted by expert, token
  rows taken into expert order and summed back with their weights;
* :func:`mx4_quantize`, :func:`mx4_dequantize`, :func:`mx4_matmul`:
  microscaled 4-bit floating point rows and their product, dense or grouped by
  expert;
* :func:`fp8_quantize`, :func:`fp8_dequantize`, :func:`fp8_matmul`: 8-bit
  floating point rows and weights with a scale for each block of 128, and their
  products, dense or grouped by expert, also with the weights transposed;
* :func:`weight_grad`: the gradient of the experts' weights; :func:`fp8_linear`:
  the 8-bit product of 16-bit rows, forward and backward;
* :func:`block_norm`, :func:`block_norm_grad`: the norms on either side of a
  block with the gate of its output and the residual scale.

``expert_route``, ``dispatch``, ``combine``, ``fp8_linear`` and ``block_norm``
take part in automatic differentiation where an input requires a gradient;
forward mode is refused.
Refused arguments raise
:class:`~weight_only_quantized_qmoe_gb300.QMoEError`.  Every call runs on the
current stream, or on ``stream=``: its outputs then belong to that stream (a
reader on another stream has to wait for it), and its inputs have to be ready
there.  Tensors whose last axis is not contiguous are copied first.

Arguments are checked and outputs allocated by the compiled module
``_ops_torch`` (csrc/qmoe_ops_torch.cpp); there is no fallback without it.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import QMoEError, binding

try:
    from . import _ops_torch as _c
except ImportError as e:   # pragma: no cover
    raise RuntimeError("_ops_torch.so is missing or does not belong to this torch: build it with "
                       "weight_only_quantized_qmoe_gb300.build.build()") from e

_DTYPES = {torch.float32: binding.QMOE_F32, torch.float16: binding.QMOE_F16, torch.bfloat16: binding.QMOE_BF16}
_SCORING = {"softmax": binding.QMOE_SCORE_SOFTMAX, "sigmoid": binding.QMOE_SCORE_SIGMOID}
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


class Route(NamedTuple):
    """The experts of T tokens, best first: ``ids`` int32 [T, k] (-1: none) and
    ``weights`` float32 [T, k]."""

    ids: torch.Tensor
    weights: torch.Tensor


class MX4Tensor(NamedTuple):
    """Microscaled 4-bit rows [..., N, cols]: ``codes`` uint8 [..., N, 16 * nb]
    and ``scales`` uint8 [..., ceil(nb / 4), N, 4], nb = ceil(cols / 32).  Codes
    past ``cols`` have to be zeros, scales past nb are not used."""

    codes: torch.Tensor
    scales: torch.Tensor
    cols: int


class FP8Tensor(NamedTuple):
    """8-bit rows [..., N, cols]: ``codes`` uint8 (E4M3) [..., N, 16 * ceil(cols /
    16)] and ``scales`` uint8 (E8M0) of 128 values of a row, [..., ceil(nb / 4), N,
    4] with nb = ceil(cols / 128), or with ``square`` of 128 x 128 blocks, [...,
    ceil(N / 128), nb].  Codes past ``cols`` and scales past nb are not used."""

    codes: torch.Tensor
    scales: torch.Tensor
    cols: int
    square: bool


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


_c.setup(QMoEError, ExpertPlan, MX4Tensor, NormStats, NormGrads, Route, FP8Tensor)


def _refuse(msg):
    raise QMoEError(binding.QMOE_ERR_INVALID_ARG, msg)


def _type_code(dtype, name):
    code = _DTYPES.get(dtype)
    if code is None:
        _refuse(f"{name} {dtype}: float32, float16 or bfloat16")
    return code


def _elsewhere(stream, call, *args):
    """call(...) on `stream`; the inputs' memory is kept until it is done there."""
    with torch.cuda.stream(stream):
        out = call(*args)
    for a in args:
        for t in a if isinstance(a, tuple) else (a,):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
    return out


def _differentiable(*tensors):
    if forward_ad._current_level >= 0:   # inside a dual level: a tangent is not to be lost without a word
        for t in tensors:
            if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
                _refuse("forward-mode differentiation is not supported")
    if torch.is_grad_enabled():
        for t in tensors:
            if getattr(t, "requires_grad", False):
                return True
    return False


def poll_status() -> int:
    """QMOE_OK, or QMOE_ERR_TIMEOUT if a bounded wait of an operator ran out
    since the last call (read and cleared; synchronises the device)."""
    return binding.qmoe_op_poll_status()


# --- the router ----------------------------------------------------------------
class _RouteFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, bias, scoring, groups, top_groups, group_best, renormalize, scale):
        r = _c.expert_route(logits, k, bias, scoring, groups, top_groups, group_best, renormalize, scale)
        ctx.save_for_backward(logits, r.ids)
        ctx.how = scoring, renormalize, scale
        ctx.mark_non_differentiable(r.ids)
        ctx.set_materialize_grads(False)
        return r.ids, r.weights

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dweights):
        logits, ids = ctx.saved_tensors
        dlogits = None if dweights is None else _c.expert_route_grad(dweights, logits, ids, *ctx.how)
        return (dlogits,) + (None,) * 8


def _scoring(scoring):
    code = _SCORING.get(scoring)
    if code is None:
        _refuse(f"scoring {scoring!r}: 'softmax' or 'sigmoid'")
    return code


def expert_route(logits, k, scoring="softmax", bias=None, groups=1, top_groups=None, group_best=1, renormalize=True, scale=1.0,
                 stream=None) -> Route:
    """The k experts of each token of logits [T, E], best first.

    Scores are the softmax or the sigmoid of the logits; with ``bias`` (float32
    [E]) experts are chosen by score + bias, but weighted by their scores.  With
    ``top_groups`` only the experts of that many of the ``groups`` equal runs of
    experts are chosen from, the groups with the largest sum of their
    ``group_best`` (1 or 2) best.  Ties go to the lower index.  Weights are scale *
    score, with ``renormalize`` divided by the sum of the chosen scores.  Experts
    with a logit of -inf are not chosen (id -1, weight 0 where none is left).  The
    weights have a gradient to the logits; the choice, and so the bias, has none."""
    if stream is not None:
        return _elsewhere(stream, expert_route, logits, k, scoring, bias, groups, top_groups, group_best, renormalize, scale)
    args = logits, k, bias, _scoring(scoring), groups, groups if top_groups is None else top_groups, group_best, renormalize, scale
    return Route(*_RouteFn.apply(*args)) if _differentiable(logits) else _c.expert_route(*args)


def expert_route_grad(dweights, logits, ids, scoring="softmax", renormalize=True, scale=1.0, stream=None):
    """The gradient of the weights of :func:`expert_route`: dlogits [T, E] of
    dweights [T, k] for the ids chosen."""
    if stream is not None:
        return _elsewhere(stream, expert_route_grad, dweights, logits, ids, scoring, renormalize, scale)
    return _c.expert_route_grad(dweights, logits, ids, _scoring(scoring), renormalize, scale)


# --- tokens sorted by expert and back -----------------------------------------
def expert_sort(ids, experts, stream=None) -> ExpertPlan:
    """Sort the routes ids [T, k] (int32 or int64) by expert, stably.  Ids
    outside [0, experts) drop their route."""
    if stream is not None:
        return _elsewhere(stream, expert_sort, ids, experts)
    return _c.expert_sort(ids, experts)


class _DispatchFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        out = _c.dispatch(x, plan)
        ctx.save_for_backward(plan.pos, plan.offsets)
        ctx.sizes = plan.k, plan.experts
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        return dispatch_grad(dxs, ExpertPlan(None, *ctx.saved_tensors, *ctx.sizes)), None


class _CombineFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, plan):
        out = _c.combine(y, weights, plan)
        ctx.save_for_backward(y, weights, plan.pos, plan.offsets)
        ctx.sizes = plan.k, plan.experts
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, weights, pos, offsets = ctx.saved_tensors
        plan = ExpertPlan(None, pos, offsets, *ctx.sizes)
        dy, dw = combine_grad(dout, y, weights, plan, ctx.needs_input_grad[0],
                              weights is not None and ctx.needs_input_grad[1])
        return dy, None if dw is None else dw.reshape(weights.shape), None


def dispatch(x, plan, stream=None):
    """Token rows x [T, H] into expert order [T * k, H] (zeros past the rows in
    use)."""
    if stream is not None:
        return _elsewhere(stream, dispatch, x, plan)
    return _DispatchFn.apply(x, plan) if _differentiable(x) else _c.dispatch(x, plan)


def dispatch_grad(dxs, plan, stream=None):
    """The gradient of :func:`dispatch`: dx [T, H] of dxs [T * k, H]."""
    if stream is not None:
        return _elsewhere(stream, dispatch_grad, dxs, plan)
    return _c.combine(dxs, None, plan)


def combine(y, weights, plan, stream=None):
    """Expert rows y [T * k, H] back to token order [T, H], weighted with
    ``weights`` (float32 [T, k], or None for ones)."""
    if stream is not None:
        return _elsewhere(stream, combine, y, weights, plan)
    return _CombineFn.apply(y, weights, plan) if _differentiable(y, weights) else _c.combine(y, weights, plan)


def combine_grad(dout, y, weights, plan, need_dy=True, need_dweights=True, stream=None):
    """The gradients of :func:`combine`: (dy [T * k, H], dweights float32 [T, k])
    of dout [T, H]; one that is not needed is None."""
    if stream is not None:
        return _elsewhere(stream, combine_grad, dout, y, weights, plan, need_dy, need_dweights)
    return _c.combine_grad(dout, y, weights, plan, need_dy, need_dweights)


# --- microscaled 4-bit floating point -----------------------------------------
def mx4_quantize(x, plan=None, activation=None, stream=None) -> MX4Tensor:
    """Quantise the rows of x [..., N, K].  With ``plan`` the rows x [T, K] are
    written in expert order [T * k, K].  With ``activation`` "swiglu" or
    "geglu" a row holds gate | up (2 K values) and act(gate) * up is quantised."""
    if stream is not None:
        return _elsewhere(stream, mx4_quantize, x, plan, activation)
    act = _ACTIVATIONS.get(activation)
    if act is None:
        _refuse(f"activation {activation!r}: None, 'swiglu' or 'geglu'")
    return _c.mx4_quantize(x, plan, act)


def mx4_dequantize(q, dtype=torch.bfloat16, stream=None):
    """The values [..., N, cols] of an :class:`MX4Tensor`."""
    if stream is not None:
        return _elsewhere(stream, mx4_dequantize, q, dtype)
    return _c.mx4_dequantize(q, _type_code(dtype, "dtype"))


def mx4_matmul(a, w, plan=None, out_dtype=torch.bfloat16, stream=None):
    """a [R, K] times the transpose of w: [N, K] for all rows, or with ``plan``
    [experts, N, K], each expert's rows with its own (zeros past the rows in
    use).  Returns [R, N]."""
    if stream is not None:
        return _elsewhere(stream, mx4_matmul, a, w, plan, out_dtype)
    return _c.mx4_matmul(a, w, plan, _type_code(out_dtype, "out_dtype"))


# --- 8-bit floating point ------------------------------------------------------
def fp8_quantize(x, plan=None, activation=None, square=False, stream=None) -> FP8Tensor:
    """Quantise the rows of x [..., N, K] in blocks of 128 values; ``plan`` and
    ``activation`` as in :func:`mx4_quantize`.  With ``square`` in blocks of 128 x
    128: weights, one copy of which serves the product and the transposed one."""
    if stream is not None:
        return _elsewhere(stream, fp8_quantize, x, plan, activation, square)
    act = _ACTIVATIONS.get(activation)
    if act is None:
        _refuse(f"activation {activation!r}: None, 'swiglu' or 'geglu'")
    return _c.fp8_quantize(x, plan, act, square)


def fp8_dequantize(q, dtype=torch.bfloat16, stream=None):
    """The values [..., N, cols] of an :class:`FP8Tensor`."""
    if stream is not None:
        return _elsewhere(stream, fp8_dequantize, q, dtype)
    return _c.fp8_dequantize(q, _type_code(dtype, "dtype"))


def fp8_matmul(a, w, plan=None, transpose=False, out_dtype=torch.bfloat16, stream=None):
    """a [R, K] times the transpose of w [N, K] (``square`` blocks), or with
    ``transpose`` a [R, N] times w; with ``plan`` w is [experts, N, K], each expert's
    rows with its own (zeros past the rows in use).  Returns [R, N] or [R, K]."""
    if stream is not None:
        return _elsewhere(stream, fp8_matmul, a, w, plan, transpose, out_dtype)
    return _c.fp8_matmul(a, w, plan, transpose, _type_code(out_dtype, "out_dtype"))


# --- gradient of the experts' weights --------------------------------------------
def weight_grad(dy, x, plan=None, out_dtype=None, stream=None):
    """The sum over the rows of dy [R, N] outer x [R, K] (both float16 or both
    bfloat16): [N, K], or with ``plan`` [experts, N, K], over each expert's rows (in
    expert order).  ``out_dtype``: the operands' by default."""
    if stream is not None:
        return _elsewhere(stream, weight_grad, dy, x, plan, out_dtype)
    return _c.weight_grad(dy, x, plan, _type_code(getattr(dy, "dtype", None) if out_dtype is None else out_dtype, "out_dtype"))


class _LinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, quantized, plan):
        if quantized is None:
            quantized = _c.fp8_quantize(w, None, binding.QMOE_ACT_NONE, True)
        y = _c.fp8_matmul(_c.fp8_quantize(x, None, binding.QMOE_ACT_NONE, False), quantized, plan, False, _DTYPES[x.dtype])
        need_w = w is not None and ctx.needs_input_grad[1]
        ctx.save_for_backward(x if need_w else None, quantized.codes, quantized.scales,
                              *((None, None) if plan is None else (plan.pos, plan.offsets)))
        ctx.sizes = quantized.cols, None if plan is None else (plan.k, plan.experts), (w.shape, _DTYPES[w.dtype]) if need_w else None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, codes, scales, pos, offsets = ctx.saved_tensors
        cols, sizes, weight = ctx.sizes
        plan = None if sizes is None else ExpertPlan(None, pos, offsets, *sizes)
        dx = dw = None
        if ctx.needs_input_grad[0]:
            q = _c.fp8_quantize(dy, None, binding.QMOE_ACT_NONE, False)
            dx = _c.fp8_matmul(q, FP8Tensor(codes, scales, cols, True), plan, True, _DTYPES[dy.dtype])
        if weight is not None:
            dw = _c.weight_grad(dy, x, plan, weight[1]).reshape(weight[0])
        return dx, dw, None, None


def fp8_linear(x, w, plan=None, stream=None):
    """y = x times the transpose of w, with rows and weights quantised to 8 bits
    on the way (:func:`fp8_quantize`, weights in square blocks; :func:`fp8_matmul`).

    ``x`` [R, K] is float16 or bfloat16, y [R, N] has its type; ``w`` [N, K], or
    with ``plan`` [experts, N, K] (x in expert order), is a tensor of any of the
    three types, quantised in each call, or an :class:`FP8Tensor`.  Gradients pass
    the roundings unchanged: dx is the product of the quantised dy with the
    quantised weights, dw (of a tensor w, in its type) the :func:`weight_grad` of
    dy and x as they are."""
    if stream is not None:
        return _elsewhere(stream, fp8_linear, x, w, plan)
    if not isinstance(x, torch.Tensor) or not isinstance(w, (torch.Tensor, FP8Tensor)):
        _refuse("x must be a CUDA tensor, w one or an FP8Tensor")
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise QMoEError(binding.QMOE_ERR_UNSUPPORTED, f"x is {x.dtype}: float16 or bfloat16")
    w, quantized = (None, w) if isinstance(w, FP8Tensor) else (w, None)
    if _differentiable(x, w):
        return _LinearFn.apply(x, w, quantized, plan)
    if quantized is None:
        quantized = _c.fp8_quantize(w, None, binding.QMOE_ACT_NONE, True)
    return _c.fp8_matmul(_c.fp8_quantize(x, None, binding.QMOE_ACT_NONE, False), quantized, plan, False, _DTYPES[x.dtype])


# --- norms around a block ------------------------------------------------------
class _BlockNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, o, gate, w_post, w_pre, residual_scale, eps):
        r, h, stats = _c.block_norm(x, o, gate, w_post, w_pre, residual_scale, eps, True)
        ctx.save_for_backward(x, o, gate, w_post, w_pre, *stats)
        ctx.residual_scale = residual_scale
        ctx.set_materialize_grads(False)
        return r, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dr, dh):
        x, o, gate, w_post, w_pre, s1, s2 = ctx.saved_tensors
        g = _c.block_norm_grad(x, o, gate, w_post, w_pre, dr, dh, s1, s2, ctx.residual_scale)
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
    if not return_stats and _differentiable(x, o, gate, w_post, w_pre):
        return _BlockNormFn.apply(x, o, gate, w_post, w_pre, residual_scale, eps)
    return _c.block_norm(x, o, gate, w_post, w_pre, residual_scale, eps, return_stats)


def block_norm_grad(dr, dh, x, o, stats, gate=None, w_post=None, w_pre=None, residual_scale=1.0, eps=None,
                    stream=None) -> NormGrads:
    """The gradients of :func:`block_norm` for the gradients ``dr`` and ``dh``
    of its outputs (None: zero) and its own arguments; ``stats`` are the
    forward's (they hold ``eps``, taken here only so that the forward's keywords
    can be passed on)."""
    if stream is not None:
        return _elsewhere(stream, block_norm_grad, dr, dh, x, o, stats, gate, w_post, w_pre, residual_scale)
    return _c.block_norm_grad(x, o, gate, w_post, w_pre, dr, dh, stats[0], stats[1], residual_scale)


__all__ = ["ExpertPlan", "Route", "MX4Tensor", "FP8Tensor", "NormStats", "NormGrads", "expert_route", "expert_route_grad",
           "fp8_quantize", "fp8_dequantize", "fp8_matmul", "fp8_linear", "weight_grad", "expert_sort", "dispatch", "dispatch_grad", "combine",
           "combine_grad", "mx4_quantize", "mx4_dequantize", "mx4_matmul", "block_norm", "block_norm_grad",
           "poll_status"]
