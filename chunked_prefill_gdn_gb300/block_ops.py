"""The operators of a layer beside its recurrence: what lies between two blocks
(norm, gate, scale, residual sum, norm, in one pass) and the gated feed-forward
block (include/gdn.h has the definitions).

    x, h, rstd_post, rstd_pre = block_norm_fwd(y, residual, gate, post_weight, scale, pre_weight)
    dy, dresidual, dgate, dpost_weight, dscale, dpre_weight = block_norm_bwd(dx, dh, y, x, rstd_post, rstd_pre, ...)
    y, gate, up = gated_ffn_fwd(x, w_gate, w_up, w_down)
    dx, dw_gate, dw_up, dw_down = gated_ffn_bwd(dy, x, w_gate, w_up, w_down, gate, up)

and with autograd: block_norm, gated_ffn.

Types, layouts, streams, `out` and version counters are those of layer_ops.
block_norm also takes rows in two levels (heads of a token that is a slice of a
wider projection).  The weights of the feed-forward block have the activations'
type, and so have their gradients.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch
from torch.autograd import forward_ad

from .layer_ops import _CODE, _On, _act, _apart, _like, _p, _raise, _row_stride, _workspace, _wrote

__all__ = ["block_norm_fwd", "block_norm_bwd", "block_norm", "gated_ffn_fwd", "gated_ffn_bwd", "gated_ffn",
           "GdnBlockNormDesc", "GdnFfnDesc", "GdnFfnPlanInfo"]

_F32, _I32 = torch.float32, torch.int32
_GATES = {"silu": 0, "sigmoid": 1}
_ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}


class GdnBlockNormDesc(ctypes.Structure):
    """gdn_block_norm_desc of include/gdn.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("y", "gate", "post_weight", "scale", "pre_weight")] +
                [(n, ctypes.c_int64) for n in ("outer", "inner", "D", "y_outer_stride", "y_inner_stride",
                                               "gate_outer_stride", "gate_inner_stride")] +
                [("eps", ctypes.c_float)] +
                [(n, ctypes.c_int32) for n in ("post_norm", "pre_norm", "gate_activation", "dtype", "w_dtype")])


class GdnFfnDesc(ctypes.Structure):
    """gdn_ffn_desc of include/gdn.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "w_gate", "w_up", "w_down")] +
                [(n, ctypes.c_int64) for n in ("x_stride", "M", "D", "F", "D_out")] +
                [(n, ctypes.c_int32) for n in ("activation", "dtype")])


class GdnFfnPlanInfo(ctypes.Structure):
    """gdn_ffn_plan_info of include/gdn.h."""
    _fields_ = [("path", ctypes.c_int32), ("tile", ctypes.c_int32 * 2), ("a_rows", ctypes.c_int32 * 2),
                ("products", ctypes.c_int32 * 2), ("parts", ctypes.c_int32 * 4 * 2)]


def bind(lib):
    """Argument types of these operators' C entry points."""
    vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
    norm, ffn = ctypes.POINTER(GdnBlockNormDesc), ctypes.POINTER(GdnFfnDesc)
    for name, res, args in (
            ("gdn_block_norm_fwd", i32, [norm, vp, i64, i64] + [vp] * 5),
            ("gdn_block_norm_bwd_workspace_size", sz, [norm]),
            ("gdn_block_norm_bwd", i32, [norm] + [vp, i64, i64] * 3 + [vp] * 9 + [sz, vp]),
            ("gdn_gated_ffn_fwd_workspace_size", sz, [ffn]),
            ("gdn_gated_ffn_fwd", i32, [ffn, vp, vp, vp, vp, vp, sz, vp]),
            ("gdn_gated_ffn_bwd_workspace_size", sz, [ffn, vp, i64]),
            ("gdn_gated_ffn_bwd", i32, [ffn, vp, i64] + [vp] * 8 + [sz, vp]),
            ("gdn_gated_ffn_debug", i32, [i32]),
            ("gdn_gated_ffn_plan_query", i32, [ffn, i32, vp, i64, ctypes.POINTER(GdnFfnPlanInfo)])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    global _bound
    _bound = lib


_bound = None   # the loaded library


def _lib():
    if _bound is None:
        from . import load_library
        load_library()
    return _bound


def _scratch(on, workspace, size):
    """The workspace; None where size is 0: arguments that the call refuses, and says why."""
    return _workspace(on, workspace, size) if size else None


def _bytes(ws):
    return ws.numel() if ws is not None else 0


def _status(on, check):
    return on.empty(1, _I32) if check else None


def _read_status(word, on, where):
    if word is None:
        return
    torch.cuda.current_stream(on.device).synchronize()   # the call's own, current until done()
    st = int(word.item())
    if st != 0:
        _raise(st, where + " (device check)")


def _plain(tensors):
    """Whether a call needs no autograd function: no gradients, and outside of dual
    levels, where there may be tangents (which those functions refuse)."""
    return getattr(forward_ad, "_current_level", 0) < 0 and not (
        torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors))


# -------------------------------------------------------- between two blocks

def _levels(name, t):
    """The rows of a [..., D] tensor as (size, stride) levels, neighbouring levels
    that run on into one another merged."""
    D = t.shape[-1]
    at = []
    for n, s in zip(t.shape[:-1], t.stride()[:-1]):
        if n == 1:
            continue
        if at and at[-1][1] == n * s:
            at[-1] = (at[-1][0] * n, s)
        else:
            at.append((n, s))
    if len(at) > 2:
        raise ValueError("%s: its rows are not equally spaced in two levels" % name)
    if any(s < D for _, s in at):
        raise ValueError("%s: rows overlap" % name)
    return at


def _row_levels(tensors):
    """A common (outer, inner) for the rows of several [..., D] tensors of one shape
    (the first is given), and their outer and inner strides one after the other."""
    first = tensors[0][1]
    D, strides = first.shape[-1], []
    if first.dim() == 2:            # plain rows: the path of a few tokens, bound by the host
        rows = first.shape[0]
        for name, t in tensors:
            s = t.stride(0) if t is not None and rows > 1 else D
            if s < D and rows:
                raise ValueError("%s: rows overlap" % name)
            strides += (s, s)
        return rows, 1, strides
    rows = first.numel() // D if D else 0
    if rows == 0 or all(t is None or t.is_contiguous() for _, t in tensors):
        return rows, 1, [D] * (2 * len(tensors))
    levels = [_levels(name, t) if t is not None else [] for name, t in tensors]
    inner = 1
    for (name, _), at in zip(tensors, levels):
        if len(at) == 2:
            if inner not in (1, at[1][0]):
                raise ValueError("%s: its rows are in levels of %d, another input's of %d" % (name, at[1][0], inner))
            inner = at[1][0]
    for at in levels:
        if len(at) == 2:
            strides += (at[0][1], at[1][1])
        else:
            s = at[0][1] if at else D
            strides += (s * inner, s)
    return rows // inner, inner, strides


def _norm_desc(y, gate, post_weight, scale, pre_weight, post_norm, pre_norm, activation, eps, others):
    """Checks the operator's inputs; returns (descriptor, strides of `others`)."""
    _act("y", y)
    shape, dev, dtype = y.shape, y.device, y.dtype
    D = shape[-1]
    tensors = (("y", y), ("gate", gate), *others)
    for name, t in tensors:
        if t is not None and not (t.shape == shape and t.dtype == dtype and t.device == dev and t.stride(-1) == 1):
            _like(name, t, shape, dtype, dev, strided=True)
    if activation not in _GATES:
        raise ValueError("activation must be 'silu' or 'sigmoid', got %r" % (activation,))
    if post_weight is not None and not post_norm:
        raise ValueError("post_weight needs post_norm")
    if pre_weight is not None and not pre_norm:
        raise ValueError("pre_weight needs pre_norm")
    wtype = None    # of the [D] parameters: float32 or the activations' type, all alike
    for name, t in (("post_weight", post_weight), ("scale", scale), ("pre_weight", pre_weight)):
        if t is None:
            continue
        if wtype is None:
            wtype = t.dtype
            if wtype != _F32 and wtype != dtype:
                raise TypeError("%s must be float32 or %s, got %s" % (name, dtype, wtype))
        _like(name, t, shape[-1:], wtype, dev)
    outer, inner, strides = _row_levels(tensors)
    return GdnBlockNormDesc(y.data_ptr(), _p(gate), _p(post_weight), _p(scale), _p(pre_weight), outer, inner, D,
                            *strides[:4], eps, 1 if post_norm else 0, 1 if pre_norm else 0,
                            _GATES[activation], _CODE[dtype], 1 if wtype is None else _CODE[wtype]), strides[4:]


def block_norm_fwd(y, residual=None, gate=None, post_weight=None, scale=None, pre_weight=None, post_norm: bool = True,
                   pre_norm: bool = True, activation: str = "silu", eps: float = 1e-5, out=None,
                   stream: Optional[torch.cuda.Stream] = None):
    """What lies between two blocks, over the last axis of y [..., D]: x = residual +
    scale * norm(y) * act(gate) and h = norm(x), norm(t) = t * (mean t^2 + eps)^-1/2 * weight;
    returns (x, h, rstd_post, rstd_pre), the last two float32 [...] for the backward pass.
    Each part may be left out: post_norm=False takes y itself, pre_norm=False makes no h
    (None); residual, gate, scale and the weights are optional.  gate and residual have
    y's shape; weights and scale are [D] in float32 or y's type.  activation: 'silu' or
    'sigmoid'.  `out` receives x."""
    desc, (ro, ri) = _norm_desc(y, gate, post_weight, scale, pre_weight, post_norm, pre_norm, activation, eps,
                                   (("residual", residual),))
    dtype, dev = y.dtype, y.device
    if out is not None:
        _like("out", out, y.shape, dtype, dev)
        _apart(out, (("y", y), ("residual", residual), ("gate", gate), ("post_weight", post_weight), ("scale", scale),
                     ("pre_weight", pre_weight)), same=("y", "residual", "gate"))
    on = _On(dev, stream)
    try:
        x = out if out is not None else on.empty(y.shape, dtype)
        h = on.empty(y.shape, dtype) if pre_norm else None
        rp = on.empty(y.shape[:-1], _F32) if post_norm else None
        rn = on.empty(y.shape[:-1], _F32) if pre_norm else None
        rc = _lib().gdn_block_norm_fwd(desc, _p(residual), ro, ri, x.data_ptr(), _p(h), _p(rp), _p(rn), on.raw)
        if rc != 0:
            _raise(rc, "gdn_block_norm_fwd")
        _wrote(None, out)
    finally:
        on.done()
    return x, h, rp, rn


def block_norm_bwd(dx, dh, y, x, rstd_post, rstd_pre, gate=None, post_weight=None, scale=None, pre_weight=None,
                   activation: str = "silu", residual: bool = True, workspace=None,
                   stream: Optional[torch.cuda.Stream] = None):
    """Gradients of block_norm_fwd from dx and dh (the gradients of x and h; dh None
    without the second norm, dx None where x is used for h only), the forward pass's y, x
    and rstd (None for a norm that was left out): (dy, dresidual, dgate, dpost_weight,
    dscale, dpre_weight).  dresidual is the gradient of x as a whole (None with
    residual=False); the parameters' gradients are float32, None for those not given."""
    post, pre = rstd_post is not None, rstd_pre is not None
    if pre and (dh is None or x is None):
        raise ValueError("the second norm's backward pass needs dh and x")
    if not pre and (dh is not None or dx is None):
        raise ValueError("without the second norm dx is needed and there is no dh")
    xs = x if pre else None
    desc, strides = _norm_desc(y, gate, post_weight, scale, pre_weight, post, pre, activation, 0.0,
                               (("dx", dx), ("dh", dh), ("x", xs)))
    D, dtype, dev = y.shape[-1], y.dtype, y.device
    for name, t in (("rstd_post", rstd_post), ("rstd_pre", rstd_pre)):
        if t is not None:
            _like(name, t, y.shape[:-1], _F32, dev)
    lib = _lib()
    on = _On(dev, stream)
    try:
        dy = on.empty(y.shape, dtype)
        dr = on.empty(y.shape, dtype) if residual else None
        dz = on.empty(y.shape, dtype) if gate is not None else None
        given = [t is not None for t in (post_weight, scale, pre_weight)]
        grads, ws = [None] * 3, None
        if any(given):
            rows = iter(on.empty((sum(given), D), _F32).unbind(0))
            grads = [next(rows) if g else None for g in given]
            ws = _scratch(on, workspace, lib.gdn_block_norm_bwd_workspace_size(desc))
        rc = lib.gdn_block_norm_bwd(desc, _p(dx), *strides[:2], _p(dh), *strides[2:4], _p(xs), *strides[4:], _p(rstd_post),
                                    _p(rstd_pre), dy.data_ptr(), _p(dr), _p(dz), *(_p(t) for t in grads), _p(ws),
                                    _bytes(ws), on.raw)
        if rc != 0:
            _raise(rc, "gdn_block_norm_bwd")
    finally:
        on.done()
    return (dy, dr, dz, *grads)


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, residual, gate, post_weight, scale, pre_weight, post_norm, pre_norm, activation, eps):
        x, h, rp, rn = block_norm_fwd(y, residual, gate, post_weight, scale, pre_weight, post_norm, pre_norm, activation,
                                      eps)
        ctx.save_for_backward(y, x if pre_norm else None, rp, rn, gate, post_weight, scale, pre_weight)
        ctx.activation, ctx.residual = activation, residual is not None
        ctx.types = [None if t is None else t.dtype for t in (post_weight, scale, pre_weight)]
        ctx.set_materialize_grads(False)
        return x, h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dx, dh):
        y, x, rp, rn, gate, post_weight, scale, pre_weight = ctx.saved_tensors
        if dx is None and dh is None:
            return (None,) * 10
        if rn is not None and dh is None:
            dh = torch.zeros(y.shape, dtype=y.dtype, device=y.device)
        dy, dr, dz, *params = block_norm_bwd(
            dx.contiguous() if dx is not None else None, dh.contiguous() if dh is not None else None, y, x, rp, rn, gate,
            post_weight, scale, pre_weight, ctx.activation, residual=ctx.residual)
        return (dy, dr, dz, *(None if g is None else g.to(t) for g, t in zip(params, ctx.types)), None, None, None, None)


def block_norm(y, residual=None, gate=None, post_weight=None, scale=None, pre_weight=None, post_norm: bool = True,
               pre_norm: bool = True, activation: str = "silu", eps: float = 1e-5):
    """block_norm_fwd with autograd (every tensor); returns (x, h), h None without
    pre_norm."""
    if _plain((y, residual, gate, post_weight, scale, pre_weight)):
        return block_norm_fwd(y, residual, gate, post_weight, scale, pre_weight, post_norm, pre_norm, activation, eps)[:2]
    return _BlockNorm.apply(y, residual, gate, post_weight, scale, pre_weight, post_norm, pre_norm, activation, eps)


# ---------------------------------------------------- the gated feed-forward block

def _ffn_desc(x, w_gate, w_up, w_down, activation):
    """Checks the block's inputs; returns (descriptor, M, F, D_out)."""
    _act("x", x)
    if w_gate.dim() != 2 or w_down.dim() != 2:
        raise ValueError("w_gate and w_up must be [F, D], w_down [D_out, F]")
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be 'silu' or 'gelu_tanh', got %r" % (activation,))
    D, F, out = x.shape[-1], w_gate.shape[0], w_down.shape[0]
    for name, w, shape in (("w_gate", w_gate, (F, D)), ("w_up", w_up, (F, D)), ("w_down", w_down, (out, F))):
        _like(name, w, shape, x.dtype, x.device)
    M = x.numel() // D if D else 0
    return GdnFfnDesc(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), _row_stride("x", x), M, D, F,
                      out, _ACTIVATIONS[activation], _CODE[x.dtype]), M, F, out


def gated_ffn_fwd(x, w_gate, w_up, w_down, activation: str = "silu", save: bool = False, out=None, workspace=None,
                  stream: Optional[torch.cuda.Stream] = None, check: bool = False):
    """The gated feed-forward block of x [..., D]: y = (act(x w_gate^T) * (x w_up^T)) w_down^T
    with w_gate, w_up [F, D] and w_down [D_out, F] in x's type; returns (y [..., D_out],
    gate, up), gate and up the two projections [..., F] for the backward pass (None without
    save).  activation: 'silu' or 'gelu_tanh'.  check=True waits for the call and raises
    GdnError where a bounded wait inside a kernel ran out (the outputs are then not those of
    the inputs); without it nothing is said."""
    desc, M, F, n_out = _ffn_desc(x, w_gate, w_up, w_down, activation)
    lead, dtype, dev = x.shape[:-1], x.dtype, x.device
    if out is not None:
        _like("out", out, (*lead, n_out), dtype, dev)
        _apart(out, (("x", x), ("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)))
    lib = _lib()
    on = _On(dev, stream)
    try:
        y = out if out is not None else on.empty((*lead, n_out), dtype)
        gate, up = (on.empty((*lead, F), dtype), on.empty((*lead, F), dtype)) if save else (None, None)
        ws = _scratch(on, workspace, lib.gdn_gated_ffn_fwd_workspace_size(desc))
        word = _status(on, check)
        rc = lib.gdn_gated_ffn_fwd(desc, y.data_ptr(), _p(gate), _p(up), _p(word), _p(ws), _bytes(ws), on.raw)
        if rc != 0:
            _raise(rc, "gdn_gated_ffn_fwd")
        _wrote(None, out)
        _read_status(word, on, "gdn_gated_ffn_fwd")
    finally:
        on.done()
    return y, gate, up


def gated_ffn_bwd(dy, x, w_gate, w_up, w_down, gate, up, activation: str = "silu", needs=(True, True, True, True),
                  workspace=None, stream: Optional[torch.cuda.Stream] = None, check: bool = False):
    """Gradients of gated_ffn_fwd: (dx, dw_gate, dw_up, dw_down) in x's type from dy and the
    forward pass's gate and up; `needs` says which are wanted (None for the others).  check as
    in gated_ffn_fwd."""
    desc, M, F, n_out = _ffn_desc(x, w_gate, w_up, w_down, activation)
    lead, dtype, dev = x.shape[:-1], x.dtype, x.device
    _like("dy", dy, (*lead, n_out), dtype, dev, strided=True)
    _like("gate", gate, (*lead, F), dtype, dev)
    _like("up", up, (*lead, F), dtype, dev)
    stride = _row_stride("dy", dy)
    lib = _lib()
    on = _On(dev, stream)
    try:
        grads = [on.empty(t.shape, dtype) if need else None for t, need in zip((x, w_gate, w_up, w_down), needs)]
        ws = _scratch(on, workspace, lib.gdn_gated_ffn_bwd_workspace_size(desc, dy.data_ptr(), stride))
        word = _status(on, check)
        rc = lib.gdn_gated_ffn_bwd(desc, dy.data_ptr(), stride, gate.data_ptr(), up.data_ptr(), *(_p(t) for t in grads),
                                   _p(word), _p(ws), _bytes(ws), on.raw)
        if rc != 0:
            _raise(rc, "gdn_gated_ffn_bwd")
        _read_status(word, on, "gdn_gated_ffn_bwd")
    finally:
        on.done()
    return tuple(grads)


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, activation, save, check):
        y, gate, up = gated_ffn_fwd(x, w_gate, w_up, w_down, activation, save=save, check=check)
        ctx.save_for_backward(x, w_gate, w_up, w_down, gate, up)
        ctx.activation, ctx.check = activation, check
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w_gate, w_up, w_down, gate, up = ctx.saved_tensors
        return (*gated_ffn_bwd(dy.contiguous(), x, w_gate, w_up, w_down, gate, up, ctx.activation,
                               needs=ctx.needs_input_grad[:4], check=ctx.check), None, None, None)


def gated_ffn(x, w_gate, w_up, w_down, activation: str = "silu", check: bool = False):
    """gated_ffn_fwd with autograd (x and the weights); returns y.  check as in gated_ffn_fwd,
    in the backward pass too."""
    tensors = x, w_gate, w_up, w_down
    if _plain(tensors):
        return gated_ffn_fwd(*tensors, activation, check=check)[0]
    save = torch.is_grad_enabled() and any(t.requires_grad for t in tensors)
    return _GatedFfn.apply(*tensors, activation, save, check)
