"""The operators of a layer's blocks beside the recurrence: the gated feed-forward
block (include/gdn.h has the definitions).

    y, gate, up = gated_ffn_fwd(x, w_gate, w_up, w_down)
    dx, dw_gate, dw_up, dw_down = gated_ffn_bwd(dy, x, w_gate, w_up, w_down, gate, up)

and with autograd: gated_ffn.

Types, layouts, streams, `out` and version counters are those of layer_ops.  The
weights of the feed-forward block have the activations' type, and so have their
gradients.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .layer_ops import _CODE, _On, _act, _apart, _like, _p, _raise, _row_stride, _workspace, _wrote

__all__ = ["gated_ffn_fwd", "gated_ffn_bwd", "gated_ffn", "GdnFfnDesc"]

_I32 = torch.int32
_ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}


class GdnFfnDesc(ctypes.Structure):
    """gdn_ffn_desc of include/gdn.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "w_gate", "w_up", "w_down")] +
                [(n, ctypes.c_int64) for n in ("x_stride", "M", "D", "F", "D_out")] +
                [(n, ctypes.c_int32) for n in ("activation", "dtype")])


def bind(lib):
    """Argument types of these operators' C entry points."""
    vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
    ffn = ctypes.POINTER(GdnFfnDesc)
    for name, res, args in (
            ("gdn_gated_ffn_fwd_workspace_size", sz, [ffn]),
            ("gdn_gated_ffn_fwd", i32, [ffn, vp, vp, vp, vp, vp, sz, vp]),
            ("gdn_gated_ffn_bwd_workspace_size", sz, [ffn, vp, i64]),
            ("gdn_gated_ffn_bwd", i32, [ffn, vp, i64] + [vp] * 8 + [sz, vp])):
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


def _status(on, check):
    return on.empty(1, _I32) if check else None


def _read_status(word, on, where):
    if word is None:
        return
    torch.cuda.current_stream(on.device).synchronize()   # the call's own, current until done()
    st = int(word.item())
    if st != 0:
        _raise(st, where + " (device check)")


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
    save).  activation: 'silu' or 'gelu_tanh'."""
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
        ws = _workspace(on, workspace, lib.gdn_gated_ffn_fwd_workspace_size(desc))
        word = _status(on, check)
        rc = lib.gdn_gated_ffn_fwd(desc, y.data_ptr(), _p(gate), _p(up), _p(word), ws.data_ptr(), ws.numel(), on.raw)
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
    forward pass's gate and up; `needs` says which are wanted (None for the others)."""
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
        ws = _workspace(on, workspace, lib.gdn_gated_ffn_bwd_workspace_size(desc, dy.data_ptr(), stride))
        word = _status(on, check)
        rc = lib.gdn_gated_ffn_bwd(desc, dy.data_ptr(), stride, gate.data_ptr(), up.data_ptr(), *(_p(t) for t in grads),
                                   _p(word), ws.data_ptr(), ws.numel(), on.raw)
        if rc != 0:
            _raise(rc, "gdn_gated_ffn_bwd")
        _read_status(word, on, "gdn_gated_ffn_bwd")
    finally:
        on.done()
    return tuple(grads)


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, activation, save):
        y, gate, up = gated_ffn_fwd(x, w_gate, w_up, w_down, activation, save=save)
        ctx.save_for_backward(x, w_gate, w_up, w_down, gate, up)
        ctx.activation = activation
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w_gate, w_up, w_down, gate, up = ctx.saved_tensors
        return (*gated_ffn_bwd(dy.contiguous(), x, w_gate, w_up, w_down, gate, up, ctx.activation,
                               needs=ctx.needs_input_grad[:4]), None, None)


def gated_ffn(x, w_gate, w_up, w_down, activation: str = "silu"):
    """gated_ffn_fwd with autograd (x and the weights); returns y."""
    save = torch.is_grad_enabled() and any(t.requires_grad for t in (x, w_gate, w_up, w_down))
    return _GatedFfn.apply(x, w_gate, w_up, w_down, activation, save)
