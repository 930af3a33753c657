"""The layer operators around the gated delta rule: layer norm, the short causal
convolution, the selective state space scan, and the single-token forms that
serve a cached state (include/gdn.h has the definitions).

    y, mean, rstd = layer_norm_fwd(x, weight, bias)
    dx, dw, db    = layer_norm_bwd(dy, x, mean, rstd, weight)
    y, state      = causal_conv_fwd(x, weight, bias, initial_state, cu_seqlens)
    dx, dw, db, d_state = causal_conv_bwd(dy, x, weight, bias, ...)
    y             = causal_conv_step(x, state, weight, bias)           # state in place
    y, state      = selective_scan_fwd(x, dt, A, B, C, D, z, dt_bias, ...)
    dx, ddt, dA, dB, dC, dD, dz, d_dt_bias, d_state = selective_scan_bwd(dy, x, dt, A, B, C, ...)
    y             = selective_scan_step(x, dt, A, B, C, state, ...)    # state in place
    o             = gated_delta_step(q, k, v, g, beta, state)          # state in place

and with autograd: layer_norm, causal_conv, selective_scan.

As in the rest of the package these functions only marshal arguments.
Activations are bfloat16 or float32; they may be strided views as long as the
last axis is contiguous (a slice of a wider projection), everything else is
contiguous.  Gradients of activations come in the activations' type, gradients
of parameters in float32.

`out` must not overlap an input (refused): only layer_norm_fwd, selective_scan_fwd
and the steps of the convolution and the scan may be given x (the scan also dt or
z) itself.

The functions run on the current stream, or on `stream`.  A given stream is not
made to wait for the one its inputs were written on, and inputs stay alive until
it has read them: that order is the caller's, as for any tensor used on another
stream than its own.

What a call writes into a tensor of the caller's (a state, `out`) counts as an
in-place operation: autograd refuses to use that tensor's earlier value in a
backward pass.  The functions with out=, the steps and the *_fwd and *_bwd forms
record nothing for autograd themselves.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version as _increment_version

__all__ = ["layer_norm_fwd", "layer_norm_bwd", "layer_norm", "causal_conv_fwd", "causal_conv_bwd", "causal_conv_step",
           "causal_conv", "selective_scan_fwd", "selective_scan_bwd", "selective_scan_step", "selective_scan",
           "gated_delta_step", "GdnScanDesc"]

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_CODE = {torch.bfloat16: 0, torch.float32: 1}


class GdnScanDesc(ctypes.Structure):
    """gdn_scan_desc of include/gdn.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "dt", "z", "B_", "C_", "A", "D_skip", "dt_bias",
                                                "initial_state", "cu_seqlens")] +
                [(n, ctypes.c_int64) for n in ("x_batch_stride", "x_token_stride", "dt_batch_stride",
                                               "dt_token_stride", "z_batch_stride", "z_token_stride",
                                               "b_batch_stride", "b_token_stride", "c_batch_stride",
                                               "c_token_stride")] +
                [(n, ctypes.c_int32) for n in ("B", "T", "D", "N", "n_seqs", "dt_softplus", "dtype", "reserved")])


def bind(lib):
    """Argument types of the layer operators' C entry points."""
    vp, sz, i32, i64, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    desc = ctypes.POINTER(GdnScanDesc)
    for name, res, args in (
            ("gdn_layer_norm_fwd", i32, [vp, i64, vp, vp, i32, f32, i64, i32, i32, vp, vp, vp, vp]),
            ("gdn_layer_norm_bwd_workspace_size", sz, [i64, i32]),
            ("gdn_layer_norm_bwd", i32, [vp, i64, vp, i64, vp, vp, vp, i32, i64, i32, i32, vp, vp, vp, vp, sz, vp]),
            ("gdn_causal_conv_fwd", i32, [vp, i64, i64, vp, vp, i32, vp, vp] + [i32] * 7 + [vp, vp, vp, vp]),
            ("gdn_causal_conv_bwd_workspace_size", sz, [i32] * 4),
            ("gdn_causal_conv_bwd", i32, [vp, i64, i64, vp, i64, i64, vp, vp, i32, vp, vp, vp] + [i32] * 7 +
             [vp] * 5 + [vp, sz, vp]),
            ("gdn_causal_conv_step", i32, [vp, i64, vp, vp, i32, vp, vp] + [i32] * 6 + [vp, vp]),
            ("gdn_selective_scan_fwd_workspace_size", sz, [i32] * 4),
            ("gdn_selective_scan_fwd", i32, [desc, vp, vp, vp, vp, sz, vp]),
            ("gdn_selective_scan_bwd_workspace_size", sz, [i32] * 4),
            ("gdn_selective_scan_bwd", i32, [desc, vp, i64, i64] + [vp] * 12 + [sz, vp]),
            ("gdn_selective_scan_step", i32, [desc, vp, vp, i32, vp, vp]),
            ("gdn_delta_step", i32, [vp, i64, vp, i64, vp, i64] + [vp] * 4 + [i32, f32] + [i32] * 6 + [vp, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    global _bound
    _bound = lib


# ------------------------------------------------------------------ arguments

_bound = None   # the loaded library


def _lib():
    if _bound is None:
        from . import load_library
        load_library()
    return _bound


def _raise(status, where):
    from . import GdnError
    raise GdnError(status, where)


def _act(name, t):
    """An activation: a CUDA tensor in bf16 or fp32 with a contiguous last axis."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor, got one on %s" % (name, t.device))
    if t.dtype not in _CODE:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s must be contiguous in its last axis" % name)


def _like(name, t, shape, dtype, device, strided=False):
    """Another tensor of the call: shape, type, device, layout."""
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if strided:
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError("%s must be contiguous in its last axis" % name)
    elif not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor" % name)


def _strides(name, t):
    """(batch, token) strides of a [B, T, D] tensor."""
    B, T, D = t.shape
    sb, st, _ = t.stride()
    if T <= 1 or t.numel() == 0:
        st = D
    elif st < D:
        raise ValueError("%s: tokens overlap (token stride %d for %d elements)" % (name, st, D))
    return (0 if B <= 1 else sb), st


def _row_stride(name, t):
    """The distance between the rows of a [..., D] tensor, when it is one."""
    D = t.shape[-1]
    if t.is_contiguous() or t.numel() == 0:
        return D
    sizes, strides = t.shape[:-1], t.stride()[:-1]
    at = [(n, s) for n, s in zip(sizes, strides) if n != 1]
    if not at:
        return D
    for (_, s0), (n1, s1) in zip(at, at[1:]):
        if s0 != n1 * s1:
            raise ValueError("%s: its rows are not equally spaced" % name)
    if at[-1][1] < D:
        raise ValueError("%s: rows overlap" % name)
    return at[-1][1]


def _head_stride(name, t):
    """The distance between the tokens of a [N, H, d] tensor whose heads lie
    next to each other."""
    N, H, d = t.shape
    st = t.stride()
    if H > 1 and st[1] != d:
        raise ValueError("%s: the heads of a token must be contiguous" % name)
    if N > 1 and st[0] < H * d:
        raise ValueError("%s: tokens overlap" % name)
    return st[0] if N > 1 else H * d


class _On:
    """The device and stream of a call, and what it allocates there.  With a
    stream of the caller's the memory comes from that stream's pool: a block of
    the current stream's pool may still be in use by work queued there, which
    the given stream does not wait for.  Tensors that go back to the caller are
    also recorded on the current stream, where they are likely to be read."""
    __slots__ = ("device", "raw", "stream", "guard", "reader")

    def __init__(self, device, stream):
        self.device, self.stream = device, stream
        self.guard = self.reader = None
        if stream is not None:
            if stream.device != device:
                raise ValueError("stream is on %s, expected %s" % (stream.device, device))
            self.reader = torch.cuda.current_stream(device)
            self.guard = torch.cuda.stream(stream)
            self.guard.__enter__()
            self.raw = stream.cuda_stream
        else:
            if device.index != torch.cuda.current_device():
                self.guard = torch.cuda.device(device)
                self.guard.__enter__()
            self.raw = _current_raw_stream(device.index)

    def empty(self, shape, dtype):
        t = torch.empty(shape, dtype=dtype, device=self.device)
        if self.reader is not None:
            t.record_stream(self.reader)
        return t

    def done(self):
        if self.guard is not None:
            self.guard.__exit__(None, None, None)
            self.guard = None


# torch.cuda.current_stream(device).cuda_stream without the Stream object in
# between (2 us of a single-token call)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _p(t):
    return t.data_ptr() if t is not None else None


def _extent(t):
    """The first byte of a tensor and the one past its last."""
    first = t.data_ptr()
    if t.numel() == 0:
        return first, first
    return first, first + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def _apart(out, inputs, same=()):
    """Refuses an `out` in the memory of an input, which other threads may still
    have to read when it is written.  Inputs of `same` may be out itself: there
    every element is read only by what writes it."""
    if out is None:
        return
    first, last = _extent(out)
    for name, t in inputs:
        if t is None:
            continue
        a, b = _extent(t)
        if max(a, first) < min(b, last) and not (
                name in same and a == first and t.shape == out.shape and t.is_contiguous()):
            raise ValueError("out overlaps %s" % name)


def _wrote(state, out):
    """Tells autograd that a kernel wrote into the caller's state or `out` (None:
    not given), as an in-place operation of torch's own does."""
    if state is not None:
        _increment_version(state)
    if out is not None:
        _increment_version(out)


def _workspace(on, workspace, size):
    if size == 0:
        _raise(1, "workspace size")
    if workspace is None:
        return on.empty(size, torch.uint8)
    _like("workspace", workspace, workspace.shape, torch.uint8, on.device)
    return workspace


def _params(D, device, dtype, weight, bias, shape):
    """Type code of weight and bias ([...] in fp32 or the activations' type)."""
    w = weight if weight is not None else bias
    if w is None:
        return 1
    if w.dtype != _F32 and w.dtype != dtype:
        raise TypeError("weight and bias must be float32 or %s, got %s" % (dtype, w.dtype))
    if weight is not None:
        _like("weight", weight, shape, w.dtype, device)
    if bias is not None:
        _like("bias", bias, (D,), w.dtype, device)
    return _CODE[w.dtype]


def _status_word(on, check, cu_seqlens):
    return on.empty(1, _I32) if check and cu_seqlens is not None else None


def _read_status(word, on, where):
    if word is None:
        return
    torch.cuda.current_stream(on.device).synchronize()   # the call's own, current until done()
    st = int(word.item())
    if st != 0:
        _raise(st, where + " (device check)")


def _sequences(cu_seqlens, B, device):
    if cu_seqlens is None:
        return B
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be 1-D with at least two entries")
    if B != 1:
        raise ValueError("cu_seqlens needs B == 1")
    _like("cu_seqlens", cu_seqlens, cu_seqlens.shape, _I32, device)
    return cu_seqlens.numel() - 1


def _slots(state, state_indices, N, device):
    if state_indices is None:
        if state.shape[0] < N:
            raise ValueError("state holds %d rows for %d tokens" % (state.shape[0], N))
    else:
        _like("state_indices", state_indices, (N,), _I32, device)


# ------------------------------------------------------------------ layer norm

def layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-5, out=None, stats: bool = True,
                   stream: Optional[torch.cuda.Stream] = None):
    """Layer norm over the last axis of x [..., D]; returns (y, mean, rstd),
    mean and rstd float32 [...] for the backward pass (None without stats).
    weight and bias: [D] in float32 or x's type, or None."""
    _act("x", x)
    D, lead, dev, dtype = x.shape[-1], x.shape[:-1], x.device, x.dtype
    wcode = _params(D, dev, dtype, weight, bias, (D,))
    stride = _row_stride("x", x)
    if out is not None:
        _like("out", out, x.shape, dtype, dev)
        _apart(out, (("x", x), ("weight", weight), ("bias", bias)), same=("x",))
    on = _On(dev, stream)
    try:
        y = out if out is not None else on.empty(x.shape, dtype)
        mean = rstd = None
        if stats:
            mean, rstd = on.empty((2, *lead), _F32).unbind(0)
        rows = y.numel() // D if D else 0
        st = _lib().gdn_layer_norm_fwd(x.data_ptr(), stride, _p(weight), _p(bias), wcode, eps, rows, D, _CODE[dtype],
                                       y.data_ptr(), _p(mean), _p(rstd), on.raw)
        if st != 0:
            _raise(st, "gdn_layer_norm_fwd")
        _wrote(None, out)
    finally:
        on.done()
    return y, mean, rstd


def layer_norm_bwd(dy, x, mean, rstd, weight=None, workspace=None, stream: Optional[torch.cuda.Stream] = None):
    """Gradients of layer_norm_fwd: (dx in x's type, dweight and dbias float32
    [D]) from dy and the forward pass's x, mean and rstd."""
    _act("x", x)
    D, dev, dtype = x.shape[-1], x.device, x.dtype
    _like("dy", dy, x.shape, dtype, dev, strided=True)
    _like("mean", mean, x.shape[:-1], _F32, dev)
    _like("rstd", rstd, x.shape[:-1], _F32, dev)
    wcode = _params(D, dev, dtype, weight, None, (D,))
    sx, sdy = _row_stride("x", x), _row_stride("dy", dy)
    lib, rows = _lib(), mean.numel()
    on = _On(dev, stream)
    try:
        dx = on.empty(x.shape, dtype)
        dw = on.empty((2, D), _F32)
        ws = _workspace(on, workspace, lib.gdn_layer_norm_bwd_workspace_size(rows, D))
        p = dw.data_ptr()
        st = lib.gdn_layer_norm_bwd(dy.data_ptr(), sdy, x.data_ptr(), sx, mean.data_ptr(), rstd.data_ptr(), _p(weight),
                                    wcode, rows, D, _CODE[dtype], dx.data_ptr(), p, p + 4 * D, ws.data_ptr(),
                                    ws.numel(), on.raw)
        if st != 0:
            _raise(st, "gdn_layer_norm_bwd")
    finally:
        on.done()
    return (dx, *dw.unbind(0))


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, stats):
        y, mean, rstd = layer_norm_fwd(x, weight, bias, eps, stats=stats)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_type = bias.dtype if bias is not None else None
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = layer_norm_bwd(dy.contiguous(), x, mean, rstd, weight)
        return (dx, dw.to(weight.dtype) if weight is not None else None,
                db.to(ctx.bias_type) if ctx.bias_type is not None else None, None, None)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm over the last axis with autograd (x, weight, bias).  Forward-mode
    derivatives are refused, as by the other operators."""
    stats = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias))
    # A tangent leaves requires_grad False, and there are tangents in dual levels only
    # (torch.func.jvp enters one): outside of them nothing is lost past the autograd
    # function, which costs 10 us of a 20 us call.
    if not stats and getattr(forward_ad, "_current_level", 0) < 0:
        return layer_norm_fwd(x, weight, bias, eps, stats=False)[0]
    return _LayerNorm.apply(x, weight, bias, eps, stats)


# ---------------------------------------------------- short causal convolution

def _silu(activation):
    if activation not in (None, "silu"):
        raise ValueError("activation must be None or 'silu', got %r" % (activation,))
    return 1 if activation else 0


def _conv_shapes(x, weight, bias, initial_state, cu_seqlens):
    _act("x", x)
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    if weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    B, T, D = x.shape
    W = weight.shape[1]
    wcode = _params(D, x.device, x.dtype, weight, bias, (D, W))
    n = _sequences(cu_seqlens, B, x.device)
    if initial_state is not None:
        _like("initial_state", initial_state, (n, W - 1, D), x.dtype, x.device)
    return B, T, D, W, n, wcode


def causal_conv_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation: Optional[str] = "silu",
                    output_final_state: bool = False, out=None, stream: Optional[torch.cuda.Stream] = None,
                    check: bool = False):
    """Short causal depthwise convolution of x [B, T, D] with weight [D, W];
    returns (y, final_state or None).  States are [n, W - 1, D], the last inputs
    of a sequence, oldest first."""
    B, T, D, W, n, wcode = _conv_shapes(x, weight, bias, initial_state, cu_seqlens)
    sb, st = _strides("x", x)
    dev, dtype, silu = x.device, x.dtype, _silu(activation)
    if out is not None:
        _like("out", out, x.shape, dtype, dev)
        _apart(out, (("x", x), ("weight", weight), ("bias", bias), ("initial_state", initial_state),
                     ("cu_seqlens", cu_seqlens)))
    on = _On(dev, stream)
    try:
        y = out if out is not None else on.empty(x.shape, dtype)
        final = on.empty((n, W - 1, D), dtype) if output_final_state else None
        word = _status_word(on, check, cu_seqlens)
        rc = _lib().gdn_causal_conv_fwd(x.data_ptr(), sb, st, weight.data_ptr(), _p(bias), wcode, _p(initial_state),
                                        _p(cu_seqlens), n, B, T, D, W, silu, _CODE[dtype], y.data_ptr(), _p(final),
                                        _p(word), on.raw)
        if rc != 0:
            _raise(rc, "gdn_causal_conv_fwd")
        _wrote(None, out)
        _read_status(word, on, "gdn_causal_conv_fwd")
    finally:
        on.done()
    return y, final


def causal_conv_bwd(dy, x, weight, bias=None, initial_state=None, cu_seqlens=None,
                    activation: Optional[str] = "silu", d_final_state=None, workspace=None,
                    stream: Optional[torch.cuda.Stream] = None, check: bool = False):
    """Gradients of causal_conv_fwd: (dx, dweight, dbias, d_initial_state) from
    dy and, where the final state is used, d_final_state; dweight [D, W] and
    dbias [D] in float32, the others in x's type."""
    B, T, D, W, n, wcode = _conv_shapes(x, weight, bias, initial_state, cu_seqlens)
    dev, dtype, silu = x.device, x.dtype, _silu(activation)
    _like("dy", dy, x.shape, dtype, dev, strided=True)
    if d_final_state is not None:
        _like("d_final_state", d_final_state, (n, W - 1, D), dtype, dev)
    gb, gt = _strides("dy", dy)
    sb, st = _strides("x", x)
    lib = _lib()
    on = _On(dev, stream)
    try:
        dx = on.empty(x.shape, dtype)
        dw, db = on.empty((D, W), _F32), on.empty((D,), _F32)
        ds = on.empty((n, W - 1, D), dtype)
        ws = _workspace(on, workspace, lib.gdn_causal_conv_bwd_workspace_size(B, T, D, W) or (16 if W in (2, 3, 4) else 0))
        word = _status_word(on, check, cu_seqlens)
        rc = lib.gdn_causal_conv_bwd(dy.data_ptr(), gb, gt, x.data_ptr(), sb, st, weight.data_ptr(), _p(bias), wcode,
                                     _p(initial_state), _p(d_final_state), _p(cu_seqlens), n, B, T, D, W, silu,
                                     _CODE[dtype], dx.data_ptr(), dw.data_ptr(), db.data_ptr(), ds.data_ptr(),
                                     _p(word), ws.data_ptr(), ws.numel(), on.raw)
        if rc != 0:
            _raise(rc, "gdn_causal_conv_bwd")
        _read_status(word, on, "gdn_causal_conv_bwd")
    finally:
        on.done()
    return dx, dw, db, ds


def causal_conv_step(x, state, weight, bias=None, activation: Optional[str] = "silu", state_indices=None, out=None,
                     stream: Optional[torch.cuda.Stream] = None):
    """One token of N sequences through the convolution: x [N, D], state
    [S, W - 1, D] updated in place (row r uses state_indices[r], or r); returns
    y [N, D].  A row whose index is outside [0, S) is padding: y is zero there."""
    _act("x", x)
    if x.dim() != 2 or weight.dim() != 2 or state.dim() != 3:
        raise ValueError("x must be [N, D], state [S, W - 1, D] and weight [D, W]")
    (N, D), W, dev, dtype = x.shape, weight.shape[1], x.device, x.dtype
    wcode = _params(D, dev, dtype, weight, bias, (D, W))
    _like("state", state, (state.shape[0], W - 1, D), dtype, dev)
    _slots(state, state_indices, N, dev)
    if out is not None:
        _like("out", out, (N, D), dtype, dev)
        _apart(out, (("x", x), ("state", state), ("weight", weight), ("bias", bias), ("state_indices", state_indices)),
               same=("x",))
    silu, stride = _silu(activation), _row_stride("x", x)
    on = _On(dev, stream)
    try:
        y = out if out is not None else on.empty((N, D), dtype)
        rc = _lib().gdn_causal_conv_step(x.data_ptr(), stride, state.data_ptr(), _p(state_indices), state.shape[0],
                                         weight.data_ptr(), _p(bias), wcode, N, D, W, silu, _CODE[dtype],
                                         y.data_ptr(), on.raw)
        if rc != 0:
            _raise(rc, "gdn_causal_conv_step")
        _wrote(state, out)
    finally:
        on.done()
    return y


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, cu_seqlens, activation):
        y, final = causal_conv_fwd(x, weight, bias, initial_state, cu_seqlens, activation, output_final_state=True)
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.activation = activation
        ctx.set_materialize_grads(False)
        return y, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, d_final):
        x, weight, bias, initial_state, cu_seqlens = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy.contiguous()
        dx, dw, db, ds = causal_conv_bwd(dy, x, weight, bias, initial_state, cu_seqlens, ctx.activation,
                                         d_final.contiguous() if d_final is not None else None)
        return (dx, dw.to(weight.dtype), db.to(bias.dtype) if bias is not None else None,
                ds if initial_state is not None else None, None, None)


def causal_conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, activation: Optional[str] = "silu",
                output_final_state: bool = False):
    """causal_conv_fwd with autograd (x, weight, bias, initial_state); returns
    (y, final_state or None)."""
    y, final = _CausalConv.apply(x, weight, bias, initial_state, cu_seqlens, activation)
    return y, (final if output_final_state else None)


# ------------------------------------------------------- selective state space scan

def _scan_desc(x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, cu_seqlens):
    """Checks the scan's inputs (activations [Bt, T, D], or [Bt, D] for one
    token) and fills the descriptor; returns (descriptor, number of sequences)."""
    _act("x", x)
    lead, dev, dtype = x.shape[:-1], x.device, x.dtype
    Dn, N = A.shape
    one = len(lead) == 1
    _like("dt", dt, x.shape, dtype, dev, strided=True)
    _like("A", A, (x.shape[-1], N), _F32, dev)
    _like("B", B, (*lead, N), dtype, dev, strided=True)
    _like("C", C, (*lead, N), dtype, dev, strided=True)
    if z is not None:
        _like("z", z, x.shape, dtype, dev, strided=True)
    if D is not None:
        _like("D", D, (Dn,), _F32, dev)
    if dt_bias is not None:
        _like("dt_bias", dt_bias, (Dn,), _F32, dev)
    Bt, T = (lead[0], 1) if one else lead
    n = _sequences(cu_seqlens, Bt, dev)
    if initial_state is not None:
        _like("initial_state", initial_state, (n, Dn, N), _F32, dev)
    if one:
        strides = (x.stride(0), Dn, dt.stride(0), Dn, z.stride(0) if z is not None else 0, Dn, B.stride(0), N,
                   C.stride(0), N)
    else:
        strides = (*_strides("x", x), *_strides("dt", dt), *(_strides("z", z) if z is not None else (0, Dn)),
                   *_strides("B", B), *_strides("C", C))
    return GdnScanDesc(x.data_ptr(), dt.data_ptr(), _p(z), B.data_ptr(), C.data_ptr(), A.data_ptr(), _p(D),
                       _p(dt_bias), _p(initial_state), _p(cu_seqlens), *strides, Bt, T, Dn, N, n,
                       1 if dt_softplus else 0, _CODE[dtype], 0), n


def selective_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = True, initial_state=None,
                       cu_seqlens=None, out=None, workspace=None, stream: Optional[torch.cuda.Stream] = None,
                       check: bool = False):
    """Selective scan of x [Bt, T, D] (dt, z alike) with A [D, N] float32 and
    B, C [Bt, T, N]; returns (y, final_state), final_state float32 [n, D, N]."""
    if x.dim() != 3 or A.dim() != 2:
        raise ValueError("x must be [B, T, D] and A [D, N]")
    desc, n = _scan_desc(x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, cu_seqlens)
    if out is not None:
        _like("out", out, x.shape, x.dtype, x.device)
        _apart(out, (("x", x), ("dt", dt), ("z", z), ("A", A), ("B", B), ("C", C), ("D", D), ("dt_bias", dt_bias),
                     ("initial_state", initial_state), ("cu_seqlens", cu_seqlens)), same=("x", "dt", "z"))
    lib = _lib()
    on = _On(x.device, stream)
    try:
        y = out if out is not None else on.empty(x.shape, x.dtype)
        final = on.empty((n, desc.D, desc.N), _F32)
        size = lib.gdn_selective_scan_fwd_workspace_size(desc.B, desc.T, desc.D, desc.N)
        ws = _workspace(on, workspace, size) if size > 16 or workspace is not None else None
        word = _status_word(on, check, cu_seqlens)
        rc = lib.gdn_selective_scan_fwd(desc, y.data_ptr(), final.data_ptr(), _p(word), _p(ws),
                                        ws.numel() if ws is not None else 0, on.raw)
        if rc != 0:
            _raise(rc, "gdn_selective_scan_fwd")
        _wrote(None, out)
        _read_status(word, on, "gdn_selective_scan_fwd")
    finally:
        on.done()
    return y, final


def selective_scan_bwd(dy, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = True,
                       initial_state=None, cu_seqlens=None, d_final_state=None, workspace=None,
                       stream: Optional[torch.cuda.Stream] = None, check: bool = False):
    """Gradients of selective_scan_fwd from dy and, where the final state is
    used, d_final_state: (dx, ddt, dA, dB, dC, dD, dz, d_dt_bias,
    d_initial_state); dz is None without z.  dA, dD, d_dt_bias and the state's
    gradient are float32, the others in x's type."""
    if x.dim() != 3 or A.dim() != 2:
        raise ValueError("x must be [B, T, D] and A [D, N]")
    desc, n = _scan_desc(x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, cu_seqlens)
    dev, dtype = x.device, x.dtype
    _like("dy", dy, x.shape, dtype, dev, strided=True)
    if d_final_state is not None:
        _like("d_final_state", d_final_state, (n, desc.D, desc.N), _F32, dev)
    gb, gt = _strides("dy", dy)
    lib = _lib()
    on = _On(dev, stream)
    try:
        dx, ddt = on.empty(x.shape, dtype), on.empty(x.shape, dtype)
        dz = on.empty(x.shape, dtype) if z is not None else None
        dB, dC = on.empty(B.shape, dtype), on.empty(C.shape, dtype)
        dA, dv, ds = on.empty(A.shape, _F32), on.empty((2, desc.D), _F32), on.empty((n, desc.D, desc.N), _F32)
        ws = _workspace(on, workspace, lib.gdn_selective_scan_bwd_workspace_size(desc.B, desc.T, desc.D, desc.N))
        word = _status_word(on, check, cu_seqlens)
        p = dv.data_ptr()
        rc = lib.gdn_selective_scan_bwd(desc, dy.data_ptr(), gb, gt, _p(d_final_state), dx.data_ptr(), ddt.data_ptr(),
                                        dA.data_ptr(), dB.data_ptr(), dC.data_ptr(), p, _p(dz), p + 4 * desc.D,
                                        ds.data_ptr(), _p(word), ws.data_ptr(), ws.numel(), on.raw)
        if rc != 0:
            _raise(rc, "gdn_selective_scan_bwd")
        _read_status(word, on, "gdn_selective_scan_bwd")
    finally:
        on.done()
    dD, db = dv.unbind(0)
    return dx, ddt, dA, dB, dC, dD, dz, db, ds


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus: bool = True,
                        state_indices=None, out=None, stream: Optional[torch.cuda.Stream] = None):
    """One token of Bt sequences through the scan: x, dt, z [Bt, D], B, C
    [Bt, N], state float32 [S, D, N] updated in place (row r uses
    state_indices[r], or r); returns y [Bt, D].  A row whose index is outside
    [0, S) is padding: y is zero there."""
    if x.dim() != 2 or A.dim() != 2:
        raise ValueError("x must be [N, D] and A [D, N]")
    desc, _ = _scan_desc(x, dt, A, B, C, D, z, dt_bias, dt_softplus, None, None)
    _like("state", state, (state.shape[0], desc.D, desc.N), _F32, x.device)
    _slots(state, state_indices, desc.B, x.device)
    if out is not None:
        _like("out", out, x.shape, x.dtype, x.device)
        _apart(out, (("x", x), ("dt", dt), ("z", z), ("A", A), ("B", B), ("C", C), ("D", D), ("dt_bias", dt_bias),
                     ("state", state), ("state_indices", state_indices)), same=("x", "dt", "z"))
    on = _On(x.device, stream)
    try:
        y = out if out is not None else on.empty(x.shape, x.dtype)
        rc = _lib().gdn_selective_scan_step(desc, state.data_ptr(), _p(state_indices), state.shape[0], y.data_ptr(),
                                            on.raw)
        if rc != 0:
            _raise(rc, "gdn_selective_scan_step")
        _wrote(state, out)
    finally:
        on.done()
    return y


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, cu_seqlens):
        y, final = selective_scan_fwd(x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, cu_seqlens)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens)
        ctx.dt_softplus = dt_softplus
        ctx.set_materialize_grads(False)
        return y, final

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, d_final):
        x, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy.contiguous()
        dx, ddt, dA, dB, dC, dD, dz, db, ds = selective_scan_bwd(
            dy, x, dt, A, B, C, D, z, dt_bias, ctx.dt_softplus, initial_state, cu_seqlens,
            d_final.contiguous() if d_final is not None else None)
        return (dx, ddt, dA, dB, dC, dD if D is not None else None, dz, db if dt_bias is not None else None, None,
                ds if initial_state is not None else None, None)


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = True, initial_state=None,
                   output_final_state: bool = False, cu_seqlens=None):
    """selective_scan_fwd with autograd (every tensor but cu_seqlens); returns
    (y, final_state or None)."""
    y, final = _SelectiveScan.apply(x, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, cu_seqlens)
    return y, (final if output_final_state else None)


# -------------------------------------------------- one token of the delta rule

def gated_delta_step(q, k, v, g, beta, state, scale=None, use_qk_l2norm_in_kernel: bool = False, state_indices=None,
                     out=None, stream: Optional[torch.cuda.Stream] = None):
    """One token of the gated delta rule for N sequences, chunk_fwd's recurrence
    on a cached state: q, k [N, H, dk], v [N, H, dv] (bf16 or fp32, each token's
    heads contiguous), g, beta [N, H] float32, state float32 [S, H, dk, dv] updated in place (row r uses
    state_indices[r], or r); returns o [N, H, dv].  A row whose index is outside
    [0, S) is padding: o is zero there."""
    _act("q", q)
    if q.dim() != 3 or v.dim() != 3 or state.dim() != 4:
        raise ValueError("q and k must be [N, H, dk], v [N, H, dv] and state [S, H, dk, dv]")
    (N, H, dk), dv, dev, dtype = q.shape, v.shape[2], q.device, q.dtype
    _like("k", k, q.shape, dtype, dev, strided=True)
    _like("v", v, (N, H, dv), dtype, dev, strided=True)
    sq, sk, sv = _head_stride("q", q), _head_stride("k", k), _head_stride("v", v)
    _like("g", g, (N, H), _F32, dev)
    _like("beta", beta, (N, H), _F32, dev)
    _like("state", state, (state.shape[0], H, dk, dv), _F32, dev)
    _slots(state, state_indices, N, dev)
    if out is not None:
        _like("out", out, v.shape, dtype, dev)
        _apart(out, (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("state", state),
                     ("state_indices", state_indices)))
    on = _On(dev, stream)
    try:
        o = out if out is not None else on.empty(v.shape, dtype)
        rc = _lib().gdn_delta_step(q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, g.data_ptr(), beta.data_ptr(),
                                   state.data_ptr(), _p(state_indices), state.shape[0],
                                   float(scale) if scale is not None else 0.0, 1 if use_qk_l2norm_in_kernel else 0,
                                   N, H, dk, dv, _CODE[dtype], o.data_ptr(), on.raw)
        if rc != 0:
            _raise(rc, "gdn_delta_step")
        _wrote(state, out)
    finally:
        on.done()
    return o
