"""Host-side refusals of the layer operators (no GPU): the C entry points
return a status before any launch, the Python functions raise for tensors that
are not on a CUDA device."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import chunked_prefill_gdn_gb300 as gdn
from chunked_prefill_gdn_gb300 import build as gdn_build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.load_library()


P = ctypes.c_void_p(4096)   # never dereferenced: the calls are refused first


def test_layer_norm_arguments(lib):
    f = lib.gdn_layer_norm_fwd
    assert f(P, 8, None, None, 1, 1e-5, 4, 0, 1, P, None, None, None) == INVALID        # no columns
    assert f(P, 7, None, None, 1, 1e-5, 4, 8, 1, P, None, None, None) == INVALID        # rows overlap
    assert f(P, 8, None, None, 1, -1.0, 4, 8, 1, P, None, None, None) == INVALID        # eps
    assert f(P, 8, None, None, 1, float("nan"), 4, 8, 1, P, None, None, None) == INVALID
    assert f(P, 8, None, None, 1, 1e-5, 4, 8, 7, P, None, None, None) == INVALID        # type
    assert f(None, 8, None, None, 1, 1e-5, 4, 8, 1, P, None, None, None) == INVALID
    assert f(ctypes.c_void_p(4098), 8, None, None, 1, 1e-5, 4, 8, 1, P, None, None, None) == INVALID   # fp32 at 2 bytes
    assert f(P, 1 << 31, None, None, 1, 1e-5, 4, (1 << 30) + 1, 1, P, None, None, None) == UNSUPPORTED
    assert f(None, 8, None, None, 1, 1e-5, 0, 8, 1, None, None, None, None) == 0        # no rows
    b = lib.gdn_layer_norm_bwd
    size = lib.gdn_layer_norm_bwd_workspace_size(4, 8)
    assert size >= 64 and lib.gdn_layer_norm_bwd_workspace_size(4, 0) == 0
    assert b(P, 8, P, 8, P, P, None, 1, 4, 8, 1, P, P, P, P, size - 1, None) == WORKSPACE
    assert b(P, 8, P, 8, P, P, None, 1, 4, 8, 1, P, P, P, None, 0, None) == INVALID
    assert b(P, 8, P, 8, None, P, None, 1, 4, 8, 1, P, P, P, P, size, None) == INVALID


def test_causal_conv_arguments(lib):
    f = lib.gdn_causal_conv_fwd

    def fwd(x=P, sb=64, st=8, w=P, wd=1, cu=None, n=0, B=1, T=8, D=8, W=4, dt=1, y=P):
        return f(x, sb, st, w, None, wd, None, cu, n, B, T, D, W, 1, dt, y, None, None, None)

    assert fwd(W=1) == UNSUPPORTED and fwd(W=5) == UNSUPPORTED
    assert fwd(st=7) == INVALID and fwd(D=0) == INVALID and fwd(T=-1) == INVALID and fwd(w=None) == INVALID
    assert fwd(x=None) == INVALID and fwd(y=None) == INVALID and fwd(dt=2) == INVALID
    assert fwd(cu=P, n=0) == INVALID and fwd(cu=P, n=2, B=2) == INVALID
    assert fwd(wd=0) == INVALID                      # bf16 weights with fp32 activations
    assert fwd(B=0) == 0
    assert fwd(T=(1 << 30) + 1) == UNSUPPORTED and fwd(B=1 << 30, T=64) == UNSUPPORTED
    size = lib.gdn_causal_conv_bwd_workspace_size(1, 8, 8, 4)
    assert size > 0 and lib.gdn_causal_conv_bwd_workspace_size(1, 8, 8, 5) == 0
    assert lib.gdn_causal_conv_bwd(P, 64, 8, P, 64, 8, P, None, 1, None, None, None, 0, 1, 8, 8, 4, 1, 1, P, P, P, None,
                                   None, P, size - 1, None) == WORKSPACE
    s = lib.gdn_causal_conv_step
    assert s(P, 8, P, None, 3, P, None, 1, 4, 8, 4, 1, 1, P, None) == INVALID     # four rows, three states
    assert s(P, 8, None, None, 4, P, None, 1, 4, 8, 4, 1, 1, P, None) == INVALID
    assert s(P, 8, P, None, 0, P, None, 1, 0, 8, 4, 1, 1, P, None) == 0


def scan_desc(**kw):
    d = gdn.GdnScanDesc(4096, 4096, None, 4096, 4096, 4096, None, None, None, None, 64, 8, 64, 8, 0, 8, 128, 16, 128, 16,
                        1, 8, 8, 16, 1, 1, 1, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_selective_scan_arguments(lib):
    f = lambda **kw: lib.gdn_selective_scan_fwd(scan_desc(**kw), P, None, None, None, 0, None)   # noqa: E731
    assert f(T=(1 << 30) + 1) == UNSUPPORTED and f(B=65536) == UNSUPPORTED
    assert f(N=65) == UNSUPPORTED and f(N=0) == INVALID and f(D=0) == INVALID
    assert f(x=None) == INVALID and f(A=None) == INVALID and f(dtype=3) == INVALID
    assert f(x_token_stride=7) == INVALID and f(b_token_stride=15) == INVALID and f(x_batch_stride=-1) == INVALID
    assert f(cu_seqlens=4096, n_seqs=0) == INVALID and f(cu_seqlens=4096, n_seqs=2, B=2) == INVALID
    assert f(B=0) == 0
    assert lib.gdn_selective_scan_fwd(None, P, None, None, None, 0, None) == INVALID
    size = lib.gdn_selective_scan_fwd_workspace_size(1, 4096, 8, 16)
    assert size > 16
    assert lib.gdn_selective_scan_fwd(scan_desc(T=4096), P, None, None, P, size - 1, None) == WORKSPACE
    size = lib.gdn_selective_scan_bwd_workspace_size(1, 64, 8, 16)
    assert size > 16 and lib.gdn_selective_scan_bwd_workspace_size(1, 64, 8, 65) == 0
    b = lambda dy=P, st=8, ws=P, size=size, dA=P, **kw: lib.gdn_selective_scan_bwd(   # noqa: E731
        scan_desc(T=64, **kw), dy, 512, st, None, P, P, dA, P, P, None, None, None, None, None, ws, size, None)
    assert b(size=size - 1) == WORKSPACE and b(ws=None) == INVALID and b(dy=None) == INVALID and b(dA=None) == INVALID
    assert b(st=7) == INVALID and b(z=4096) == INVALID and b(N=65) == UNSUPPORTED     # a gate without dz
    s = lib.gdn_selective_scan_step
    assert s(scan_desc(T=2), P, None, 1, P, None) == INVALID
    assert s(scan_desc(T=1), P, None, 0, P, None) == INVALID


@pytest.mark.parametrize("T", [0, 5, 16, 17, 64, 4096])
def test_scan_plans_an_empty_batch(lib, T):
    """No batch rows, however long: the size queries answer (in a process of
    their own, which an integer division by zero would end)."""
    code = ("import chunked_prefill_gdn_gb300 as gdn\n"
            "lib = gdn.load_library()\n"
            "for D, N in ((1, 1), (64, 16), (1024, 24), (40, 64)):\n"
            "    print(lib.gdn_selective_scan_fwd_workspace_size(0, %d, D, N),\n"
            "          lib.gdn_selective_scan_bwd_workspace_size(0, %d, D, N))\n" % (T, T))
    run = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-500:]
    sizes = [int(v) for v in run.stdout.split()]
    assert len(sizes) == 8 and all(v >= 16 for v in sizes) and all(v == 16 for v in sizes[::2])
    assert lib.gdn_selective_scan_fwd(scan_desc(B=0, T=T), P, None, None, None, 0, None) == 0


def test_delta_step_arguments(lib):
    def f(q=P, n=2, N=2, H=2, dk=32, dv=32, dt=1, st=64, state=P):
        return lib.gdn_delta_step(q, st, P, 64, P, 64, P, P, state, None, n, 0.0, 0, N, H, dk, dv, dt, P, None)

    assert f(dk=48) == UNSUPPORTED and f(dv=256) == UNSUPPORTED
    assert f(q=None) == INVALID and f(n=1) == INVALID and f(H=0) == INVALID and f(dt=9) == INVALID
    assert f(q=ctypes.c_void_p(4098)) == INVALID and f(state=ctypes.c_void_p(4100)) == INVALID and f(st=63) == INVALID
    assert f(N=0, n=0) == 0


def test_python_functions_refuse_host_tensors(lib):
    x = torch.zeros(1, 4, 8)
    w = torch.zeros(8, 4)
    with pytest.raises(ValueError):
        gdn.layer_norm_fwd(x)
    with pytest.raises(ValueError):
        gdn.causal_conv_fwd(x, w)
    with pytest.raises(ValueError):
        gdn.causal_conv_step(x[0], torch.zeros(4, 3, 8), w)
    with pytest.raises(ValueError):
        gdn.selective_scan_fwd(x, x, w, x, x)
    with pytest.raises(ValueError):
        gdn.gated_delta_step(x, x, x, x, x, torch.zeros(1, 4, 8, 8))


def test_overlapping_memory_is_found():
    """What counts as `out` in an input's memory: any shared byte of their extents,
    but for an input that may be out itself."""
    apart = gdn.layer_ops._apart
    buf = torch.zeros(100)
    x, out = buf[:48].view(6, 8), buf[48:96].view(6, 8)
    apart(None, [("x", x)])
    apart(out, [("x", x), ("bias", None), ("empty", buf[50:50])])
    apart(out, [("cu", torch.zeros(3, dtype=torch.int32))])
    for t in (out, out[5], out.t(), buf[47:49], buf[95:], buf.view(20, 5)[9:], buf[::7], buf[48:96].view(torch.int32)):
        with pytest.raises(ValueError, match="overlaps x"):
            apart(out, [("x", t)])
    apart(out, [("x", out)], same=("x",))
    for t in (out[:5], buf[49:97].view(6, 8), out.view(8, 6), buf[48:96].view(8, 6).t()):   # not out itself
        with pytest.raises(ValueError, match="overlaps x"):
            apart(out, [("x", t)], same=("x",))


def test_layer_norm_refuses_forward_mode(monkeypatch):
    """A tangent of any input reaches the autograd function, which has no forward
    mode and raises; it is never dropped.  (The kernel is replaced by torch's
    arithmetic: no GPU.)"""
    from torch.autograd import forward_ad

    calls = []

    def kernel(x, weight=None, bias=None, eps=1e-5, out=None, stats=True, stream=None):
        calls.append(stats)
        mean = x.mean(-1)
        rstd = (x.var(-1, unbiased=False) + eps).rsqrt()
        y = (x - mean[..., None]) * rstd[..., None]
        y = y * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
        return y, *((mean, rstd) if stats else (None, None))

    monkeypatch.setattr(gdn.layer_ops, "layer_norm_fwd", kernel)
    x, w, b = torch.randn(3, 8), torch.randn(8), torch.randn(8)
    for args in ((x,), (x, w, b)):
        with pytest.raises(RuntimeError):
            torch.func.jvp(gdn.layer_norm, args, tuple(torch.ones_like(t) for t in args))
    for grads in (True, False):
        for i in range(3):
            with forward_ad.dual_level(), torch.set_grad_enabled(grads):
                args = [x, w, b]
                args[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
                with pytest.raises(RuntimeError):
                    gdn.layer_norm(*args)
    # nested, with the tangent of the outer level in a captured tensor
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda u: torch.func.jvp(lambda t: t.sum() * gdn.layer_norm(u), (x,), (x,))[0], (x,), (x,))
    # without tangents: the values, and statistics only where a backward pass will ask for them
    del calls[:]
    want = kernel(x, w, b)[0]
    assert torch.equal(gdn.layer_norm(x, w, b), want) and calls[-1] is False
    leaf = w.clone().requires_grad_()
    y = gdn.layer_norm(x, leaf, b)
    assert y.requires_grad and calls[-1] is True
    with torch.no_grad():
        y = gdn.layer_norm(x, leaf, b)
        assert not y.requires_grad and calls[-1] is False
