"""Host-side refusals and plans of the block norm and the gated feed-forward block
(no GPU): the C entry points return a status before any launch, the Python
functions raise for tensors that are not on a CUDA device."""
import ctypes

import pytest
import torch

import chunked_prefill_gdn_gb300 as gdn
from chunked_prefill_gdn_gb300 import block_ops
from chunked_prefill_gdn_gb300 import build as gdn_build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.load_library()


P = ctypes.c_void_p(4096)   # never dereferenced: the calls are refused first
ODD = ctypes.c_void_p(4098)


def norm_desc(**kw):
    d = gdn.GdnBlockNormDesc(4096, 4096, 4096, 4096, 4096, 6, 1, 64, 64, 64, 64, 64, 1e-5, 1, 1, 0, 1, 1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_block_norm_arguments(lib):
    def f(r=P, rs=64, x=P, h=P, rp=P, rn=P, **kw):
        return lib.gdn_block_norm_fwd(norm_desc(**kw), r, rs, rs, x, h, rp, rn, None)

    assert lib.gdn_block_norm_fwd(None, P, 64, 64, P, P, P, P, None) == INVALID
    for kw in (dict(D=0), dict(outer=-1), dict(inner=0), dict(eps=-1.0), dict(eps=float("nan")), dict(dtype=2), dict(w_dtype=7),
               dict(w_dtype=0), dict(gate_activation=2), dict(y=None), dict(y=4098), dict(post_weight=4097), dict(y_outer_stride=63),
               dict(inner=3, y_inner_stride=63), dict(gate_outer_stride=8), dict(rs=8), dict(x=None), dict(h=None), dict(rp=None),
               dict(rn=None), dict(post_norm=0), dict(pre_norm=0), dict(x=ODD)):
        assert f(**kw) == INVALID, kw
    assert f(D=(1 << 30) + 1) == UNSUPPORTED and f(outer=1 << 31) == UNSUPPORTED and f(outer=1 << 20, inner=1 << 11) == UNSUPPORTED
    assert f(outer=0, y=None, x=None) == 0
    size = lib.gdn_block_norm_bwd_workspace_size(norm_desc())
    assert size >= 2 * 64 * 4 and lib.gdn_block_norm_bwd_workspace_size(norm_desc(D=0)) == 0

    def b(dx=P, dh=P, x=P, st=64, rp=P, rn=P, dy=P, dz=P, ws=P, n=size, **kw):
        return lib.gdn_block_norm_bwd(norm_desc(**kw), dx, st, st, dh, 64, 64, x, 64, 64, rp, rn, dy, P, dz, P, P, P, ws, n, None)

    for kw in (dict(dh=None), dict(x=None), dict(rp=None), dict(rn=None), dict(dy=None), dict(dz=None), dict(ws=None), dict(st=8),
               dict(dx=None, pre_norm=0, pre_weight=None), dict(dy=ODD)):
        assert b(**kw) == INVALID, kw
    assert b(n=size - 1) == WORKSPACE


def ffn_desc(**kw):
    d = gdn.GdnFfnDesc(4096, 4096, 4096, 4096, 64, 40, 64, 128, 64, 0, 1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_gated_ffn_arguments(lib):
    size = lib.gdn_gated_ffn_fwd_workspace_size(ffn_desc())

    def f(y=P, gate=None, up=None, ws=P, n=size, **kw):
        return lib.gdn_gated_ffn_fwd(ffn_desc(**kw), y, gate, up, None, ws, n, None)

    assert lib.gdn_gated_ffn_fwd(None, P, None, None, None, P, size, None) == INVALID
    for kw in (dict(M=-1), dict(D=0), dict(F=0), dict(D_out=0), dict(x_stride=63), dict(activation=2), dict(dtype=3), dict(x=None),
               dict(w_gate=None), dict(w_down=None), dict(w_up=4098), dict(y=None), dict(y=ODD), dict(gate=P), dict(ws=None),
               dict(ws=ctypes.c_void_p(8))):
        assert f(**kw) == INVALID, kw
    assert f(n=size - 1) == WORKSPACE
    for kw in (dict(M=(1 << 24) + 1), dict(F=(1 << 24) + 1), dict(M=1 << 20, F=1 << 20), dict(x_stride=1 << 37),
               dict(M=1 << 20, x_stride=1 << 20)):
        assert f(**kw) == UNSUPPORTED and lib.gdn_gated_ffn_fwd_workspace_size(ffn_desc(**kw)) == 0, kw
    assert f(M=0, x=None, y=None, ws=None, n=0) == 0
    size = lib.gdn_gated_ffn_bwd_workspace_size(ffn_desc(), P, 64)

    def b(dy=P, st=64, gate=P, up=P, dx=P, ws=P, n=size, **kw):
        return lib.gdn_gated_ffn_bwd(ffn_desc(**kw), dy, st, gate, up, dx, P, P, P, None, ws, n, None)

    for kw in (dict(dy=None), dict(st=63), dict(gate=None), dict(up=None), dict(dx=ODD), dict(ws=None), dict(w_up=None)):
        assert b(**kw) == INVALID, kw
    assert b(n=size - 1) == WORKSPACE and lib.gdn_gated_ffn_bwd_workspace_size(ffn_desc(), P, 63) == 0
    assert b(st=1 << 37) == UNSUPPORTED and lib.gdn_gated_ffn_bwd_workspace_size(ffn_desc(), P, 1 << 37) == 0
    one = ffn_desc(M=1, x_stride=0)
    assert lib.gdn_gated_ffn_fwd(one, P, None, None, None, P, 0, None) == WORKSPACE          # a row's stride does not matter


def test_gated_ffn_workspace_follows_what_has_to_be_laid_out(lib):
    """bf16 rows that are 16-byte aligned are read in place; others, and fp32, are laid out."""
    size = lib.gdn_gated_ffn_fwd_workspace_size
    M, D, F = 512, 1024, 4096
    kw = dict(M=M, D=D, F=F, D_out=D, x_stride=D)
    h = M * F * 2
    assert h <= size(ffn_desc(dtype=0, **kw)) <= h + 40 * M * D * 4 + 4096                 # h, and parts of split sums
    assert size(ffn_desc(dtype=0, **{**kw, "x_stride": D + 4})) >= h + M * D * 2            # x too
    assert size(ffn_desc(dtype=0, w_up=4098, **kw)) >= h + F * D * 2
    assert size(ffn_desc(dtype=1, **kw)) >= 3 * (h + 2 * (M * D + 3 * D * F))               # three planes of all
    assert size(ffn_desc(M=0)) == 16


def test_python_refusals_without_a_gpu():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.block_norm_fwd(x)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gated_ffn_fwd(x, x, x, x)


def test_levels_of_rows():
    """How a tensor's leading axes become one or two levels of rows."""
    t = torch.zeros(4, 6, 10, 16)
    assert block_ops._levels("t", t) == [(240, 16)]
    assert block_ops._levels("t", t[..., :8]) == [(240, 16)]
    assert block_ops._levels("t", t[:, :, :4]) == [(24, 160), (4, 16)]
    assert block_ops._levels("t", t[:1, :1, :1]) == []
    with pytest.raises(ValueError, match="two levels"):
        block_ops._levels("t", t[:, :3, :4])
    with pytest.raises(ValueError, match="overlap"):
        block_ops._levels("t", t.view(-1).as_strided((5, 16), (8, 1)))
    heads = t[:, :, :4]
    outer, inner, strides = block_ops._row_levels((("a", heads), ("b", heads.contiguous()), ("c", None)))
    assert (outer, inner) == (24, 4) and strides == [160, 16, 64, 16, 64, 16]
    assert block_ops._row_levels((("a", t[0, 0]), ("b", None))) == (10, 1, [16, 16, 16, 16])
    assert block_ops._row_levels((("a", torch.zeros(8, 32)[:, :16]), ("b", torch.zeros(8, 16)))) == (8, 1, [32, 32, 16, 16])
    with pytest.raises(ValueError, match="levels of"):
        block_ops._row_levels((("a", heads), ("b", torch.zeros(4, 12, 4, 16)[:, :6])))
