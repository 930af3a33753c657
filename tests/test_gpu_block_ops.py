"""GPU parity of the block norm and the gated feed-forward block against the fp64
oracle, element by element, at the sizes, layouts and parts where they can go wrong.

Bars, with U = 2^-24 and M the sum of the absolute values of the terms behind an
element (the oracle on absolute values):
  rounding       a result in bf16 is within half a step, 2^-8 of the exact value
  block norm     sums of 16 + 9 + 16 terms deep, rsqrt, the sigmoid (its argument is
                 rounded at |z| U): K = 64 for |z| up to 20, on M of x; h follows
                 x's error and, through rstd_pre, the row's; the backward pass sums
                 the same way twice: K = 128; sums over rows K = 128 + rows
  feed-forward   bf16: h (backward: dgate, dup, h) is rounded to bf16 between two
                 products, so the second one is off by 2^-8 of the sum of its terms'
                 absolute values, and its own sums by less than 2^-14 of that: the
                 tensor cores add 16 products at a time, K / 16 of them one after the
                 other, each addition off by at most 2^-22 of the sum so far (K up to
                 4096 here: 256 2^-22 = 2^-14).  fp32: three bf16 terms hold 24 bits;
                 what is left out of a product is 4 U, the tensor cores' sums are 6 x 32
                 additions deep (2^-22 each at most), those over K another K / 512:
                 1024 U covers both products of up to 4096 terms
  besides, relative L2 errors: 5e-3 for bf16 as for the whole package (roundings of
  2^-8 at most, 2^-9.8 rms, up to four of them: 4.5e-3), 1e-5 for fp32.
"""
import numpy as np
import pytest
import torch

import chunked_prefill_gdn_gb300 as gdn
import oracle
from chunked_prefill_gdn_gb300 import build as gdn_build
from oracle import block_ops as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {"bf16": 2.0 ** -8, "f32": 0.0}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def lib():
    gdn_build.build()
    return gdn.load_library()


def rng(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, std=1.0, to="f32"):
    return (torch.randn(*shape, generator=g) * std).to(TORCH[to]).cuda()


def plain(t):
    return t


def wide(t, left=8, right=16):
    """The same values as a slice of wider rows (16-byte aligned, strided)."""
    buf = torch.full((*t.shape[:-1], left + t.shape[-1] + right), float("nan"), dtype=t.dtype, device=t.device)
    view = buf[..., left:left + t.shape[-1]]
    view.copy_(t)
    return view


def odd(t):
    """The same values at an address that only its element type aligns."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    view = buf[1:].view(t.shape)
    view.copy_(t)
    return view


def num(t):
    return None if t is None else oracle.to_f64(t)


def rows_of(t):
    return None if t is None else num(t).reshape(-1, t.shape[-1])


def close(name, got, want, mag, K, dtype="f32", extra=0.0):
    got = num(got).reshape(want.shape)
    err, tol = np.abs(got - want), ROUND[dtype] * np.abs(want) + K * U * mag + extra + 1e-37
    assert np.isfinite(got).all(), name
    assert (err <= tol).all(), "%s: error %.3e at a bar of %.3e" % (name, err.flat[np.argmax(err / tol)],
                                                                    tol.flat[np.argmax(err / tol)])


# ------------------------------------------------------------------ block norm

NORM = [(1, 1), (3, 7), (37, 33), (9, 64), (33, 128), (5, 130), (5, 256), (9, 264), (17, 512), (4, 513), (3, 1000),
        (5, 1024), (3, 2049), (700, 96), (2, 4096), (3, 4100), (2, 8192), (2, 8193), (3, 9001), (5, 9008), (2, 20000)]


class Norm:
    """One case: `parts` of p (norm after), g (gate), r (residual), s (scale), n (norm before)."""

    def __init__(self, rows, D, dtype, wtype, parts, layout=plain, lead=None, activation="silu", seed=0):
        g = rng(seed + 10007 * rows + D)
        shape = (*lead, D) if lead else (rows, D)
        act = lambda std=1.0: layout(normal(g, *shape, std=std, to=dtype))   # noqa: E731
        self.dtype, self.parts, self.activation = dtype, parts, activation
        self.y, self.dx, self.dh = act(1.5), act(), act() if "n" in parts else None
        self.z = act(3.0) if "g" in parts else None
        self.r = act(2.0) if "r" in parts else None
        vec = lambda on: (1 + 0.3 * torch.randn(D, generator=g)).to(TORCH[wtype]).cuda() if on and wtype else None   # noqa: E731
        self.wp, self.sc, self.wn = vec("p" in parts), vec("s" in parts), vec("n" in parts)

    def forward(self, fn=gdn.block_norm_fwd, **kw):
        return fn(self.y, self.r, self.z, self.wp, self.sc, self.wn, post_norm="p" in self.parts,
                  pre_norm="n" in self.parts, activation=self.activation, eps=1e-5, **kw)

    def backward(self, x, rp, rn, dx="given", **kw):
        return gdn.block_norm_bwd(self.dx if isinstance(dx, str) else dx, self.dh, self.y, x, rp, rn, self.z, self.wp, self.sc,
                                  self.wn, activation=self.activation, residual="r" in self.parts, **kw)

    def check_forward(self, got):
        args = [rows_of(self.y), rows_of(self.r), rows_of(self.z), num(self.wp), num(self.sc), num(self.wn)]
        x0, h0, rp0, rn0 = ref.block_norm(*args, "p" in self.parts, "n" in self.parts, self.activation)
        x, h, rp, rn = got
        branch = x0 - (0.0 if args[1] is None else args[1])
        mag = np.abs(branch) + (0.0 if args[1] is None else np.abs(args[1]))
        close("x", x, x0, mag, 64, self.dtype)
        assert (rp is None) == ("p" not in self.parts) and (h is None) == (rn is None) == ("n" not in self.parts)
        if rp is not None:
            close("rstd_post", rp, rp0, rp0, 64)
        if rn is not None:
            spread = 1 + np.sqrt((mag ** 2).mean(-1)) * rn0       # the row's error, relative to its rms
            close("rstd_pre", rn, rn0, rn0 * spread, 64)
            w = 1.0 if args[5] is None else np.abs(args[5])
            close("h", h, h0, w * rn0[:, None] * (mag + np.abs(x0) * spread[:, None]), 64, self.dtype)

    def check_backward(self, got, x, rp, rn, dx="given"):
        flat = lambda t: None if t is None else num(t).reshape(-1)   # noqa: E731
        dx = self.dx if isinstance(dx, str) else dx
        tail = [rows_of(self.z), num(self.wp), num(self.sc), num(self.wn)]
        head = [rows_of(dx), rows_of(self.dh), rows_of(self.y), rows_of(x), flat(rp), flat(rn)]
        want = ref.block_norm_backward(*head, *tail, self.activation)
        ab = lambda t: None if t is None else np.abs(t)   # noqa: E731
        mag = ref.block_norm_backward(*(ab(t) for t in head), tail[0], *(ab(t) for t in tail[1:]), self.activation, magnitude=True)
        R = head[2].shape[0]
        there = [True, self.r is not None, self.z is not None, self.wp is not None, self.sc is not None, self.wn is not None]
        for name, a, b, m, on, per_row in zip(("dy", "dr", "dz", "dpost", "dscale", "dpre"), got, want, mag, there, [1] * 3 + [0] * 3):
            assert (a is not None) == on, name
            if on:
                close(name, a, b, m, 128 if per_row else 128 + R, self.dtype if per_row else "f32")


@pytest.mark.parametrize("dtype,wtype,layout,parts", [
    ("bf16", "f32", plain, "pgrsn"), ("bf16", "bf16", wide, "pgrsn"), ("f32", "f32", odd, "pgrsn"), ("f32", None, wide, "prn"),
    ("bf16", "f32", odd, "pg"), ("f32", "f32", plain, "rsn"), ("bf16", "f32", wide, "grs"), ("f32", "f32", plain, "gn")])
@pytest.mark.parametrize("rows,D", NORM)
def test_block_norm(rows, D, dtype, wtype, layout, parts):
    c = Norm(rows, D, dtype, wtype, parts, layout)
    x, h, rp, rn = got = c.forward()
    c.check_forward(got)
    c.check_backward(c.backward(x, rp, rn), x, rp, rn)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 100, 128, 256])
@pytest.mark.parametrize("B,T,H", [(2, 37, 3), (1, 700, 5), (3, 1, 7)])
def test_gated_norm_of_heads_that_are_slices(B, T, H, D, dtype):
    """The recurrence's output [B, T, H, D] and a gate that is half of a projection: rows in two levels."""
    c = Norm(B * T * H, D, dtype, "f32", "pg", lead=(B, T, H), activation="sigmoid" if D == 64 else "silu")
    both = torch.full((B, T, 2 * H * D + 8), float("nan"), dtype=TORCH[dtype], device="cuda")
    both[..., :H * D] = c.z.flatten(-2)
    c.z = both[..., :H * D].unflatten(-1, (H, D))
    x, h, rp, rn = got = c.forward()
    c.check_forward(got)
    c.check_backward(c.backward(x, rp, rn), x, rp, rn)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", [(5000, 128), (3000, 256), (2011, 1024), (1400, 4096), (700, 8192), (3001, 100)])
def test_block_norm_more_rows_than_the_grid(rows, D, dtype):
    """Several rows per block: the copies' stages go round, sums over a block's rows."""
    c = Norm(rows, D, dtype, "f32", "pgrsn")
    x, h, rp, rn = got = c.forward()
    c.check_forward(got)
    c.check_backward(c.backward(x, rp, rn), x, rp, rn)


def test_block_norm_without_dx_and_repeatable():
    """x used for h alone: dx None is a zero gradient; the same inputs give the same bits."""
    c = Norm(300, 512, "bf16", "f32", "pgrsn")
    x, _, rp, rn = c.forward()
    a = c.backward(x, rp, rn, dx=None)
    c.check_backward(a, x, rp, rn, dx=None)
    b = c.backward(x, rp, rn, dx=torch.zeros_like(c.dx))
    again = c.backward(x, rp, rn, dx=None)
    for u, v, w in zip(a, b, again):
        assert torch.equal(u, v) and torch.equal(u, w)


@pytest.mark.parametrize("D", [96, 640, 4095, 9001])
def test_block_norm_rows_stand_alone(D):
    """A row with a NaN or an infinity spoils its own outputs only; zero rows stay zero."""
    c = Norm(9, D, "f32", "f32", "pgrsn")
    clean = c.forward()
    cleang = c.backward(clean[0], clean[2], clean[3])
    c.y, c.r = c.y.clone(), c.r.clone()
    c.y[2, 17], c.r[5, D - 1] = float("nan"), float("inf")
    c.y[7] = 0.0
    c.r[7] = 0.0
    got = c.forward()
    keep = [0, 1, 3, 4, 6, 8]
    for a, b in zip(got, clean):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(got[1][2]).all() and not torch.isfinite(got[0][5, D - 1]) and torch.isfinite(got[0][5, 0])
    assert (got[0][7] == 0).all() and (got[1][7] == 0).all()
    gotg = c.backward(got[0], got[2], got[3])
    for a, b in zip(gotg[:3], cleang[:3]):
        assert torch.equal(a[keep], b[keep]) and torch.isfinite(a[7]).all()


@pytest.mark.parametrize("D", [128, 2048, 9000])
def test_block_norm_in_place(D):
    """out in the memory of y, residual or gate; shifted memory is refused."""
    want = Norm(50, D, "bf16", "f32", "pgrsn").forward()
    for name in ("y", "r", "z"):
        c = Norm(50, D, "bf16", "f32", "pgrsn")
        t = getattr(c, name)
        got = c.forward(out=t)
        assert got[0] is t
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    c = Norm(50, D, "bf16", "f32", "pgrsn")
    buf = torch.zeros(51 * D, dtype=torch.bfloat16, device="cuda")
    c.y = buf[:50 * D].view(50, D)
    with pytest.raises(ValueError, match="overlaps y"):
        c.forward(out=buf[D:].view(50, D))


def test_block_norm_no_rows():
    c = Norm(0, 40, "bf16", "f32", "pgrsn")
    x, h, rp, rn = c.forward()
    assert x.shape == h.shape == (0, 40) and rp.numel() == rn.numel() == 0
    dy, dr, dz, *params = c.backward(x, rp, rn)
    assert dy.shape == dr.shape == dz.shape == (0, 40) and all((p == 0).all() and p.shape == (40,) for p in params)


def test_block_norm_autograd_matches_torch():
    """Gradients through the autograd function against torch's own in 64 bits, a second
    use of x, and parameters in bf16."""
    c = Norm(65, 200, "f32", "f32", "pgrsn")
    leaves = [t.clone().requires_grad_() for t in (c.y, c.r, c.z, c.wp, c.sc, c.wn)]
    x, h = gdn.block_norm(*leaves, eps=1e-5)
    got = torch.autograd.grad((x * c.dx).sum() + (h * c.dh).sum(), leaves)
    w = [t.double().requires_grad_() for t in (c.y, c.r, c.z, c.wp, c.sc, c.wn)]
    n = w[0] * torch.rsqrt(w[0].square().mean(-1, keepdim=True) + 1e-5) * w[3]
    xx = w[1] + w[4] * n * torch.nn.functional.silu(w[2])
    hh = xx * torch.rsqrt(xx.square().mean(-1, keepdim=True) + 1e-5) * w[5]
    want = torch.autograd.grad((xx * c.dx).sum() + (hh * c.dh).sum(), w, retain_graph=True)
    for a, b in zip(got, want):
        assert a.dtype == torch.float32 and (a - b).norm() <= 1e-5 * b.norm()
    # x alone and h alone
    for pick in (0, 1):
        out = gdn.block_norm(*leaves, eps=1e-5)[pick]
        got = torch.autograd.grad(out.sum(), leaves, allow_unused=True)
        want = torch.autograd.grad((xx, hh)[pick].sum(), w, retain_graph=True, allow_unused=True)
        for a, b in zip(got, want):
            if b is not None:
                assert (a - b).norm() <= 1e-5 * b.norm() + 1e-9
    half = [t.bfloat16().requires_grad_() for t in (c.y, c.wp)]
    x, h = gdn.block_norm(half[0], post_weight=half[1], pre_norm=False)
    assert h is None
    g = torch.autograd.grad(x.float().sum(), half)
    assert all(t.dtype == torch.bfloat16 for t in g)


# ------------------------------------------------------- gated feed-forward block

FFN = [(1, 1, 1, 1), (1, 8, 8, 8), (1, 256, 520, 256), (2, 64, 64, 200), (5, 77, 135, 51), (16, 512, 1024, 512), (64, 128, 256, 64),
       (127, 72, 136, 72), (128, 64, 128, 128), (129, 64, 129, 65), (256, 256, 256, 256), (257, 320, 200, 264), (300, 33, 517, 30),
       (700, 130, 70, 257), (1100, 512, 300, 512),
       (300, 1, 1, 1), (300, 8, 8, 8), (40, 3, 5, 7), (33, 4097, 9, 2), (35, 2, 4099, 16)]


class Ffn:
    def __init__(self, M, D, F, O, dtype, layout=plain, seed=0):
        g = rng(seed + 31 * M + 7 * D + F)
        self.dtype = dtype
        self.x, self.dy = layout(normal(g, M, D, to=dtype)), layout(normal(g, M, O, to=dtype))
        self.w = [normal(g, F, D, std=D ** -0.5, to=dtype), normal(g, F, D, std=D ** -0.5, to=dtype),
                  normal(g, O, F, std=F ** -0.5, to=dtype)]
        if layout is odd:
            self.w = [odd(t) for t in self.w]

    def off(self, second):
        """Beside the last rounding: what roundings between the products leave, K and the fp32 part."""
        return (2.0 ** -8 + 2.0 ** -14) * second if self.dtype == "bf16" else 1024 * U * second

    def rel(self, name, got, want):
        e = np.linalg.norm(num(got) - want) / max(np.linalg.norm(want), 1e-300)
        assert e <= (5e-3 if self.dtype == "bf16" else 1e-5), "%s: relative error %.2e" % (name, e)

    def check_forward(self, y, gate, up, act):
        X, W = num(self.x), [num(t) for t in self.w]
        y0, g0, u0, h0 = ref.gated_ffn(X, *W, act)
        aX, aW = np.abs(X), [np.abs(t) for t in W]
        mg, mu = aX @ aW[0].T, aX @ aW[1].T
        first = 2.0 ** -14 if self.dtype == "bf16" else 1024 * U
        if gate is not None:
            close("gate", gate, g0, mg, 0, self.dtype, first * mg)
            close("up", up, u0, mu, 0, self.dtype, first * mu)
        # |act'| < 1.13, |act(g)| <= |g|: how far h may be off before it is rounded
        dh = first * (1.13 * mg * np.abs(u0) + np.abs(g0) * mu) + 16 * U * np.abs(h0)
        close("y", y, y0, 0.0, 0, self.dtype, self.off(np.abs(h0) @ aW[2].T) + 1.01 * dh @ aW[2].T)
        self.rel("y", y, y0)

    def check_backward(self, got, gate, up, act):
        X, DY, W = num(self.x), num(self.dy), [num(t) for t in self.w]
        want, (dg, du, h) = ref.gated_ffn_backward(DY, X, *W, num(gate), num(up), act)
        first = 2.0 ** -14 if self.dtype == "bf16" else 1024 * U
        mdh = np.abs(DY) @ np.abs(W[2])
        a, slope = ref.ffn_activation(num(gate), act)
        edg, edu = first * mdh * np.abs(num(up)) * (np.abs(slope) + 0.01), first * mdh * (np.abs(a) + 0.01)
        adg, adu, ah = np.abs(dg) + edg, np.abs(du) + edu, np.abs(h)
        terms = [(adg @ np.abs(W[0]) + adu @ np.abs(W[1]), edg @ np.abs(W[0]) + edu @ np.abs(W[1])),
                 (adg.T @ np.abs(X), edg.T @ np.abs(X)), (adu.T @ np.abs(X), edu.T @ np.abs(X)), (np.abs(DY).T @ ah, 0.0)]
        for name, p, q, (m, e) in zip(("dx", "dw_gate", "dw_up", "dw_down"), got, want, terms):
            close(name, p, q, 0.0, 0, self.dtype, self.off(m) + 1.01 * e)
            self.rel(name, p, q)


@pytest.mark.parametrize("dtype,layout,act", [("bf16", plain, "silu"), ("bf16", wide, "gelu_tanh"), ("bf16", odd, "silu"),
                                              ("f32", plain, "gelu_tanh"), ("f32", odd, "silu")])
@pytest.mark.parametrize("M,D,F,O", FFN)
def test_gated_ffn(M, D, F, O, dtype, layout, act):
    c = Ffn(M, D, F, O, dtype, layout)
    y, gate, up = gdn.gated_ffn_fwd(c.x, *c.w, activation=act, save=True, check=True)
    c.check_forward(y, gate, up, act)
    y2, none, _ = gdn.gated_ffn_fwd(c.x, *c.w, activation=act, check=True)
    assert none is None and torch.equal(y, y2)
    got = gdn.gated_ffn_bwd(c.dy, c.x, *c.w, gate, up, activation=act, check=True)
    c.check_backward(got, gate, up, act)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,F,O", [(2500, 512, 4000, 520), (40, 4096, 1000, 256), (4096, 64, 160, 64), (600, 2048, 640, 1030),
                                     (12, 4096, 6000, 4096)])
def test_gated_ffn_many_tiles(M, D, F, O, dtype):
    """More tiles than the GPU holds at once, long sums, sums in parts."""
    c = Ffn(M, D, F, O, dtype)
    y, gate, up = gdn.gated_ffn_fwd(c.x, *c.w, save=True, check=True)
    c.check_forward(y, gate, up, "silu")
    got = gdn.gated_ffn_bwd(c.dy, c.x, *c.w, gate, up, check=True)
    c.check_backward(got, gate, up, "silu")
    for a, b in zip(got, gdn.gated_ffn_bwd(c.dy, c.x, *c.w, gate, up)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [0, 1, 7, 300])
def test_gated_ffn_gradients_that_are_not_wanted(M, dtype):
    c = Ffn(M, 72, 200, 40, dtype)
    y, gate, up = gdn.gated_ffn_fwd(c.x, *c.w, save=True)
    assert y.shape == (M, 40)
    full = gdn.gated_ffn_bwd(c.dy, c.x, *c.w, gate, up)
    if M == 0:
        assert full[0].shape == (0, 72) and all((t == 0).all() for t in full[1:])
    for needs in [(True, False, False, False), (False, True, False, False), (False, False, True, True), (False, False, False, True)]:
        got = gdn.gated_ffn_bwd(c.dy, c.x, *c.w, gate, up, needs=needs)
        for a, b, need in zip(got, full, needs):
            assert (a is not None) == need
            assert not need or torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [3, 200])
def test_gated_ffn_rows_stand_alone(M, dtype):
    """A row that is not finite spoils its own outputs only; memory behind an output stays."""
    c = Ffn(M, 200, 264, 136, dtype)
    clean = gdn.gated_ffn_fwd(c.x, *c.w, save=True)
    bad = c.x.clone()
    bad[1, 3] = float("nan")
    buf = torch.full((M + 1, 136), 7.0, dtype=c.x.dtype, device="cuda")
    got = gdn.gated_ffn_fwd(bad, *c.w, save=True, out=buf[:M])
    assert (buf[M] == 7).all()
    keep = [i for i in range(M) if i != 1]
    for a, b in zip(got, clean):
        assert torch.equal(a[keep], b[keep]) and torch.isnan(a[1]).all()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_ffn_far_values(act):
    """Projections of +-1e4: the activation is 0 or the identity, its slope 0 or 1, nothing overflows."""
    x = torch.tensor([[1e4], [-1e4], [90.0], [-90.0], [0.0]], device="cuda")
    w = [torch.ones(1, 1, device="cuda") for _ in range(3)]
    y, gate, up = gdn.gated_ffn_fwd(x, *w, activation=act, save=True)
    want = torch.where(x > 0, x * x, torch.zeros_like(x))
    assert torch.allclose(y, want, rtol=1e-6, atol=1e-25)
    dx = gdn.gated_ffn_bwd(torch.ones_like(y), x, *w, gate, up, activation=act)[0]
    assert torch.allclose(dx, torch.where(x > 0, 2 * x, torch.zeros_like(x)), rtol=1e-6, atol=1e-25)
    # where g^2 overflows too: act'(g) is 1 or 0
    far = torch.tensor([[3e25], [-3e25]], device="cuda")
    one = torch.ones_like(far)
    dx, _, _, _ = gdn.gated_ffn_bwd(one, one, *w, far, one, activation=act)
    assert torch.allclose(dx, torch.tensor([[1.0 + 3e25], [0.0]], device="cuda"), rtol=1e-6, atol=0.0)


def test_gated_ffn_autograd_matches_torch():
    c = Ffn(130, 48, 100, 56, "f32")
    leaves = [t.clone().requires_grad_() for t in (c.x.view(2, 65, 48), *c.w)]
    y = gdn.gated_ffn(*leaves, activation="gelu_tanh")
    assert y.shape == (2, 65, 56)
    got = torch.autograd.grad(y, leaves, c.dy.view(2, 65, 56))
    w = [t.detach().double().requires_grad_() for t in leaves]
    h = torch.nn.functional.gelu(w[0] @ w[1].t(), approximate="tanh") * (w[0] @ w[2].t())
    want = torch.autograd.grad(h @ w[3].t(), w, c.dy.view(2, 65, 56).double())
    for a, b in zip(got, want):
        assert (a - b).norm() <= 1e-5 * b.norm()
    frozen = [t.detach() for t in leaves]
    assert not gdn.gated_ffn(*frozen).requires_grad


def test_offsets_beyond_32_bits():
    """Tensors of more than 2^31 elements: the first, a middle and the last rows."""
    g = rng(3)
    rows, D = 525000, 4096
    base = normal(g, 1000, D, to="bf16")
    y = base.repeat(rows // 1000, 1)
    w = 1 + normal(g, D, std=0.2)
    x, h, rp, rn = gdn.block_norm_fwd(y, y, y, w, w, w)
    want = gdn.block_norm_fwd(base, base, base, w, w, w)
    grads = gdn.block_norm_bwd(x, h, y, x, rp, rn, y, w, w, w)
    small = gdn.block_norm_bwd(want[0], want[1], base, *(want[0], want[2], want[3]), base, w, w, w)
    for at in (0, 1000 * 262, rows - 1000):
        for a, b in zip((x, h, rp, rn), want):
            assert torch.equal(a[at:at + 1000], b)
        for a, b in zip(grads[:3], small[:3]):
            assert torch.equal(a[at:at + 1000], b)
    for a, b in zip(grads[3:], small[3:]):
        assert (a / (rows // 1000) - b).norm() <= 1e-5 * b.norm()
    del y, x, h, grads
    M, D, F = 70000, 64, 32768
    base = normal(g, 1000, D, to="bf16")
    ws = [normal(g, F, D, std=D ** -0.5, to="bf16"), normal(g, F, D, std=D ** -0.5, to="bf16"), normal(g, D, F, std=F ** -0.5, to="bf16")]
    X = base.repeat(M // 1000, 1)
    y, gate, up = gdn.gated_ffn_fwd(X, *ws, save=True)
    dx = gdn.gated_ffn_bwd(X, X, *ws, gate, up, needs=(True, False, False, False))[0]
    c = Ffn.__new__(Ffn)
    c.dtype, c.x, c.dy, c.w = "bf16", base[:40], base[:40], ws
    for at in (0, 35000, M - 1000):
        c.check_forward(y[at:at + 40], gate[at:at + 40], up[at:at + 40], "silu")
        want = ref.gated_ffn_backward(num(base[:40]), num(base[:40]), *(num(t) for t in ws), num(gate[at:at + 40]), num(up[at:at + 40]))[0][0]
        c.rel("dx", dx[at:at + 40], want)


@pytest.mark.parametrize("M", [2, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_ffn_every_count_of_tokens_beside_a_limit(M, dtype):
    """Around the counts at which the products change their kernel, rows of an odd pitch among them."""
    for D, F, O in ((520, 1032, 264), (131, 257, 45)):
        c = Ffn(M, D, F, O, dtype)
        y, gate, up = gdn.gated_ffn_fwd(c.x, *c.w, save=True, check=True)
        c.check_forward(y, gate, up, "silu")


def test_single_row_without_a_leading_axis():
    c = Ffn(1, 64, 128, 72, "bf16")
    y, gate, up = gdn.gated_ffn_fwd(c.x[0], *c.w, save=True)
    assert y.shape == (72,) and gate.shape == up.shape == (128,)
    assert torch.equal(y, gdn.gated_ffn_fwd(c.x, *c.w)[0][0])
    n = Norm(1, 64, "f32", "f32", "pgrsn")
    want = n.forward()
    n.y, n.r, n.z = n.y[0], n.r[0], n.z[0]
    for a, b in zip(n.forward(), want):
        assert torch.equal(a, b[0])


# ----------------------------------------------------------------- both together

def test_two_calls_at_once():
    """Calls on two streams at the same time give what they give alone."""
    cs = [Ffn(900, 256, 1000, 256, "bf16", seed=1), Ffn(700, 300, 800, 200, "f32", seed=2)]
    ns = [Norm(4000, 512, "bf16", "f32", "pgrsn", seed=1), Norm(3000, 130, "f32", "f32", "pg", seed=2)]

    def run(c, n, stream=None):
        y, gate, up = gdn.gated_ffn_fwd(c.x, *c.w, save=True, stream=stream)
        x, h, rp, rn = n.forward(stream=stream)
        return (y, *gdn.gated_ffn_bwd(c.dy, c.x, *c.w, gate, up, stream=stream), x, *n.backward(x, rp, rn, stream=stream))

    want = [run(c, n) for c, n in zip(cs, ns)]
    streams = [torch.cuda.Stream() for _ in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(3):
        for i, (c, n) in enumerate(zip(cs, ns)):
            got[i].append(run(c, n, streams[i]))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for i in range(2):
        for again in got[i]:
            for a, b in zip(again, want[i]):
                assert (a is None and b is None) or torch.equal(a, b)


def test_training_step_in_a_graph():
    """Forward and backward through autograd, captured and replayed on new inputs."""
    g = rng(21)
    M, D, F = 150, 128, 320
    w = [normal(g, F, D, std=D ** -0.5), normal(g, F, D, std=D ** -0.5), normal(g, D, F, std=F ** -0.5), 1 + normal(g, D, std=0.1)]
    w = [t.requires_grad_() for t in w]
    x = normal(g, M, D)

    def step():
        r, h = gdn.block_norm(x, x, x, w[3], w[3], w[3])
        y, _ = gdn.block_norm(gdn.gated_ffn(h, *w[:3]), r, None, w[3], pre_norm=False)
        return torch.autograd.grad(y.square().sum(), w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.copy_(normal(g, M, D))
    graph.replay()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)

def test_layer_on_another_stream_and_in_a_graph():
    """norm -> feed-forward -> norm, on a stream of its own and replayed from a captured
    graph on new inputs: the same bits as the plain calls."""
    g = rng(11)
    M, D, F = 70, 256, 640
    y, r, z = (normal(g, M, D, to="bf16") for _ in range(3))
    w = [normal(g, F, D, std=D ** -0.5, to="bf16"), normal(g, F, D, std=D ** -0.5, to="bf16"), normal(g, D, F, std=F ** -0.5, to="bf16")]
    wn = 1 + normal(g, D, std=0.1)

    def layer(y, r, z, stream=None):
        x, h, _, _ = gdn.block_norm_fwd(y, r, z, wn, wn, wn, stream=stream)
        f, gate, up = gdn.gated_ffn_fwd(h, *w, save=True, stream=stream)
        x2, h2, rp, rn = gdn.block_norm_fwd(f, x, None, wn, None, wn, stream=stream)
        d = gdn.block_norm_bwd(x2, h2, f, x2, rp, rn, None, wn, None, wn, stream=stream)
        return (x2, h2, *d[:2], *gdn.gated_ffn_bwd(d[0], h, *w, gate, up, stream=stream))

    want = layer(y, r, z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer(y, r, z, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    iy, ir, iz = y.clone(), r.clone(), z.clone()
    with torch.cuda.stream(side):
        layer(iy, ir, iz)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(iy, ir, iz)
    ny, nr, nz = (normal(g, M, D, to="bf16") for _ in range(3))
    for t, n in ((iy, ny), (ir, nr), (iz, nz)):
        t.copy_(n)
    graph.replay()
    for a, b in zip(out, layer(ny, nr, nz)):
        assert torch.equal(a, b)


def test_written_outputs_move_their_version():
    c = Norm(4, 64, "f32", "f32", "pgrsn")
    before = c.y._version
    c.forward(out=c.y)
    assert c.y._version > before
    f = Ffn(4, 64, 64, 64, "f32")
    out = torch.empty(4, 64, device="cuda")
    before = out._version
    gdn.gated_ffn_fwd(f.x, *f.w, out=out)
    assert out._version > before


# ----------------------------------------------------------------------- refusals

def test_block_norm_refuses():
    c = Norm(6, 32, "bf16", "f32", "pgrsn")
    y, w = c.y, c.wp
    for bad, what in [((y.half(),), TypeError), ((y.cpu(),), ValueError), ((y.t(),), ValueError), ((y, y[:3]), ValueError),
                      ((y, y.float()), TypeError), ((y, None, y.float()), TypeError), ((y, None, None, w[:5]), ValueError),
                      ((y, None, None, w.double()), TypeError), ((y, None, None, w, w.bfloat16()), TypeError)]:
        with pytest.raises(what):
            gdn.block_norm_fwd(*bad)
    with pytest.raises(ValueError, match="activation"):
        gdn.block_norm_fwd(y, activation="relu")
    with pytest.raises(ValueError, match="post_norm"):
        gdn.block_norm_fwd(y, post_weight=w, post_norm=False)
    with pytest.raises(ValueError, match="pre_norm"):
        gdn.block_norm_fwd(y, pre_weight=w, pre_norm=False)
    with pytest.raises(gdn.GdnError):
        gdn.block_norm_fwd(y, eps=-1.0)
    with pytest.raises(ValueError, match="overlap"):
        gdn.block_norm_fwd(torch.zeros(100, device="cuda").as_strided((6, 32), (8, 1)))
    three = torch.zeros(4, 6, 8, 32, device="cuda")[::2, ::2, ::2]
    with pytest.raises(ValueError, match="two levels"):
        gdn.block_norm_fwd(three)
    x, _, rp, rn = c.forward()
    with pytest.raises(ValueError):
        gdn.block_norm_bwd(c.dx, None, y, x, rp, rn)
    with pytest.raises(ValueError):
        gdn.block_norm_bwd(None, None, y, x, rp, None)
    with pytest.raises(ValueError):
        gdn.block_norm_bwd(c.dx, c.dh, y, x, rp[:2], rn)
    with pytest.raises(gdn.GdnError):
        c.backward(x, rp, rn, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    # only the backward pass in reverse mode is there
    with pytest.raises(Exception):
        torch.func.jvp(lambda t: gdn.block_norm(t)[0], (c.y.float(),), (c.y.float(),))


def test_two_host_threads():
    """Calls from two threads, each on a stream of its own, give what they give alone."""
    import threading
    cs = [Ffn(400, 256, 520, 264, "bf16", seed=5), Ffn(90, 130, 300, 70, "f32", seed=6)]
    want = [gdn.gated_ffn_fwd(c.x, *c.w, save=True) for c in cs]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                got[i].append(gdn.gated_ffn_fwd(cs[i].x, *cs[i].w, save=True, stream=stream))
            stream.synchronize()
        except Exception as e:   # pragma: no cover
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for i in range(2):
        for again in got[i]:
            for a, b in zip(again, want[i]):
                assert torch.equal(a, b)


def test_gated_ffn_refuses():
    c = Ffn(6, 32, 64, 40, "bf16")
    x, (wg, wu, wd) = c.x, c.w
    for bad, what in [((x.half(), wg, wu, wd), TypeError), ((x.cpu(), wg, wu, wd), ValueError), ((x, wg.float(), wu, wd), TypeError),
                      ((x, wg, wu[:5], wd), ValueError), ((x, wg, wu, wd.t()), ValueError), ((x[:, :8], wg, wu, wd), ValueError),
                      ((x, wg[0], wu, wd), ValueError)]:
        with pytest.raises(what):
            gdn.gated_ffn_fwd(*bad)
    with pytest.raises(ValueError, match="activation"):
        gdn.gated_ffn_fwd(x, wg, wu, wd, activation="relu")
    with pytest.raises(ValueError, match="overlaps x"):
        gdn.gated_ffn_fwd(x, wg, wu, wd[:32].contiguous(), out=x)
    with pytest.raises(gdn.GdnError):
        gdn.gated_ffn_fwd(x, wg, wu, wd, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    y, gate, up = gdn.gated_ffn_fwd(x, wg, wu, wd, save=True)
    with pytest.raises(ValueError):
        gdn.gated_ffn_bwd(c.dy, x, wg, wu, wd, gate[:2], up)
    with pytest.raises(ValueError):
        gdn.gated_ffn_bwd(c.dy[:, :8], x, wg, wu, wd, gate, up)
    with pytest.raises(gdn.GdnError):
        gdn.gated_ffn_bwd(c.dy, x, wg, wu, wd, gate, up, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(Exception):
        torch.func.jvp(lambda t: gdn.gated_ffn(t, wg, wu, wd), (x,), (x,))
