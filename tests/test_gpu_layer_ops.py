"""GPU parity of the layer operators against the fp64 oracle, element by
element, at the sizes, layouts and masks where they can go wrong.

Bars.  A result that is rounded to bf16 is within 2^-8 of the exact value
relative to it (one rounding is at most 2^-9); fp32 arithmetic adds K U M, with
U = 2^-24, M the sum of the absolute values of the terms behind the element
(the oracle run on absolute values) and K the number of roundings on the
longest path:
  layer norm     the mean's sum is at most 16 + 5 + 16 additions deep: K = 64
                 on rstd max|x| (the mean's error) and on |xh|; the backward
                 pass sums the same way; its sums over rows are `rows` deep
  convolution    W products, the sigmoid (exp of an argument rounded at about
                 |u| U, a reciprocal): K = 64; its derivative moves by half of
                 u's error, so M takes |dy| (2 + |u|); sums over tokens 64 + 4 +
                 8 + groups deep: K = 256
  scan           every step multiplies by an exponential that is off by at most
                 2^-21 relatively (2^-22 of ex2, the argument's roundings
                 weighted by the exponent), so K = 8 (T + 8); in the backward
                 pass both recurrences and the sum over tokens: K = 8 (3 T + 32),
                 and over channels for B and C, which that covers
  delta step     sums over dk: K = dk + 32
"""
import numpy as np
import pytest
import torch

import chunked_prefill_gdn_gb300 as gdn
import oracle
from chunked_prefill_gdn_gb300 import build as gdn_build
from oracle import layer_ops as ref

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


def close(name, got, want, mag, K, dtype="f32"):
    got = num(got).reshape(want.shape)
    err, tol = np.abs(got - want), ROUND[dtype] * np.abs(want) + K * U * mag + 1e-37
    assert np.isfinite(got).all(), name
    assert (err <= tol).all(), "%s: error %.3e at a bar of %.3e" % (name, err.flat[np.argmax(err / tol)],
                                                                    tol.flat[np.argmax(err / tol)])


# ------------------------------------------------------------------ layer norm

NORM = [(1, 1), (3, 7), (37, 33), (5, 256), (9, 264), (17, 512), (4, 513), (3, 1000), (5, 1024), (3, 2049), (700, 96),
        (2, 4096), (3, 4100), (2, 8192), (2, 8193), (3, 9001)]


def norm_case(rows, D, dtype, wtype, layout, seed=0, shift=0.0):
    g = rng(seed + rows * 10007 + D)
    x = normal(g, rows, D, std=1.5) + shift + torch.linspace(-1, 1, rows).cuda()[:, None]
    x = layout(x.to(TORCH[dtype]))
    w = None if wtype is None else (1 + 0.3 * torch.randn(D, generator=g)).to(TORCH[wtype]).cuda()
    b = None if wtype is None else normal(g, D, std=0.2, to=wtype)
    return x, w, b, normal(g, rows, D, to=dtype)


@pytest.mark.parametrize("dtype,wtype,layout", [("bf16", "f32", lambda t: t), ("bf16", "bf16", wide),
                                                ("f32", "f32", odd), ("f32", None, wide), ("bf16", None, odd)])
@pytest.mark.parametrize("rows,D", NORM)
def test_layer_norm(rows, D, dtype, wtype, layout):
    x, w, b, dy = norm_case(rows, D, dtype, wtype, layout)
    y, mean, rstd = gdn.layer_norm_fwd(x, w, b, eps=1e-5)
    y0, m0, r0 = ref.layer_norm(num(x), num(w), num(b))
    w0 = np.ones(D) if w is None else num(w)
    top = np.abs(num(x)).max(-1, keepdims=True)
    xh = np.abs((num(x) - m0[:, None]) * r0[:, None])
    mag = np.abs(w0) * (r0[:, None] * top + xh) + (0.0 if b is None else np.abs(num(b)))
    close("y", y, y0, mag, 64, dtype)
    close("mean", mean, m0, top[:, 0], 64)
    close("rstd", rstd, r0, r0 * (1 + r0 * top[:, 0]), 64)
    # backward, from the forward's own statistics
    dx, dw, db = gdn.layer_norm_bwd(dy, x, mean, rstd, w)
    dx0, dw0, db0 = ref.layer_norm_backward(num(dy), num(x), num(mean), num(rstd), num(w))
    r = num(rstd)[:, None]
    h = np.abs((num(x) - num(mean)[:, None]) * r)
    gm = np.abs(num(dy)) * np.abs(w0)
    mag = r * (gm + gm.mean(-1, keepdims=True) + h * (gm * h).mean(-1, keepdims=True))
    close("dx", dx, dx0, mag, 64, dtype)
    close("dw", dw, dw0, (np.abs(num(dy)) * h).sum(0), 16 + rows)
    close("db", db, db0, np.abs(num(dy)).sum(0), 16 + rows)


def test_layer_norm_keeps_a_small_spread_on_a_large_mean():
    """Rows of mean 1000 and spread 1: the variance is taken around the mean."""
    x, w, b, _ = norm_case(13, 4096, "f32", "f32", lambda t: t, shift=1000.0)
    y, mean, rstd = gdn.layer_norm_fwd(x, w, b)
    y0, _, r0 = ref.layer_norm(num(x), num(w), num(b))
    top = np.abs(num(x)).max(-1, keepdims=True)
    close("y", y, y0, np.abs(num(w)) * r0[:, None] * top + np.abs(y0) + np.abs(num(b)), 64)
    close("rstd", rstd, r0, r0 * (1 + r0 * top[:, 0]), 64)


def test_layer_norm_rows_stand_alone():
    """A row with a NaN or an infinity spoils its own outputs only; a constant
    row gives the bias; no rows give zero sums."""
    x = normal(rng(5), 9, 640)
    clean = gdn.layer_norm_fwd(x)[0]
    bad = x.clone()
    bad[2, 17], bad[5, 600] = float("nan"), float("inf")
    bad[7] = 3.25
    b = normal(rng(6), 640)
    y, _, rstd = gdn.layer_norm_fwd(bad, None, b)
    keep = [0, 1, 3, 4, 6, 8]
    assert torch.equal(y[keep], gdn.layer_norm_fwd(x, None, b)[0][keep]) and not torch.isfinite(y[[2, 5]]).any()
    assert torch.equal(y[7], b) and abs(float(rstd[7]) - 1e-5 ** -0.5) < 1e-2
    assert torch.equal(clean[keep], gdn.layer_norm_fwd(bad)[0][keep])
    e = torch.empty(0, 640, device="cuda")
    dx, dw, db = gdn.layer_norm_bwd(e, e, e[:, 0], e[:, 0])
    assert dx.shape == (0, 640) and not dw.any() and not db.any()


# more rows than the blocks of a full GPU take at once (8 rows per block up to 512
# columns, else one; 6 to 1 blocks per SM): five to seven turns of every block
MANY_ROWS = [(96, 21893), (264, 18001), (512, 15003), (520, 5001), (1000, 5500), (1536, 2500), (2056, 2203), (4096, 1999),
             (4100, 901), (8192, 777), (8200, 611), (8193, 600)]


@pytest.mark.parametrize("dtype,wtype,layout", [("bf16", "f32", lambda t: t), ("f32", "f32", lambda t: t),
                                                ("bf16", "bf16", odd)])
@pytest.mark.parametrize("D,rows", MANY_ROWS)
def test_layer_norm_many_rows(D, rows, dtype, wtype, layout):
    """Every block takes several rows in turn: the stages of rows in flight go round,
    the sums of dw and db gather over a block's rows.  A sum over rows is at most 7
    turns, 8 warps, 15 + 32 partial rows and 8 roundings of a term deep: K = 80,
    which one row missing or taken twice exceeds."""
    g = rng(D * 3 + rows)
    x = layout((normal(g, rows, D, std=1.5) + torch.linspace(-1, 1, rows).cuda()[:, None]).to(TORCH[dtype]))
    w, b = (1 + 0.3 * torch.randn(D, generator=g)).to(TORCH[wtype]).cuda(), normal(g, D, std=0.2, to=wtype)
    dy = layout(normal(g, rows, D, to=dtype))
    y, mean, rstd = gdn.layer_norm_fwd(x, w, b, eps=1e-5)
    x0, w0, dy0 = num(x), num(w), num(dy)
    y0, m0, r0 = ref.layer_norm(x0, w0, num(b))
    top = np.abs(x0).max(-1, keepdims=True)
    close("y", y, y0, np.abs(w0) * (r0[:, None] * top + np.abs((x0 - m0[:, None]) * r0[:, None])) + np.abs(num(b)), 64, dtype)
    close("mean", mean, m0, top[:, 0], 64)
    close("rstd", rstd, r0, r0 * (1 + r0 * top[:, 0]), 64)
    dx, dw, db = gdn.layer_norm_bwd(dy, x, mean, rstd, w)
    dx0, dw0, db0 = ref.layer_norm_backward(dy0, x0, num(mean), num(rstd), w0)
    r = num(rstd)[:, None]
    h, gm = np.abs((x0 - num(mean)[:, None]) * r), np.abs(dy0) * np.abs(w0)
    close("dx", dx, dx0, r * (gm + gm.mean(-1, keepdims=True) + h * (gm * h).mean(-1, keepdims=True)), 64, dtype)
    close("dw", dw, dw0, (np.abs(dy0) * h).sum(0), 80)
    close("db", db, db0, np.abs(dy0).sum(0), 80)


@pytest.mark.parametrize("dtype,layout", [("bf16", lambda t: t), ("bf16", odd), ("f32", lambda t: t), ("f32", odd)])
@pytest.mark.parametrize("D", [5, 64, 128, 300, 520, 1000, 1536, 2052, 4100, 8200])
def test_layer_norm_backward_of_a_constant_row_on_a_huge_mean(D, dtype, layout):
    """Every deviation is zero, mean x rstd is past fp32's range: columns that a
    thread holds past the row's end stay out of its sums."""
    g = rng(51 + D)
    x = layout(torch.full((3, D), 2.0 ** 120, dtype=TORCH[dtype], device="cuda"))
    mean, rstd = torch.full((3,), 2.0 ** 120, device="cuda"), torch.full((3,), 2.0 ** 9, device="cuda")
    dy, w = layout(normal(g, 3, D, to=dtype)), 1 + 0.3 * normal(g, D)
    dx, dw, db = gdn.layer_norm_bwd(dy, x, mean, rstd, w)
    gw = num(dy) * num(w)
    close("dx", dx, 512.0 * (gw - gw.mean(-1, keepdims=True)), 512.0 * (np.abs(gw) + np.abs(gw).mean(-1, keepdims=True)), 64, dtype)
    assert not dw.any()
    close("db", db, num(dy).sum(0), np.abs(num(dy)).sum(0), 19)


def test_layer_norm_autograd_and_determinism():
    x, w, b, dy = norm_case(1500, 384, "bf16", "f32", lambda t: t)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    gdn.layer_norm(*leaves).backward(dy)
    _, mean, rstd = gdn.layer_norm_fwd(x, w, b)
    first = gdn.layer_norm_bwd(dy, x, mean, rstd, w)
    again = gdn.layer_norm_bwd(dy, x, mean, rstd, w)
    for leaf, a, c in zip(leaves, first, again):
        assert torch.equal(a, c) and torch.equal(leaf.grad, a)
    y, none, _ = gdn.layer_norm_fwd(x, w, b, stats=False)
    assert none is None and torch.equal(y, gdn.layer_norm(x, w, b)) and torch.equal(y, gdn.layer_norm_fwd(x, w, b)[0])


# ---------------------------------------------------- short causal convolution

CONV = [  # B, T, D, W, cu
    (1, 1, 1, 2, None), (2, 5, 3, 4, None), (3, 64, 132, 4, None), (1, 70, 260, 3, None), (2, 131, 40, 2, None),
    (1, 300, 8, 4, None), (1, 20, 12, 4, [0, 0, 1, 3, 3, 20]), (1, 200, 64, 4, [0, 1, 2, 66, 130, 131, 133, 200, 200]),
    (1, 190, 5, 3, [0, 64, 128, 190]), (1, 77, 136, 2, [0, 7, 71, 72, 77]), (1, 4, 16, 4, [0, 1, 2, 3, 4]),
]


def conv_case(B, T, D, W, cu, dtype, wtype, seed=1):
    g = rng(seed + T * 31 + D)
    n = B if cu is None else len(cu) - 1
    dev = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    return dict(x=normal(g, B, T, D, to=dtype), w=normal(g, D, W, std=0.6, to=wtype), b=normal(g, D, std=0.3, to=wtype),
                s=normal(g, n, W - 1, D, to=dtype), dy=normal(g, B, T, D, to=dtype), dl=normal(g, n, W - 1, D, to=dtype),
                cu=dev, seqs=ref.spans(B, T, cu))


@pytest.mark.parametrize("dtype,wtype,layout", [("bf16", "bf16", lambda t: t), ("bf16", "f32", wide), ("f32", "f32", odd),
                                                ("f32", "f32", lambda t: t)])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("case", CONV)
def test_causal_conv(case, silu, dtype, wtype, layout):
    c = conv_case(*case, dtype, wtype)
    W, act = case[3], "silu" if silu else None
    x, dy = layout(c["x"]), layout(c["dy"])
    y, last = gdn.causal_conv_fwd(x, c["w"], c["b"], c["s"], c["cu"], act, output_final_state=True, check=True)
    a = [num(t) for t in (x, c["w"], c["b"], c["s"])]
    y0, last0 = ref.causal_conv(*a, c["seqs"], silu)
    m, _ = ref.causal_conv(*[np.abs(t) for t in a], c["seqs"], False)
    close("y", y, y0, m, 64, dtype)
    assert np.array_equal(num(last), last0)
    dx, dw, db, ds = gdn.causal_conv_bwd(dy, x, c["w"], c["b"], c["s"], c["cu"], act, c["dl"], check=True)
    want = ref.causal_conv_backward(num(dy), *a, c["seqs"], silu, num(c["dl"]))
    mags = ref.causal_conv_backward(np.abs(num(dy)) * (2 + m), *[np.abs(t) for t in a], c["seqs"], False,
                                    np.abs(num(c["dl"])))
    for name, got, w0, mg, K, t in zip(("dx", "dw", "db", "dstate"), (dx, dw, db, ds), want, mags, (64, 256, 256, 64),
                                       (dtype, "f32", "f32", dtype)):
        close(name, got, w0, mg, K, t)


# large enough that a warp's run of tokens (8 at least) is several times the rows
# that are loaded ahead; on 152 SMs, forward / backward:
LONG_RUNS = [
    (1, 700, 12000, 4, [0, 1, 24, 25, 47, 64, 65, 95, 97, 97, 192, 224, 226, 255, 256, 288, 500, 698, 700]),   # 24 / 32
    (2, 1000, 4096, 3, None),                                                                                # 20 / 32
    (1, 1999, 4096, 2, [0, 28, 61, 240, 243, 1000, 1997, 1999]),                                              # 20 / 28
    (1, 1200, 4099, 4, [0, 40, 41, 52, 129, 700, 1200]),              # one channel per thread: 52 / 76
]


@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("case", LONG_RUNS)
def test_causal_conv_long_runs(case, dtype, wtype):
    """The ring of rows refilled many times, on and off the path without boundaries,
    sequences that start and end at the edges of runs and around them.  Sums over
    tokens are a run's 128, 8 warps, 8 + 8 groups and 10 roundings of a term deep:
    K = 256 covers them."""
    c = conv_case(*case, dtype, wtype)
    y, last = gdn.causal_conv_fwd(c["x"], c["w"], c["b"], c["s"], c["cu"], "silu", output_final_state=True, check=True)
    a = [num(c[k]) for k in ("x", "w", "b", "s")]
    y0, last0 = ref.causal_conv(*a, c["seqs"], True)
    m, _ = ref.causal_conv(*[np.abs(t) for t in a], c["seqs"], False)
    close("y", y, y0, m, 64, dtype)
    assert np.array_equal(num(last), last0)
    got = gdn.causal_conv_bwd(c["dy"], c["x"], c["w"], c["b"], c["s"], c["cu"], "silu", c["dl"], check=True)
    want = ref.causal_conv_backward(num(c["dy"]), *a, c["seqs"], True, num(c["dl"]))
    mags = ref.causal_conv_backward(np.abs(num(c["dy"])) * (2 + m), *[np.abs(t) for t in a], c["seqs"], False,
                                    np.abs(num(c["dl"])))
    for name, x, w0, mg, K, t in zip(("dx", "dw", "db", "dstate"), got, want, mags, (64, 256, 256, 64),
                                     (dtype, "f32", "f32", dtype)):
        close(name, x, w0, mg, K, t)


def test_causal_conv_without_bias_and_state():
    c = conv_case(1, 40, 24, 4, [0, 3, 3, 40], "f32", "f32")
    y, last = gdn.causal_conv_fwd(c["x"], c["w"], cu_seqlens=c["cu"], activation=None, output_final_state=True)
    y0, last0 = ref.causal_conv(num(c["x"]), num(c["w"]), None, None, c["seqs"], False)
    m, _ = ref.causal_conv(np.abs(num(c["x"])), np.abs(num(c["w"])), None, None, c["seqs"], False)
    close("y", y, y0, m, 64)
    assert np.array_equal(num(last), last0) and not last[1].any()
    assert gdn.causal_conv_fwd(c["x"], c["w"])[1] is None
    dx, dw, db, ds = gdn.causal_conv_bwd(c["dy"], c["x"], c["w"], cu_seqlens=c["cu"], activation=None)
    want = ref.causal_conv_backward(num(c["dy"]), num(c["x"]), num(c["w"]), None, None, c["seqs"], False)
    mags = ref.causal_conv_backward(np.abs(num(c["dy"])), np.abs(num(c["x"])), np.abs(num(c["w"])), None, None, c["seqs"], False)
    for name, got, w0, mg in zip(("dx", "dw", "db", "dstate"), (dx, dw, db, ds), want, mags):
        close(name, got, w0, mg, 256)


def test_causal_conv_of_no_tokens_hands_the_state_on():
    s, dl = normal(rng(2), 2, 3, 6), normal(rng(3), 2, 3, 6)
    w, x = normal(rng(4), 6, 4), torch.empty(2, 0, 6, device="cuda")
    y, last = gdn.causal_conv_fwd(x, w, None, s, output_final_state=True)
    assert y.shape == (2, 0, 6) and torch.equal(last, s)
    _, dw, db, ds = gdn.causal_conv_bwd(x, x, w, None, s, d_final_state=dl)
    assert torch.equal(ds, dl) and not dw.any() and not db.any()
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    _, last = gdn.causal_conv_fwd(x[:1], w, None, s, cu, output_final_state=True, check=True)
    assert torch.equal(last, s)


@pytest.mark.parametrize("dtype,D,W", [("bf16", 264, 4), ("f32", 7, 3), ("bf16", 130, 2)])
def test_causal_conv_steps_continue_a_prompt(dtype, D, W):
    """A prompt's last state and single tokens in permuted cache rows, with a
    padded row, against the convolution of the whole sequence."""
    g = rng(7)
    x, w, b = normal(g, 3, 9, D, to=dtype), normal(g, D, W, std=0.6, to=dtype), normal(g, D, std=0.3, to=dtype)
    y0, last0 = ref.causal_conv(num(x), num(w), num(b))
    m, _ = ref.causal_conv(np.abs(num(x)), np.abs(num(w)), np.abs(num(b)), silu=False)
    _, state = gdn.causal_conv_fwd(x[:, :4], w, b, output_final_state=True)
    pool = torch.full((5, W - 1, D), float("nan"), dtype=x.dtype, device="cuda")
    rows = [4, 0, 2]
    pool[rows] = state
    idx = torch.tensor([rows[0], -1, rows[1], rows[2], 5], dtype=torch.int32, device="cuda")
    before = pool.clone()
    for t in range(4, 9):
        xt = torch.full((5, D), float("nan"), dtype=x.dtype, device="cuda")
        xt[[0, 2, 3]] = x[:, t]
        y = gdn.causal_conv_step(xt, pool, w, b, state_indices=idx)
        close("y", y[[0, 2, 3]], y0[:, t], m[:, t], 64, dtype)
        assert not y[[1, 4]].any()
    assert np.array_equal(num(pool[rows]), last0)
    assert torch.equal(pool[[1, 3]].isnan(), before[[1, 3]].isnan())


def test_causal_conv_autograd_through_the_state():
    c = conv_case(1, 33, 20, 4, [0, 2, 33], "f32", "f32")
    leaves = [c[k].clone().requires_grad_() for k in ("x", "w", "b", "s")]
    y, last = gdn.causal_conv(*leaves, c["cu"], output_final_state=True)
    ((y * c["dy"]).sum() + (last * c["dl"]).sum()).backward()
    want = gdn.causal_conv_bwd(c["dy"], c["x"], c["w"], c["b"], c["s"], c["cu"], "silu", c["dl"])
    for leaf, g in zip(leaves, want):
        assert torch.equal(leaf.grad, g)


# ------------------------------------------------------- selective state space scan

SCAN = [  # B, T, D, N, cu
    (1, 1, 1, 1, None), (2, 5, 3, 4, None), (2, 33, 40, 16, None), (1, 300, 20, 16, None), (3, 100, 65, 8, None),
    (1, 97, 24, 17, None), (1, 64, 16, 64, None), (2, 40, 10, 33, None), (1, 130, 8, 3, [0, 0, 1, 32, 64, 64, 65, 130]),
    (1, 200, 72, 16, [0, 5, 133, 200, 200]), (1, 96, 33, 24, [0, 31, 33, 96]), (1, 70, 9, 16, [0, 70]),
]


def scan_case(B, T, D, N, cu, dtype, seed=1):
    g = rng(seed + T * 31 + D * 7 + N)
    n = B if cu is None else len(cu) - 1
    c = dict(x=normal(g, B, T, D, to=dtype), dt=normal(g, B, T, D, std=0.5, to=dtype), B=normal(g, B, T, N, to=dtype),
             C=normal(g, B, T, N, to=dtype), D=normal(g, D), z=normal(g, B, T, D, to=dtype),
             bias=normal(g, D, std=0.7) - 2.0, s=normal(g, n, D, N), dy=normal(g, B, T, D, to=dtype), dl=normal(g, n, D, N))
    c["A"] = -(torch.arange(1, N + 1, dtype=torch.float32).cuda() * torch.exp(normal(g, D, N, std=0.2)))
    c["cu"] = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    c["seqs"] = ref.spans(B, T, cu)
    return c


def scan_kw(c, softplus=True, gate=True):
    return dict(D=c["D"], z=c["z"] if gate else None, dt_bias=c["bias"], dt_softplus=softplus, initial_state=c["s"],
                cu_seqlens=c["cu"])


def scan_ref(c, f=lambda t: t, **k):
    t = {n: f(num(c[n])) for n in ("x", "B", "C", "D", "s")}
    return dict(x=t["x"], dt=num(c["dt"]), A=num(c["A"]), B=t["B"], C=t["C"], D=t["D"], bias=num(c["bias"]), state=t["s"],
                seqs=c["seqs"], **k)


def silu(z):
    return z * ref.sigmoid(z)


@pytest.mark.parametrize("dtype,layout", [("bf16", lambda t: t), ("bf16", wide), ("f32", odd), ("f32", lambda t: t)])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("case", SCAN)
def test_selective_scan(case, gate, dtype, layout):
    c = scan_case(*case, dtype)
    T = case[1]
    for k in ("x", "dt", "z", "B", "C"):
        c[k] = layout(c[k])
    y, last = gdn.selective_scan_fwd(c["x"], c["dt"], c["A"], c["B"], c["C"], **scan_kw(c, gate=gate), check=True)
    y0, last0 = ref.selective_scan(**scan_ref(c), z=num(c["z"]) if gate else None)
    ym, lm = ref.selective_scan(**scan_ref(c, np.abs))
    close("y", y, y0, ym * (np.abs(silu(num(c["z"]))) if gate else 1.0), 8 * (T + 8), dtype)
    close("state", last, last0, lm, 8 * (T + 8))


GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dstate")


def check_scan_grads(c, got, dtype, T, gate=True, softplus=True, with_final=True):
    want = ref.selective_scan_backward(num(c["dy"]), **scan_ref(c, use_softplus=softplus), z=num(c["z"]) if gate else None,
                                       d_last=num(c["dl"]) if with_final else None)
    g = np.abs(num(c["dy"])) * (np.abs(silu(num(c["z"]))) if gate else 1.0)
    mags = list(ref.selective_scan_backward(g, **scan_ref(c, np.abs, use_softplus=softplus), magnitude=True,
                                            d_last=np.abs(num(c["dl"])) if with_final else None))
    ym, _ = ref.selective_scan(**scan_ref(c, np.abs, use_softplus=softplus))
    mags[6] = 1.1 * np.abs(num(c["dy"])) * ym
    types = (dtype, dtype, "f32", dtype, dtype, "f32", dtype, "f32", "f32")
    for name, x, w, m, t in zip(GRADS, got, want, mags, types):
        if name == "dz" and not gate:
            assert x is None
            continue
        close(name, x, w, m, 8 * (3 * T + 32), t)


@pytest.mark.parametrize("dtype,layout", [("bf16", lambda t: t), ("bf16", wide), ("f32", odd), ("f32", lambda t: t)])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("case", SCAN)
def test_selective_scan_backward(case, gate, dtype, layout):
    c = scan_case(*case, dtype)
    for k in ("x", "dt", "z", "B", "C", "dy"):
        c[k] = layout(c[k])
    got = gdn.selective_scan_bwd(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"], **scan_kw(c, gate=gate),
                                 d_final_state=c["dl"], check=True)
    check_scan_grads(c, got, dtype, case[1], gate)


# several tiles of 16 tokens per block; segments of the row x tiles on 152 SMs
MANY_TILES = [
    (1, 96, 16000, 16, [0, 16, 17, 48, 50, 96]),         # 2 x 3, starting at a tile's edge, inside, at the segment's
    (1, 70, 17056, 16, [0, 3, 32, 33, 70]),              # 1 x 5
    (1, 203, 17057, 8, [0, 100, 101, 203]),              # 1 x 13, an odd number of channels
    (1, 150, 8000, 24, None),                            # 2 x 5
    (1, 100, 4900, 64, [0, 40, 64, 64, 100]),            # 1 x 7
    (2, 333, 4000, 16, None),                            # 4 x 6
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", MANY_TILES)
def test_selective_scan_many_tiles(case, dtype):
    """A block walks several tiles: rows on their way in three stages, steps prepared
    and outputs finished beside the scan, states carried from tile to tile and into
    segments of several tiles.  The oracle takes every 61st channel and the last 40."""
    c = scan_case(*case, dtype)
    T, D = case[1], case[2]
    y, last = gdn.selective_scan_fwd(c["x"], c["dt"], c["A"], c["B"], c["C"], **scan_kw(c), check=True)
    pick = torch.tensor(sorted(set(range(0, D, 61)) | set(range(D - 40, D))), device="cuda")
    p = dict(c, A=c["A"][pick], D=c["D"][pick], bias=c["bias"][pick], s=c["s"][:, pick],
             **{k: c[k][..., pick] for k in ("x", "dt", "z")})
    y0, last0 = ref.selective_scan(**scan_ref(p), z=num(p["z"]))
    ym, lm = ref.selective_scan(**scan_ref(p, np.abs))
    longest = max(t1 - t0 for _, t0, t1 in c["seqs"])
    close("y", y[..., pick], y0, ym * np.abs(silu(num(p["z"]))), 8 * (longest + 8), dtype)
    close("state", last[:, pick], last0, lm, 8 * (longest + 8))
    assert torch.isfinite(y).all() and torch.isfinite(last).all()


# segments x tiles of the main kernel, segments per block of the maps on 152 SMs
MANY_TILES_BWD = [
    ("bf16", (1, 500, 4096, 16, [0, 16, 41, 64, 128, 200, 201, 256, 300, 300, 460, 500])),   # 8 x 4, 2
    ("f32", (1, 500, 4096, 16, [0, 16, 41, 64, 128, 200, 201, 256, 300, 300, 460, 500])),
    ("f32", (1, 595, 4096, 16, None)),                        # 19 x 2, 3
    ("bf16", (1, 300, 4096, 24, [0, 80, 81, 170, 300])),      # 4 x 5, 1
    ("f32", (1, 333, 2047, 40, [0, 333])),                    # 7 x 3, 1
    ("bf16", (2, 300, 4096, 8, None)),                        # 19 x 1, 7
    ("f32", (1, 400, 8192, 8, [0, 48, 49, 144, 150, 400])),   # 9 x 3, 3
]


@pytest.mark.parametrize("dtype,case", MANY_TILES_BWD)
def test_selective_scan_backward_many_tiles(dtype, case):
    """Segments of several tiles and blocks of the maps of several segments: every
    tile's kept start state, the gradient carried from tile to tile, sequences that
    start and end at the edges of tiles, of segments and of blocks and inside."""
    c = scan_case(*case, dtype)
    got = gdn.selective_scan_bwd(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"], **scan_kw(c), d_final_state=c["dl"],
                                 check=True)
    check_scan_grads(c, got, dtype, case[1])


def test_selective_scan_backward_over_many_blocks():
    """More channels than a block of any kernel holds and longer than a segment,
    twice with the same bits; plain steps without a bias."""
    c = scan_case(1, 150, 300, 16, [0, 40, 150], "f32")
    c["bias"] = torch.zeros_like(c["bias"])
    c["dt"] = 0.3 * c["dt"].abs()
    run = lambda: gdn.selective_scan_bwd(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"], **scan_kw(c, softplus=False),   # noqa: E731
                                         d_final_state=c["dl"])
    got, again = run(), run()
    check_scan_grads(c, got, "f32", 150, softplus=False)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


def test_selective_scan_autograd():
    c = scan_case(1, 70, 40, 16, [0, 3, 70], "f32")
    names = ("x", "dt", "A", "B", "C", "D", "z", "bias")
    leaves = [c[k].clone().requires_grad_() for k in names] + [c["s"].clone().requires_grad_()]
    y, last = gdn.selective_scan(*leaves[:8], True, leaves[8], True, c["cu"])
    ((y * c["dy"]).sum() + (last * c["dl"]).sum()).backward()
    want = gdn.selective_scan_bwd(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"], **scan_kw(c), d_final_state=c["dl"])
    for leaf, g in zip(leaves, want):
        assert torch.equal(leaf.grad, g)
    # without options, through y alone
    leaves = [c[k].clone().requires_grad_() for k in ("x", "dt", "A", "B", "C")]
    y, last = gdn.selective_scan(*leaves)
    assert last is None
    (y * c["dy"]).sum().backward()
    want = gdn.selective_scan_bwd(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"])
    for leaf, g in zip(leaves, want):
        assert torch.equal(leaf.grad, g)


def test_selective_scan_backward_of_no_tokens():
    c = scan_case(2, 40, 8, 16, None, "f32")
    e = lambda t: t[:, :0]   # noqa: E731
    got = gdn.selective_scan_bwd(e(c["dy"]), e(c["x"]), e(c["dt"]), c["A"], e(c["B"]), e(c["C"]), D=c["D"],
                                 initial_state=c["s"], d_final_state=c["dl"])
    assert torch.equal(got[8], c["dl"]) and not got[2].any() and not got[5].any() and not got[7].any()


def test_no_sequences_give_zero_parameter_gradients():
    c = scan_case(2, 5, 8, 16, None, "f32")
    none = lambda t: t[:0]   # noqa: E731
    y, last = gdn.selective_scan_fwd(none(c["x"]), none(c["dt"]), c["A"], none(c["B"]), none(c["C"]))
    assert y.shape == (0, 5, 8) and last.shape == (0, 8, 16)
    got = gdn.selective_scan_bwd(none(c["dy"]), none(c["x"]), none(c["dt"]), c["A"], none(c["B"]), none(c["C"]))
    assert not got[2].any() and not got[5].any() and not got[7].any()
    x, w = torch.empty(0, 5, 8, device="cuda"), normal(rng(1), 8, 4)
    assert gdn.causal_conv_fwd(x, w)[0].shape == (0, 5, 8)
    _, dw, db, _ = gdn.causal_conv_bwd(x, x, w)
    assert not dw.any() and not db.any()
    assert gdn.causal_conv_step(x[:, 0], torch.empty(0, 3, 8, device="cuda"), w).shape == (0, 8)
    q = torch.empty(0, 2, 32, device="cuda")
    assert gdn.gated_delta_step(q, q, q, q[..., 0], q[..., 0], torch.empty(0, 2, 32, 32, device="cuda")).shape == (0, 2, 32)


@pytest.mark.parametrize("T", [17, 40, 600])
def test_no_sequences_of_many_tokens(T):
    """No batch rows of more than one tile: empty outputs, zero gradients of the
    parameters."""
    c = scan_case(1, 3, 40, 16, None, "f32")
    e, bc = torch.empty(0, T, 40, device="cuda"), torch.empty(0, T, 16, device="cuda")
    y, last = gdn.selective_scan_fwd(e, e, c["A"], bc, bc, D=c["D"], dt_bias=c["bias"])
    assert y.shape == (0, T, 40) and last.shape == (0, 40, 16)
    got = gdn.selective_scan_bwd(e, e, e, c["A"], bc, bc, D=c["D"], dt_bias=c["bias"])
    assert got[0].shape == (0, T, 40) and got[3].shape == (0, T, 16) and got[8].shape == (0, 40, 16)
    assert not got[2].any() and not got[5].any() and not got[7].any()


@pytest.mark.parametrize("N", [16, 24])
def test_selective_scan_channels_stand_alone(N):
    """A NaN in one channel's input, or an infinite one, leaves the others' outputs,
    states and gradients as they are."""
    c = scan_case(1, 60, 40, N, [0, 20, 60], "f32")
    run = lambda: gdn.selective_scan_fwd(c["x"], c["dt"], c["A"], c["B"], c["C"], **scan_kw(c))   # noqa: E731
    grads = lambda: gdn.selective_scan_bwd(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"], **scan_kw(c))   # noqa: E731
    (y, last), g = run(), grads()
    c["x"][0, 30, 7], c["dt"][0, 31, 9] = float("nan"), float("inf")
    (y2, last2), g2 = run(), grads()
    others = [i for i in range(40) if i not in (7, 9)]
    assert torch.equal(y[..., others], y2[..., others]) and torch.equal(last[:, others], last2[:, others])
    assert torch.equal(y[:, :20], y2[:, :20])                 # and the sequence before
    assert not torch.isfinite(y2[0, 30:, 7]).any()
    for i in (0, 1, 6):
        assert torch.equal(g[i][..., others], g2[i][..., others])
    assert torch.equal(g[2][others], g2[2][others]) and torch.equal(g[8][:, others], g2[8][:, others])


def test_selective_scan_plain_steps_and_no_options():
    """dt used as it is (positive and zero steps, no bias), no skip, no gate, no state."""
    c = scan_case(2, 70, 12, 16, None, "f32")
    c["dt"] = c["dt"].abs() * (c["dt"] > -0.2)
    y, last = gdn.selective_scan_fwd(c["x"], c["dt"], c["A"], c["B"], c["C"], dt_softplus=False)
    a = dict(dt=num(c["dt"]), A=num(c["A"]), use_softplus=False)
    y0, last0 = ref.selective_scan(num(c["x"]), B=num(c["B"]), C=num(c["C"]), **a)
    ym, lm = ref.selective_scan(np.abs(num(c["x"])), B=np.abs(num(c["B"])), C=np.abs(num(c["C"])), **a)
    close("y", y, y0, ym, 8 * 78)
    close("state", last, last0, lm, 8 * 78)


def test_selective_scan_of_no_tokens_and_of_closed_steps():
    """No tokens: the state is handed on.  dt = -inf (a masked token): the step is
    zero, the state stays; dt far below or above: softplus's own limits."""
    c = scan_case(2, 40, 8, 16, None, "f32")
    e = lambda t: t[:, :0]   # noqa: E731
    y, last = gdn.selective_scan_fwd(e(c["x"]), e(c["dt"]), c["A"], e(c["B"]), e(c["C"]), initial_state=c["s"])
    assert y.shape == (2, 0, 8) and torch.equal(last, c["s"])
    dt = torch.full_like(c["dt"], float("-inf"))
    y, last = gdn.selective_scan_fwd(c["x"], dt, c["A"], c["B"], c["C"], initial_state=c["s"])
    assert torch.equal(last, c["s"])
    y0 = np.einsum("bdn,btn->btd", num(c["s"]), num(c["C"]))
    close("y", y, y0, np.einsum("bdn,btn->btd", np.abs(num(c["s"])), np.abs(num(c["C"]))), 64)
    dt = torch.where(c["dt"] > 0, 25.0, -25.0).float()
    y, _ = gdn.selective_scan_fwd(c["x"], dt, c["A"], c["B"], c["C"])
    a = dict(dt=num(dt), A=num(c["A"]))
    y0, _ = ref.selective_scan(num(c["x"]), B=num(c["B"]), C=num(c["C"]), **a)
    ym, _ = ref.selective_scan(np.abs(num(c["x"])), B=np.abs(num(c["B"])), C=np.abs(num(c["C"])), **a)
    close("y", y, y0, ym, 8 * 48)


@pytest.mark.parametrize("dtype,D,N", [("bf16", 72, 16), ("f32", 5, 24), ("bf16", 33, 3), ("f32", 16, 64)])
def test_selective_scan_steps_continue_a_prompt(dtype, D, N):
    c = scan_case(3, 9, D, N, None, dtype)
    y0, last0 = ref.selective_scan(**scan_ref(c), z=num(c["z"]))
    ym, lm = ref.selective_scan(**scan_ref(c, np.abs))
    ym = ym * np.abs(silu(num(c["z"])))
    cut = lambda t, a, b: t[:, a:b]   # noqa: E731
    _, state = gdn.selective_scan_fwd(*(cut(c[k], 0, 4) for k in ("x", "dt")), c["A"],
                                      *(cut(c[k], 0, 4) for k in ("B", "C")), D=c["D"], z=cut(c["z"], 0, 4),
                                      dt_bias=c["bias"], initial_state=c["s"])
    pool = torch.full((5, D, N), float("nan"), device="cuda")
    rows, at = [4, 0, 2], [0, 2, 3]
    pool[rows] = state
    idx = torch.tensor([rows[0], -1, rows[1], rows[2], 7], dtype=torch.int32, device="cuda")

    def padded(t):
        p = torch.full((5, t.shape[-1]), float("nan"), dtype=t.dtype, device="cuda")
        p[at] = t
        return p

    for t in range(4, 9):
        y = gdn.selective_scan_step(padded(c["x"][:, t]), padded(c["dt"][:, t]), c["A"], padded(c["B"][:, t]),
                                    padded(c["C"][:, t]), pool, D=c["D"], z=padded(c["z"][:, t]), dt_bias=c["bias"],
                                    state_indices=idx)
        close("y", y[at], y0[:, t], ym[:, t], 8 * 17, dtype)
        assert not y[[1, 4]].any()
    close("state", pool[rows], last0, lm, 8 * 17)
    assert pool[[1, 3]].isnan().all()


# ------------------------------------------------------------- outputs and inputs

def test_out_in_an_inputs_memory_is_refused():
    """Where a value is read by others than the thread that writes in its place."""
    g = rng(41)
    buf = normal(g, 2, 40, 32)
    x = buf[:, :32].contiguous()
    flat = torch.cat([x.flatten(), x.flatten()[:64]])
    xs, later = flat[:2048].view(2, 32, 32), flat[64:].view(2, 32, 32)      # two rows apart
    w, s = normal(g, 32, 4), normal(g, 2, 3, 32)
    A, bc = -normal(g, 32, 32).abs(), normal(g, 2, 32, 32)
    for call in (lambda: gdn.causal_conv_fwd(x, w, out=x), lambda: gdn.causal_conv_fwd(xs, w, out=later),
                 lambda: gdn.causal_conv_fwd(normal(g, 1, 3, 32), w, initial_state=s[:1], out=s[:1]),
                 lambda: gdn.layer_norm_fwd(xs, out=later), lambda: gdn.layer_norm_fwd(x, x[0, 0], out=x),
                 lambda: gdn.selective_scan_fwd(xs, xs, A, bc, bc, out=later),
                 lambda: gdn.selective_scan_fwd(x, x, A, bc, bc, out=bc),
                 lambda: gdn.causal_conv_step(x[:, 0].contiguous(), s, w, out=s.view(-1)[:64].view(2, 32)),
                 lambda: gdn.causal_conv_step(xs[0, :2], s, w, out=flat[16:80].view(2, 32)),
                 lambda: gdn.selective_scan_step(xs[0, :2], xs[0, :2], A, bc[0, :2], bc[0, :2], normal(g, 2, 32, 32),
                                                 out=flat[16:80].view(2, 32))):
        with pytest.raises(ValueError, match="overlaps"):
            call()
    q, gate, S = normal(g, 2, 2, 64), -normal(g, 2, 2).abs(), normal(g, 2, 2, 64, 64)
    k, v = normal(g, 2, 2, 64), normal(g, 2, 2, 64)
    before = S.clone()
    for out in (q, k, v, S.view(-1)[:256].view(2, 2, 64)):
        with pytest.raises(ValueError, match="overlaps"):
            gdn.gated_delta_step(q, k, v, gate, gate, S, out=out)
    assert torch.equal(S, before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(1, 40), (70, 33), (200, 512)])
def test_out_may_be_the_input_where_that_is_allowed(T, D, dtype):
    c = scan_case(2, T, D, 16, None, dtype)
    want = gdn.layer_norm_fwd(c["x"], c["D"])[0]
    x = c["x"].clone()
    assert torch.equal(gdn.layer_norm_fwd(x, c["D"], out=x)[0], want) and torch.equal(x, want)
    run = lambda t, out: gdn.selective_scan_fwd(t["x"], t["dt"], c["A"], c["B"], c["C"], **scan_kw(dict(c, z=t["z"])), out=out)   # noqa: E731
    want, last = run(c, None)
    for k in ("x", "dt", "z"):
        t = {n: c[n].clone() for n in ("x", "dt", "z")}
        got, end = run(t, t[k])
        assert got is t[k] and torch.equal(got, want) and torch.equal(end, last)
    one = {n: c[n][:, 0].contiguous() for n in ("x", "dt", "z", "B", "C")}
    step = lambda t, S, out: gdn.selective_scan_step(t["x"], t["dt"], c["A"], t["B"], t["C"], S, z=t["z"], out=out)   # noqa: E731
    S0 = c["s"].clone()
    want = step(one, S0, None)
    for k in ("x", "dt", "z"):
        t, S = {n: v.clone() for n, v in one.items()}, c["s"].clone()
        assert torch.equal(step(t, S, t[k]), want) and torch.equal(S, S0)
    w, s0, s1 = normal(rng(3), D, 4), normal(rng(4), 2, 3, D, to=dtype), normal(rng(4), 2, 3, D, to=dtype)
    want, x = gdn.causal_conv_step(one["x"], s0, w), one["x"].clone()
    assert torch.equal(gdn.causal_conv_step(x, s1, w, out=x), want) and torch.equal(s0, s1)


# ------------------------------------------------------- writes that autograd sees

def test_written_tensors_count_as_modified():
    """Every state and every out= moves its version counter; nothing else does."""
    g = rng(31)
    x, w = normal(g, 2, 32), normal(g, 32, 4)
    x3, A, bc = normal(g, 1, 6, 32), -normal(g, 32, 8).abs(), normal(g, 1, 6, 8)
    q, gate, beta = normal(g, 2, 1, 32), -normal(g, 2, 1).abs(), torch.sigmoid(normal(g, 2, 1))
    conv, ssm, delta = normal(g, 2, 3, 32), normal(g, 2, 32, 8), normal(g, 2, 1, 32, 32)
    b2, c2 = normal(g, 2, 8), normal(g, 2, 8)
    like = torch.empty_like
    calls = [
        ((), lambda out: gdn.layer_norm_fwd(x, out=out), like(x)),
        ((), lambda out: gdn.causal_conv_fwd(x3, w, out=out), like(x3)),
        ((), lambda out: gdn.selective_scan_fwd(x3, x3, A, bc, bc, out=out), like(x3)),
        ((conv,), lambda out: gdn.causal_conv_step(x, conv, w, out=out), like(x)),
        ((ssm,), lambda out: gdn.selective_scan_step(x, x, A, b2, c2, ssm, out=out), like(x)),
        ((delta,), lambda out: gdn.gated_delta_step(q, q, q, gate, beta, delta, out=out), like(q)),
    ]
    inputs = (x, w, x3, A, bc, q, gate, beta, b2, c2)
    versions = [t._version for t in inputs]
    for states, call, out in calls:
        before = [t._version for t in (*states, out)]
        call(out)
        assert all(t._version > v for t, v in zip((*states, out), before))
        before = [t._version for t in states]
        call(None)
        assert all(t._version > v for t, v in zip(states, before))
    assert [t._version for t in inputs] == versions


def test_a_state_moved_on_is_not_used_in_a_backward_pass():
    """A step on a state that a recorded call has read: torch's error, not the
    gradient at the overwritten value."""
    g = rng(32)
    x, w, s = normal(g, 1, 6, 32), normal(g, 32, 4).requires_grad_(), normal(g, 1, 3, 32)
    y, _ = gdn.causal_conv(x, w, initial_state=s)
    gdn.causal_conv_step(x[:, 0], s, w.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    A, bc, h = (-normal(g, 32, 8).abs()).requires_grad_(), normal(g, 1, 6, 8), normal(g, 1, 32, 8)
    y, _ = gdn.selective_scan(x, x, A, bc, bc, initial_state=h)
    gdn.selective_scan_step(x[:, 0], x[:, 0], A.detach(), bc[:, 0], bc[:, 0], h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    wn, v = normal(g, 32).requires_grad_(), normal(g, 4, 32)
    y = gdn.layer_norm(v, wn)
    gdn.layer_norm_fwd(normal(g, 4, 32), out=v)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


# -------------------------------------------------- one token of the delta rule

@pytest.mark.parametrize("N,H,dk,dv,dtype,norm", [
    (1, 1, 128, 128, "bf16", False), (2, 32, 128, 128, "bf16", True), (12, 32, 128, 128, "f32", False), (3, 5, 32, 32, "f32", True),
    (2, 3, 32, 128, "bf16", False), (1, 7, 128, 32, "f32", False), (3, 2, 64, 64, "bf16", False), (40, 9, 64, 128, "f32", True),
    (2, 2, 64, 32, "bf16", True), (300, 2, 32, 64, "f32", False)])
def test_delta_step(N, H, dk, dv, dtype, norm):
    g = rng(N * 100 + dk)
    q, k, v = normal(g, N, H, dk, to=dtype), normal(g, N, H, dk, to=dtype), normal(g, N, H, dv, to=dtype)
    if not norm:
        q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(t.dtype) for t in (q, k))
    gate, beta = -normal(g, N, H).abs(), torch.sigmoid(normal(g, N, H))
    rows = torch.randperm(N + 3, generator=g)[:N].tolist()
    pool = normal(g, N + 3, H, dk, dv)
    start = pool.clone()
    idx = torch.tensor(rows, dtype=torch.int32, device="cuda")
    if N > 2:
        idx[1] = -1
    live = [i for i in range(N) if not (N > 2 and i == 1)]
    o = gdn.gated_delta_step(q, k, v, gate, beta, pool, use_qk_l2norm_in_kernel=norm, state_indices=idx)
    a = [num(t) for t in (q, k, v, gate, beta, start[rows])]
    o0, S0 = ref.delta_step(*a, l2norm=norm)
    b = [np.abs(t) for t in a]
    b[3] = a[3]
    # |u| <= beta (|v| + |k|.|S'|): with v negated the oracle adds the magnitudes
    kn, qn = b[1], b[0]
    if norm:
        kn, qn = (t / np.sqrt((t * t).sum(-1, keepdims=True) + 1e-6) for t in (kn, qn))
    Sm = b[5] * np.exp(a[3])[..., None, None]
    um = b[4][..., None] * (b[2] + np.einsum("nhj,nhji->nhi", kn, Sm))
    Sm = Sm + kn[..., None] * um[..., None, :]
    om = np.einsum("nhj,nhji->nhi", qn, Sm) * dk ** -0.5
    close("o", o[live], o0[live], om[live], dk + 32, dtype)
    close("state", pool[rows][live], S0[live], Sm[live], dk + 32)
    others = [i for i in range(N + 3) if i not in [rows[j] for j in live]]
    assert torch.equal(pool[others], start[others])
    if N > 2:
        assert not o[1].any()


def test_delta_step_takes_slices_of_one_projection():
    g = rng(21)
    N, H, d = 5, 3, 64
    qkv = normal(g, N, 3, H, d, to="bf16")
    gate, beta, S = -normal(g, N, H).abs(), torch.sigmoid(normal(g, N, H)), normal(g, N, H, d, d)
    S2 = S.clone()
    o = gdn.gated_delta_step(*qkv.unbind(1), gate, beta, S, use_qk_l2norm_in_kernel=True)
    o2 = gdn.gated_delta_step(*(t.contiguous() for t in qkv.unbind(1)), gate, beta, S2, use_qk_l2norm_in_kernel=True)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    with pytest.raises(ValueError):
        gdn.gated_delta_step(*(normal(g, N, H, 2 * d)[..., :d] for _ in range(3)), gate, beta, S)   # heads apart


def test_delta_steps_continue_a_prompt():
    """chunk_fwd's final state goes on token by token as the longer prompt does
    (the parity bar of the prefill path: 5e-3 relative, 2e-2 largest)."""
    g = rng(11)
    N, T, H, d = 2, 70, 3, 128
    q, k, v = (normal(g, N, T, H, d, to="bf16") for _ in range(3))
    q, k = (torch.nn.functional.normalize(t.float(), dim=-1).bfloat16() for t in (q, k))
    gate, beta = -0.2 * normal(g, N, T, H).abs(), torch.sigmoid(normal(g, N, T, H))
    o_all, s_all = gdn.chunk_fwd(q, k, v, gate, beta)
    cut = lambda t, a, b: t[:, a:b].contiguous()   # noqa: E731
    _, state = gdn.chunk_fwd(*(cut(t, 0, 66) for t in (q, k, v, gate, beta)))
    for t in range(66, 70):
        o = gdn.gated_delta_step(*(x[:, t].contiguous() for x in (q, k, v, gate, beta)), state)
        d_o = num(o) - num(o_all[:, t])
        assert np.linalg.norm(d_o) <= 1e-2 * np.linalg.norm(num(o)) and np.abs(d_o).max() <= 2e-2
    assert np.linalg.norm(num(state) - num(s_all)) <= 5e-3 * np.linalg.norm(num(s_all))


def test_delta_step_in_a_cache_past_32_bits():
    """The last rows of a cache of more than 2^32 elements."""
    H, d = 64, 128
    P = 2 ** 32 // (H * d * d) + 2
    if torch.cuda.mem_get_info()[0] < 4 * P * H * d * d + 2 ** 31:
        pytest.skip("not enough memory free")
    pool = torch.empty(P, H, d, d, device="cuda")
    g = rng(12)
    q, k, v = (normal(g, 1, H, d) for _ in range(3))
    gate, beta, S = -normal(g, 1, H).abs(), torch.sigmoid(normal(g, 1, H)), normal(g, 1, H, d, d)
    pool[P - 1] = S[0]
    idx = torch.tensor([P - 1], dtype=torch.int32, device="cuda")
    o = gdn.gated_delta_step(q, k, v, gate, beta, pool, use_qk_l2norm_in_kernel=True, state_indices=idx)
    small = S.clone()
    assert torch.equal(o, gdn.gated_delta_step(q, k, v, gate, beta, small, use_qk_l2norm_in_kernel=True))
    assert torch.equal(pool[P - 1], small[0])


# ------------------------------------------------------------ streams and graphs

def test_operators_follow_the_stream_they_are_given():
    """Inputs made on one stream, the call on another: an event orders them, and
    what the call allocates stays its own while it runs."""
    side = torch.cuda.Stream()
    x, w, b, dy = norm_case(4000, 1024, "bf16", "f32", lambda t: t)
    c = conv_case(1, 200, 64, 4, None, "bf16", "bf16")
    want = gdn.layer_norm_fwd(x, w, b), gdn.causal_conv_fwd(c["x"], c["w"], c["b"])
    want_b = gdn.layer_norm_bwd(dy, x, want[0][1], want[0][2], w)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = gdn.layer_norm_fwd(x, w, b, stream=side)
    got_b = gdn.layer_norm_bwd(dy, x, mean, rstd, w, stream=side)
    yc, _ = gdn.causal_conv_fwd(c["x"], c["w"], c["b"], stream=side)
    junk = [torch.full((2 ** 20,), 7.0, device="cuda") for _ in range(8)]   # would reuse freed memory
    side.synchronize()
    assert torch.equal(y, want[0][0]) and torch.equal(yc, want[1][0]) and len(junk) == 8
    assert all(torch.equal(a, d) for a, d in zip(got_b, want_b))


def test_outputs_on_a_given_stream_are_not_blocks_of_the_current_one():
    """A block freed on the current stream may still be written by work queued
    there; what a call on another stream allocates is not such a block, its
    workspace included."""
    side = torch.cuda.Stream()
    x, w, b, dy = norm_case(4000, 1024, "bf16", "f32", lambda t: t)
    y, mean, rstd = gdn.layer_norm_fwd(x, w, b)
    want = gdn.layer_norm_bwd(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    blocks = [torch.empty_like(x) for _ in range(4)]
    freed = {t.data_ptr() for t in blocks}
    for t in blocks:
        t.fill_(7.0)
    side.wait_stream(torch.cuda.current_stream())
    del blocks, t
    out = gdn.layer_norm_fwd(x, w, b, stream=side)
    got = gdn.layer_norm_bwd(dy, x, mean, rstd, w, stream=side)
    assert out[0].data_ptr() not in freed and got[0].data_ptr() not in freed
    assert torch.cuda.current_stream() != side
    torch.cuda.synchronize()
    assert torch.equal(out[0], y) and all(torch.equal(a, d) for a, d in zip(got, want))
    ran = torch.cuda.current_stream()
    with pytest.raises(gdn.GdnError):
        gdn.layer_norm_fwd(torch.zeros(2, 0, device="cuda"), stream=side)
    assert torch.cuda.current_stream() == ran


def test_steps_run_in_a_graph():
    c = scan_case(2, 1, 64, 16, None, "bf16")
    x, w, b = normal(rng(1), 2, 64, to="bf16"), normal(rng(2), 64, 4, to="bf16"), normal(rng(3), 64, to="bf16")
    cs, ss = normal(rng(4), 2, 3, 64, to="bf16"), c["s"].clone()

    def token(cs, ss):
        h = gdn.causal_conv_step(x, cs, w, b)
        return gdn.selective_scan_step(h, c["dt"][:, 0], c["A"], c["B"][:, 0], c["C"][:, 0], ss, D=c["D"],
                                       dt_bias=c["bias"])

    ref_cs, ref_ss = cs.clone(), ss.clone()
    want = [token(ref_cs, ref_ss).clone() for _ in range(3)]
    g_cs, g_ss = cs.clone(), ss.clone()
    token(cs.clone(), ss.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(g_cs, g_ss)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
    assert torch.equal(g_cs, ref_cs) and torch.equal(g_ss, ref_ss)


# ------------------------------------------------------------------- refusals

def test_layer_ops_refuse_bad_arguments():
    g = rng(1)
    x, w = normal(g, 4, 32), normal(g, 32)
    xc, wc = normal(g, 1, 6, 32), normal(g, 32, 4)
    with pytest.raises(ValueError):
        gdn.layer_norm_fwd(x, w[:16])
    with pytest.raises(TypeError):
        gdn.layer_norm_fwd(x.half())
    with pytest.raises(ValueError):
        gdn.layer_norm_fwd(x.t())
    with pytest.raises(ValueError):
        gdn.layer_norm_fwd(x.expand(3, 4, 32))
    with pytest.raises(TypeError):
        gdn.layer_norm_fwd(x.bfloat16(), w.half())
    with pytest.raises(gdn.GdnError):
        gdn.layer_norm_fwd(x, eps=-1.0)
    with pytest.raises(gdn.GdnError):                       # five taps
        gdn.causal_conv_fwd(xc, normal(g, 32, 5))
    with pytest.raises(ValueError):
        gdn.causal_conv_fwd(xc, wc, activation="relu")
    with pytest.raises(ValueError):
        gdn.causal_conv_fwd(xc, wc, initial_state=normal(g, 1, 4, 32))
    with pytest.raises(TypeError):
        gdn.causal_conv_fwd(xc, wc, cu_seqlens=torch.tensor([0, 6], device="cuda"))
    with pytest.raises(ValueError):
        gdn.causal_conv_step(x, normal(g, 3, 3, 32), wc)    # fewer states than rows
    with pytest.raises(gdn.GdnError):                       # more states than a channel may have
        gdn.selective_scan_fwd(xc, xc, normal(g, 32, 65), normal(g, 1, 6, 65), normal(g, 1, 6, 65))
    with pytest.raises(ValueError):
        gdn.selective_scan_fwd(xc, xc, normal(g, 32, 8), normal(g, 1, 6, 8), normal(g, 1, 5, 8))
    with pytest.raises(gdn.GdnError):                       # head size
        gdn.gated_delta_step(*(normal(g, 1, 2, 48) for _ in range(3)), normal(g, 1, 2), normal(g, 1, 2), normal(g, 1, 2, 48, 48))


@pytest.mark.parametrize("cu", [[1, 6], [0, 5], [0, 4, 3, 6], [0, 9, 6], [0, -3, 6], [5, 0, 6]])
def test_bad_cu_seqlens_is_reported(cu):
    """Found on the device and read back with check=True; nothing outside the
    tensors is touched (every index is clamped to them)."""
    g = rng(1)
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    n = cu.numel() - 1
    x, w = normal(g, 1, 6, 32), normal(g, 32, 4)
    s = normal(g, n, 3, 32)
    with pytest.raises(gdn.GdnError) as e:
        gdn.causal_conv_fwd(x, w, None, s, cu, output_final_state=True, check=True)
    assert e.value.status == 5
    with pytest.raises(gdn.GdnError) as e:
        gdn.causal_conv_bwd(x, x, w, None, s, cu, check=True)
    assert e.value.status == 5
    B, A = normal(g, 1, 6, 8), -normal(g, 32, 8).abs()
    with pytest.raises(gdn.GdnError) as e:
        gdn.selective_scan_fwd(x, x, A, B, B, initial_state=normal(g, n, 32, 8), cu_seqlens=cu, check=True)
    assert e.value.status == 5
    with pytest.raises(gdn.GdnError) as e:
        gdn.selective_scan_bwd(x, x, x, A, B, B, initial_state=normal(g, n, 32, 8), cu_seqlens=cu, check=True)
    assert e.value.status == 5
