"""The feed-forward block where its sums are long: gradients of the weights over millions of
tokens, against 64 bits.

All terms are positive, so that what an addition cuts off adds up instead of cancelling.
Bar for bf16, relative to the value: 2^-8 for the last rounding, 2^-8 for that of dgate, dup
or h before the product, and 2^-10 for the sums: 8192 additions of 16 products in one part at
most, each off by at most 2^-22 of the sum so far, which on average is half the final one.  The
reference takes the rounded h, dgate and dup where they are known (h, dup), and so their
rounding drops out.  fp32: 1024 U as for shorter sums: 6 x 16 additions in tensor memory of up to
2^-22 (384 U), then 512 of U within a part (512 U), then 33 parts of U."""
import pytest
import torch

import chunked_prefill_gdn_gb300 as gdn
from chunked_prefill_gdn_gb300 import build as gdn_build

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def lib():
    gdn_build.build()
    return gdn.load_library()


def positive(g, *shape, to):
    return (torch.rand(*shape, generator=g, device="cuda") + 0.5).to(TORCH[to])


def within(name, got, want, bar):
    err = ((got.double() - want) / want).abs().max().item()
    assert err <= bar, "%s: relative error %.2e at a bar of %.2e" % (name, err, bar)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,F,O", [(2 ** 21 + 5, 8, 16, 8), (2 ** 22, 24, 8, 40), (2 ** 20 + 77, 5, 3, 7)])
def test_gradients_of_weights_over_millions_of_tokens(M, D, F, O, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + D)
    x, dy, gate, up = (positive(g, M, n, to=dtype) for n in (D, O, F, F))
    w = [positive(g, *s, to=dtype) for s in ((F, D), (F, D), (O, F))]
    _, dwg, dwu, dwd = got = gdn.gated_ffn_bwd(dy, x, *w, gate, up, check=True)
    gd, ud, dh = gate.double(), up.double(), dy.double() @ w[2].double()
    s = torch.sigmoid(gd)
    a, slope = gd * s, s + gd * s * (1 - s)
    bf16 = dtype == "bf16"
    between = (lambda t: t.bfloat16().double()) if bf16 else lambda t: t   # noqa: E731
    sums = 2.0 ** -8 + 2.0 ** -10 if bf16 else 1024 * U
    # dh is rounded nowhere, but its own sums' error may move dup's and dgate's rounding by a step
    within("dw_down", dwd, dy.double().t() @ between(a * ud), sums)
    within("dw_up", dwu, between(dh * a).t() @ x.double(), sums + (2.0 ** -12 if bf16 else 0.0))
    within("dw_gate", dwg, (dh * ud * slope).t() @ x.double(), sums + (2.0 ** -8 if bf16 else 0.0))
    for p, q in zip(got, gdn.gated_ffn_bwd(dy, x, *w, gate, up)):
        assert torch.equal(p, q)


# (M, D, F, D_out): weights of which one side passes 2^19, with few tokens and many
LONG = [(4, 64, 600000, 64), (16, 8, 600008, 9), (40, 24, 600000, 16), (200, 8, 530001, 8), (1, 2 ** 21, 24, 16), (3, 2 ** 20 + 8, 7, 5),
        (40, 2 ** 21, 24, 16), (5, 16, 24, 2 ** 21 + 3), (130, 16, 24, 700000), (1, 8, 2 ** 21, 8)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,F,O", LONG)
def test_long_sides_of_weights(M, D, F, O, dtype):
    """Bars on the sum of the absolute values of a result's terms: a sum in tensor memory 2^-9
    (8192 additions of 2^-22), and fp32 as above with K / 256 additions of U for a few tokens;
    what lies between the products is off by as much in its terms, and rounded (bf16)."""
    bf16 = dtype == "bf16"
    g = torch.Generator(device="cuda").manual_seed(F + D + O)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(TORCH[dtype])   # noqa: E731
    x, dy = n(M, D), n(M, O)
    w = [n(F, D, std=D ** -0.5), n(F, D, std=D ** -0.5), n(O, F, std=F ** -0.5)]
    y, gate, up = gdn.gated_ffn_fwd(x, *w, save=True, check=True)
    assert torch.equal(y, gdn.gated_ffn_fwd(x, *w)[0])
    half = 2.0 ** -8 if bf16 else 0.0
    part = lambda K: 2.0 ** -9 if bf16 else (1024 + K / 256) * U   # noqa: E731

    def check(name, got, want, mag, K, before=0.0):
        tol = half * want.abs() + part(K) * mag + before
        assert ((got.double() - want).abs() <= tol + 1e-37).all(), name
        assert (got.double() - want).norm() <= (5e-3 if bf16 else 1e-5) * want.norm(), name

    X, DY, (WG, WU, WD) = x.double(), dy.double(), (t.double() for t in w)
    G, V = X @ WG.t(), X @ WU.t()
    mg, mu = X.abs() @ WG.abs().t(), X.abs() @ WU.abs().t()
    check("gate", gate, G, mg, D)
    check("up", up, V, mu, D)
    h = G * torch.sigmoid(G) * V
    dh = part(D) * (1.13 * mg * V.abs() + G.abs() * mu) + 16 * U * h.abs() + half * h.abs()
    check("y", y, h @ WD.t(), h.abs() @ WD.abs().t(), F, 1.01 * dh @ WD.abs().t())
    del G, V, mg, mu, h, dh
    got = gdn.gated_ffn_bwd(dy, x, *w, gate, up, check=True)
    G, V = gate.double(), up.double()
    s = torch.sigmoid(G)
    a, slope = G * s, s + G * s * (1 - s)
    dh, mdh = DY @ WD, DY.abs() @ WD.abs()
    dg, du, h = dh * V * slope, dh * a, a * V
    edg = part(O) * mdh * V.abs() * (slope.abs() + 0.01) + half * dg.abs() + 16 * U * dg.abs()
    edu = part(O) * mdh * (a.abs() + 0.01) + half * du.abs() + 16 * U * du.abs()
    eh = (half + 16 * U) * h.abs()
    adg, adu, ah = dg.abs() + edg, du.abs() + edu, h.abs() + eh
    check("dx", got[0], dg @ WG + du @ WU, adg @ WG.abs() + adu @ WU.abs(), 2 * F, edg @ WG.abs() + edu @ WU.abs())
    check("dw_gate", got[1], dg.t() @ X, adg.t() @ X.abs(), M, edg.t() @ X.abs())
    check("dw_up", got[2], du.t() @ X, adu.t() @ X.abs(), M, edu.t() @ X.abs())
    check("dw_down", got[3], DY.t() @ h, DY.abs().t() @ ah, M, DY.abs().t() @ eh)
    for p, q in zip(got, gdn.gated_ffn_bwd(dy, x, *w, gate, up)):
        assert torch.equal(p, q)
