"""The gated feed-forward block against 64 bits on the GPU, element by element, for sizes at
which the CPU's oracle takes too long.

Bars on the sum of the absolute values of a result's terms, by the length K of its sums.  bf16:
the tensor cores add 16 products at a time, each addition off by at most 2^-22 of the sum so far,
and no sum there is longer than 2^17.  fp32: three bf16 terms hold 24 bits and leave 4 U out of a
product; sums of 256 of K are 6 x 16 additions of 2^-22 (384 U), those over K another K / 256 of
U; 1024 U + K / 256 U covers them.  To that come the last rounding to bf16 (2^-8 of the value),
and what lies between the products: as far off as its own sums, and rounded."""
import torch

import chunked_prefill_gdn_gb300 as gdn

U = 2.0 ** -24
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def sums(K, dtype):
    return (min(K, 2 ** 17) / 16 + 1) * 2.0 ** -22 if dtype == "bf16" else (1024 + K / 256) * U


def activation(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    c = (2.0 / torch.pi) ** 0.5
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def check_ffn(M, D, F, O, dtype, act="silu"):
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    g = torch.Generator(device="cuda").manual_seed(7 * M + F + D + O)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(TORCH[dtype])   # noqa: E731
    x, dy = n(M, D), n(M, O)
    w = [n(F, D, std=D ** -0.5), n(F, D, std=D ** -0.5), n(O, F, std=F ** -0.5)]
    y, gate, up = gdn.gated_ffn_fwd(x, *w, activation=act, save=True, check=True)
    assert torch.equal(y, gdn.gated_ffn_fwd(x, *w, activation=act)[0])

    def check(name, got, want, mag, K, before=0.0):
        err, tol = (got.double() - want).abs(), half * want.abs() + sums(K, dtype) * mag + before + 1e-37
        assert (err <= tol).all(), "%s: %.2f of its bar" % (name, (err / tol).max().item())   # NaN fails too
        assert err.norm() <= (5e-3 if dtype == "bf16" else 1e-5) * want.norm(), name

    X, DY, (WG, WU, WD) = x.double(), dy.double(), (t.double() for t in w)
    G, V = X @ WG.t(), X @ WU.t()
    mg, mu = X.abs() @ WG.abs().t(), X.abs() @ WU.abs().t()
    check("gate", gate, G, mg, D)
    check("up", up, V, mu, D)
    a, _ = activation(G, act)
    h = a * V
    # |act'| < 1.13, |act(g)| <= |g|
    dh = sums(D, dtype) * (1.13 * mg * V.abs() + G.abs() * mu) + (half + 16 * U) * h.abs()
    check("y", y, h @ WD.t(), h.abs() @ WD.abs().t(), F, 1.01 * dh @ WD.abs().t())
    del G, V, mg, mu, h, dh

    got = gdn.gated_ffn_bwd(dy, x, *w, gate, up, activation=act, check=True)
    G, V = gate.double(), up.double()
    a, slope = activation(G, act)
    dh, mdh = DY @ WD, DY.abs() @ WD.abs()
    dg, du, h = dh * V * slope, dh * a, a * V
    edg = sums(O, dtype) * mdh * V.abs() * (slope.abs() + 0.01) + (half + 16 * U) * dg.abs()
    edu = sums(O, dtype) * mdh * (a.abs() + 0.01) + (half + 16 * U) * du.abs()
    eh = (half + 16 * U) * h.abs()
    adg, adu, ah = dg.abs() + edg, du.abs() + edu, h.abs() + eh
    check("dx", got[0], dg @ WG + du @ WU, adg @ WG.abs() + adu @ WU.abs(), 2 * F, 1.01 * (edg @ WG.abs() + edu @ WU.abs()))
    check("dw_gate", got[1], dg.t() @ X, adg.t() @ X.abs(), M, 1.01 * edg.t() @ X.abs())
    check("dw_up", got[2], du.t() @ X, adu.t() @ X.abs(), M, 1.01 * edu.t() @ X.abs())
    check("dw_down", got[3], DY.t() @ h, DY.abs().t() @ ah, M, 1.01 * DY.abs().t() @ eh)
    for p, q in zip(got, gdn.gated_ffn_bwd(dy, x, *w, gate, up, activation=act)):
        assert torch.equal(p, q)
