"""Pins for the fp64 oracle of the block norm and the gated feed-forward block:
gradients against central differences, closed forms, and autograd of torch in 64
bits."""
import numpy as np
import pytest
import torch

from oracle import block_ops as ref

RNG = np.random.default_rng


def difference(f, x, at, step=1e-6):
    hi, lo = x.copy(), x.copy()
    hi[at] += step
    lo[at] -= step
    return (f(hi) - f(lo)) / (2 * step)


@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
@pytest.mark.parametrize("post,pre,gate,res", [(True, True, True, True), (True, False, True, False), (False, True, False, True),
                                               (False, False, True, True), (True, True, False, False)])
def test_block_norm_gradients_against_differences(post, pre, gate, res, activation):
    g = RNG(3)
    R, D = 4, 7
    y, r, z = (g.standard_normal((R, D)) for _ in range(3))
    wp, sc, wn = (1 + 0.3 * g.standard_normal(D) for _ in range(3))
    r, z = r if res else None, z if gate else None
    dx, dh = g.standard_normal((R, D)), g.standard_normal((R, D)) if pre else None

    def loss(y=y, r=r, z=z, wp=wp, sc=sc, wn=wn):
        x, h, _, _ = ref.block_norm(y, r, z, wp, sc, wn, post, pre, activation)
        return (x * dx).sum() + (0.0 if h is None else (h * dh).sum())

    x, _, rp, rn = ref.block_norm(y, r, z, wp, sc, wn, post, pre, activation)
    dy, dr, dz, dwp, ds, dwn = ref.block_norm_backward(dx, dh, y, x, rp, rn, z, wp if post else None, sc,
                                                       wn if pre else None, activation)
    for at in [(0, 0), (1, 3), (3, 6)]:
        assert abs(difference(lambda v: loss(y=v), y, at) - dy[at]) < 1e-7
        if res:
            assert abs(difference(lambda v: loss(r=v), r, at) - dr[at]) < 1e-7
        if gate:
            assert abs(difference(lambda v: loss(z=v), z, at) - dz[at]) < 1e-7
    for at in (0, 5):
        if post:
            assert abs(difference(lambda v: loss(wp=v), wp, at) - dwp[at]) < 1e-7
        assert abs(difference(lambda v: loss(sc=v), sc, at) - ds[at]) < 1e-7
        if pre:
            assert abs(difference(lambda v: loss(wn=v), wn, at) - dwn[at]) < 1e-7


def test_block_norm_closed_forms():
    """A constant row has rstd 1 / |c| (eps 0); a zero gate leaves the residual; h has
    a mean square of one."""
    y = np.full((2, 5), -3.0)
    x, h, rp, rn = ref.block_norm(y, pre=False, eps=0.0)
    assert h is None and rn is None and np.allclose(x, -1.0) and np.allclose(rp, 1 / 3)
    r = RNG(0).standard_normal((2, 5))
    x, h, _, _ = ref.block_norm(y, r, np.zeros((2, 5)), eps=0.0)
    assert np.array_equal(x, r) and np.allclose((h * h).mean(-1), 1.0)
    half = ref.block_norm(y, z=np.zeros((2, 5)), activation="sigmoid", pre=False, eps=0.0)[0]
    assert np.allclose(half, -0.5)


@pytest.mark.parametrize("activation", ["silu", "gelu_tanh"])
def test_gated_ffn_against_autograd(activation):
    gen = torch.Generator().manual_seed(1)
    x, wg, wu, wd, dy = (torch.randn(*s, generator=gen, dtype=torch.float64) for s in ((5, 6), (9, 6), (9, 6), (4, 9), (5, 4)))
    leaf = [t.clone().requires_grad_() for t in (x, wg, wu, wd)]
    g, u = leaf[0] @ leaf[1].t(), leaf[0] @ leaf[2].t()
    a = torch.nn.functional.silu(g) if activation == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    y = (a * u) @ leaf[3].t()
    want = torch.autograd.grad(y, leaf, dy)
    num = lambda t: t.detach().numpy()   # noqa: E731
    y0, g0, u0, _ = ref.gated_ffn(num(x), num(wg), num(wu), num(wd), activation)
    assert np.allclose(y0, num(y)) and np.allclose(g0, num(g)) and np.allclose(u0, num(u))
    got, _ = ref.gated_ffn_backward(num(dy), num(x), num(wg), num(wu), num(wd), g0, u0, activation)
    for a, b in zip(got, want):
        assert np.allclose(a, num(b), rtol=1e-10, atol=1e-10)
