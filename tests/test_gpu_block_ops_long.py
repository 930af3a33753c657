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

from ffn_check import TORCH, U, check_ffn

pytestmark = pytest.mark.gpu

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
    check_ffn(M, D, F, O, dtype)
