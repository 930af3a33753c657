"""The feed-forward block's bounded waits: when they run out (about 2 s a launch, without a
fault or a hang) the call says so, and the next one is unaffected."""
import pytest
import torch

import chunked_prefill_gdn_gb300 as gdn
from chunked_prefill_gdn_gb300 import build as gdn_build

from ffn_plans import plan

pytestmark = pytest.mark.gpu

PROBE, TIMEOUT = 1, 6


@pytest.fixture
def lib():
    gdn_build.build()
    lib = gdn.load_library()
    yield lib
    assert lib.gdn_gated_ffn_debug(0) == 0


# pairs of CTAs that leave at once; single CTAs; fp32 in parts
@pytest.mark.parametrize("dtype,M,D,F,O,tiles", [("bf16", 291, 760, 1928, 32, 0), ("bf16", 300, 64, 136, 64, 1), ("f32", 198, 72, 352, 40, 2)])
def test_waits_that_run_out_are_reported(lib, dtype, M, D, F, O, tiles):
    assert plan(lib, M, D, F, O, dtype, 0).tile[0] == tiles
    g = torch.Generator().manual_seed(M)
    n = lambda *s: (torch.randn(*s, generator=g) / s[-1] ** 0.5).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()   # noqa: E731
    x, w = n(M, D), [n(F, D), n(F, D), n(O, F)]
    want = gdn.gated_ffn(x, *w, check=True)
    assert lib.gdn_gated_ffn_debug(PROBE) == 0
    with pytest.raises(gdn.GdnError, match="GDN_ERR_TIMEOUT") as e:
        gdn.gated_ffn(x, *w, check=True)
    assert e.value.status == TIMEOUT
    assert lib.gdn_gated_ffn_debug(0) == 0
    assert torch.equal(gdn.gated_ffn(x, *w, check=True), want)


def test_the_backward_pass_checks_too(lib, monkeypatch):
    """check goes on to the backward pass of the autograd function."""
    from chunked_prefill_gdn_gb300 import block_ops
    seen = []
    backward = block_ops.gated_ffn_bwd
    monkeypatch.setattr(block_ops, "gated_ffn_bwd", lambda *a, **kw: seen.append(kw["check"]) or backward(*a, **kw))
    x, w = torch.ones(40, 8, device="cuda", requires_grad=True), torch.ones(8, 8, device="cuda")
    for check in (False, True):
        gdn.gated_ffn(x, w, w, w, check=check).sum().backward()
    assert seen == [False, True]


def test_other_debug_bits_are_refused(lib):
    assert lib.gdn_gated_ffn_debug(2) == 1 and lib.gdn_gated_ffn_debug(-1) == 1
