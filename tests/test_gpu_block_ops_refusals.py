"""What the block operators' tensor functions say when they refuse: the status of the call
itself, also where it is the size of the workspace that cannot be given."""
import pytest
import torch

import chunked_prefill_gdn_gb300 as gdn
from chunked_prefill_gdn_gb300 import build as gdn_build

pytestmark = pytest.mark.gpu

UNSUPPORTED = 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    gdn_build.build()
    return gdn.load_library()


def zeros(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")


def test_too_many_tokens():
    x = zeros((1 << 24) + 1, 1)
    w = zeros(1, 1)
    with pytest.raises(gdn.GdnError, match="GDN_ERR_UNSUPPORTED in gdn_gated_ffn_fwd") as e:
        gdn.gated_ffn_fwd(x, w, w, w)
    assert e.value.status == UNSUPPORTED
    with pytest.raises(gdn.GdnError, match="GDN_ERR_UNSUPPORTED in gdn_gated_ffn_bwd"):
        gdn.gated_ffn_bwd(x, x, w, w, w, x, x)
    x.requires_grad_()
    with pytest.raises(gdn.GdnError, match="GDN_ERR_UNSUPPORTED"):
        gdn.gated_ffn(x, w, w, w)


def test_no_columns():
    x = zeros(40, 0)
    w = zeros(8, 0)
    with pytest.raises(gdn.GdnError, match="GDN_ERR_INVALID_ARG in gdn_gated_ffn_fwd"):
        gdn.gated_ffn_fwd(x, w, w, zeros(8, 8))


def test_rows_too_wide_for_the_norm():
    v = zeros((1 << 30) + 8)
    y, one = v.view(1, -1), torch.ones(1, device="cuda")
    with pytest.raises(gdn.GdnError, match="GDN_ERR_UNSUPPORTED in gdn_block_norm_fwd"):
        gdn.block_norm_fwd(y, post_norm=False, pre_norm=False, scale=v)
    with pytest.raises(gdn.GdnError, match="GDN_ERR_UNSUPPORTED in gdn_block_norm_bwd"):
        gdn.block_norm_bwd(y, None, y, None, one, None, scale=v)
