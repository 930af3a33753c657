"""Parity of the feed-forward block with 64 bits at the sizes that run every way of launching its
products (test_ffn_plans_host.py holds them to that)."""
import pytest

import chunked_prefill_gdn_gb300 as gdn
from chunked_prefill_gdn_gb300 import build as gdn_build

from ffn_check import check_ffn
from ffn_plans import SHAPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    gdn_build.build()
    return gdn.load_library()


@pytest.mark.parametrize("dtype,size", [(t, s) for t, sizes in SHAPES.items() for s in sizes])
def test_gated_ffn_on_every_way(dtype, size):
    check_ffn(*size, dtype, act="gelu_tanh" if size[0] % 3 == 0 else "silu")
