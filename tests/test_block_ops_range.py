"""The sizes that the feed-forward block takes, as its header states them: M, D, F and D_out
up to 2^24, tensors of up to 2^38 elements (host side, no GPU)."""
import ctypes

import pytest

import chunked_prefill_gdn_gb300 as gdn
from chunked_prefill_gdn_gb300 import build as gdn_build

P = ctypes.c_void_p(4096)   # never dereferenced: only sizes are asked for
MOST = 1 << 24


@pytest.fixture(scope="module")
def lib():
    gdn_build.build()
    return gdn.load_library()


def sizes(lib, M, D, F, O, dtype):
    d = gdn.GdnFfnDesc(4096, 4096, 4096, 4096, D, M, D, F, O, 0, dtype)
    return lib.gdn_gated_ffn_fwd_workspace_size(d), lib.gdn_gated_ffn_bwd_workspace_size(d, P, O)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("M,D,F,O", [(4, 64, 600000, 64), (40, 64, 600000, 64), (1, MOST, 8, 8), (30, 8, MOST, 8), (7, 8, 8, MOST),
                                     (MOST, 8, 8, 8), (3, 1 << 14, MOST, 5), (1 << 20, 1 << 18, 64, 64), (2, 5, 1 << 14, MOST)])
def test_sizes_within_the_stated_range(lib, M, D, F, O, dtype):
    fwd, bwd = sizes(lib, M, D, F, O, dtype)
    assert fwd >= M * F * (4 if dtype else 2) and bwd >= 3 * M * F * (6 if dtype else 2)


@pytest.mark.parametrize("M,D,F,O", [(4, 64, MOST + 1, 64), (4, MOST + 1, 8, 8), (4, 8, 8, MOST + 1), (MOST + 1, 8, 8, 8),
                                     (3, (1 << 14) + 1, MOST, 5), (1 << 20, 64, 64, (1 << 18) + 1), (1 << 20, (1 << 18) + 1, 64, 64),
                                     (1 << 20, 64, (1 << 18) + 1, 64), (2, 5, (1 << 14) + 1, MOST)])
def test_sizes_beyond_it(lib, M, D, F, O):
    assert sizes(lib, M, D, F, O, 0) == (0, 0)
    d = gdn.GdnFfnDesc(4096, 4096, 4096, 4096, D, M, D, F, O, 0, 0)
    assert lib.gdn_gated_ffn_fwd(d, P, None, None, None, P, 1 << 40, None) == 2
    assert lib.gdn_gated_ffn_bwd(d, P, O, P, P, P, P, P, P, None, P, 1 << 40, None) == 2
