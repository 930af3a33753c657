"""The detail behind a CUDA error of the feed-forward block: where a tensor map cannot be
encoded it is the encoder's, not that of a launch that never was.

Without a driver the encoder is missing, so this runs on machines without a GPU only: the
pointers are not of device memory."""
import ctypes

import pytest
import torch

import chunked_prefill_gdn_gb300 as gdn
from chunked_prefill_gdn_gb300 import build as gdn_build

P = ctypes.c_void_p(4096)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the encoder is there")
def test_the_encoders_error_is_kept():
    gdn_build.build()
    lib = gdn.load_library()
    d = gdn.GdnFfnDesc(4096, 4096, 4096, 4096, 64, 40, 64, 128, 64, 0, 0)
    assert lib.gdn_gated_ffn_fwd(d, P, None, None, None, P, 1 << 30, None) == 4
    assert "cuTensorMapEncodeTiled" in gdn.gdn_last_error_detail()
    assert lib.gdn_gated_ffn_bwd(d, P, 64, P, P, P, P, P, P, None, P, 1 << 30, None) == 4
    assert "cuTensorMapEncodeTiled" in gdn.gdn_last_error_detail()
