"""Refusals of the block norm's Python calls, and rules its sources keep."""
import os
import re

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import bwd_rms_norm_gb300 as lib
    from bwd_rms_norm_gb300 import build
    if not os.path.exists(lib.LIB_PATH):
        build.build()
    lib.load_library()
    return lib


@pytest.mark.parametrize("offset", [0.5, 1.9, -0.5, 2, -1, float("nan"), "1"])
def test_offsets_that_are_neither_0_nor_1(L, offset):
    """Refused as such, not cut to a whole number."""
    x, w, s = torch.zeros(4, 8), torch.ones(8), torch.ones(4)
    for call in (lambda: L.rms_norm_block_fwd(x, x, w, None, w, 1e-6, offset),
                 lambda: L.rms_norm_block(x, x, w, None, w, 1e-6, offset),
                 lambda: L.rms_norm_block_bwd(x, x, x, x, s, s, w, None, w, offset)):
        with pytest.raises(L.RMSNormError, match="offset") as e:
            call()
        assert e.value.status == 8


@pytest.mark.parametrize("offset", [0, 1, 0.0, 1.0, True, False])
def test_offsets_that_are_0_or_1(L, offset):
    x, w = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(RuntimeError, match="CUDA"):              # past the offset
        L.rms_norm_block_fwd(x, x, w, None, w, 1e-6, offset)
